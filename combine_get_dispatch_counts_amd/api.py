"""Thin torch binding over libepx: tensors in, tensors out.

Every step of the path runs in the HIP kernels behind the C ABI; this module
only allocates output tensors with torch (device memory), takes the current
HIP stream, and marshals pointers and sizes. Names follow the C ABI
(epx_get_dispatch_layout -> get_dispatch_layout, and so on).

Shapes: x [T,h] bf16; topk_idx [T,K] int64 (-1 = no route); topk_weights
[T,K] fp32. Destination ranks are logical partitions of the experts:
rank r holds experts [r*L, (r+1)*L), L = num_experts // num_ranks.

No call takes part in autograd: tensors that require a gradient are read like
others, and outputs have no history. The gradients are calls of their own
(rms_norm_backward, route_backward, combine_backward); dispatch's is a combine
of the rows' gradient with weights of one.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import EpxError, check

_contexts: dict[int, ctypes.c_void_p] = {}


def _ctx(device: torch.device) -> ctypes.c_void_p:
    idx = device.index if device.index is not None else torch.cuda.current_device()
    if idx not in _contexts:
        h = ctypes.c_void_p()
        check(_lib.load().epx_create(ctypes.byref(h), idx), "epx_create")
        _contexts[idx] = h
    return _contexts[idx]


def _stream(device: torch.device) -> ctypes.c_void_p:
    idx = device.index if device.index is not None else torch.cuda.current_device()
    # the handle alone takes a fraction of a Stream object's time (some 1 us a
    # call less), but is not a public name of torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return ctypes.c_void_p(raw(idx) if raw else torch.cuda.current_stream(idx).cuda_stream)


def _p(t: torch.Tensor | None) -> ctypes.c_void_p | None:
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor | None, dtype: torch.dtype, name: str, ndim: int | None = None,
          shape: tuple | None = None, device: torch.device | None = None):
    """Reject what the kernels cannot take: the C ABI sees bare pointers and
    row counts, so every buffer's dtype, shape and device is checked here."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _nbytes(ws: torch.Tensor, dev: torch.device) -> int:
    if not ws.is_cuda or ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return ws.numel() * ws.element_size()


def _check_layout(lay: "Layout", T: int, K: int, E: int, R: int, C: int | None,
                  dev: torch.device) -> None:
    i32 = torch.int32
    _need(lay.num_tokens_per_expert, i32, "num_tokens_per_expert", shape=(E,), device=dev)
    _need(lay.num_tokens_per_rank, i32, "num_tokens_per_rank", shape=(R,), device=dev)
    _need(lay.is_token_in_rank, torch.uint8, "is_token_in_rank", shape=(T, R), device=dev)
    _need(lay.rank_off, i32, "rank_off", shape=(R + 1,), device=dev)
    _need(lay.exp_off, i32, "exp_off", shape=(E + 1,), device=dev)
    _need(lay.pos_in_rank, i32, "pos_in_rank", shape=(T, R), device=dev)
    _need(lay.slot_in_expert, i32, "slot_in_expert", shape=(T, K), device=dev)
    _need(lay.totals, i32, "totals", shape=(2,), device=dev)
    if C:
        _need(lay.channel_prefix, i32, "channel_prefix", shape=(R, C), device=dev)


def _check_dispatch_out(out: dict, T: int, h: int, K: int, fp8: bool,
                        dev: torch.device) -> None:
    """``out`` as alloc_dispatch makes it (row slices of those tensors
    included): the send arrays share send_x's row count, the receive
    arrays recv_x's."""
    dt = torch.uint8 if fp8 else torch.bfloat16
    _need(out.get("send_x"), dt, "send_x", ndim=2, device=dev)
    _need(out.get("recv_x"), dt, "recv_x", ndim=2, device=dev)
    ns, nr = out["send_x"].shape[0], out["recv_x"].shape[0]
    _need(out["send_x"], dt, "send_x", shape=(ns, h))
    _need(out["recv_x"], dt, "recv_x", shape=(nr, h))
    _need(out.get("send_src"), torch.int32, "send_src", shape=(ns,), device=dev)
    _need(out.get("send_topk_idx"), torch.int64, "send_topk_idx", shape=(ns, K), device=dev)
    _need(out.get("send_topk_w"), torch.float32, "send_topk_w", shape=(ns, K), device=dev)
    _need(out.get("recv_src"), torch.int32, "recv_src", shape=(nr,), device=dev)
    _need(out.get("pos_exp"), torch.int32, "pos_exp", shape=(T, K), device=dev)
    if fp8:
        st = scale_stride(h)
        _need(out.get("send_scales"), torch.float32, "send_scales", shape=(ns, st), device=dev)
        _need(out.get("recv_scales"), torch.float32, "recv_scales", shape=(nr, st), device=dev)


_workspaces: dict[tuple[int, int], torch.Tensor] = {}


def _layout_workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    """A zero-filled layout workspace of >= nbytes for this device and
    stream, kept for later calls (the layout call leaves it reusable)."""
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    key = (idx, torch.cuda.current_stream(dev).cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


def workspace_size(T: int, K: int, E: int, R: int) -> int:
    n = ctypes.c_size_t()
    check(_lib.load().epx_workspace_size(T, K, E, R, ctypes.byref(n)), "epx_workspace_size")
    return n.value


def ll_size_hint(max_tokens_per_rank: int, h: int, R: int, E: int, fp8: bool) -> int:
    return int(_lib.load().epx_ll_size_hint(max_tokens_per_rank, h, R, E, int(fp8)))


def set_sweep_rate(bf16_gbps: int, fp8_gbps: int, device: torch.device | None = None) -> None:
    """Rate (GB/s of destination rows) of the high-throughput dispatch's
    paced store sweep for bf16 and FP8 rows; 0 turns pacing off. Outputs do
    not depend on it (see epx_set_sweep_rate in include/epx.h)."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    check(_lib.load().epx_set_sweep_rate(_ctx(device), int(bf16_gbps), int(fp8_gbps)),
          "epx_set_sweep_rate")


def get_sweep_rate(device: torch.device | None = None) -> tuple[int, int]:
    """The context's current sweep rates (bf16, FP8) in GB/s."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    b, f = ctypes.c_int(), ctypes.c_int()
    check(_lib.load().epx_get_sweep_rate(_ctx(device), ctypes.byref(b), ctypes.byref(f)),
          "epx_get_sweep_rate")
    return b.value, f.value


def calibrate_sweep_rate(scratch: torch.Tensor) -> int:
    """Set the sweep rates from a fill of ``scratch`` (a contiguous GPU tensor
    of at least 512 MiB, overwritten) timed on the current stream; waits for
    the stream. Returns the measured fill rate in GB/s."""
    if not scratch.is_cuda or not scratch.is_contiguous():
        raise ValueError("scratch must be a contiguous GPU tensor")
    dev = scratch.device
    fill = ctypes.c_int()
    check(_lib.load().epx_calibrate_sweep_rate(_ctx(dev), _p(scratch),
                                               scratch.numel() * scratch.element_size(),
                                               ctypes.byref(fill), _stream(dev)),
          "epx_calibrate_sweep_rate")
    return fill.value


def get_error(device: torch.device | None = None) -> int:
    """Synchronise the current stream, return and clear the device error bits."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    flags = ctypes.c_int()
    rc = _lib.load().epx_get_error(_ctx(device), ctypes.byref(flags), _stream(device))
    if rc not in (_lib.EPX_OK, _lib.EPX_EDEVICE):
        check(rc, "epx_get_error")
    return flags.value


@dataclass
class Layout:
    num_tokens_per_expert: torch.Tensor  # [E] int32
    num_tokens_per_rank: torch.Tensor    # [R] int32
    is_token_in_rank: torch.Tensor       # [T,R] uint8
    rank_off: torch.Tensor               # [R+1] int32
    exp_off: torch.Tensor                # [E+1] int32
    pos_in_rank: torch.Tensor            # [T,R] int32
    slot_in_expert: torch.Tensor         # [T,K] int32
    channel_prefix: torch.Tensor | None  # [R,C] int32
    totals: torch.Tensor                 # [2] int32 (send rows, recv rows)
    num_experts: int
    num_ranks: int


def alloc_layout(T: int, K: int, E: int, R: int, num_channels: int | None,
                 device: torch.device) -> Layout:
    """Output tensors for get_dispatch_layout (reusable across calls)."""
    i32 = dict(dtype=torch.int32, device=device)
    return Layout(
        num_tokens_per_expert=torch.empty(E, **i32),
        num_tokens_per_rank=torch.empty(R, **i32),
        is_token_in_rank=torch.empty((T, R), dtype=torch.uint8, device=device),
        rank_off=torch.empty(R + 1, **i32),
        exp_off=torch.empty(E + 1, **i32),
        pos_in_rank=torch.empty((T, R), **i32),
        slot_in_expert=torch.empty((T, K), **i32),
        channel_prefix=torch.empty((R, num_channels), **i32) if num_channels else None,
        totals=torch.empty(2, **i32),
        num_experts=E, num_ranks=R)


def get_dispatch_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int,
                        num_channels: int | None = None, workspace: torch.Tensor | None = None,
                        totals_host: torch.Tensor | None = None,
                        out: Layout | None = None) -> Layout:
    """Counts, is_token_in_rank and receive offsets for topk_idx. ``out``
    (from alloc_layout with the same shapes) avoids allocating; ``workspace``
    must hold workspace_size(T, K, E, R) bytes and be zero-filled before its
    first use (each call leaves it ready for the next; without one, a cached
    workspace per device and stream is used); ``totals_host`` (pinned int32
    [2]) also receives the totals, readable after a stream synchronisation."""
    _need(topk_idx, torch.int64, "topk_idx", 2)
    dev = topk_idx.device
    T, K = topk_idx.shape
    E, R = num_experts, num_ranks
    lay = out if out is not None else alloc_layout(T, K, E, R, num_channels, dev)
    _check_layout(lay, T, K, E, R, num_channels, dev)
    if workspace is None:
        workspace = _layout_workspace(dev, workspace_size(T, K, E, R))
    ws_bytes = _nbytes(workspace, dev)
    if totals_host is not None and not (totals_host.is_pinned() and totals_host.numel() >= 2
                                        and totals_host.dtype == torch.int32):
        raise ValueError("totals_host must be a pinned int32 tensor of >= 2 elements")
    cp = lay.channel_prefix if num_channels else None
    rc = _lib.load().epx_get_dispatch_layout(
        _ctx(dev), _p(topk_idx), T, K, E, R, num_channels or 0,
        _p(lay.num_tokens_per_expert), _p(lay.num_tokens_per_rank), _p(lay.is_token_in_rank),
        _p(lay.rank_off), _p(lay.exp_off), _p(lay.pos_in_rank), _p(lay.slot_in_expert),
        _p(cp), _p(lay.totals), _p(totals_host), _p(workspace),
        ws_bytes, _stream(dev))
    check(rc, "epx_get_dispatch_layout")
    return lay


def get_dispatch_layout_noalloc(topk_idx: torch.Tensor, num_experts: int, num_ranks: int,
                                num_channels: int | None = None,
                                totals_host: torch.Tensor | None = None,
                                out: Layout | None = None) -> Layout:
    """get_dispatch_layout with the library's own fixed device scratch as
    the workspace (no allocation by the library; with ``out`` given, none
    here either). Calls on one GPU share that scratch and must not overlap."""
    _need(topk_idx, torch.int64, "topk_idx", 2)
    dev = topk_idx.device
    T, K = topk_idx.shape
    E, R = num_experts, num_ranks
    lay = out if out is not None else alloc_layout(T, K, E, R, num_channels, dev)
    _check_layout(lay, T, K, E, R, num_channels, dev)
    if totals_host is not None and not (totals_host.is_pinned() and totals_host.numel() >= 2
                                        and totals_host.dtype == torch.int32):
        raise ValueError("totals_host must be a pinned int32 tensor of >= 2 elements")
    cp = lay.channel_prefix if num_channels else None
    rc = _lib.load().epx_get_dispatch_layout_noalloc(
        _ctx(dev), _p(topk_idx), T, K, E, R, num_channels or 0,
        _p(lay.num_tokens_per_expert), _p(lay.num_tokens_per_rank), _p(lay.is_token_in_rank),
        _p(lay.rank_off), _p(lay.exp_off), _p(lay.pos_in_rank), _p(lay.slot_in_expert),
        _p(cp), _p(lay.totals), _p(totals_host), _stream(dev))
    check(rc, "epx_get_dispatch_layout_noalloc")
    return lay


def scale_stride(h: int) -> int:
    """fp32 entries per FP8 scale row: h/128 rounded up to whole 128-byte
    lines; the entries past h/128 are written as +0.0."""
    n = _lib.load().epx_scale_stride(h)
    if n <= 0:  # the code epx_dispatch gives for such an h with fp8
        bad_h = h < 8 or h % 8 != 0
        raise EpxError(_lib.EPX_EINVAL if bad_h else _lib.EPX_EUNSUPPORTED,
                       f"FP8 rows need h % 128 == 0 (h = {h})")
    return n


@dataclass
class Dispatched:
    """Dispatch outputs. FP8 scales are [rows, scale_stride(h)]: the group
    scales of row i are ``send_scales[i, :h // 128]``."""
    send_x: torch.Tensor          # [rows, h] bf16, or uint8 codes with fp8
    send_scales: torch.Tensor | None
    send_src: torch.Tensor        # [rows] int32
    send_topk_idx: torch.Tensor   # [rows, K] int64
    send_topk_w: torch.Tensor     # [rows, K] fp32
    recv_x: torch.Tensor          # [rows, h] expert-major
    recv_scales: torch.Tensor | None
    recv_src: torch.Tensor        # [rows] int32
    pos_exp: torch.Tensor         # [T, K] int32 -- the handle for combine
    layout: Layout


def alloc_dispatch(T: int, h: int, K: int, send_rows: int, recv_rows: int, fp8: bool,
                   device: torch.device) -> dict:
    """Output buffers for dispatch with the given row capacities."""
    dt = torch.uint8 if fp8 else torch.bfloat16
    f32 = dict(dtype=torch.float32, device=device)
    return dict(
        send_x=torch.empty((send_rows, h), dtype=dt, device=device),
        send_scales=torch.empty((send_rows, scale_stride(h)), **f32) if fp8 else None,
        send_src=torch.empty(send_rows, dtype=torch.int32, device=device),
        send_topk_idx=torch.empty((send_rows, K), dtype=torch.int64, device=device),
        send_topk_w=torch.empty((send_rows, K), **f32),
        recv_x=torch.empty((recv_rows, h), dtype=dt, device=device),
        recv_scales=torch.empty((recv_rows, scale_stride(h)), **f32) if fp8 else None,
        recv_src=torch.empty(recv_rows, dtype=torch.int32, device=device),
        pos_exp=torch.empty((T, K), dtype=torch.int32, device=device))


def dispatch(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
             num_experts: int, num_ranks: int, fp8: bool = False, layout: Layout | None = None,
             out: dict | None = None, exact: bool = True) -> Dispatched:
    """Rank-deduplicated pack + expert-major permute (+ FP8).

    Buffers: ``out`` (from alloc_dispatch) if given; else, with ``exact``,
    one host wait on the layout totals sizes them exactly (the pages' CPU
    wait before allocating the receive tensor); otherwise worst-case sizes
    T*min(K,R) and T*K rows are used and no wait happens."""
    _need(x, torch.bfloat16, "x", 2)
    dev = x.device
    T, h = x.shape
    _need(topk_idx, torch.int64, "topk_idx", 2, device=dev)
    K = topk_idx.shape[1]
    _need(topk_idx, torch.int64, "topk_idx", shape=(T, K))
    _need(topk_weights, torch.float32, "topk_weights", shape=(T, K), device=dev)
    if layout is None:
        layout = get_dispatch_layout(topk_idx, num_experts, num_ranks)
    _check_layout(layout, T, K, num_experts, num_ranks, None, dev)
    if out is None:
        if exact:
            n_send, n_recv = (int(v) for v in layout.totals.cpu())
        else:
            n_send, n_recv = T * min(K, num_ranks), T * K
        out = alloc_dispatch(T, h, K, n_send, n_recv, fp8, dev)
    _check_dispatch_out(out, T, h, K, fp8, dev)
    rc = _lib.load().epx_dispatch(
        _ctx(dev), _p(x), h, _p(topk_idx), _p(topk_weights), T, K, num_experts, num_ranks,
        _p(layout.rank_off), _p(layout.exp_off), _p(layout.pos_in_rank),
        _p(layout.slot_in_expert), int(fp8),
        _p(out["send_x"]), _p(out["send_scales"]), _p(out["send_src"]),
        _p(out["send_topk_idx"]), _p(out["send_topk_w"]), out["send_x"].shape[0],
        _p(out["recv_x"]), _p(out["recv_scales"]), _p(out["recv_src"]), out["recv_x"].shape[0],
        _p(out["pos_exp"]), _stream(dev))
    check(rc, "epx_dispatch")
    return Dispatched(layout=layout, **out)


@dataclass
class Received:
    """A receiver's rows arranged into per-local-expert blocks."""
    x: torch.Tensor                # [N*K cap, h'] rows, expert-major (row order inside a block)
    scales: torch.Tensor | None    # FP8 scale rows, arranged alike
    src_row: torch.Tensor          # [rows] the received row each output row came from
    pos: torch.Tensor              # [N, K] output row of (received row, k), or -1
    layout: Layout                 # counts / offsets over the local experts


def recv_permute(rows: torch.Tensor, local_topk_idx: torch.Tensor, num_local_experts: int,
                 scales: torch.Tensor | None = None) -> Received:
    """The receiver's side of the high-throughput mode: its received rows
    (one per source token, in source then token order) into contiguous
    per-local-expert blocks, row order kept inside each block. ``rows`` are
    bf16 [N, h], or FP8 codes uint8 [N, h] with ``scales`` [N, stride] fp32;
    ``local_topk_idx`` [N, K] int64 holds each row's local expert indices
    (-1 for entries of other ranks), as dispatch's send_topk_idx does. The
    layout of those indices, then one epx_permute launch that moves each row
    and its scale row, bit for bit."""
    dev = rows.device
    _need(local_topk_idx, torch.int64, "local_topk_idx", 2, device=dev)
    N, K = local_topk_idx.shape
    L = num_local_experts
    for name, pl in (("rows", rows), ("scales", scales)):
        if pl is None:
            continue
        if not pl.is_cuda or pl.device != dev or not pl.is_contiguous() or pl.dim() != 2 \
                or pl.shape[0] != N:
            raise ValueError(f"{name} must be a contiguous 2-d tensor on {dev} with one row "
                             "per received row")
    lay = get_dispatch_layout(local_topk_idx, L, 1)
    cap = N * K
    row_bytes = rows.shape[1] * rows.element_size()
    side_bytes = scales.shape[1] * scales.element_size() if scales is not None else 0
    out = torch.empty((cap, rows.shape[1]), dtype=rows.dtype, device=dev)
    out_side = (torch.empty((cap, scales.shape[1]), dtype=scales.dtype, device=dev)
                if scales is not None else None)
    pos = torch.empty((N, K), dtype=torch.int32, device=dev)
    src_row = torch.empty(cap, dtype=torch.int32, device=dev)
    rc = _lib.load().epx_permute(
        _ctx(dev), _p(rows), row_bytes, _p(scales), side_bytes, _p(local_topk_idx), N, K, L,
        _p(lay.exp_off), _p(lay.slot_in_expert), _p(out), _p(out_side), _p(src_row), cap,
        _p(pos), _stream(dev))
    check(rc, "epx_permute")
    return Received(x=out, scales=out_side, src_row=src_row, pos=pos, layout=lay)


def fused_workspace_size(T: int, K: int, E: int, R: int) -> int:
    n = ctypes.c_size_t()
    check(_lib.load().epx_fused_workspace_size(T, K, E, R, ctypes.byref(n)),
          "epx_fused_workspace_size")
    return n.value


def fused_launches(T: int, h: int, K: int, E: int, R: int, fp8: bool = False,
                   device: torch.device | None = None) -> int:
    """How many launches dispatch_fused takes for this shape: 1 for small
    batches (T <= 1024) and while the tiled grid covers every compute unit
    and fits on the device at once, else 2."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    n = ctypes.c_int()
    check(_lib.load().epx_fused_launches(_ctx(device), T, h, K, E, R, int(fp8), ctypes.byref(n)),
          "epx_fused_launches")
    return n.value


def dispatch_fused(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                   num_experts: int, num_ranks: int, fp8: bool = False,
                   num_channels: int | None = None, layout: Layout | None = None,
                   out: dict | None = None, workspace: torch.Tensor | None = None,
                   totals_host: torch.Tensor | None = None) -> Dispatched:
    """get_dispatch_layout and dispatch in one launch (two outside the
    shapes fused_launches reports as one; no host wait either way): the same
    outputs as the two calls. ``layout`` (from alloc_layout) and
    ``out`` (from alloc_dispatch) avoid allocating; without ``out`` the
    buffers get the worst-case capacities T*min(K,R) and T*K rows.
    ``workspace`` must hold fused_workspace_size(T, K, E, R) bytes and be
    zero-filled before its first use (without one, a cached workspace per
    device and stream is used)."""
    _need(x, torch.bfloat16, "x", 2)
    dev = x.device
    T, h = x.shape
    _need(topk_idx, torch.int64, "topk_idx", 2, device=dev)
    K = topk_idx.shape[1]
    _need(topk_idx, torch.int64, "topk_idx", shape=(T, K))
    _need(topk_weights, torch.float32, "topk_weights", shape=(T, K), device=dev)
    E, R = num_experts, num_ranks
    lay = layout if layout is not None else alloc_layout(T, K, E, R, num_channels, dev)
    _check_layout(lay, T, K, E, R, num_channels, dev)
    if out is None:
        out = alloc_dispatch(T, h, K, T * min(K, R), T * K, fp8, dev)
    _check_dispatch_out(out, T, h, K, fp8, dev)
    if workspace is None:
        workspace = _layout_workspace(dev, fused_workspace_size(T, K, E, R))
    ws_bytes = _nbytes(workspace, dev)
    if totals_host is not None and not (totals_host.is_pinned() and totals_host.numel() >= 2
                                        and totals_host.dtype == torch.int32):
        raise ValueError("totals_host must be a pinned int32 tensor of >= 2 elements")
    cp = lay.channel_prefix if num_channels else None
    rc = _lib.load().epx_dispatch_fused(
        _ctx(dev), _p(x), h, _p(topk_idx), _p(topk_weights), T, K, E, R, num_channels or 0,
        _p(lay.num_tokens_per_expert), _p(lay.num_tokens_per_rank), _p(lay.is_token_in_rank),
        _p(lay.rank_off), _p(lay.exp_off), _p(lay.pos_in_rank), _p(lay.slot_in_expert),
        _p(cp), _p(lay.totals), _p(totals_host), _p(workspace), ws_bytes, int(fp8),
        _p(out["send_x"]), _p(out["send_scales"]), _p(out["send_src"]),
        _p(out["send_topk_idx"]), _p(out["send_topk_w"]), out["send_x"].shape[0],
        _p(out["recv_x"]), _p(out["recv_scales"]), _p(out["recv_src"]), out["recv_x"].shape[0],
        _p(out["pos_exp"]), _stream(dev))
    check(rc, "epx_dispatch_fused")
    return Dispatched(layout=lay, **out)


def combine(expert_out: torch.Tensor, pos: torch.Tensor, topk_weights: torch.Tensor,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = bf16(sum over valid k, in k order, of w[t,k] * expert_out[pos[t,k]])."""
    _need(expert_out, torch.bfloat16, "expert_out", 2)
    dev = expert_out.device
    _need(pos, torch.int32, "pos", 2, device=dev)
    T, K = pos.shape
    h = expert_out.shape[1]
    _need(topk_weights, torch.float32, "topk_weights", shape=(T, K), device=dev)
    if out is None:
        out = torch.empty((T, h), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out", shape=(T, h), device=dev)
    rc = _lib.load().epx_combine(_ctx(dev), _p(expert_out), expert_out.shape[0], h,
                                 _p(topk_weights), _p(pos), T, K, _p(out), _stream(dev))
    check(rc, "epx_combine")
    return out


def combine_partial(expert_out: torch.Tensor, dispatched: Dispatched,
                    out: torch.Tensor | None = None,
                    num_rows: torch.Tensor | None = None) -> torch.Tensor:
    """Stage 1 of the two-stage combine: one bf16 partial row per rank-major
    row of ``dispatched`` (its rank's experts reduced with the token's
    weights). Rows past the layout's send-row total are not written."""
    _need(expert_out, torch.bfloat16, "expert_out", 2)
    dev = expert_out.device
    d = dispatched
    _need(d.send_topk_idx, torch.int64, "send_topk_idx", 2, device=dev)
    cap, K = d.send_topk_idx.shape
    _need(d.pos_exp, torch.int32, "pos_exp", 2, device=dev)
    T = d.pos_exp.shape[0]
    h = expert_out.shape[1]
    _need(d.pos_exp, torch.int32, "pos_exp", shape=(T, K))
    _need(d.send_src, torch.int32, "send_src", shape=(cap,), device=dev)
    _need(d.send_topk_w, torch.float32, "send_topk_w", shape=(cap, K), device=dev)
    if out is None:
        out = torch.empty((cap, h), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out", shape=(cap, h), device=dev)
    if num_rows is None:
        num_rows = d.layout.totals[:1]
    _need(num_rows, torch.int32, "num_rows", shape=(1,), device=dev)
    rc = _lib.load().epx_combine_partial(
        _ctx(dev), _p(expert_out), expert_out.shape[0], h, _p(d.send_src), _p(d.send_topk_idx),
        _p(d.send_topk_w), _p(d.pos_exp), T, K, cap, _p(num_rows), _p(out), _stream(dev))
    check(rc, "epx_combine_partial")
    return out


def combine_final(partial: torch.Tensor, layout: Layout,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Stage 2: each token's partial rows summed in rank order (fp32) into bf16."""
    _need(partial, torch.bfloat16, "partial", 2)
    dev = partial.device
    _need(layout.pos_in_rank, torch.int32, "pos_in_rank", 2, device=dev)
    T, R = layout.pos_in_rank.shape
    _need(layout.rank_off, torch.int32, "rank_off", shape=(R + 1,), device=dev)
    h = partial.shape[1]
    if out is None:
        out = torch.empty((T, h), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out", shape=(T, h), device=dev)
    rc = _lib.load().epx_combine_final(_ctx(dev), _p(partial), partial.shape[0], h,
                                       _p(layout.rank_off), _p(layout.pos_in_rank), T, R, _p(out),
                                       _stream(dev))
    check(rc, "epx_combine_final")
    return out


def ll_reset(ll_count: torch.Tensor) -> None:
    _need(ll_count, torch.int32, "ll_count")
    dev = ll_count.device
    check(_lib.load().epx_ll_reset(_ctx(dev), _p(ll_count), ll_count.numel(), _stream(dev)),
          "epx_ll_reset")


@dataclass
class LowLatency:
    ll_x: torch.Tensor              # [E*R_buf*cap, h] bf16 or uint8
    ll_scales: torch.Tensor | None  # [E*R_buf*cap, scale_stride(h)] fp32
    ll_src: torch.Tensor            # [E*R_buf*cap] int32
    ll_count: torch.Tensor          # [E*R_buf] int32
    pos_ll: torch.Tensor            # [T,K] int32 -- the handle for combine


def alloc_ll(E: int, R_buf: int, cap: int, h: int, T: int, K: int, fp8: bool,
             device: torch.device) -> LowLatency:
    rows = E * R_buf * cap
    buf = LowLatency(
        ll_x=torch.empty((rows, h), dtype=torch.uint8 if fp8 else torch.bfloat16, device=device),
        ll_scales=torch.empty((rows, scale_stride(h)), dtype=torch.float32,
                              device=device) if fp8 else None,
        ll_src=torch.empty(rows, dtype=torch.int32, device=device),
        ll_count=torch.empty(E * R_buf, dtype=torch.int32, device=device),
        pos_ll=torch.empty((T, K), dtype=torch.int32, device=device))
    ll_reset(buf.ll_count)
    return buf


def ll_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, num_experts: int, num_ranks: int,
                src_rank: int, cap: int, R_buf: int | None = None, fp8: bool = True,
                buf: LowLatency | None = None, next_buf: LowLatency | None = None,
                stats: torch.Tensor | None = None) -> LowLatency:
    """Fixed-slot low-latency dispatch (one launch, no host wait). ``buf``
    must come from alloc_ll (its counts start at -1). ``next_buf``, the
    other buffer of a ping-pong pair, gets its counts reset to -1 by the same
    launch; ``stats`` (int32 [2] on the device) receives the entries routed
    and the fullest region's count."""
    _need(x, torch.bfloat16, "x", 2)
    dev = x.device
    T, h = x.shape
    _need(topk_idx, torch.int64, "topk_idx", 2, device=dev)
    K = topk_idx.shape[1]
    _need(topk_idx, torch.int64, "topk_idx", shape=(T, K))
    R_buf = num_ranks if R_buf is None else R_buf
    if buf is None:
        buf = alloc_ll(num_experts, R_buf, cap, h, T, K, fp8, dev)
    rows = num_experts * R_buf * cap
    _need(buf.ll_x, torch.uint8 if fp8 else torch.bfloat16, "ll_x", shape=(rows, h), device=dev)
    if fp8:
        _need(buf.ll_scales, torch.float32, "ll_scales", shape=(rows, scale_stride(h)),
              device=dev)
    _need(buf.ll_src, torch.int32, "ll_src", shape=(rows,), device=dev)
    _need(buf.ll_count, torch.int32, "ll_count", shape=(num_experts * R_buf,), device=dev)
    _need(buf.pos_ll, torch.int32, "pos_ll", shape=(T, K), device=dev)
    if stats is not None:
        _need(stats, torch.int32, "stats", device=dev)
        if stats.numel() < 2:
            raise ValueError("stats needs 2 int32 entries")
    nxt = next_buf.ll_count if next_buf is not None else None
    if nxt is not None:
        _need(nxt, torch.int32, "next_buf.ll_count", device=dev)
    rc = _lib.load().epx_ll_dispatch(
        _ctx(dev), _p(x), h, _p(topk_idx), T, K, num_experts, num_ranks, src_rank, cap, R_buf,
        int(fp8), _p(buf.ll_x), _p(buf.ll_scales), _p(buf.ll_src), _p(buf.ll_count),
        _p(buf.pos_ll), _p(nxt), nxt.numel() if nxt is not None else 0, _p(stats), _stream(dev))
    check(rc, "epx_ll_dispatch")
    return buf


def quantize_weights(w: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None
                     ) -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 expert weights [E, N, K] (K a multiple of 128) into e4m3 codes
    (uint8 [E, N, K]) and one fp32 scale per 128 x 128 block
    ([E, ceil(N/128), K/128]): the weight format of grouped_gemm,
    grouped_swiglu and moe_decode. ``out`` (codes, scales) avoids allocating."""
    _need(w, torch.bfloat16, "w", 3)
    dev = w.device
    E, N, K = w.shape
    if K % 128:
        raise EpxError(_lib.EPX_EUNSUPPORTED, f"FP8 weights need K % 128 == 0 (K = {K})")
    if out is None:
        codes = w.new_empty((E, N, K), dtype=torch.uint8)
        scales = w.new_empty((E, -(-N // 128), K // 128), dtype=torch.float32)
    else:
        codes, scales = out
        _need(codes, torch.uint8, "codes", shape=(E, N, K), device=dev)
        _need(scales, torch.float32, "scales", shape=(E, -(-N // 128), K // 128), device=dev)
    check(_lib.load().epx_quantize_weights(_ctx(dev), _p(w), E, N, K, _p(codes), _p(scales),
                                           _stream(dev)), "epx_quantize_weights")
    return codes, scales


def _grouped_operands(x, w, x_scales, w_scales, gated: bool):
    """Dtypes and shapes of a product's operands: (device, rows, K, experts,
    output columns, fp8)."""
    if x is None or not x.is_cuda or x.dim() != 2:
        raise ValueError("x must be a 2-d GPU tensor")
    dev, fp8 = x.device, x.dtype == torch.uint8
    dt = torch.uint8 if fp8 else torch.bfloat16
    _need(x, dt, "x", 2)
    _need(w, dt, "w", 3, device=dev)
    n, K = x.shape
    L, rows_w, K_w = w.shape
    if K_w != K:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected {(L, rows_w, K)}")
    if gated and rows_w % 2:
        raise ValueError("w must hold the gate rows, then as many up rows")
    if fp8:
        _need(x_scales, torch.float32, "x_scales", shape=(n, scale_stride(K)), device=dev)
        _need(w_scales, torch.float32, "w_scales", shape=(L, -(-rows_w // 128), K // 128),
              device=dev)
    elif x_scales is not None or w_scales is not None:
        raise ValueError("scales go with FP8 operands (uint8 codes)")
    return dev, n, K, L, rows_w // 2 if gated else rows_w, fp8


def _swiglu_out(n: int, f: int, fp8: bool, out, out_scales, dev):
    dt = torch.uint8 if fp8 else torch.bfloat16
    if out is None:
        out = torch.empty((n, f), dtype=dt, device=dev)
    else:
        _need(out, dt, "out", shape=(n, f), device=dev)
    if fp8:
        if out_scales is None:
            out_scales = torch.empty((n, scale_stride(f)), dtype=torch.float32, device=dev)
        else:
            _need(out_scales, torch.float32, "out_scales", shape=(n, scale_stride(f)), device=dev)
    elif out_scales is not None:
        raise ValueError("out_scales goes with FP8 operands (uint8 codes)")
    return out, out_scales


def grouped_gemm(x: torch.Tensor, w: torch.Tensor, exp_off: torch.Tensor,
                 x_scales: torch.Tensor | None = None, w_scales: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """out[r] = x[r] @ w[e].T in bf16 for the rows [exp_off[e], exp_off[e+1])
    of each expert e: x [rows, K] expert-major (dispatch's recv_x), w
    [L, N, K], exp_off int32 [L+1] on the device. bf16 operands, or uint8 e4m3
    codes with x_scales [rows, scale_stride(K)] (dispatch's recv_scales) and
    w_scales [L, ceil(N/128), K/128] (quantize_weights'). Rows of no expert
    are not written."""
    dev, n, K, L, N, fp8 = _grouped_operands(x, w, x_scales, w_scales, False)
    _need(exp_off, torch.int32, "exp_off", shape=(L + 1,), device=dev)
    if out is None:
        out = torch.empty((n, N), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, torch.bfloat16, "out", shape=(n, N), device=dev)
    check(_lib.load().epx_grouped_gemm(_ctx(dev), _p(x), _p(x_scales), n, K, _p(w), _p(w_scales),
                                       L, N, int(fp8), _p(exp_off), _p(out), _stream(dev)),
          "epx_grouped_gemm")
    return out


def grouped_swiglu(x: torch.Tensor, w: torch.Tensor, exp_off: torch.Tensor,
                   x_scales: torch.Tensor | None = None, w_scales: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, out_scales: torch.Tensor | None = None
                   ) -> tuple[torch.Tensor, torch.Tensor | None]:
    """grouped_gemm with w [L, 2f, K] (gate rows, then up rows) and the gated
    activation silu(gate) * up applied: (act, scales), act [rows, f] bf16 and
    scales None, or with FP8 operands e4m3 codes and scales [rows,
    scale_stride(f)] in dispatch's format, ready for grouped_gemm."""
    dev, n, K, L, f, fp8 = _grouped_operands(x, w, x_scales, w_scales, True)
    _need(exp_off, torch.int32, "exp_off", shape=(L + 1,), device=dev)
    out, out_scales = _swiglu_out(n, f, fp8, out, out_scales, dev)
    check(_lib.load().epx_grouped_swiglu(_ctx(dev), _p(x), _p(x_scales), n, K, _p(w),
                                         _p(w_scales), L, f, int(fp8), _p(exp_off), _p(out),
                                         _p(out_scales), _stream(dev)), "epx_grouped_swiglu")
    return out, out_scales


def _ll_regions(n: int, L: int, ll_count: torch.Tensor, cap: int, dev) -> int:
    """Regions per expert of a low-latency buffer of n rows."""
    _need(ll_count, torch.int32, "ll_count", 1, device=dev)
    R_buf = ll_count.numel() // L if L else 0
    if L < 1 or R_buf < 1 or ll_count.numel() != L * R_buf:
        raise ValueError(f"ll_count has {ll_count.numel()} entries for {L} experts")
    if cap < 1 or n != L * R_buf * cap:
        raise ValueError(f"x has {n} rows, the regions {L * R_buf} x {cap}")
    return R_buf


def ll_grouped_gemm(x: torch.Tensor, w: torch.Tensor, ll_count: torch.Tensor, cap: int,
                    x_scales: torch.Tensor | None = None, w_scales: torch.Tensor | None = None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """grouped_gemm over low-latency regions: x [L*R_buf*cap, K] (ll_dispatch's
    ll_x), ll_count int32 [L*R_buf] on the device (negative: none), of which
    R_buf consecutive regions belong to each expert. Rows past a region's
    count are neither read nor written."""
    dev, n, K, L, N, fp8 = _grouped_operands(x, w, x_scales, w_scales, False)
    R_buf = _ll_regions(n, L, ll_count, cap, dev)
    if out is None:
        out = torch.empty((n, N), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, torch.bfloat16, "out", shape=(n, N), device=dev)
    check(_lib.load().epx_ll_grouped_gemm(_ctx(dev), _p(x), _p(x_scales), K, _p(w), _p(w_scales),
                                          L, N, int(fp8), _p(ll_count), R_buf, cap, _p(out),
                                          _stream(dev)), "epx_ll_grouped_gemm")
    return out


def ll_grouped_swiglu(x: torch.Tensor, w: torch.Tensor, ll_count: torch.Tensor, cap: int,
                      x_scales: torch.Tensor | None = None,
                      w_scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      out_scales: torch.Tensor | None = None
                      ) -> tuple[torch.Tensor, torch.Tensor | None]:
    """grouped_swiglu over low-latency regions (see ll_grouped_gemm)."""
    dev, n, K, L, f, fp8 = _grouped_operands(x, w, x_scales, w_scales, True)
    R_buf = _ll_regions(n, L, ll_count, cap, dev)
    out, out_scales = _swiglu_out(n, f, fp8, out, out_scales, dev)
    check(_lib.load().epx_ll_grouped_swiglu(_ctx(dev), _p(x), _p(x_scales), K, _p(w),
                                            _p(w_scales), L, f, int(fp8), _p(ll_count), R_buf,
                                            cap, _p(out), _p(out_scales), _stream(dev)),
          "epx_ll_grouped_swiglu")
    return out, out_scales


def moe_decode_workspace(T: int, K: int, f: int) -> int:
    return int(_lib.load().epx_moe_decode_workspace(T, K, f))


def moe_decode(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
               w13: torch.Tensor, w2: torch.Tensor, w13_scales: torch.Tensor | None = None,
               w2_scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The whole expert layer for up to 64 tokens, in two launches: out[t] =
    sum over k of topk_weights[t,k] * w2[e] (silu(gate) * up), e =
    topk_idx[t,k] (-1: none), gate and up the halves of w13[e] x[t]. x [T,h]
    bf16; w13 [E,2f,h] and w2 [E,h,f] bf16, or uint8 e4m3 codes with
    quantize_weights' scales. ``workspace`` (moe_decode_workspace(T, K, f)
    bytes; calls that share one must not overlap) and ``out`` avoid
    allocating."""
    _need(x, torch.bfloat16, "x", 2)
    dev = x.device
    T, h = x.shape
    _need(topk_idx, torch.int64, "topk_idx", 2, device=dev)
    K = topk_idx.shape[1]
    _need(topk_idx, torch.int64, "topk_idx", shape=(T, K))
    _need(topk_weights, torch.float32, "topk_weights", shape=(T, K), device=dev)
    fp8 = w13 is not None and w13.dtype == torch.uint8
    dt = torch.uint8 if fp8 else torch.bfloat16
    _need(w13, dt, "w13", 3, device=dev)
    E, f = w13.shape[0], w13.shape[1] // 2
    _need(w13, dt, "w13", shape=(E, 2 * f, h))
    _need(w2, dt, "w2", shape=(E, h, f), device=dev)
    if fp8:
        _need(w13_scales, torch.float32, "w13_scales", shape=(E, -(-2 * f // 128), h // 128),
              device=dev)
        _need(w2_scales, torch.float32, "w2_scales", shape=(E, -(-h // 128), f // 128),
              device=dev)
    elif w13_scales is not None or w2_scales is not None:
        raise ValueError("scales go with FP8 weights (uint8 codes)")
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, torch.bfloat16, "out", shape=(T, h), device=dev)
    if workspace is None:
        ws_bytes = max(moe_decode_workspace(T, K, f), 16)
        workspace = x.new_empty(ws_bytes, dtype=torch.uint8)
    else:
        ws_bytes = _nbytes(workspace, dev)
    check(_lib.load().epx_moe_decode(_ctx(dev), _p(x), h, _p(topk_idx), _p(topk_weights), T, K, E,
                                     _p(w13), _p(w13_scales), _p(w2), _p(w2_scales), f, int(fp8),
                                     _p(workspace), ws_bytes, _p(out), _stream(dev)),
          "epx_moe_decode")
    return out


def _arg(t: torch.Tensor | None, dtype: torch.dtype, name: str, shape: tuple,
         dev: torch.device) -> int:
    """The address of a tensor that _need takes (with everything right, half
    of the time that _need and _p take)."""
    if (t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != dev.index
            or not t.is_contiguous()):
        _need(t, dtype, name, shape=shape, device=dev)
    return t.data_ptr()


def _rows(t: torch.Tensor | None, dtype: torch.dtype, name: str) -> tuple[torch.device, int, int]:
    """Device and shape of a call's first matrix."""
    if t is None or t.dtype is not dtype or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        _need(t, dtype, name, 2)
    T, n = t.shape
    return t.device, T, n


def _weight(w: torch.Tensor, h: int, dev: torch.device) -> tuple[int, int]:
    """Address of the norm's weight, and 1 if it is fp32, 0 if bf16."""
    f32 = w is not None and w.dtype is torch.float32
    return _arg(w, torch.float32 if f32 else torch.bfloat16, "weight", (h,), dev), int(f32)


@dataclass
class Normed:
    out: torch.Tensor | None = None       # [T,h] bf16
    residual: torch.Tensor | None = None  # [T,h] bf16: x + residual
    codes: torch.Tensor | None = None     # [T,h] uint8, e4m3 codes
    scales: torch.Tensor | None = None    # [T, scale_stride(h)] fp32


def alloc_norm(T: int, h: int, residual: bool, bf16: bool, fp8: bool,
               device: torch.device) -> Normed:
    rows = dict(dtype=torch.bfloat16, device=device)
    return Normed(
        out=torch.empty((T, h), **rows) if bf16 else None,
        residual=torch.empty((T, h), **rows) if residual else None,
        codes=torch.empty((T, h), dtype=torch.uint8, device=device) if fp8 else None,
        scales=torch.empty((T, scale_stride(h)), dtype=torch.float32,
                           device=device) if fp8 else None)


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: torch.Tensor | None = None, bf16: bool = True, fp8: bool = False,
             buf: Normed | None = None) -> Normed:
    """y = v / sqrt(mean(v^2) + eps) * weight per row of v = x + residual (x
    alone without one), x and residual [T,h] bf16, weight [h] bf16 or fp32.
    Returns v in bf16 (``residual``, where one was given), y in bf16 (``out``,
    with ``bf16``) and y as FP8 rows in dispatch's format (``codes`` and
    ``scales``, with ``fp8``), what grouped_gemm and grouped_swiglu read for an
    expert that every token visits (dispatch takes bf16 rows). ``buf``
    (alloc_norm's, or any tensors of those shapes) avoids allocating and says
    by its members which outputs there are; its residual may be ``residual``
    or ``x`` itself, and its out one of them that its residual is not."""
    dev, T, h = _rows(x, torch.bfloat16, "x")
    w, f32 = _weight(weight, h, dev)
    b16, shape = torch.bfloat16, (T, h)
    r = None if residual is None else _arg(residual, b16, "residual", shape, dev)
    if buf is None:
        buf = alloc_norm(T, h, residual is not None, bf16, fp8, dev)
    rout = out = codes = scales = None
    if residual is not None:
        rout = _arg(buf.residual, b16, "buf.residual", shape, dev)
    elif buf.residual is not None:
        raise ValueError("buf.residual goes with a residual")
    if buf.out is not None:
        out = _arg(buf.out, b16, "buf.out", shape, dev)
    if buf.codes is not None:
        codes = _arg(buf.codes, torch.uint8, "buf.codes", shape, dev)
        scales = _arg(buf.scales, torch.float32, "buf.scales", (T, (h // 128 + 31) // 32 * 32), dev)
    elif buf.scales is not None:
        raise ValueError("buf.scales goes with buf.codes")
    elif out is None:
        raise ValueError("rms_norm needs out or codes to write")
    check(_lib.load().epx_rms_norm(_ctx(dev), x.data_ptr(), r, w, f32, T, h, eps, rout, out, codes,
                                   scales, _stream(dev)), "epx_rms_norm")
    return buf


def rms_norm_backward_workspace(T: int, h: int) -> int:
    return int(_lib.load().epx_rms_norm_backward_workspace(T, h))


def _workspace(ws: torch.Tensor | None, nbytes: int, like: torch.Tensor
               ) -> tuple[torch.Tensor | None, int | None, int]:
    """The caller's workspace, or one for this call (to be held until the
    launch), its address and size."""
    if ws is not None:
        return ws, ws.data_ptr(), _nbytes(ws, like.device)
    if nbytes == 0:
        return None, None, 0
    ws = like.new_empty(nbytes, dtype=torch.uint8)
    return ws, ws.data_ptr(), nbytes


def rms_norm_backward(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                      eps: float = 1e-6, dresidual: torch.Tensor | None = None,
                      out: tuple[torch.Tensor, torch.Tensor] | None = None,
                      workspace: torch.Tensor | None = None
                      ) -> tuple[torch.Tensor, torch.Tensor]:
    """rms_norm's gradient: (dx [T,h] bf16, dweight [h] fp32) from dout [T,h]
    bf16 and x [T,h] bf16, what was normed (rms_norm's ``residual`` where it
    had one). ``dresidual`` [T,h] bf16, the gradient that reaches that sum by
    its other ways, is added to dx, which is the gradient of rms_norm's x and
    of its residual alike. ``out`` (dx, dweight; dx may be dout or dresidual)
    and ``workspace`` (rms_norm_backward_workspace(T, h) bytes; calls that
    share one must not overlap) avoid allocating."""
    dev, T, h = _rows(x, torch.bfloat16, "x")
    b16, shape = torch.bfloat16, (T, h)
    d = _arg(dout, b16, "dout", shape, dev)
    w, f32 = _weight(weight, h, dev)
    r = None if dresidual is None else _arg(dresidual, b16, "dresidual", shape, dev)
    if out is None:
        out = torch.empty_like(x), x.new_empty(h, dtype=torch.float32)
    dx, dweight = out
    px = _arg(dx, b16, "dx", shape, dev)
    pw = _arg(dweight, torch.float32, "dweight", (h,), dev)
    lib = _lib.load()
    held, ws, ws_bytes = _workspace(workspace, lib.epx_rms_norm_backward_workspace(T, h), x)
    check(lib.epx_rms_norm_backward(_ctx(dev), d, x.data_ptr(), w, f32, r, T, h, eps, ws, ws_bytes,
                                    px, pw, _stream(dev)), "epx_rms_norm_backward")
    return out


_SCORING = {"softmax": 0, "sigmoid": 1}


def _scoring(name: str) -> int:
    if name not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {name!r}")
    return _SCORING[name]


def route(logits: torch.Tensor, topk: int, scoring: str = "softmax",
          bias: torch.Tensor | None = None, num_groups: int = 1, topk_groups: int = 1,
          normalize: bool = True, scale: float = 1.0, mask: torch.Tensor | None = None,
          out: tuple[torch.Tensor, torch.Tensor] | None = None
          ) -> tuple[torch.Tensor, torch.Tensor]:
    """The router's choice: (topk_idx [T,topk] int64, topk_weights [T,topk]
    fp32) from logits [T,E] fp32, as dispatch, moe_decode and combine read
    them. Scores are the softmax or the sigmoids of the logits; the experts
    of the largest score + ``bias`` ([E] fp32, for the choice alone) are
    taken, largest first, ties to the lower expert; the weights are their
    scores, over their sum with ``normalize``, times ``scale``. With
    ``num_groups`` > 1 only the experts of the ``topk_groups`` best groups
    (sum of the two best) can be chosen. A logit of -inf keeps an expert
    from being chosen, and a bias of -inf keeps it from all tokens (a large
    finite one only puts it last, and slows the call); ``mask`` [T] bool (or uint8) is False for padding,
    which gets -1 and 0 everywhere, as entries do for which no expert is
    left. ``out`` (topk_idx, topk_weights) avoids allocating."""
    dev, T, E = _rows(logits, torch.float32, "logits")
    b = m = None
    if bias is not None:
        b = _arg(bias, torch.float32, "bias", (E,), dev)
    if mask is not None:
        m = _arg(mask, torch.uint8 if mask.dtype is torch.uint8 else torch.bool, "mask", (T,), dev)
    if out is None:
        out = logits.new_empty((T, topk), dtype=torch.int64), logits.new_empty((T, topk))
    idx, w = out
    pi = _arg(idx, torch.int64, "topk_idx", (T, topk), dev)
    pw = _arg(w, torch.float32, "topk_weights", (T, topk), dev)
    check(_lib.load().epx_route(_ctx(dev), logits.data_ptr(), b, m, T, E, topk, _scoring(scoring),
                                num_groups, topk_groups, int(normalize), scale, pi, pw,
                                _stream(dev)), "epx_route")
    return out


@dataclass
class Balance:
    loss: torch.Tensor        # [1] fp32
    counts: torch.Tensor      # [S,E] int32: entries per expert
    probs: torch.Tensor       # [S,E] fp32: mean share per expert
    num_tokens: torch.Tensor  # [S+1] int32: tokens that count, then sequences that have any


def alloc_balance(S: int, E: int, device: torch.device) -> Balance:
    return Balance(loss=torch.empty(1, dtype=torch.float32, device=device),
                   counts=torch.empty((S, E), dtype=torch.int32, device=device),
                   probs=torch.empty((S, E), dtype=torch.float32, device=device),
                   num_tokens=torch.empty(S + 1, dtype=torch.int32, device=device))


def balance_workspace(T: int, E: int, S: int) -> int:
    return int(_lib.load().epx_balance_workspace(T, E, S))


def _sequences(seq_off: torch.Tensor | None, dev: torch.device) -> tuple[int | None, int]:
    """Address of the sequences' offsets and how many there are."""
    if seq_off is None:
        return None, 1
    _need(seq_off, torch.int32, "seq_off", 1, device=dev)
    if seq_off.numel() < 2:
        raise ValueError("seq_off needs an entry per sequence and one more")
    return seq_off.data_ptr(), seq_off.numel() - 1


def _choice(topk_idx: torch.Tensor, T: int, dev: torch.device) -> tuple[int, int]:
    """Address of topk_idx and its entries per token."""
    K = topk_idx.shape[1] if topk_idx is not None and topk_idx.dim() == 2 else 0
    return _arg(topk_idx, torch.int64, "topk_idx", (T, K), dev), K


def balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, scoring: str = "softmax",
                 seq_off: torch.Tensor | None = None, out: Balance | None = None,
                 workspace: torch.Tensor | None = None) -> Balance:
    """Balance loss, per-expert counts and mean shares of logits [T,E] fp32 and
    topk_idx [T,K] int64 (-1: no route; tokens without any do not count). Per
    sequence of n tokens loss_s = E / (K n) * sum over experts of counts *
    probs; the loss is the mean over the sequences that have tokens.
    ``seq_off`` int32 [S+1]: the sequences' first tokens, and where the last
    ends (None: one sequence of all tokens). ``out`` (alloc_balance) and
    ``workspace`` (balance_workspace(T, E, S) bytes; calls that share one must
    not overlap) avoid allocating."""
    dev, T, E = _rows(logits, torch.float32, "logits")
    idx, K = _choice(topk_idx, T, dev)
    off, S = _sequences(seq_off, dev)
    if out is None:
        out = alloc_balance(S, E, dev)
    loss = _arg(out.loss, torch.float32, "loss", (1,), dev)
    counts = _arg(out.counts, torch.int32, "counts", (S, E), dev)
    probs = _arg(out.probs, torch.float32, "probs", (S, E), dev)
    seen = _arg(out.num_tokens, torch.int32, "num_tokens", (S + 1,), dev)
    lib = _lib.load()
    held, ws, ws_bytes = _workspace(workspace, lib.epx_balance_workspace(T, E, S), logits)
    check(lib.epx_balance_loss(_ctx(dev), logits.data_ptr(), idx, off, T, E, K, S,
                               _scoring(scoring), loss, counts, probs, seen, ws, ws_bytes,
                               _stream(dev)), "epx_balance_loss")
    return out


def route_backward(logits: torch.Tensor, topk_idx: torch.Tensor, scoring: str = "softmax",
                   normalize: bool = True, scale: float = 1.0,
                   dtopk_weights: torch.Tensor | None = None, balance: Balance | None = None,
                   dloss: torch.Tensor | None = None, seq_off: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient with respect to the logits (dlogits [T,E] fp32) of route's
    weights (``dtopk_weights`` [T,K] fp32, as combine_backward gives it), of
    the balance loss (``balance`` as balance_loss left it, ``dloss`` [1] fp32
    on the device, and the ``seq_off`` it was given), or of both in one pass.
    logits, topk_idx, scoring, normalize and scale as in the forward calls;
    the choice and the counts are constants. ``out`` avoids allocating."""
    dev, T, E = _rows(logits, torch.float32, "logits")
    idx, K = _choice(topk_idx, T, dev)
    if dtopk_weights is None and balance is None:
        raise ValueError("route_backward needs dtopk_weights, balance or both")
    d = counts = seen = pl = off = None
    S = 1
    if dtopk_weights is not None:
        d = _arg(dtopk_weights, torch.float32, "dtopk_weights", (T, K), dev)
    if balance is not None:
        off, S = _sequences(seq_off, dev)
        counts = _arg(balance.counts, torch.int32, "counts", (S, E), dev)
        seen = _arg(balance.num_tokens, torch.int32, "num_tokens", (S + 1,), dev)
        _need(dloss, torch.float32, "dloss", device=dev)
        if dloss.numel() != 1:
            raise ValueError(f"dloss has {dloss.numel()} entries, expected 1")
        pl = dloss.data_ptr()
    elif dloss is not None or seq_off is not None:
        raise ValueError("dloss and seq_off go with balance")
    if out is None:
        out = torch.empty_like(logits)
    dl = _arg(out, torch.float32, "out", (T, E), dev)
    check(_lib.load().epx_route_backward(_ctx(dev), logits.data_ptr(), idx, T, E, K,
                                         _scoring(scoring), int(normalize), scale, d, counts, seen,
                                         pl, off, S, dl, _stream(dev)), "epx_route_backward")
    return out


def combine_backward(dout: torch.Tensor, expert_out: torch.Tensor | None, pos: torch.Tensor,
                     topk_weights: torch.Tensor,
                     out: tuple[torch.Tensor | None, torch.Tensor | None] | None = None
                     ) -> tuple[torch.Tensor | None, torch.Tensor | None]:
    """combine's gradient: (d_expert_out [rows,h] bf16, d_topk_weights [T,K]
    fp32) from dout [T,h] bf16 and what combine was given. Rows of
    d_expert_out that no entry of ``pos`` names are not written. ``out``
    (either may be None: that gradient is left out) avoids allocating; without
    d_topk_weights expert_out is not read, but still says how many rows there
    are (None: as many as out[0] has)."""
    dev, T, h = _rows(dout, torch.bfloat16, "dout")
    K = pos.shape[1] if pos is not None and pos.dim() == 2 else 0
    p = _arg(pos, torch.int32, "pos", (T, K), dev)
    w = _arg(topk_weights, torch.float32, "topk_weights", (T, K), dev)
    rows_of = expert_out if expert_out is not None or out is None else out[0]
    n = rows_of.shape[0] if rows_of is not None and rows_of.dim() == 2 else 0
    y = _arg(rows_of, torch.bfloat16, "expert_out", (n, h), dev)
    if out is None:
        out = torch.empty_like(expert_out), torch.empty_like(topk_weights)
    dy, dw = out
    py = pw = None
    if dy is not None:
        py = _arg(dy, torch.bfloat16, "d_expert_out", (n, h), dev)
    if dw is not None:
        pw = _arg(dw, torch.float32, "d_topk_weights", (T, K), dev)
        if expert_out is None:
            raise ValueError("d_topk_weights needs expert_out")
    elif dy is None:
        raise ValueError("combine_backward needs an output")
    check(_lib.load().epx_combine_backward(_ctx(dev), dout.data_ptr(), y, n, h, w, p, T, K, py, pw,
                                           _stream(dev)), "epx_combine_backward")
    return out


__all__ = ["EpxError", "Layout", "Dispatched", "LowLatency", "workspace_size", "ll_size_hint",
           "scale_stride", "get_error", "alloc_layout", "get_dispatch_layout", "alloc_dispatch",
           "get_dispatch_layout_noalloc", "dispatch", "combine", "combine_partial",
           "combine_final", "ll_reset", "alloc_ll",
           "ll_dispatch", "Received", "recv_permute", "fused_workspace_size",
           "fused_launches", "dispatch_fused", "set_sweep_rate", "get_sweep_rate",
           "calibrate_sweep_rate", "quantize_weights", "grouped_gemm", "grouped_swiglu",
           "ll_grouped_gemm", "ll_grouped_swiglu", "moe_decode_workspace", "moe_decode", "Normed",
           "alloc_norm", "rms_norm", "rms_norm_backward_workspace", "rms_norm_backward", "route",
           "Balance", "alloc_balance", "balance_workspace", "balance_loss", "route_backward",
           "combine_backward"]
