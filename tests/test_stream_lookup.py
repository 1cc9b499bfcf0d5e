"""The binding's lookup of the current stream: torch's handle of it, by the
public way where the short one is missing."""
import types

import pytest
import torch


def test_public_lookup_where_the_short_one_is_missing(monkeypatch):
    from combine_get_dispatch_counts_amd import api

    seen = []

    def current(device):
        seen.append(device)
        return types.SimpleNamespace(cuda_stream=4096)

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", current)
    assert api._stream(torch.device("cuda", 3)).value == 4096
    assert seen == [3]


@pytest.mark.gpu
def test_both_lookups_agree(monkeypatch):
    from combine_get_dispatch_counts_amd import api

    dev = torch.device("cuda", 0)
    streams = [torch.cuda.default_stream(dev), torch.cuda.Stream(dev), torch.cuda.Stream(dev)]

    def handles():
        out = []
        for s in streams:
            with torch.cuda.stream(s):
                out.append((api._stream(dev).value, api._stream(torch.device("cuda")).value))
        return out

    want = [(s.cuda_stream or None,) * 2 for s in streams]
    assert handles() == want
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert handles() == want
