"""Counts near 2^31, which the operators over the state cache step through in 31 bits, are refused on the host
(no GPU: nothing here gets as far as a launch); so are sizes past a C int by the binding. And how that finds
the current stream."""
import types

import pytest
import torch

from context_scan_gb300 import gdn
from test_operators_host import FAKE, L, P, recurrent  # noqa: F401

TOP = 2**31 - 1
ROOM = 1 << 62


@pytest.mark.parametrize("num,n", [(2**30 + 1, 3), (TOP - 8191, 3), (TOP, 3), (8, 2**30 + 1), (8, TOP - 1023),
                                   (8, TOP), (TOP, TOP)])
def test_cache_counts_past_30_bits(L, num, n):  # noqa: F811
    head, ws = (FAKE, 2, num, 16), (FAKE, ROOM, None)
    assert L.gdn_cache_copy(*head, n, FAKE, FAKE, *ws) == 2
    assert L.gdn_cache_fork(*head, FAKE, n, FAKE, FAKE, 0, *ws) == 2
    assert L.gdn_cache_compact(*head, FAKE, n, FAKE, None, None, *ws) == 2
    assert L.gdn_cache_free(num, FAKE, n, FAKE, *ws) == 2
    W = L.gdn_cache_workspace_bytes
    assert W(num, n) == 0 and W(2**30, 0) > 0 and W(1, 2**30) > 0


def test_binding_refuses_sizes_past_a_c_int():
    # (on the meta device: no memory behind them)
    def meta(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="meta")

    with pytest.raises(ValueError, match="length of a row"):
        gdn._rows(meta(1, 2**32 + 64), meta(1, 2**32 + 64), {})
    with pytest.raises(ValueError, match="length of src"):
        gdn._indexes(src=meta(2**32 + 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="number of pages"):
        gdn._pages(meta(1, 2**32 + 8, 4))
    with pytest.raises(ValueError, match="number of layers"):
        gdn._pages(meta(2**31, 8, 4))


@pytest.mark.parametrize("per_token", [0, 1])
@pytest.mark.parametrize("prob,nseq,cu", [
    (P(B=1, T=TOP), 2, FAKE), (P(B=1, T=TOP - 1023), 2, FAKE), (P(B=1, T=TOP), 1, None),
    (P(B=TOP, T=1, H=1), TOP, None), (P(B=1, T=TOP - 4095), 3, FAKE),
])
def test_recurrent_tokens_near_31_bits(L, prob, nseq, cu, per_token):  # noqa: F811
    assert recurrent(L, prob=prob, nseq=nseq, cu=cu, per_token=per_token, Hqk=1, n=ROOM) == 2
    if cu is not None:   # (one fewer than the limit is looked at further: here, the missing workspace)
        assert recurrent(L, prob=P(B=1, T=TOP - 4096), nseq=nseq, cu=cu, per_token=per_token, ws=None) == 5


@pytest.mark.parametrize("raw", [True, False])
def test_binding_finds_the_current_stream(monkeypatch, raw):
    # with torch's short way to the handle and, in a torch that lacks it, by the stream object
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=1234))
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    if raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    assert gdn._stream(None) == (1003 if raw else 1234)
    assert gdn._stream(77) == 77 and gdn._stream(types.SimpleNamespace(cuda_stream=5)) == 5


def test_binding_hands_on_a_missing_workspace():
    # (the library refuses it with GDN_ERR_WORKSPACE, as for the calls that were there before)
    assert gdn._room(None) == (None, 0)
    w = torch.empty(8, dtype=torch.int32)
    assert gdn._room(w) == (w.data_ptr(), 32)
