"""The operators over the state cache and of the outputs' normalisation refuse bad calls on the host,
before anything is launched (no GPU: nothing here gets as far as a launch)."""
import ctypes

import pytest
import torch

from context_scan_gb300 import _build, gdn


@pytest.fixture(scope="module")
def L():
    _build.build_cuda()
    return gdn.lib()


FAKE = ctypes.c_void_p(1 << 20)          # never dereferenced: every case fails validation first
ODD = ctypes.c_void_p((1 << 20) + 8)
BYTE = ctypes.c_void_p((1 << 20) + 2)


def P(**kw):
    d = dict(B=2, T=3, H=4, K=128, V=128, chunk=64, in_dtype=1, out_dtype=0, decay_first=0, gate_k=0)
    d.update(kw)
    return gdn.Problem(**d)


def recurrent(L, prob=None, Hqk=2, nseq=2, cu=None, q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE,
              state=FAKE, slots=5, sin=FAKE, sout=FAKE, per_token=0, o=FAKE, ws=FAKE, n=1 << 20):
    return L.gdn_recurrent_fwd(ctypes.byref(prob or P()), Hqk, nseq, cu, q, k, v, g, beta, state, slots,
                               sin, sout, per_token, o, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(prob=P(B=0)), 1), (dict(prob=P(T=-1)), 1), (dict(prob=P(H=0)), 1), (dict(nseq=0), 1),
    (dict(nseq=3), 1),                              # B sequences without cu_seqlens
    (dict(cu=FAKE), 1),                             # B == 1 with it
    (dict(Hqk=0), 1), (dict(Hqk=3), 2), (dict(Hqk=8), 2),
    (dict(slots=-1), 1), (dict(per_token=2), 1),
    (dict(prob=P(decay_first=2)), 1), (dict(prob=P(gate_k=-1)), 1),
    (dict(prob=P(K=96)), 2), (dict(prob=P(V=32)), 2), (dict(prob=P(V=256)), 2),
    (dict(prob=P(in_dtype=2)), 3), (dict(prob=P(out_dtype=99)), 3),
    (dict(prob=P(B=1 << 16, T=1 << 15), nseq=1 << 16), 2),
    (dict(prob=P(B=1 << 28, T=1), nseq=1 << 28), 2),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(g=None), 1), (dict(beta=None), 1),
    (dict(o=None), 1), (dict(state=None), 1),
    (dict(ws=None), 5), (dict(n=256), 5),
    (dict(q=ODD), 4), (dict(k=ODD), 4), (dict(v=ODD), 4), (dict(g=ODD), 4), (dict(beta=ODD), 4),
    (dict(state=ODD), 4), (dict(o=ODD), 4), (dict(ws=ODD), 4), (dict(sin=BYTE), 4),
    (dict(sout=BYTE), 4), (dict(prob=P(B=1), cu=BYTE), 4),
])
def test_recurrent_refusals(L, kw, status):
    assert recurrent(L, **kw) == status


def test_recurrent_workspace(L):
    assert L.gdn_recurrent_workspace_bytes(-1) == 0
    assert L.gdn_recurrent_workspace_bytes(0) == 256
    assert L.gdn_recurrent_workspace_bytes(1) == 512
    assert L.gdn_recurrent_workspace_bytes(64) == 512
    assert L.gdn_recurrent_workspace_bytes(65) == 768
    with pytest.raises(gdn.GdnError):
        gdn.alloc_recurrent_workspace(-1, device="cpu")


def test_recurrent_binding_refuses_tensors_off_the_device(L):
    q, v, gate = torch.zeros(1, 1, 1, 64), torch.zeros(1, 1, 2, 64), torch.zeros(1, 1, 2)
    state, slots = torch.zeros(3, 2, 64, 64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="is on cpu"):
        gdn.gdn_recurrent_fwd(q, q, v, gate, gate, state, slots, slots, v.clone(),
                              torch.zeros(512, dtype=torch.uint8))


def test_cache_workspace(L):
    W = L.gdn_cache_workspace_bytes
    assert W(0, 1) == 0 and W(1, -1) == 0
    # header, an int a page, eight bytes a job (pairs, or at most half of the pages), an int a request
    assert W(1, 0) == 256 + 256 + 256
    assert W(1000, 0) == 256 + 4096 + 4096
    assert W(1000, 700) == 256 + 4096 + 5632 + 2816
    with pytest.raises(gdn.GdnError):
        gdn.alloc_cache_workspace(0, device="cpu")


PAGES = dict(pages=FAKE, layers=2, num=8, bytes=4096)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=None), 1), (dict(layers=0), 1), (dict(num=0), 1), (dict(n=-1), 1),
    (dict(bytes=0), 2), (dict(bytes=24), 2), (dict(bytes=1 << 40), 2), (dict(pages=ODD), 4),
    (dict(ws=None), 5), (dict(room=256), 5), (dict(ws=ODD), 4),
    (dict(a=None), 1), (dict(b=None), 1), (dict(a=BYTE), 4), (dict(b=BYTE), 4),
    (dict(refs=None), 1), (dict(refs=BYTE), 4), (dict(share=2), 1), (dict(remap=BYTE), 4),
    (dict(live=BYTE), 4),
])
def test_cache_refusals(L, kw, status):
    a = dict(PAGES, n=3, a=FAKE, b=FAKE, refs=FAKE, share=0, remap=None, live=None, ws=FAKE, room=1 << 20)
    a.update(kw)
    head, ws = (a["pages"], a["layers"], a["num"], a["bytes"]), (a["ws"], a["room"], None)
    only = set(kw)
    if not only & {"refs", "share", "remap", "live"}:
        assert L.gdn_cache_copy(*head, a["n"], a["a"], a["b"], *ws) == status
    if not only & {"remap", "live"}:
        assert L.gdn_cache_fork(*head, a["refs"], a["n"], a["a"], a["b"], a["share"], *ws) == status
    if not only & {"b", "share"}:
        assert L.gdn_cache_compact(*head, a["refs"], a["n"], a["a"], a["remap"], a["live"], *ws) == status
    if only <= {"num", "n", "ws", "room", "a", "refs"}:
        assert L.gdn_cache_free(a["num"], a["refs"], a["n"], a["a"], *ws) == status


def test_cache_binding_refuses_tensors_off_the_device(L):
    pages, idx = torch.zeros(1, 4, 16), torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    for call in (lambda: gdn.gdn_cache_copy(pages, idx, idx, ws),
                 lambda: gdn.gdn_cache_fork(pages, idx, idx, idx, ws),
                 lambda: gdn.gdn_cache_free(idx, idx, ws),
                 lambda: gdn.gdn_cache_compact(pages, idx, None, None, None, ws)):
        with pytest.raises(ValueError, match="is on cpu"):
            call()


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(N=0), 1), (dict(rms=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(N=8193), 2), (dict(rows=1 << 40), 2), (dict(xt=2), 3), (dict(yt=-1), 3),
    (dict(x=None), 1), (dict(y=None), 1), (dict(x=ODD), 4), (dict(w=ODD), 4), (dict(b=ODD), 4),
    (dict(z=ODD), 4), (dict(y=ODD), 4), (dict(dy=None), 1), (dict(dy=ODD), 4), (dict(dz=ODD), 4),
    (dict(z=None, dz=FAKE), 1), (dict(dw=ODD), 4), (dict(db=ODD), 4), (dict(ws=None), 5), (dict(room=256), 5),
    (dict(ws=ODD), 4),
])
def test_norm_refusals(L, kw, status):
    a = dict(rows=4, N=64, xt=0, yt=1, rms=1, eps=1e-6, x=FAKE, w=FAKE, b=FAKE, z=FAKE, y=FAKE, dy=FAKE,
             dz=FAKE, dw=FAKE, db=FAKE, ws=FAKE, room=1 << 25)
    a.update(kw)
    head = [a[k] for k in ("rows", "N", "xt", "yt", "rms", "eps")]
    if not set(kw) & {"dy", "dz", "dw", "db", "ws", "room"}:
        assert L.gdn_norm_fwd(*head, a["x"], a["w"], a["b"], a["z"], a["y"], None) == status
    assert L.gdn_norm_bwd(*head, a["x"], a["w"], a["b"], a["z"], a["dy"], a["y"], a["dz"], a["dw"], a["db"],
                          a["ws"], a["room"], None) == status


def test_norm_workspace(L):
    W = L.gdn_norm_bwd_workspace_bytes
    assert W(-1, 8) == 0 and W(1, 0) == 0 and W(1, 8193) == 0
    assert W(0, 64) == 256
    assert W(1, 64) == 256 + 512                      # one block's sums of dw and db
    assert max(W(1 << 24, n) for n in (1, 128, 256, 257, 2048, 4096, 8192)) <= 17 << 20   # 2 * 8192 * 4 B * 256 blocks


def test_norm_binding_refuses_tensors_off_the_device(L):
    x, w = torch.zeros(2, 64), torch.zeros(64)
    with pytest.raises(ValueError, match="is on cpu"):
        gdn.gdn_norm_fwd(x, w, None, None, x.clone())
    with pytest.raises(ValueError, match="is on cpu"):
        gdn.gdn_norm_bwd(x, w, None, None, x, x.clone(), None, w.clone(), None, torch.zeros(4096, dtype=torch.uint8))
