"""Linear attention with a decay for each head and the query and key heads' norm refuse bad calls on the host, before
anything is launched (no GPU: nothing here gets as far as a launch); what the binding refuses."""
import ctypes

import pytest
import torch

from context_scan_gb300 import _build, gdn
from test_operators_host import BYTE, FAKE, ODD, P

TOP = 2**31 - 1
ROOM = 1 << 62


@pytest.fixture(scope="module")
def L():
    _build.build_cuda()
    return gdn.lib()


def args(**kw):
    a = dict(prob=P(), Hqk=2, nseq=2, cu=None, q=FAKE, k=FAKE, v=FAKE, decay=FAKE, h0=FAKE, o=FAKE, ht=FAKE, do=FAKE,
             dht=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, dh0=FAKE, ws=FAKE, room=ROOM, state=FAKE, slots=5, sin=FAKE, sout=FAKE,
             per_token=0)
    a.update(kw)
    return a


def fwd(L, a):
    return L.gdn_linear_fwd(ctypes.byref(a["prob"]), a["Hqk"], a["nseq"], a["cu"], *(a[n] for n in (
        "q", "k", "v", "decay", "h0", "o", "ht", "ws", "room")), None)


def bwd(L, a):
    return L.gdn_linear_bwd(ctypes.byref(a["prob"]), a["Hqk"], a["nseq"], a["cu"], *(a[n] for n in (
        "q", "k", "v", "decay", "h0", "do", "dht", "dq", "dk", "dv", "dh0", "ws", "room")), None)


def rec(L, a):
    return L.gdn_linear_recurrent_fwd(ctypes.byref(a["prob"]), a["Hqk"], a["nseq"], a["cu"], *(a[n] for n in (
        "q", "k", "v", "decay", "state", "slots", "sin", "sout", "per_token", "o", "ws", "room")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(prob=P(B=0)), 1), (dict(prob=P(T=-1)), 1), (dict(prob=P(H=0)), 1), (dict(nseq=0), 1), (dict(nseq=3), 1),
    (dict(cu=FAKE), 1), (dict(Hqk=0), 1), (dict(Hqk=3), 2), (dict(Hqk=8), 2),
    (dict(prob=P(decay_first=1)), 1), (dict(prob=P(gate_k=1)), 1),
    (dict(prob=P(K=96)), 2), (dict(prob=P(V=32)), 2), (dict(prob=P(V=256)), 2),
    (dict(prob=P(in_dtype=2)), 3), (dict(prob=P(out_dtype=99)), 3),
    (dict(prob=P(B=1 << 16, T=1 << 15), nseq=1 << 16), 2), (dict(prob=P(B=1, T=TOP - 4095), nseq=1), 2),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(decay=None), 1),
    (dict(ws=None), 5), (dict(room=255), 5), (dict(q=ODD), 4), (dict(k=ODD), 4), (dict(v=ODD), 4), (dict(decay=BYTE), 4),
    (dict(ws=ODD), 4), (dict(prob=P(B=1), cu=BYTE), 4),
])
def test_refusals(L, kw, status):
    a = args(**kw)
    assert fwd(L, a) == status and bwd(L, a) == status and rec(L, a) == status


@pytest.mark.parametrize("kw,status,calls", [
    (dict(o=None), 1, (fwd, rec)), (dict(o=ODD), 4, (fwd, rec)), (dict(h0=ODD), 4, (fwd, bwd)), (dict(ht=ODD), 4, (fwd,)),
    (dict(do=None), 1, (bwd,)), (dict(dq=None), 1, (bwd,)), (dict(dk=None), 1, (bwd,)), (dict(dv=None), 1, (bwd,)),
    (dict(do=ODD), 4, (bwd,)), (dict(dht=ODD), 4, (bwd,)), (dict(dq=ODD), 4, (bwd,)), (dict(dk=ODD), 4, (bwd,)),
    (dict(dv=ODD), 4, (bwd,)), (dict(dh0=ODD), 4, (bwd,)),
    (dict(prob=P(B=1 << 26, T=1), nseq=1 << 26), 2, (fwd, bwd)), (dict(prob=P(B=1 << 28, T=1), nseq=1 << 28), 2, (rec,)),
    (dict(state=None), 1, (rec,)), (dict(slots=-1), 1, (rec,)), (dict(per_token=2), 1, (rec,)), (dict(state=ODD), 4, (rec,)),
    (dict(sin=BYTE), 4, (rec,)), (dict(sout=BYTE), 4, (rec,)),
])
def test_refusals_of_some(L, kw, status, calls):
    for call in calls:
        assert call(L, args(**kw)) == status


def test_workspace(L):
    W = L.gdn_linear_workspace_bytes
    # (no GPU here: no sequence is cut. Packed, there is an entry of 16 bytes a sequence.)
    assert W(ctypes.byref(P(B=2)), 4, 2, 0) == 256
    assert W(ctypes.byref(P(B=1)), 4, 40, 0) == 256 + 768
    # gradients of shared heads: every head's own, for q and for k
    assert W(ctypes.byref(P(B=2)), 2, 2, 1) == 256 + 2 * (2 * 3 * 4 * 128 * 4)
    assert W(ctypes.byref(P(B=2)), 4, 2, 1) == 256
    assert W(ctypes.byref(P(B=2)), 3, 2, 0) == 0 and W(ctypes.byref(P(K=32)), 2, 2, 0) == 0 and W(None, 2, 2, 0) == 0


def test_linear_binding(L):
    q, v, decay = torch.zeros(1, 3, 1, 64), torch.zeros(1, 3, 2, 64), torch.zeros(2)
    ws = torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: gdn.gdn_linear_fwd(q, q, v, decay, None, v.clone(), None, ws),
                 lambda: gdn.gdn_linear_bwd(q, q, v, decay, None, v, None, q.clone(), q.clone(), v.clone(), None, ws),
                 lambda: gdn.gdn_linear_recurrent_fwd(q, q, v, decay, None, None, None, v.clone(), ws)):
        with pytest.raises(ValueError, match="is on cpu"):
            call()
    for kw, what in ((dict(k=q[:, :2]), "k is"), (dict(q=q.bfloat16()), "q is"), (dict(decay=torch.zeros(3)), "decay"),
                     (dict(o=v[..., :32]), "o is"), (dict(cu=torch.zeros(2)), "cu_seqlens"),
                     (dict(states=dict(h0=torch.zeros(1, 2, 64, 32))), "h0"), (dict(v=v[0]), "v ")):
        a = dict(q=q, k=q, v=v, decay=decay, o=v, cu=None, states={})
        a.update(kw)
        with pytest.raises(ValueError, match=what):
            gdn._linear(*a.values())
    with pytest.raises(gdn.GdnError):
        gdn.alloc_linear_workspace(torch.zeros(1, 3, 1, 48), torch.zeros(1, 3, 2, 64))
    with pytest.raises(ValueError, match="more than the library counts"):
        gdn._linear(*[torch.empty(1, 2**31, 1, 64, device="meta")] * 3, None, None, None, {})


def Q(**kw):
    d = dict(B=2, T=3, Hq=4, Hk=2, K=128, R=64, interleaved=0, x_dtype=1, y_dtype=1, eps=1e-6, q_stride=512, k_stride=256)
    d.update(kw)
    return gdn.QkProblem(**d)


def qk(L, a):
    return (L.gdn_qk_norm_fwd(ctypes.byref(a["p"]), *(a[n] for n in ("q", "k", "wq", "wk", "freq", "pos", "yq", "yk")), None),
            L.gdn_qk_norm_bwd(ctypes.byref(a["p"]), *(a[n] for n in (
                "q", "k", "wq", "wk", "freq", "pos", "dyq", "dyk", "dq", "dk", "dwq", "dwk", "ws", "room")), None))


ONE = ctypes.c_void_p((1 << 20) + 1)


@pytest.mark.parametrize("kw,status,which", [
    (dict(p=Q(B=0)), 1, 3), (dict(p=Q(T=-1)), 1, 3), (dict(p=Q(Hq=0)), 1, 3), (dict(p=Q(Hk=0)), 1, 3), (dict(p=Q(K=0)), 1, 3),
    (dict(p=Q(R=-2)), 1, 3), (dict(p=Q(interleaved=2)), 1, 3), (dict(p=Q(eps=-1.0)), 1, 3), (dict(p=Q(eps=float("inf"))), 1, 3),
    (dict(p=Q(eps=float("nan"))), 1, 3), (dict(p=Q(K=127)), 2, 3), (dict(p=Q(K=258, q_stride=2000, k_stride=2000)), 2, 3),
    (dict(p=Q(R=63)), 2, 3), (dict(p=Q(R=130)), 2, 3), (dict(p=Q(q_stride=511)), 1, 3), (dict(p=Q(k_stride=255)), 1, 3),
    (dict(p=Q(q_stride=1 << 31)), 2, 3), (dict(p=Q(Hq=4097, q_stride=1 << 20)), 2, 3), (dict(p=Q(B=1 << 16, T=1 << 15)), 2, 3),
    (dict(p=Q(x_dtype=2)), 3, 3), (dict(p=Q(y_dtype=-1)), 3, 3),
    (dict(q=None), 1, 3), (dict(k=None), 1, 3), (dict(freq=None), 1, 3), (dict(yq=None), 1, 1), (dict(yk=None), 1, 1),
    (dict(dyq=None), 1, 2), (dict(dyk=None), 1, 2), (dict(dq=None), 1, 2), (dict(dk=None), 1, 2),
    (dict(q=ONE), 4, 3), (dict(k=ONE), 4, 3), (dict(wq=BYTE), 4, 3), (dict(wk=BYTE), 4, 3), (dict(freq=BYTE), 4, 3),
    (dict(pos=BYTE), 4, 3), (dict(yq=ONE), 4, 1), (dict(yk=ONE), 4, 1), (dict(dyq=ONE), 4, 2), (dict(dq=ONE), 4, 2),
    (dict(dk=ONE), 4, 2), (dict(dwq=BYTE), 4, 2), (dict(dwk=BYTE), 4, 2), (dict(p=Q(x_dtype=0), q=BYTE), 4, 3),
    (dict(ws=None), 5, 2), (dict(room=1000), 5, 2), (dict(ws=ODD), 4, 2),
])
def test_qk_norm_refusals(L, kw, status, which):
    a = {n: FAKE for n in ("q", "k", "wq", "wk", "freq", "pos", "yq", "yk", "dyq", "dyk", "dq", "dk", "dwq", "dwk", "ws")}
    a |= dict(p=Q(), room=1 << 30)
    a.update(kw)
    got = qk(L, a)
    assert (which == 2 or got[0] == status) and (which == 1 or got[1] == status)


def test_qk_norm_workspace(L):
    W = L.gdn_qk_norm_bwd_workspace_bytes
    assert W(1) == 0 and W(127) == 0 and W(258) == 0 and W(0) == 0
    assert 0 < W(2) <= W(256) <= 3 << 20


def test_qk_norm_binding(L):
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64)
    with pytest.raises(ValueError, match="is on cpu"):
        gdn.gdn_qk_norm_fwd(q, k, None, None, None, q.clone(), k.clone())
    with pytest.raises(ValueError, match="is on cpu"):
        gdn.gdn_qk_norm_bwd(q, k, None, None, None, q, k, q.clone(), k.clone(), None, None, torch.zeros(9, dtype=torch.uint8))
    with pytest.raises(gdn.GdnError):
        gdn.alloc_qk_norm_bwd_workspace(torch.zeros(1, 1, 1, 300))
    rows = torch.zeros(2, 3, 8 * 64)
    S = gdn._head_stride
    assert S("q", q) == 256 and S("q", rows[..., :256].unflatten(-1, (4, 64))) == 512
    assert S("q", rows[:, :1, 64:320].unflatten(-1, (4, 64))) == 3 * 512        # one token a sequence
    assert S("q", torch.zeros(1, 1, 4, 64)) == 256 and S("q", torch.zeros(2, 0, 4, 64)) >= 256
    assert S("q", torch.zeros(2, 6, 4, 64)[:, ::2]) == 512        # every other token: evenly apart all the same
    for bad in (q.transpose(1, 2), q[..., ::2], q[0], torch.zeros(3, 2, 4, 64).transpose(0, 1),
                torch.zeros(2, 1, 1, 64).expand(2, 3, 4, 64)):
        with pytest.raises(ValueError):
            S("q", bad)
