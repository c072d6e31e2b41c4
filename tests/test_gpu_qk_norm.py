"""GPU parity of the query and key heads' norm with the position rotation (gdn_qk_norm_fwd, gdn_qk_norm_bwd) against the plain
64-bit form and its gradients by differentiation.

Tolerances, derived. Forward: the sum of K squares in pairs of chains of at most 16 and five exchanges is good to 22 steps
of 2^-24, its root to half of that, the reciprocal root's instruction to 2, the products with s, w, cos and sin and their sum to
one each, sin and cos to 2 steps and their angle (31 bits of a turn as fp32) to one more: 24 steps of 2^-24 of |u_a| + |u_b|, the
pair's values. A bf16 result adds half a step, 2^-8 of itself. Backward: with e the turned dy (8 steps of its pair), dx = s (e w -
x s m): m, a sum over K of products good to 40 steps of the sum of their absolute values; 64 steps of s (|e w| + |x s| M), M that
sum over K. dw: its n rows' terms pass 40 roundings each and a sum of n / 1000 + 100 in a chain.
"""
import pytest
import torch

import plain64_linear as plain
from context_scan_gb300 import gdn
from gpu_util import record

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
STEP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


def make(B, T, Hq, Hk, K, R, x=BF, y=BF, fused=False, offset=0, far=1000, weights=True, positions=True, seed=0):
    gen = torch.Generator().manual_seed(900 + seed)
    normal = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {}
    if fused:
        rows = normal(B, T, (Hq + 2 * Hk) * K + offset).to(x).cuda()
        d["q"] = rows[..., offset:offset + Hq * K].unflatten(-1, (Hq, K))
        d["k"] = rows[..., offset + Hq * K:offset + (Hq + Hk) * K].unflatten(-1, (Hk, K))
    else:
        d["q"], d["k"] = normal(B, T, Hq, K).to(x).cuda(), normal(B, T, Hk, K).to(x).cuda()
    d["wq"] = (1 + 0.2 * normal(K)).cuda() if weights else None
    d["wk"] = (1 + 0.2 * normal(K)).cuda() if weights else None
    d["freq"] = (10000.0 ** (-torch.arange(R // 2).double() * 2 / max(R, 1))).float().cuda() if R else None
    d["pos"] = torch.randint(0, far, (B, T), generator=gen, dtype=torch.int32).cuda() if positions else None
    d["dyq"], d["dyk"] = normal(B, T, Hq, K).to(y).cuda(), normal(B, T, Hk, K).to(y).cuda()
    d["y"], d["x"] = y, x
    return d


def call(d, il, eps=1e-6, stream=None):
    yq = torch.full(d["q"].shape, float("nan"), dtype=d["y"], device="cuda")
    yk = torch.full(d["k"].shape, float("nan"), dtype=d["y"], device="cuda")
    gdn.gdn_qk_norm_fwd(d["q"], d["k"], d["wq"], d["wk"], d["freq"], yq, yk, positions=d["pos"], eps=eps, interleaved=il,
                        stream=stream)
    torch.cuda.synchronize()
    return yq, yk


def positions(d):
    B, T = d["q"].shape[:2]
    return d["pos"].cpu() if d["pos"] is not None else torch.arange(T).expand(B, T)


def pairs(x, R, il):
    """|u_a| + |u_b| at both members of every rotated pair, |u| elsewhere."""
    x = x.abs()
    out = x.clone()
    if il:
        s = x[..., 0:R:2] + x[..., 1:R:2]
        out[..., 0:R:2] = out[..., 1:R:2] = s
    else:
        s = x[..., :R // 2] + x[..., R // 2:R]
        out[..., :R // 2] = out[..., R // 2:R] = s
    return out


def freq64(d):
    return None if d["freq"] is None else d["freq"].double().cpu()


CASES = {
    # B, T, Hq, Hk, K, R, interleaved, options
    "decode": (3, 1, 4, 2, 128, 128, False, {}),
    "one_row": (1, 1, 1, 1, 64, 64, True, {}),
    "prompt": (2, 33, 8, 2, 128, 128, False, dict(positions=False)),
    "interleaved": (2, 17, 3, 3, 128, 128, True, {}),
    "fused": (2, 19, 6, 2, 128, 128, False, dict(fused=True)),
    "fused_interleaved": (2, 19, 6, 2, 64, 64, True, dict(fused=True)),
    "fused_decode": (5, 1, 6, 2, 128, 64, True, dict(fused=True)),
    "fused_odd_offset": (2, 9, 3, 1, 64, 64, False, dict(fused=True, offset=1)),
    "fused_even_offset": (2, 9, 3, 1, 64, 64, True, dict(fused=True, offset=2)),
    "partial": (1, 40, 4, 4, 128, 64, False, {}),
    "partial_interleaved": (1, 40, 4, 4, 96, 32, True, {}),
    "norm_alone": (1, 21, 3, 5, 128, 0, False, {}),
    "no_weights": (1, 21, 3, 5, 80, 80, False, dict(weights=False)),
    "k2": (1, 5, 2, 1, 2, 2, False, {}),
    "k6": (2, 5, 2, 1, 6, 4, True, {}),
    "k18": (2, 5, 3, 2, 18, 10, False, {}),
    "k72": (2, 5, 3, 2, 72, 72, False, {}),
    "k254": (1, 7, 2, 2, 254, 254, False, {}),
    "k250_interleaved": (1, 7, 2, 2, 250, 100, True, {}),
    "k256": (1, 7, 2, 2, 256, 256, False, {}),
    "k256_interleaved": (1, 7, 2, 2, 256, 128, True, dict(x=F32, y=F32)),
    "fp32": (2, 13, 4, 2, 128, 128, False, dict(x=F32, y=F32)),
    "fp32_96": (13, 1, 16, 16, 96, 96, True, dict(x=F32, y=F32, far=1 << 20)),
    "fp32_to_bf16": (2, 13, 4, 2, 64, 64, False, dict(x=F32, y=BF)),
    "bf16_to_fp32": (2, 13, 4, 2, 64, 32, True, dict(x=BF, y=F32)),
    "many_heads": (1, 3, 70, 33, 64, 64, False, {}),
    "many_tokens": (3, 700, 5, 3, 64, 64, True, {}),
    "many_tokens_few_heads": (2, 4000, 1, 1, 128, 128, False, {}),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_forward(name):
    B, T, Hq, Hk, K, R, il, kw = CASES[name]
    d = make(B, T, Hq, Hk, K, R, **kw)
    for got, x, w in zip(call(d, il), (d["q"], d["k"]), (d["wq"], d["wk"])):
        w = None if w is None else w.double().cpu()
        x = x.double().cpu()
        ref = plain.qk_norm(x, w, freq64(d), positions(d), il, 1e-6)
        u = plain.qk_norm(x, w, None, None, il, 1e-6)
        tol = 24 * STEP * pairs(u, R, il) + (2.0 ** -8 if d["y"] == BF else 0.0) * ref.abs()
        off = (got.double().cpu() - ref).abs()
        record(float((off / tol.clamp(min=1e-30)).max()), "y")
        assert (off <= tol + 1e-30).all()


def run_bwd(d, il, dw=True):
    K = d["q"].shape[-1]
    g = {}
    for n in ("q", "k"):
        t = d[n]
        # (the same strides, in memory of its own)
        size = t.shape[0] * max(t.stride(0), t.shape[1] * t.stride(1)) + t.shape[2] * K
        g[n] = torch.full((size,), float("nan"), dtype=t.dtype, device="cuda").as_strided(t.shape, t.stride())
    dw = [torch.full((K,), float("nan"), device="cuda") if dw else None for _ in range(2)]
    ws = gdn.alloc_qk_norm_bwd_workspace(d["q"], d["k"])
    ws.fill_(255)
    gdn.gdn_qk_norm_bwd(d["q"], d["k"], d["wq"], d["wk"], d["freq"], d["dyq"], d["dyk"], g["q"], g["k"], *dw, ws,
                        positions=d["pos"], interleaved=il)
    torch.cuda.synchronize()
    return g["q"], g["k"], dw[0], dw[1]


@pytest.mark.parametrize("name", sorted(CASES))
def test_backward(name):
    B, T, Hq, Hk, K, R, il, kw = CASES[name]
    d = make(B, T, Hq, Hk, K, R, **kw)
    got = run_bwd(d, il)
    for dx, dw, x, w, dy in ((got[0], got[2], d["q"], d["wq"], d["dyq"]), (got[1], got[3], d["k"], d["wk"], d["dyk"])):
        x = x.double().cpu().requires_grad_()
        w = (torch.ones(K) if w is None else w.cpu()).double().requires_grad_()
        dy = dy.double().cpu()
        y = plain.qk_norm(x, w, freq64(d), positions(d), il, 1e-6)
        rx, rw = torch.autograd.grad(y, (x, w), dy)
        x, w = x.detach(), w.detach()
        s = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        e = pairs(dy, R, il)
        M = (e * w.abs() * (x * s).abs()).mean(-1, keepdim=True)
        tol = 64 * STEP * s * (e * w.abs() + (x * s).abs() * M) + (2.0 ** -8 if d["x"] == BF else 0.0) * rx.abs()
        off = (dx.double().cpu() - rx).abs()
        record(float((off / tol.clamp(min=1e-30)).max()), "dx")
        assert (off <= tol + 1e-30).all()
        n = x.shape[0] * x.shape[1] * x.shape[2]
        tol = (40 + n / 1000 + 100) * STEP * (e * (x * s).abs()).sum((0, 1, 2))
        off = (dw.double().cpu() - rw).abs()
        record(float((off / tol.clamp(min=1e-30)).max()), "dw")
        assert (off <= tol).all()


def test_without_weight_gradients():
    d = make(2, 9, 3, 2, 64, 64)
    a, b = run_bwd(d, False), run_bwd(d, False, dw=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_what_lies_between_the_rows_stays():
    d = make(2, 9, 3, 2, 64, 64, fused=True)
    width = (3 + 4) * 64
    rows = torch.full((2, 9, width), 7.0, dtype=BF, device="cuda")
    dq, dk = rows[..., :192].unflatten(-1, (3, 64)), rows[..., 192:320].unflatten(-1, (2, 64))
    ws = gdn.alloc_qk_norm_bwd_workspace(d["q"])
    gdn.gdn_qk_norm_bwd(d["q"], d["k"], d["wq"], d["wk"], d["freq"], d["dyq"], d["dyk"], dq, dk, None, None, ws, positions=d["pos"])
    a = run_bwd(d, False)
    assert torch.equal(dq, a[0]) and torch.equal(dk, a[1]) and (rows[..., 320:] == 7.0).all()


@pytest.mark.parametrize("il", [False, True])
def test_far_and_negative_positions(il):
    d = make(1, 8, 1, 1, 64, 64, x=F32, y=F32)
    d["pos"] = torch.tensor([[0, -1, 2**31 - 1, -2**31, 10**9 + 7, 123456789, 2**24 + 1, -(10**6)]], dtype=torch.int32).cuda()
    yq, _ = call(d, il)
    x = d["q"].double().cpu()
    ref = plain.qk_norm(x, d["wq"].double().cpu(), freq64(d), positions(d), il, 1e-6)
    u = plain.qk_norm(x, d["wq"].double().cpu(), None, None, il, 1e-6)
    # (the 64-bit angle itself is good to 2^31 2^-52 of a turn on either side, 3e-6 of a radian)
    assert ((yq.double().cpu() - ref).abs() <= (24 * STEP + 6e-6) * pairs(u, 64, il)).all()


def test_rows_of_zeros_and_no_tokens():
    d = make(1, 3, 2, 2, 64, 64, x=F32, y=F32)
    d["q"][0, 1] = 0
    yq, yk = call(d, False)
    assert (yq[0, 1] == 0).all() and torch.isfinite(yk).all()
    g = run_bwd(d, False)
    assert all(torch.isfinite(x).all() for x in g)
    d = make(2, 0, 2, 2, 64, 64)
    call(d, False)
    g = run_bwd(d, False)
    assert (g[2] == 0).all() and (g[3] == 0).all()


def test_same_bits_graph_and_stream():
    d = make(3, 500, 6, 2, 128, 128, fused=True)
    a = run_bwd(d, False)
    b = run_bwd(d, False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    side = torch.cuda.Stream()
    yq, yk = call(d, False)
    zq, zk = torch.empty_like(yq), torch.empty_like(yk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gdn.gdn_qk_norm_fwd(d["q"], d["k"], d["wq"], d["wk"], d["freq"], zq, zk, positions=d["pos"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(zq, yq) and torch.equal(zk, yk)
    with torch.cuda.stream(side):
        again = call(d, False)
    assert torch.equal(again[0], yq)


def test_l2_normalisation():
    # as the header says: w = 1 / sqrt(K) and eps / K give the L2 norm that the delta rule takes
    d = make(1, 20, 4, 4, 128, 0, x=F32, y=F32)
    d["wq"] = d["wk"] = torch.full((128,), 128.0 ** -0.5, device="cuda")
    yq, _ = call(d, False, eps=1e-12 / 128)
    ref = torch.nn.functional.normalize(d["q"].double(), dim=-1)
    assert ((yq.double() - ref).abs() <= 24 * STEP * ref.abs() + 1e-30).all()
