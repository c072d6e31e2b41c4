"""The operators as a layer runs them, in training and in serving: a projection's rows -> heads' norm with the position
rotation -> linear attention with a decay for each head -> gated norm of its outputs, the gradients back through all three, and
a prompt, forks of it and single tokens over a state cache.

Tolerances, derived: in fp32 every operator is good to some 1e-5 of its results' RMS (its own tests), the chain of three to the
sum of theirs, carried through Jacobians of norms around 1: 1e-4. In bf16 each rounding of an activation, 2^-8 / sqrt(3) of its
RMS, counts once: seven of them forward and back, in quadrature 2^-8 sqrt(7 / 3) = 6e-3; 2e-2, the library's bf16 bar.
"""
import pytest
import torch

import plain64
import plain64_linear as plain
from context_scan_gb300 import gdn
from gpu_util import TOL_BF16, record

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from context_scan_gb300 import _build
    _build.build_cuda()
    gdn.lib()


class Layer:
    """Weights of one layer and its three operators."""

    def __init__(self, H, Hqk, K, V, dtype, seed=0):
        gen = torch.Generator().manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.H, self.Hqk, self.K, self.V, self.dtype = H, Hqk, K, V, dtype
        self.wq, self.wk = ((1 + 0.2 * normal(K)) / K ** 0.5).cuda(), ((1 + 0.2 * normal(K)) / K ** 0.5).cuda()
        self.freq = (10000.0 ** (-torch.arange(K // 4).double() * 4 / K)).float().cuda()      # half of the channels turn
        self.decay = (-(2.0 ** (-8.0 * (torch.arange(H) + 1) / H))).cuda()
        self.w = (1 + 0.2 * normal(V)).cuda()

    def rows(self, B, T, seed):
        """What the projection gives: q, k, v and the gate z in one row a token."""
        gen = torch.Generator().manual_seed(seed)
        n = 2 * self.Hqk * self.K + 2 * self.H * self.V
        return torch.randn(B, T, n, generator=gen).to(self.dtype).cuda()

    def split(self, rows):
        a, b = self.Hqk * self.K, self.H * self.V
        parts = rows.split([a, a, b, b], -1)
        return [x.unflatten(-1, (h, -1)) for x, h in zip(parts, (self.Hqk, self.Hqk, self.H, self.H))]

    def heads(self, rows, positions=None):
        q, k, v, z = self.split(rows)
        yq, yk = (torch.empty(q.shape, dtype=self.dtype, device="cuda") for _ in range(2))
        gdn.gdn_qk_norm_fwd(q, k, self.wq, self.wk, self.freq, yq, yk, positions=positions)
        return yq, yk, v.contiguous(), z.contiguous()

    def forward(self, rows, h0=None, positions=None):
        q, k, v, z = self.heads(rows, positions)
        o, y = torch.empty_like(v), torch.empty_like(v)
        ht = torch.empty(rows.shape[0], self.H, self.K, self.V, device="cuda")
        gdn.gdn_linear_fwd(q, k, v, self.decay, h0, o, ht, gdn.alloc_linear_workspace(k, v))
        gdn.gdn_norm_fwd(o, self.w, None, z, y)
        return y, ht, (q, k, v, z, o)

    def backward(self, rows, saved, dy, h0=None, dht=None):
        q, k, v, z, o = saved
        do, dz, dw = torch.empty_like(o), torch.empty_like(z), torch.empty_like(self.w)
        gdn.gdn_norm_bwd(o, self.w, None, z, dy, do, dz, dw, None, gdn.alloc_norm_bwd_workspace(o.numel() // self.V, self.V))
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dh0 = None if h0 is None else torch.empty_like(h0)
        gdn.gdn_linear_bwd(q, k, v, self.decay, h0, do, dht, dq, dk, dv, dh0, gdn.alloc_linear_workspace(k, v, backward=True))
        grad = torch.empty_like(rows)
        gq, gk, gv, gz = self.split(grad)
        dwq, dwk = torch.empty_like(self.wq), torch.empty_like(self.wk)
        rq, rk = self.split(rows)[:2]
        gdn.gdn_qk_norm_bwd(rq, rk, self.wq, self.wk, self.freq, dq, dk, gq, gk, dwq, dwk, gdn.alloc_qk_norm_bwd_workspace(rq))
        gv.copy_(dv)
        gz.copy_(dz)
        return grad, dwq, dwk, dw, dh0

    def plain(self, rows, wq, wk, w, h0=None):
        """The layer in 64 bits, differentiable; rows [B, T, *] on the CPU."""
        B, T = rows.shape[:2]
        q, k, v, z = self.split(rows)
        pos = torch.arange(T).expand(B, T)
        freq = self.freq.double().cpu()
        q = plain.qk_norm(q, wq, freq, pos, False, 1e-6).repeat_interleave(self.H // self.Hqk, 2)
        k = plain.qk_norm(k, wk, freq, pos, False, 1e-6).repeat_interleave(self.H // self.Hqk, 2)
        gap = torch.arange(T)[:, None] - torch.arange(T)
        g = self.decay.double().cpu()[:, None, None]
        D = torch.where(gap >= 0, torch.exp(g * gap.clamp(min=0)), 0.0)
        o = torch.einsum("bihk,bjhk,hij,bjhv->bihv", q, k, D, v)
        t = torch.arange(T)
        ht = torch.einsum("bjhk,bjhv,hj->bhkv", k, v, torch.exp(g[:, 0] * (T - 1 - t)))
        if h0 is not None:
            o = o + torch.einsum("bihk,bhkv,hi->bihv", q, h0, torch.exp(g[:, 0] * (t + 1)))
            ht = ht + torch.exp(g * T) * h0
        return plain64.norm(o, w, None, z, True, 1e-6), ht


def off(got, ref, label):
    return record(float((got.double().cpu() - ref).square().mean().sqrt() / ref.square().mean().sqrt()), label)


@pytest.mark.parametrize("dtype,bar", [(F32, 1e-4), (BF, TOL_BF16)])
@pytest.mark.parametrize("H,Hqk,K,V,T", [(4, 2, 128, 128, 300), (2, 2, 64, 64, 77), (4, 1, 64, 128, 200)])
def test_training_step(H, Hqk, K, V, T, dtype, bar):
    layer = Layer(H, Hqk, K, V, dtype)
    rows = layer.rows(2, T, 3)
    gen = torch.Generator().manual_seed(9)
    dy = torch.randn(2, T, H, V, generator=gen).to(dtype).cuda()
    h0, dht = (0.3 * torch.randn(2, H, K, V, generator=gen).cuda() for _ in range(2))
    y, ht, saved = layer.forward(rows, h0)
    got = (y, ht) + layer.backward(rows, saved, dy, h0, dht)
    leaf = [x.double().cpu().requires_grad_() for x in (rows, layer.wq, layer.wk, layer.w, h0)]
    y64, ht64 = layer.plain(*leaf)
    loss = (y64 * dy.double().cpu()).sum() + (ht64 * dht.double().cpu()).sum()
    ref = (y64.detach(), ht64.detach()) + torch.autograd.grad(loss, leaf)
    for name, a, b in zip(("y", "ht", "rows", "wq", "wk", "w", "h0"), got, ref):
        assert off(a, b, name) <= bar, name


@pytest.mark.parametrize("dtype,bar", [(F32, 1e-4), (BF, TOL_BF16)])
def test_prompt_forks_and_single_tokens(dtype, bar):
    # one prompt in chunks; its state forked to three sequences, which go on by single tokens of their own; the whole of
    # each against the 64-bit layer
    layer = Layer(4, 2, 128, 128, dtype, seed=1)
    prompt, n = layer.rows(1, 261, 5), 6
    tails = layer.rows(3, n, 6)
    y, ht, _ = layer.forward(prompt)
    pages = torch.zeros(1, 8, 4, 128, 128, device="cuda")
    pages[0, 0] = ht[0]
    refs = torch.zeros(8, dtype=torch.int32, device="cuda")
    refs[0] = 1
    children = torch.empty(3, dtype=torch.int32, device="cuda")
    cws = gdn.alloc_cache_workspace(8, 3)
    gdn.gdn_cache_fork(pages, refs, torch.zeros(3, dtype=torch.int32, device="cuda"), children, cws)
    ws = gdn.alloc_recurrent_workspace(8)
    outs = []
    for t in range(n):
        pos = torch.full((3, 1), 261 + t, dtype=torch.int32, device="cuda")
        q, k, v, z = layer.heads(tails[:, t:t + 1], pos)
        o, out = torch.empty_like(v), torch.empty_like(v)
        gdn.gdn_linear_recurrent_fwd(q, k, v, layer.decay, pages[0], children, children, o, ws)
        gdn.gdn_norm_fwd(o, layer.w, None, z, out)
        outs.append(out)
    assert gdn.gdn_check_device_error(ws)[0] == 0 and gdn.gdn_check_device_error(cws)[0] == 0
    params = [x.double().cpu() for x in (layer.wq, layer.wk, layer.w)]
    whole = torch.cat([prompt.expand(3, -1, -1), tails], 1).double().cpu()
    y64, ht64 = layer.plain(whole, *params)
    assert off(torch.cat([y.expand(3, -1, -1, -1)] + outs, 1), y64, "y") <= bar
    assert off(torch.cat(outs, 1), y64[:, 261:], "tail") <= bar
    assert off(pages[0][children.long()], ht64, "state") <= bar


def test_graphs_of_a_training_step():
    # forward and backward captured once, replayed on other rows, beside an eager step on another stream
    layer = Layer(4, 4, 128, 128, BF)
    rows, dy = layer.rows(2, 500, 1), torch.randn(2, 500, 4, 128, device="cuda").to(BF)
    want = []
    for seed in (11, 12):
        rows.copy_(layer.rows(2, 500, seed))
        y, ht, saved = layer.forward(rows)
        want.append([x.clone() for x in (y, ht) + layer.backward(rows, saved, dy)[:4]])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, ht, saved = layer.forward(rows)
        got = (y, ht) + layer.backward(rows, saved, dy)[:4]
    side = torch.cuda.Stream()
    for i, seed in enumerate((11, 12)):
        rows.copy_(layer.rows(2, 500, seed))
        other = layer.rows(2, 500, 11)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            y2, ht2, saved2 = layer.forward(other)
            eager = (y2, ht2) + layer.backward(other, saved2, dy)[:4]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[0]))
