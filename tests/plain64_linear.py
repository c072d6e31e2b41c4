"""Plain 64-bit forms of linear attention with a decay for each head and of the query and key heads' norm with the position
rotation, for the tests: written from the formulas, on the CPU, one token at a time. The same forms on absolute
values bound what roundings can add up to."""
import torch


def _f(x):
    return None if x is None else x.detach().double().cpu()


def _states(n, h0, shape):
    return torch.zeros(n, *shape, dtype=torch.float64) if h0 is None else _f(h0).clone()


def starts(lens):
    return [sum(lens[:i]) for i in range(len(lens))]


def forward(q, k, v, decay, h0, lens, keep=None):
    """o [tokens, H, V] and the last states [nseq, H, K, V]; q, k [tokens, Hqk, K], v [tokens, H, V]; `keep`: a list that
    receives the state after every token."""
    q, k, v = _f(q), _f(k), _f(v)
    rep = v.shape[1] // k.shape[1]
    w = torch.exp(_f(decay))[:, None, None]
    H = _states(len(lens), h0, (v.shape[1], k.shape[2], v.shape[2]))
    o = torch.zeros(v.shape, dtype=torch.float64)
    for s, lo in enumerate(starts(lens)):
        for t in range(lo, lo + lens[s]):
            kt, qt = k[t].repeat_interleave(rep, 0), q[t].repeat_interleave(rep, 0)
            H[s] = w * H[s] + kt[:, :, None] * v[t][:, None, :]
            o[t] = (qt[:, :, None] * H[s]).sum(1)
            if keep is not None:
                keep.append(H[s].clone())
    return o, H


def backward(q, k, v, decay, h0, do, dht, lens):
    """dq, dk [tokens, Hqk, K], dv [tokens, H, V], dh0 by the formulas."""
    q, k, v, do = _f(q), _f(k), _f(v), _f(do)
    Hqk, H = k.shape[1], v.shape[1]
    rep = H // Hqk
    w = torch.exp(_f(decay))[:, None, None]
    S = _states(len(lens), h0, (H, k.shape[2], v.shape[2]))
    D = _states(len(lens), dht, (H, k.shape[2], v.shape[2]))
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    share = lambda x: x.view(Hqk, rep, -1).sum(1)  # noqa: E731
    for s, lo in enumerate(starts(lens)):
        for t in range(lo, lo + lens[s]):
            S[s] = w * S[s] + k[t].repeat_interleave(rep, 0)[:, :, None] * v[t][:, None, :]
            dq[t] = share((S[s] * do[t][:, None, :]).sum(2))
        for t in reversed(range(lo, lo + lens[s])):
            D[s] = D[s] + q[t].repeat_interleave(rep, 0)[:, :, None] * do[t][:, None, :]   # the gradient of the state after t
            dk[t] = share((D[s] * v[t][:, None, :]).sum(2))
            dv[t] = (k[t].repeat_interleave(rep, 0)[:, :, None] * D[s]).sum(1)
            D[s] = w * D[s]
    return dq, dk, dv, D


def qk_norm(x, w, freq, pos, interleaved, eps):
    """y in float64 (differentiable in x and w): x [B, T, H, K], pos [B, T]."""
    K = x.shape[-1]
    u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        u = u * w
    R = 0 if freq is None else 2 * freq.numel()
    if R == 0:
        return u
    t = pos.double()[..., None, None] * freq.double()
    if interleaved:
        a, b = u[..., 0:R:2], u[..., 1:R:2]
    else:
        a, b = u[..., :R // 2], u[..., R // 2:R]
    ya, yb = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
    y = torch.stack([ya, yb], -1).flatten(-2) if interleaved else torch.cat([ya, yb], -1)
    return torch.cat([y, u[..., R:]], -1) if R < K else y
