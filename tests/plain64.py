"""Plain 64-bit forms of the operators around the chunked rule, for the tests: written from the
formulas, on the CPU, one token (row, page) at a time."""
import torch


def recurrence(q, k, v, g, beta, state, slots_in, slots_out, lens, per_token=False, decay_first=False):
    """o [tokens, H, V] and the cache after the call, in float64. q, k [tokens, Hqk, K], v [tokens, H,
    V], g [tokens, H] or [tokens, H, K], beta [tokens, H]; slots as lists (None: no array)."""
    q, k, v, g, beta = (x.detach().double().cpu() for x in (q, k, v, g, beta))
    before = state.detach().double().cpu()
    after = before.clone()
    H = v.shape[1]
    rep = H // k.shape[1]
    o = torch.zeros(v.shape, dtype=torch.float64)
    t = 0
    for s, n in enumerate(lens):
        a = slots_in[s] if slots_in is not None else -1
        S = before[a].clone() if a >= 0 else torch.zeros(before.shape[1:], dtype=torch.float64)
        for _ in range(n):
            kt, qt = k[t].repeat_interleave(rep, 0), q[t].repeat_interleave(rep, 0)
            e = torch.exp(g[t])
            E = e[:, :, None] if g.dim() == 3 else e[:, None, None]
            read = torch.einsum("hk,hkv->hv", kt, E * S if decay_first else S)
            r = beta[t][:, None] * (v[t] - read)
            S = E * S + kt[:, :, None] * r[:, None, :]
            o[t] = torch.einsum("hk,hkv->hv", qt, S)
            if per_token and slots_out is not None and slots_out[t] >= 0:
                after[slots_out[t]] = S
            t += 1
        if not per_token and slots_out is not None and slots_out[s] >= 0:
            after[slots_out[s]] = S
    return o, after


def cache_copy(pages, src, dst):
    """pages [layers, num_pages, ...] after the copy; pairs that the call refuses are left out, and
    whether any was."""
    after, bad = pages.clone(), False
    num = pages.shape[1]
    for i, (a, b) in enumerate(zip(src, dst)):
        others = [(x, y) for j, (x, y) in enumerate(zip(src, dst)) if j != i]
        if a >= num or b >= num or (b >= 0 and any(b in pair for pair in others)):
            bad = True
        elif b >= 0:
            after[:, b] = pages[:, a] if a >= 0 else 0
    return after, bad


def cache_fork(pages, refs, parents):
    """(pages, refs, children, code of the error word) after a fork."""
    pages, refs, before = pages.clone(), list(refs), list(refs)
    free = [p for p, r in enumerate(refs) if r <= 0]
    children, code = [], 0
    for a in parents:
        if a >= len(refs) or (a >= 0 and before[a] <= 0):
            children.append(-1)
            code = 1   # (recorded before a full cache is)
        elif not free:
            children.append(-1)
            code = code or 9
        else:
            child = free.pop(0)
            pages[:, child] = pages[:, a] if a >= 0 else 0
            refs[child] = 1
            children.append(child)
    return pages, refs, children, code


def cache_compact(pages, refs, table):
    """(pages, refs, table, remap, live) after a compaction."""
    pages, refs = pages.clone(), list(refs)
    num = len(refs)
    live = sum(r > 0 for r in refs)
    remap = [p if refs[p] > 0 else -1 for p in range(num)]
    holes = [p for p in range(live) if refs[p] <= 0]
    for p in range(live, num):
        if refs[p] > 0:
            to = holes.pop(0)
            pages[:, to], refs[to], refs[p], remap[p] = pages[:, p], refs[p], 0, to
    table = [t if t < 0 else remap[t] if t < num else -1 for t in table]
    return pages, refs, table, remap, live


def norm(x, w, b, z, rms, eps):
    """y in float64 (differentiable)."""
    m = 0.0 if rms else x.mean(-1, keepdim=True)
    var = ((x - m) ** 2).mean(-1, keepdim=True)
    y = (x - m) / torch.sqrt(var + eps)
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y if z is None else y * z * torch.sigmoid(z)


def norm_grads(x, w, b, z, dy, rms, eps):
    """(dx, dz, dw, db) by the formulas, in float64; the parameters' gradients also where they are None."""
    x, dy = x.double(), dy.double()
    n = x.shape[-1]
    w = torch.ones(n, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(n, dtype=torch.float64) if b is None else b.double()
    xm = x if rms else x - x.mean(-1, keepdim=True)
    s = 1.0 / torch.sqrt((xm * xm).mean(-1, keepdim=True) + eps)
    xh, d, dz = xm * s, dy, None
    if z is not None:
        z = z.double()
        sg = torch.sigmoid(z)
        dz = dy * (xh * w + b) * sg * (1 + z * (1 - sg))
        d = dy * z * sg
    dw, db = (d * xh).sum(0), d.sum(0)
    dxh = d * w
    dx = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if not rms:
        dx = dx - dxh.mean(-1, keepdim=True)
    return dx * s, dz, dw, db
