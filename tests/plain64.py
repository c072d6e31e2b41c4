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
