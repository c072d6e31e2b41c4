"""Cases and plain forms of linear attention with a decay for each head -- the chunked form for prompts, its
gradients, the recurrent form over a state cache -- and of the norm of every query and key head with the position
rotation, with its gradients.

``run`` computes a case with elementary torch operations in 32 bits, or, where ``own`` is true, with
the library's kernels through ``context_scan_gb300.gdn``; ``exact`` gives the same in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-6
CHUNK = 128     # of the plain form


# ---------------------------------------------------------------------------------------- cases

def linear(op, nseq, lo, hi, h, hqk, k, v, dtype="bf16", start=True, name=None):
    """nseq sequences of lo..hi tokens (lo == hi: all alike, no cu_seqlens; else packed); `start`: from given
    states, else from zeros."""
    c = dict(op=op, nseq=nseq, lo=lo, hi=hi, h=h, hqk=hqk, k=k, v=v, dtype=dtype, start=start)
    return dict(c, name=name) if name else c


def recurrent(nseq, lo, hi, h, hqk, k, v, dtype="bf16", per_token=False, fresh=0, name=None):
    """The recurrent form over a state cache; `fresh`: every so many sequences one starts from a zero state;
    `per_token`: the state is kept after every token."""
    c = dict(op="recurrent", nseq=nseq, lo=lo, hi=hi, h=h, hqk=hqk, k=k, v=v, dtype=dtype,
             per_token=per_token, fresh=fresh)
    return dict(c, name=name) if name else c


def heads(op, b, t, hq, hk, k, r, dtype="bf16", interleaved=False, fused=False, far=0, name=None):
    """b sequences of t tokens of hq query and hk key heads of k channels, of which r are rotated; `fused`: queries and
    keys lie in the rows of one projection; positions start at up to `far`."""
    c = dict(op=op, b=b, t=t, hq=hq, hk=hk, k=k, r=r, dtype=dtype, interleaved=interleaved, fused=fused, far=far)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the chunked rule's headline batch, with its heads: training, or the long prompts of two requests
        linear("fwd", 2, 32768, 32768, 32, 32, 128, 128, name="fwd_long"),
        # packed prompts of different lengths, 5 of them, 7760 tokens, two value heads a key head
        linear("fwd", 5, 700, 2220, 16, 8, 128, 128, start=False, name="fwd_packed"),
        # one prompt of odd length: few heads' chains to spread over the machine
        linear("fwd", 1, 8001, 8001, 16, 16, 128, 128, name="fwd_one"),
        # short fp32 prompts of a small model
        linear("fwd", 5, 130, 130, 2, 2, 64, 64, dtype="f32", name="fwd_small_f32"),
        # the gradients of a training batch
        linear("bwd", 2, 8192, 8192, 32, 32, 128, 128, name="bwd_train"),
        # gradients of packed sequences with shared key heads, narrow keys
        linear("bwd", 7, 1, 1500, 16, 4, 64, 128, start=False, name="bwd_packed_grouped"),
        # one sequence, one new token: the latency of a decode step
        recurrent(1, 1, 1, 32, 16, 128, 128, name="decode_1seq"),
        # a full decode batch: one new token for each of 256 sequences
        recurrent(256, 1, 1, 32, 16, 128, 128, name="decode_256seq"),
        # draft tokens under verification: 1 to 8 a sequence, the state kept after each
        recurrent(48, 1, 8, 32, 16, 128, 128, per_token=True, name="draft_48seq"),
        # the queries and keys of 32768 tokens, in the rows of one projection
        heads("norm_fwd", 4, 8192, 32, 8, 128, 128, fused=True, far=131072, name="heads_fwd"),
        # those of a decode step's 13 sequences at far positions, fp32
        heads("norm_fwd", 13, 1, 16, 16, 96, 96, dtype="f32", interleaved=True, far=1 << 20, name="heads_decode_f32"),
        # the gradients for 8192 tokens, a part of each head rotated
        heads("norm_bwd", 2, 4096, 32, 32, 128, 64, name="heads_bwd"),
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def one_case(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "recurrent", "recurrent", "norm_fwd", "norm_bwd"))
    if op.startswith("norm"):
        k = rng.choice((64, 128, 2 * spread(rng, 8, 128), 8 * spread(rng, 2, 32)))
        r = rng.choice((k, k, k // 4 * 2, 0))
        return heads(op, spread(rng, 1, 16), spread(rng, 1, 16384), spread(rng, 1, 64), spread(rng, 1, 32), k, r,
                     dtype=rng.choice(("bf16", "bf16", "f32")), interleaved=rng.random() < 0.5,
                     fused=rng.random() < 0.5, far=spread(rng, 1, 1 << 22))
    hqk = spread(rng, 1, 16)
    h = hqk * rng.choice((1, 1, 2, 4))
    k, v = rng.choice((64, 128, 128)), rng.choice((64, 128, 128))
    if op == "recurrent":
        hi = spread(rng, 1, 100)
        return recurrent(spread(rng, 1, 300), rng.choice((0, 1, hi)), hi, h, hqk, k, v,
                         dtype=rng.choice(("bf16", "bf16", "f32")), per_token=rng.random() < 0.3,
                         fresh=rng.choice((0, 1, 3)))
    hi = spread(rng, 1, 32768)
    return linear(op, spread(rng, 1, 40), rng.choice((0, hi // 3, hi)), hi, h, hqk, k, v,
                  dtype=rng.choice(("bf16", "bf16", "bf16", "f32")), start=rng.random() < 0.5)


def draw(rng):
    while True:
        c = one_case(rng)
        if not c["op"].startswith("norm") and not sum(lens(c)):
            continue
        w = work(c)
        if c["op"] in ("fwd", "bwd"):
            # (the padded rows of the plain form; fp32 for small models)
            rows = c["nseq"] * c["hi"] * c["h"]
            if rows > (2 ** 21 if c["op"] == "fwd" else 2 ** 19) or (c["dtype"] == "f32" and rows > 2 ** 16):
                continue
        if c["op"] == "recurrent" and c["nseq"] * c["hi"] * c["h"] * c["k"] * c["v"] * (8 if c["per_token"] else 1) > 2 ** 31:
            continue
        if w["bytes"] <= (2.2e9 if c["op"] in ("fwd", "recurrent") else 1.1e9):
            return c


def lens(c):
    """The sequences' lengths, a plain spread over lo..hi in no order."""
    n = c["hi"] - c["lo"] + 1
    return [c["lo"] + (i * (n * 19 // 31 + 1) + n // 3) % n for i in range(c["nseq"])]


def packed(c):
    return c["lo"] != c["hi"]


def is_fresh(c, i):
    return c["fresh"] > 0 and i % c["fresh"] == 0


def page(c):
    return 4 * c["h"] * c["k"] * c["v"]


def work(c):
    es = BYTES[c["dtype"]]
    if c["op"].startswith("norm"):
        e = c["b"] * c["t"] * (c["hq"] + c["hk"]) * c["k"]
        if c["op"] == "norm_fwd":
            return {"bytes": 2 * e * es + 8 * c["k"], "flops": 8 * e}
        return {"bytes": 3 * e * es + 16 * c["k"], "flops": 16 * e}
    t, qk, v = sum(lens(c)), c["hqk"] * c["k"], c["h"] * c["v"]
    kv = c["h"] * c["k"] * c["v"]
    if c["op"] == "recurrent":
        reads = sum(not is_fresh(c, i) for i in range(c["nseq"]))
        writes = t if c["per_token"] else c["nseq"]
        return {"bytes": (reads + writes) * page(c) + t * es * 2 * (qk + v), "flops": 5 * t * kv}
    states = c["nseq"] * page(c)
    if c["op"] == "fwd":
        return {"bytes": t * es * 2 * (qk + v) + (2 if c["start"] else 1) * states, "flops": 4 * t * kv}
    return {"bytes": t * es * (4 * qk + 3 * v) + 3 * states, "flops": 10 * t * kv}


# --------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype="f32", mean=0.0, sd=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(sd).add_(mean).to(DTYPES[dtype])

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    c, d = case, case["dtype"]
    s = {"case": c}
    if c["op"].startswith("norm"):
        b, t, hq, hk, k = (c[n] for n in ("b", "t", "hq", "hk", "k"))
        if c["fused"]:
            # the rows of a projection of queries, keys and values
            rows = normal(b, t, (hq + 2 * hk) * k, dtype=d)
            s["q"] = rows[..., :hq * k].unflatten(-1, (hq, k))
            s["k"] = rows[..., hq * k:(hq + hk) * k].unflatten(-1, (hk, k))
        else:
            s["q"], s["k"] = normal(b, t, hq, k, dtype=d), normal(b, t, hk, k, dtype=d)
        s["wq"], s["wk"] = normal(k, mean=1.0, sd=0.2), normal(k, mean=1.0, sd=0.2)
        s["freq"] = (10000.0 ** (-torch.arange(c["r"] // 2, dtype=torch.float64) * 2 / max(1, c["r"]))).float().cuda()
        first = torch.randint(0, c["far"] + 1, (b, 1), generator=gen, device="cuda")
        s["pos"] = (first + torch.arange(t, device="cuda")).to(torch.int32)
        if c["op"] == "norm_bwd":
            s["dyq"], s["dyk"] = normal(b, t, hq, k, dtype=d), normal(b, t, hk, k, dtype=d)
        if own:
            # the buffers and the workspace that a training or serving program keeps
            from context_scan_gb300 import gdn
            if c["op"] == "norm_fwd":
                s["yq"], s["yk"] = torch.empty_like(s["q"], memory_format=torch.contiguous_format), torch.empty_like(
                    s["k"], memory_format=torch.contiguous_format)
            else:
                s["dq"], s["dk"] = torch.empty_like(s["dyq"]), torch.empty_like(s["dyk"])
                if c["fused"]:   # gradients in the rows of the projection's
                    grad = torch.empty(b, t, (hq + 2 * hk) * k, dtype=DTYPES[d], device="cuda")
                    s["dq"] = grad[..., :hq * k].unflatten(-1, (hq, k))
                    s["dk"] = grad[..., hq * k:(hq + hk) * k].unflatten(-1, (hk, k))
                s["dwq"], s["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
                s["ws"] = gdn.alloc_qk_norm_bwd_workspace(s["q"], s["k"])
        return s
    L = lens(c)
    t = sum(L)
    lead = (1, t) if packed(c) else (c["nseq"], c["hi"])
    unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1).to(x.dtype)  # noqa: E731
    s["q"] = unit(normal(*lead, c["hqk"], c["k"], dtype=d))
    s["k"] = unit(normal(*lead, c["hqk"], c["k"], dtype=d))
    s["v"] = normal(*lead, c["h"], c["v"], dtype=d)
    # slopes from about one e-fold in one token to one in some hundreds, a little off for each layer
    slope = -(2.0 ** (-8.0 * (torch.arange(c["h"], device="cuda") + 1) / c["h"]))
    s["decay"] = slope * torch.empty(c["h"], device="cuda").uniform_(0.8, 1.2, generator=gen)
    s["cu"] = ints([sum(L[:i]) for i in range(len(L) + 1)]) if packed(c) else None
    # where each token of each sequence lies (-1: none), for the plain form
    at = torch.full((c["nseq"], max(L + [1])), -1, dtype=torch.int64)
    n = 0
    for i, m in enumerate(L):
        at[i, :m] = torch.arange(n, n + m)
        n += m
    s["at"], s["len"] = at.cuda(), torch.tensor(L, device="cuda")
    if c["op"] == "recurrent":
        # a cache of state pages whose numbers are in no order; a state is read from one page and written
        # to another, as for a sequence that starts from a shared prefix (and so that a pass can be repeated)
        outs = t if c["per_token"] else c["nseq"]
        slots = c["nseq"] + outs + 1
        order = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
        s["state"] = normal(slots, c["h"], c["k"], c["v"], sd=0.3)
        stay = ints([0 if is_fresh(c, i) else 1 for i in range(c["nseq"])])
        s["slots_in"] = torch.where(stay > 0, order[:c["nseq"]], -1).to(torch.int32)
        s["slots_out"] = order[c["nseq"]:c["nseq"] + outs].contiguous()
    else:
        s["h0"] = normal(c["nseq"], c["h"], c["k"], c["v"], sd=0.3) if c["start"] else None
        if c["op"] == "bwd":
            s["do"] = normal(*lead, c["h"], c["v"], dtype=d)
            s["dht"] = normal(c["nseq"], c["h"], c["k"], c["v"], sd=0.3)
    if own:
        from context_scan_gb300 import gdn
        s["o"] = torch.empty_like(s["v"])
        if c["op"] == "recurrent":
            s["ws"] = gdn.alloc_recurrent_workspace(s["state"].shape[0])
        else:
            s["ht"] = torch.empty(c["nseq"], c["h"], c["k"], c["v"], device="cuda")
            s["ws"] = gdn.alloc_linear_workspace(s["k"], s["v"], cu_seqlens=s["cu"], backward=c["op"] == "bwd")
            if c["op"] == "bwd":
                s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[n]) for n in ("q", "k", "v"))
    return s


# ----------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return run_own(s)
    return {"fwd": plain_fwd, "bwd": plain_bwd, "recurrent": plain_recurrent, "norm_fwd": plain_norm_fwd,
            "norm_bwd": plain_norm_bwd}[s["case"]["op"]](s)


def run_own(s):
    from context_scan_gb300 import gdn
    c = s["case"]
    if c["op"] == "fwd":
        gdn.gdn_linear_fwd(s["q"], s["k"], s["v"], s["decay"], s["h0"], s["o"], s["ht"], s["ws"], cu_seqlens=s["cu"])
        return {"o": s["o"], "h_final": s["ht"]}
    if c["op"] == "bwd":
        gdn.gdn_linear_bwd(s["q"], s["k"], s["v"], s["decay"], s["h0"], s["do"], s["dht"], s["dq"], s["dk"], s["dv"],
                           s["ht"], s["ws"], cu_seqlens=s["cu"])
        return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"], "dh0": s["ht"]}
    if c["op"] == "recurrent":
        gdn.gdn_linear_recurrent_fwd(s["q"], s["k"], s["v"], s["decay"], s["state"], s["slots_in"], s["slots_out"],
                                     s["o"], s["ws"], cu_seqlens=s["cu"], per_token=c["per_token"])
        return {"o": s["o"], "state": s["state"]}
    freq = s["freq"] if c["r"] else None
    if c["op"] == "norm_fwd":
        gdn.gdn_qk_norm_fwd(s["q"], s["k"], s["wq"], s["wk"], freq, s["yq"], s["yk"], positions=s["pos"], eps=EPS,
                            interleaved=c["interleaved"])
        return {"yq": s["yq"], "yk": s["yk"]}
    gdn.gdn_qk_norm_bwd(s["q"], s["k"], s["wq"], s["wk"], freq, s["dyq"], s["dyk"], s["dq"], s["dk"], s["dwq"],
                        s["dwk"], s["ws"], positions=s["pos"], eps=EPS, interleaved=c["interleaved"])
    return {n: s[n] for n in ("dq", "dk", "dwq", "dwk")}


def rows(s, name, rep=1, flip=False):
    """Tokens as [sequence, place, head, channel] in 32 bits, zeros behind the sequences' ends; `flip`: the last
    token first; `rep`: heads repeated."""
    x = s[name]
    x = x.reshape(-1, *x.shape[2:])
    at = s["at"]
    if flip:
        last = (s["len"][:, None] - 1 - torch.arange(at.shape[1], device="cuda"))
        at = torch.where(last >= 0, at.gather(1, last.clamp(min=0)), -1)
    y = x[at.clamp(min=0)].float() * (at >= 0)[..., None, None]
    return y if rep == 1 else y.repeat_interleave(rep, 2)


def unrows(s, y, dtype, flip=False):
    """The tokens of rows() back in their places."""
    at = s["at"]
    if flip:
        last = (s["len"][:, None] - 1 - torch.arange(at.shape[1], device="cuda"))
        at = torch.where(last >= 0, at.gather(1, last.clamp(min=0)), -1)
    out = torch.empty(int(s["v"].shape[0] * s["v"].shape[1]), *y.shape[2:], device="cuda")
    out[at[at >= 0]] = y[at >= 0]
    return out.view(*s["v"].shape[:2], *y.shape[2:]).to(dtype)


def power(decay, n):
    """e^(decay n) over the heads (last), 0 where n is negative; in 64 bits before it is rounded."""
    x = torch.exp(decay.double() * n.clamp(min=0)[..., None].double())
    return (x * (n >= 0)[..., None]).float()


def attend(a, b, c, decay, start, length, shift):
    """out_i = sum over j <= i of w^(i - j) (a_i . b_j) c_j + w^(i + 1 - shift) a_i start, w = e^decay, in chunks, and
    w^length start + sum of w^(length - 1 - j + shift) b_j c_j^T. a, b, c [N, L, H, *], start [N, H, *, *] or None."""
    N, L, H, _ = a.shape
    C = min(CHUNK, L)
    pad = -L % C
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(N, -1, C, H, x.shape[-1]) for x in (a, b, c))
    n, i = torch.arange(a.shape[1], device="cuda"), torch.arange(C, device="cuda")
    P = torch.einsum("nmihk,nmjhk->nmhij", a, b) * power(decay, i[:, None] - i).permute(2, 0, 1)
    out = torch.einsum("nmhij,nmjhv->nmihv", P, c)
    del P
    # the state before each chunk, and with it the rest
    own_ = torch.einsum("nmjhk,nmjhv->nmhkv", b * power(decay, C - 1 - i + shift)[:, :, None], c)
    before = torch.einsum("xmh,nmhkv->nxhkv", power(decay, C * (n[:, None] - 1 - n)), own_)
    if start is not None:
        before = before + power(decay, C * n)[:, :, None, None] * start[:, None]
    out = out + torch.einsum("nmihk,nmhkv->nmihv", a * power(decay, i + 1 - shift)[:, :, None], before)
    del before, own_
    j = torch.arange(L, device="cuda")
    weight = power(decay, torch.where(j < length[:, None], length[:, None] - 1 - j + shift, -1))
    last = torch.einsum("nlhk,nlhv->nhkv", b.flatten(1, 2)[:, :L] * weight[..., None], c.flatten(1, 2)[:, :L])
    if start is not None:
        last = last + power(decay, length)[..., None, None] * start
    return out.flatten(1, 2)[:, :L], last


def plain_fwd(s):
    rep = s["case"]["h"] // s["case"]["hqk"]
    o, last = attend(rows(s, "q", rep), rows(s, "k", rep), rows(s, "v"), s["decay"], s["h0"], s["len"], 0)
    return {"o": unrows(s, o, s["v"].dtype), "h_final": last}


def plain_bwd(s):
    """With o = A(q, k, v): dq = A(dO, v, k) from the transposed state, and from the end on, with the gradient of the
    last state for a start, dk = A(v, dO, q) and dv = A(k, q, dO)."""
    c = s["case"]
    rep = c["h"] // c["hqk"]
    group = lambda x: x.unflatten(2, (c["hqk"], rep)).sum(3)  # noqa: E731
    h0 = None if s["h0"] is None else s["h0"].transpose(-1, -2)
    dq, _ = attend(rows(s, "do"), rows(s, "v"), rows(s, "k", rep), s["decay"], h0, s["len"], 0)
    dq = unrows(s, group(dq), s["q"].dtype)
    q, k, v, do = (rows(s, n, m, True) for n, m in (("q", rep), ("k", rep), ("v", 1), ("do", 1)))
    dk, _ = attend(v, do, q, s["decay"], s["dht"].transpose(-1, -2), s["len"], 1)
    dk = unrows(s, group(dk), s["k"].dtype, True)
    dv, dh0 = attend(k, q, do, s["decay"], s["dht"], s["len"], 1)
    return {"dq": dq, "dk": dk, "dv": unrows(s, dv, s["v"].dtype, True), "dh0": dh0}


def plain_recurrent(s):
    c = s["case"]
    rep = c["h"] // c["hqk"]
    slots_in, slots_out = s["slots_in"].long(), s["slots_out"].long()
    start = s["state"][slots_in.clamp(min=0)] * (slots_in >= 0).view(-1, 1, 1, 1)
    k, v = rows(s, "k", rep), rows(s, "v")
    o, last = attend(rows(s, "q", rep), k, v, s["decay"], start, s["len"], 0)
    if not c["per_token"]:
        s["state"][slots_out] = last
    else:
        i = torch.arange(k.shape[1], device="cuda")
        kept = torch.einsum("tjh,njhk,njhv->nthkv", power(s["decay"], i[:, None] - i), k, v)
        kept = kept + power(s["decay"], i + 1)[:, :, None, None] * start[:, None]
        s["state"][slots_out[s["at"][s["at"] >= 0]]] = kept[s["at"] >= 0]
    return {"o": unrows(s, o, s["v"].dtype), "state": s["state"]}


def angles(s):
    """cos and sin [B, T, 1, R / 2], of angles in 64 bits."""
    a = s["pos"].double()[..., None, None] * s["freq"].double()
    return a.cos().float(), a.sin().float()


def halves(c, x):
    """The first and the second member of every rotated pair, and the channels that are not rotated."""
    r = c["r"]
    if c["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def rotate(c, x, cos, sin):
    a, b, rest = halves(c, x)
    y = [a * cos - b * sin, b * cos + a * sin]
    y = torch.stack(y, -1).flatten(-2) if c["interleaved"] else torch.cat(y, -1)
    return torch.cat([y, rest], -1)


def plain_norm_fwd(s):
    c = s["case"]
    cos, sin = angles(s)

    def one(x, w):
        u = x.float()
        u = u * (u.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
        return rotate(c, u, cos, sin).to(x.dtype)

    return {"yq": one(s["q"], s["wq"]), "yk": one(s["k"], s["wk"])}


def plain_norm_bwd(s):
    c = s["case"]
    cos, sin = angles(s)

    def one(x, w, dy):
        u = x.float()
        rstd = (u.square().mean(-1, keepdim=True) + EPS).rsqrt()
        u = u * rstd
        e = rotate(c, dy.float(), cos, -sin)
        dw = (e * u).flatten(0, 2).sum(0, dtype=torch.float64).float()   # (a long sum: in 64 bits)
        d = e * w
        return ((d - u * (d * u).mean(-1, keepdim=True)) * rstd).to(x.dtype), dw

    dq, dwq = one(s["q"], s["wq"], s["dyq"])
    dk, dwk = one(s["k"], s["wk"], s["dyk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# -------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"].startswith("norm"):
        return exact_norm(c, s)
    if c["nseq"] * c["h"] * c["k"] * c["v"] * c["hi"] > 1.5e11:
        return None
    return exact_recurrent(c, s) if c["op"] == "recurrent" else exact_linear(c, s)


def exact_norm(c, s):
    got = {}
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[..., None, None] * s["freq"].double())
    half = c["r"] // 2
    if c["interleaved"]:
        first = torch.arange(half, device="cuda") * 2
        second = first + 1
    else:
        first = torch.arange(half, device="cuda")
        second = first + half
    for n in ("q", "k"):
        x = s[n].double().requires_grad_()
        w = s["w" + n].double().requires_grad_()
        u = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["k"] + EPS) * w
        z = torch.complex(u[..., first], u[..., second]) * turn
        y = u.index_copy(-1, first, z.real).index_copy(-1, second, z.imag)
        if c["op"] == "norm_fwd":
            got["y" + n] = y.detach()
        else:
            got["d" + n], got["dw" + n] = torch.autograd.grad(y, (x, w), s["dy" + n].double())
    return got


def exact_recurrent(c, s):
    group = torch.arange(c["h"], device="cuda") // (c["h"] // c["hqk"])
    flat = {n: s[n].reshape(-1, *s[n].shape[2:]) for n in ("q", "k", "v")}
    state = s["state"].double()
    w = torch.exp(s["decay"].double())[:, None, None]
    o = torch.zeros(flat["v"].shape, dtype=torch.float64, device="cuda")
    ins, outs = s["slots_in"].tolist(), s["slots_out"].tolist()
    t = 0
    for i, m in enumerate(lens(c)):
        H = state[ins[i]].clone() if ins[i] >= 0 else torch.zeros_like(state[0])   # [h, k, v]
        for _ in range(m):
            q, k = flat["q"][t][group].double(), flat["k"][t][group].double()
            H = w * H + k[:, :, None] * flat["v"][t].double()[:, None, :]
            o[t] = (q[:, :, None] * H).sum(1)
            if c["per_token"]:
                state[outs[t]] = H
            t += 1
        if not c["per_token"]:
            state[outs[i]] = H
    return {"o": o.view(s["v"].shape), "state": state}


def exact_linear(c, s):
    """Token by token, all sequences at once."""
    group = torch.arange(c["h"], device="cuda") // (c["h"] // c["hqk"])
    flat = {n: s[n].reshape(-1, *s[n].shape[2:]) for n in ("q", "k", "v", "do") if n in s}
    w = torch.exp(s["decay"].double())[:, None, None]
    L = lens(c)
    H = torch.zeros(c["nseq"], c["h"], c["k"], c["v"], dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        H += s["h0"].double()
    starts = [sum(L[:i]) for i in range(len(L))]
    tokens = sum(L)
    out = torch.zeros(tokens, c["h"], c["v"] if c["op"] == "fwd" else c["k"], dtype=torch.float64, device="cuda")
    order = sorted(range(c["nseq"]), key=lambda i: -L[i])     # the sequences still running come first
    H = H[order]
    first = torch.tensor([starts[i] for i in order], device="cuda")
    counts = [sum(m > t for m in L) for t in range(max(L + [0]))]

    def at(name, where):
        x = flat[name][where].double()
        return x if name in ("v", "do") else x[:, group]

    for t, n in enumerate(counts):
        here = first[:n] + t
        H[:n].mul_(w).addcmul_(at("k", here)[..., None], at("v", here)[..., None, :])
        if c["op"] == "fwd":
            out[here] = torch.matmul(at("q", here)[..., None, :], H[:n])[..., 0, :]
        else:
            out[here] = torch.matmul(H[:n], at("do", here)[..., None])[..., 0]
    lead = s["v"].shape[:2]
    back = torch.tensor(order, device="cuda").argsort()
    if c["op"] == "fwd":
        return {"o": out.view(*lead, *out.shape[1:]), "h_final": H[back]}
    share = lambda x: x.view(*lead, c["hqk"], -1, x.shape[-1]).sum(3)  # noqa: E731
    dk, dv = torch.zeros_like(out), torch.zeros(tokens, c["h"], c["v"], dtype=torch.float64, device="cuda")
    D = s["dht"].double()[order]
    for t in range(len(counts) - 1, -1, -1):
        n = counts[t]
        here = first[:n] + t
        D[:n].addcmul_(at("q", here)[..., None], at("do", here)[..., None, :])   # the gradient of the state after t
        dk[here] = torch.matmul(D[:n], at("v", here)[..., None])[..., 0]
        dv[here] = torch.matmul(at("k", here)[..., None, :], D[:n])[..., 0, :]
        D[:n].mul_(w)
    return {"dq": share(out), "dk": share(dk), "dv": dv.view(*lead, *dv.shape[1:]), "dh0": D[back]}
