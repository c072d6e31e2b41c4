"""Cases and plain forms of the serving and training operators around the chunked gated delta rule:
the recurrent form over a state cache, the cache's page operations, and the (gated) normalisation
of the rule's outputs with its gradients.

``run`` computes a case with elementary torch operations in 32 bits, or, where ``own`` is true, with
the library's kernels through ``context_scan_gb300.gdn``; ``exact`` gives the same in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-6


# ---------------------------------------------------------------------------------------- cases

def recurrent(nseq, lo, hi, h, hqk, k, v, dtype="bf16", out="bf16", gate_k=False, decay_first=False,
              per_token=False, fresh=0, name=None):
    """nseq sequences of lo..hi tokens (lo == hi: all alike, no cu_seqlens); `fresh`: every so many
    sequences one starts from a zero state; `per_token`: the state is kept after every token."""
    c = dict(op="recurrent", nseq=nseq, lo=lo, hi=hi, h=h, hqk=hqk, k=k, v=v, dtype=dtype, out=out,
             gate_k=gate_k, decay_first=decay_first, per_token=per_token, fresh=fresh)
    return dict(c, name=name) if name else c


def norm(op, rows, n, x, y, rms, gated, name=None):
    """rows of n values; x (and dx) of type x, the gate z, y and their gradients of type y. The
    layer norm has a weight and a bias, the root-mean-square norm a weight."""
    c = dict(op=op, rows=rows, n=n, x=x, y=y, rms=rms, gated=gated)
    return dict(c, name=name) if name else c


def cache(op, layers, pages, h, k, v, n, name=None):
    """A state cache of `layers` arrays of `pages` pages [h, k, v]; n pages copied or forked (every
    seventh made anew, of zeros), or (compaction) n pages in use, scattered over the cache."""
    c = dict(op=op, layers=layers, pages=pages, h=h, k=k, v=v, n=n)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence, one new token: the latency of a decode step
        recurrent(1, 1, 1, 32, 16, 128, 128, name="decode_1seq"),
        # a full decode batch: one new token for each of 256 sequences
        recurrent(256, 1, 1, 32, 16, 128, 128, name="decode_256seq"),
        # draft tokens under verification: 1 to 8 a sequence, the state kept after each so that
        # the rejected ones can be dropped
        recurrent(48, 1, 8, 32, 16, 128, 128, out="f32", per_token=True, name="draft_48seq"),
        # the ends of prompts, 0 to 63 tokens behind the last whole chunk, gates per key channel
        recurrent(37, 0, 63, 16, 16, 128, 128, out="f32", gate_k=True, decay_first=True, fresh=5,
                  name="tails_kda_37seq"),
        # short fp32 prompts of a small model, run from zero states
        recurrent(5, 130, 130, 2, 2, 64, 64, dtype="f32", out="f32", fresh=1, name="small_f32_5seq"),
        # the outputs of 32768 tokens, 32 heads, normalised head by head and gated
        norm("norm_fwd", 32768 * 32, 128, "f32", "bf16", True, True, name="head_norm_fwd"),
        # layer norm over a hidden size that is no multiple of a vector
        norm("norm_fwd", 7300, 1999, "bf16", "bf16", False, False, name="layer_norm_fwd_odd"),
        # the gradients of the first of these, for 8192 tokens of 32 heads
        norm("norm_bwd", 8192 * 32, 128, "f32", "bf16", True, True, name="head_norm_bwd"),
        # layer norm over a hidden size of 2048, in training
        norm("norm_bwd", 8192, 2048, "bf16", "bf16", False, False, name="layer_norm_bwd"),
        # a batch's states saved before a risky step, some pages cleared for new sequences
        cache("cache_copy", 12, 128, 32, 128, 128, 48, name="copy_48pages"),
        # four beams of one sequence forked from their parents and dropped again
        cache("cache_fork", 12, 64, 32, 128, 128, 4, name="fork_4pages"),
        # a cache two thirds full after its sequences ended in no order
        cache("cache_compact", 12, 192, 32, 128, 128, 128, name="compact_192pages"),
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def one_case(rng):
    op = rng.choice(("recurrent", "recurrent", "norm_fwd", "norm_bwd", "cache_copy", "cache_fork",
                     "cache_compact"))
    if op == "recurrent":
        hi = spread(rng, 1, 200)
        lo = rng.choice((0, 1, hi))
        hqk, kv = spread(rng, 1, 16), rng.choice((64, 128))
        h = hqk * rng.choice((1, 1, 2, 4))
        return recurrent(spread(rng, 1, 300), lo, hi, h, hqk, kv, kv, dtype=rng.choice(("bf16", "bf16", "f32")),
                         out=rng.choice(("f32", "bf16")), gate_k=rng.random() < 0.3,
                         decay_first=rng.random() < 0.5, per_token=rng.random() < 0.3,
                         fresh=rng.choice((0, 1, 3)))
    if op.startswith("norm"):
        n = rng.choice((64, 128, spread(rng, 16, 8192), 8 * spread(rng, 2, 1024)))
        return norm(op, spread(rng, 1, 1 << 20), n, rng.choice(("f32", "bf16")),
                    rng.choice(("f32", "bf16")), rng.random() < 0.5, rng.random() < 0.5)
    pages, kv = spread(rng, 2, 2000), rng.choice((64, 128))
    return cache(op, spread(rng, 1, 24), pages, spread(rng, 1, 32), kv, kv, rng.randint(1, max(1, pages // 2)))


def draw(rng):
    while True:
        c = one_case(rng)
        w = work(c)
        most = 4.6e8 if c["op"] == "norm_bwd" else 1.07e9   # the largest listed ones'
        if c["op"] == "recurrent" and c["nseq"] * c["hi"] > 4096:
            continue
        if c["op"].startswith("cache"):
            most = 2.1e9
            if c["layers"] * c["pages"] * page_bytes(c) > 4.9e9:
                continue
        if w["bytes"] <= most and w["flops"] <= 3e10:
            return c


def lens(c):
    """The sequences' lengths, a plain spread over lo..hi in no order."""
    return [c["lo"] + (i * 29 + 7) % (c["hi"] - c["lo"] + 1) for i in range(c["nseq"])]


def is_fresh(c, i):
    return c["fresh"] > 0 and i % c["fresh"] == 0


def page_bytes(c):
    return 4 * c["h"] * c["k"] * c["v"]


def moved(c):
    """How many of n pages in use, at the places that `in_use` gives, lie behind the first n."""
    return sum(p >= c["n"] for p in in_use(c))


def in_use(c):
    """The pages in use: n of them, spread over the cache in no order."""
    step = next(s for s in range(int(c["pages"] * 0.618) + 1, 2 * c["pages"] + 2) if math.gcd(s, c["pages"]) == 1)
    return [(i * step + 1) % c["pages"] for i in range(c["n"])]


def work(c):
    if c["op"] == "recurrent":
        L = lens(c)
        t, es = sum(L), BYTES[c["dtype"]]
        page = page_bytes(c)
        reads = sum(not is_fresh(c, i) for i in range(c["nseq"]))
        writes = t if c["per_token"] else c["nseq"]
        token = es * (2 * c["hqk"] * c["k"] + c["h"] * (c["v"] + 1 + (c["k"] if c["gate_k"] else 1)))
        token += BYTES[c["out"]] * c["h"] * c["v"]
        return {"bytes": (reads + writes) * page + t * token, "flops": 7 * t * c["h"] * c["k"] * c["v"]}
    if c["op"].startswith("norm"):
        e, x, y = c["rows"] * c["n"], BYTES[c["x"]], BYTES[c["y"]]
        params = 4 * c["n"] * (1 if c["rms"] else 2)
        if c["op"] == "norm_fwd":
            return {"bytes": e * (x + y + (y if c["gated"] else 0)) + params, "flops": 8 * e}
        return {"bytes": e * (2 * x + y + (2 * y if c["gated"] else 0)) + 2 * params, "flops": 16 * e}
    n = moved(c) if c["op"] == "cache_compact" else c["n"]
    return {"bytes": 2 * n * c["layers"] * page_bytes(c) + 4 * c["pages"], "flops": 0}


# --------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype="f32", mean=0.0, sd=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(sd).add_(mean).to(DTYPES[dtype])

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    c = case
    s = {"case": c}
    if c["op"] == "recurrent":
        # the layouts of a user's program: tokens of all sequences in a row, a cache of state pages
        # whose numbers are in no order; a state is read from one page and written to another, as
        # for a sequence that starts from a shared prefix (and so that a pass can be repeated)
        L = lens(c)
        t, d = sum(L), c["dtype"]
        lead = (c["nseq"], c["hi"]) if c["lo"] == c["hi"] else (1, t)
        unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1).to(x.dtype)  # noqa: E731
        s["q"] = unit(normal(*lead, c["hqk"], c["k"], dtype=d))
        s["k"] = unit(normal(*lead, c["hqk"], c["k"], dtype=d))
        s["v"] = normal(*lead, c["h"], c["v"], dtype=d)
        g = normal(*lead, c["h"], *((c["k"],) if c["gate_k"] else ()), mean=2.0)
        s["g"] = torch.nn.functional.logsigmoid(g).to(DTYPES[d])
        s["beta"] = torch.sigmoid(normal(*lead, c["h"])).to(DTYPES[d])
        s["cu"] = None
        if c["lo"] != c["hi"]:
            s["cu"] = ints([sum(L[:i]) for i in range(len(L) + 1)])
        outs = t if c["per_token"] else c["nseq"]
        slots = c["nseq"] + outs + 1
        order = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
        s["state"] = normal(slots, c["h"], c["k"], c["v"], sd=0.3)
        stay = ints([0 if is_fresh(c, i) else 1 for i in range(c["nseq"])])
        s["slots_in"] = torch.where(stay > 0, order[:c["nseq"]], -1).to(torch.int32)
        s["slots_out"] = order[c["nseq"]:c["nseq"] + outs].contiguous()
        s["o"] = torch.empty(*lead, c["h"], c["v"], dtype=DTYPES[c["out"]], device="cuda")
        # where each token of each sequence lies (-1: none), for the plain form
        at = torch.full((c["nseq"], max(L + [0])), -1, dtype=torch.int64)
        n = 0
        for i, m in enumerate(L):
            at[i, :m] = torch.arange(n, n + m)
            n += m
        s["at"] = at.cuda()
    elif c["op"].startswith("norm"):
        rows, n = c["rows"], c["n"]
        s["x"] = normal(rows, n, dtype=c["x"], mean=0.2)
        s["w"] = normal(n, mean=1.0, sd=0.2)
        s["b"] = None if c["rms"] else normal(n, sd=0.2)
        s["z"] = normal(rows, n, dtype=c["y"]) if c["gated"] else None
        if c["op"] == "norm_fwd":
            s["y"] = torch.empty(rows, n, dtype=DTYPES[c["y"]], device="cuda")
        else:
            s["dy"] = normal(rows, n, dtype=c["y"])
            s["dx"] = torch.empty_like(s["x"])
            s["dz"] = None if s["z"] is None else torch.empty_like(s["z"])
            s["dw"] = torch.empty_like(s["w"])
            s["db"] = None if s["b"] is None else torch.empty_like(s["b"])
    else:
        s["pages"] = normal(c["layers"], c["pages"], c["h"], c["k"], c["v"])
        used = in_use(c) if c["op"] == "cache_compact" else in_use(dict(c, n=c["pages"] // 2))
        refs = torch.zeros(c["pages"], dtype=torch.int32)
        refs[used] = 1
        s["refs"] = refs.cuda()
        order = torch.randperm(len(used), generator=gen, device="cuda")
        s["used"] = ints(used)[order].contiguous()
        if c["op"] == "cache_copy":
            s["src"] = torch.where(torch.arange(c["n"], device="cuda") % 7 == 6, -1, s["used"][:c["n"]])
            s["src"] = s["src"].to(torch.int32)
            s["dst"] = ints([p for p in range(c["pages"]) if refs[p] == 0][:c["n"]])
        elif c["op"] == "cache_fork":
            parents = s["used"].repeat(c["n"] // max(1, len(used)) + 1)[:c["n"]]
            s["parents"] = torch.where(torch.arange(c["n"], device="cuda") % 7 == 6, -1, parents)
            s["parents"] = s["parents"].to(torch.int32)
            s["children"] = torch.empty(c["n"], dtype=torch.int32, device="cuda")
        else:
            s["refs0"], s["table0"] = s["refs"].clone(), s["used"]
            s["table"] = s["used"].clone()
            s["remap"] = torch.empty(c["pages"], dtype=torch.int32, device="cuda")
            s["live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    if own:
        # the workspace that a user's program allocates once for its shapes
        from context_scan_gb300 import gdn
        if c["op"] == "recurrent":
            s["ws"] = gdn.alloc_recurrent_workspace(s["state"].shape[0])
        elif c["op"] == "norm_bwd":
            s["ws"] = gdn.alloc_norm_bwd_workspace(c["rows"], c["n"])
        elif c["op"].startswith("cache"):
            s["ws"] = gdn.alloc_cache_workspace(c["pages"], c["n"])
    return s


# ----------------------------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        return run_own(s)
    if c["op"] == "recurrent":
        return plain_recurrent(s)
    if c["op"] == "norm_fwd":
        return plain_norm_fwd(s)
    if c["op"] == "norm_bwd":
        return plain_norm_bwd(s)
    return plain_cache(s)


def run_own(s):
    from context_scan_gb300 import gdn
    c = s["case"]
    if c["op"] == "recurrent":
        gdn.gdn_recurrent_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["slots_in"],
                              s["slots_out"], s["o"], s["ws"], cu_seqlens=s["cu"],
                              per_token=c["per_token"], decay_first=c["decay_first"])
        return {"o": s["o"], "state": s["state"]}
    if c["op"] == "norm_fwd":
        gdn.gdn_norm_fwd(s["x"], s["w"], s["b"], s["z"], s["y"], eps=EPS, rms=c["rms"])
        return {"y": s["y"]}
    if c["op"] == "norm_bwd":
        gdn.gdn_norm_bwd(s["x"], s["w"], s["b"], s["z"], s["dy"], s["dx"], s["dz"], s["dw"], s["db"],
                         s["ws"], eps=EPS, rms=c["rms"])
        return {"dx": s["dx"], "dz": s["dz"], "dw": s["dw"], "db": s["db"]}
    if c["op"] == "cache_copy":
        gdn.gdn_cache_copy(s["pages"], s["src"], s["dst"], s["ws"])
        return {"pages": s["pages"]}
    if c["op"] == "cache_fork":
        gdn.gdn_cache_fork(s["pages"], s["refs"], s["parents"], s["children"], s["ws"])
        gdn.gdn_cache_free(s["refs"], s["children"], s["ws"])
        return {"pages": s["pages"], "children": s["children"], "refs": s["refs"]}
    s["refs"].copy_(s["refs0"])     # a pass can be repeated: the pages themselves stay where they were
    s["table"].copy_(s["table0"])
    gdn.gdn_cache_compact(s["pages"], s["refs"], s["table"], s["remap"], s["live"], s["ws"])
    return {k: s[k] for k in ("pages", "refs", "table", "remap", "live")}


def plain_recurrent(s):
    c = s["case"]
    rep = c["h"] // c["hqk"]
    flat = lambda x: x.reshape(-1, *x.shape[2:])  # noqa: E731
    q, k, v, g, beta = (flat(s[n]) for n in ("q", "k", "v", "g", "beta"))
    o = torch.zeros(v.shape, device="cuda")
    slots_in, slots_out = s["slots_in"].long(), s["slots_out"].long()
    h = s["state"][slots_in.clamp(min=0)] * (slots_in >= 0).view(-1, 1, 1, 1)
    kept = s["state"]
    for t in range(s["at"].shape[1]):
        at = s["at"][:, t]
        on = (at >= 0).nonzero().flatten() if s["cu"] is not None else slice(None)
        at = at[on]
        kt = k[at].float().repeat_interleave(rep, 1)
        qt = q[at].float().repeat_interleave(rep, 1)
        e = g[at].float().exp()
        e = e[..., None] if c["gate_k"] else e[..., None, None]
        prev = h[on]
        next_ = prev * e
        read = torch.einsum("nhk,nhkv->nhv", kt, next_ if c["decay_first"] else prev)
        r = beta[at].float()[..., None] * (v[at].float() - read)
        next_ = next_ + kt[..., None] * r[..., None, :]
        o[at] = torch.einsum("nhk,nhkv->nhv", qt, next_)
        h[on] = next_
        if c["per_token"]:
            kept[slots_out[at]] = next_
    if not c["per_token"]:
        kept[slots_out] = h
    return {"o": o.to(s["o"].dtype).view(s["o"].shape), "state": kept}


def plain_norm_fwd(s):
    c, x = s["case"], s["x"].float()
    if not c["rms"]:
        x = x - x.mean(-1, keepdim=True)
    y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z / (1 + (-z).exp())
    return {"y": y.to(DTYPES[c["y"]])}


def plain_norm_bwd(s):
    c, x, d = s["case"], s["x"].float(), s["dy"].float()
    if not c["rms"]:
        x = x - x.mean(-1, keepdim=True)
    rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    x = x * rstd
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1 / (1 + (-z).exp())
        y = x * s["w"] if s["b"] is None else x * s["w"] + s["b"]
        dz = (d * y * sig * (1 + z * (1 - sig))).to(s["z"].dtype)
        d = d * z * sig
    # (the columns' sums are long: in 64 bits)
    dw = (d * x).sum(0, dtype=torch.float64).float()
    db = None if s["b"] is None else d.sum(0, dtype=torch.float64).float()
    d = d * s["w"]
    dx = d - x * (d * x).mean(-1, keepdim=True)
    if not c["rms"]:
        dx = dx - d.mean(-1, keepdim=True)
    return {"dx": (dx * rstd).to(s["x"].dtype), "dz": dz, "dw": dw, "db": db}


def plain_cache(s):
    c, pages = s["case"], s["pages"]
    if c["op"] == "cache_copy":
        src = s["src"].long()
        pages[:, s["dst"].long()] = pages[:, src.clamp(min=0)] * (src >= 0).view(1, -1, 1, 1, 1)
        return {"pages": pages}
    if c["op"] == "cache_fork":
        children = torch.argsort((s["refs"] != 0).to(torch.uint8), stable=True)[:c["n"]]
        s["refs"][children] = 1
        src = s["parents"].long()
        pages[:, children] = pages[:, src.clamp(min=0)] * (src >= 0).view(1, -1, 1, 1, 1)
        s["refs"][children] -= 1
        return {"pages": pages, "children": children.to(torch.int32), "refs": s["refs"]}
    refs = s["refs0"]
    live = refs > 0
    count = live.sum()
    at = torch.arange(c["pages"], device="cuda")
    old = (live & (at >= count)).nonzero().flatten()
    new = (~live & (at < count)).nonzero().flatten()
    pages[:, new] = pages[:, old]
    remap = torch.where(live, at, -1)
    remap[old] = new
    s["refs"].copy_(refs)
    s["refs"][new] = refs[old]
    s["refs"][old] = 0
    s["table"].copy_(remap[s["table0"].long()])
    return {"pages": pages, "refs": s["refs"], "table": s["table"], "remap": remap.to(torch.int32),
            "live": count.to(torch.int32).view(1)}


# -------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "recurrent":
        return exact_recurrent(c, s)
    if c["op"].startswith("norm"):
        leaf = {n: s[n].double().requires_grad_() for n in ("x", "w", "b", "z") if s[n] is not None}
        x = leaf["x"]
        mean = 0.0 if c["rms"] else x.sum(-1, keepdim=True) / c["n"]
        var = ((x - mean) ** 2).sum(-1, keepdim=True) / c["n"]
        y = (x - mean) / torch.sqrt(var + EPS) * leaf["w"] + leaf.get("b", 0.0)
        if "z" in leaf:
            y = y * leaf["z"] * torch.sigmoid(leaf["z"])
        if c["op"] == "norm_fwd":
            return {"y": y.detach()}
        names = sorted(leaf)
        grads = dict(zip(names, torch.autograd.grad(y, [leaf[n] for n in names], s["dy"].double())))
        return {"d" + n: grads.get(n) for n in ("x", "z", "w", "b")}
    refs = s["refs"].tolist()
    pages = s["pages"].double()
    if c["op"] == "cache_copy":
        before = s["pages"]
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pages[:, b] = before[:, a].double() if a >= 0 else 0.0
        return {"pages": pages}
    if c["op"] == "cache_fork":
        free = [p for p, r in enumerate(refs) if r == 0]
        for a, b in zip(s["parents"].tolist(), free):
            pages[:, b] = pages[:, a] if a >= 0 else 0.0
        return {"pages": pages, "children": None, "refs": None}
    count = sum(r > 0 for r in refs)
    holes = [p for p in range(count) if refs[p] == 0]
    for p in range(count, c["pages"]):
        if refs[p] > 0:
            pages[:, holes.pop(0)] = pages[:, p]
    return {"pages": pages, "refs": None, "table": None, "remap": None, "live": None}


def exact_recurrent(c, s):
    group = torch.arange(c["h"], device="cuda") // (c["h"] // c["hqk"])
    flat = {n: s[n].reshape(-1, *s[n].shape[2:]) for n in ("q", "k", "v", "g", "beta")}
    state = s["state"].double()
    o = torch.zeros(flat["v"].shape, dtype=torch.float64, device="cuda")
    ins, outs = s["slots_in"].tolist(), s["slots_out"].tolist()
    t = 0
    for i, m in enumerate(lens(c)):
        H = state[ins[i]].clone() if ins[i] >= 0 else torch.zeros_like(state[0])   # [h, k, v]
        for _ in range(m):
            q, k = flat["q"][t][group].double(), flat["k"][t][group].double()
            decay = torch.exp(flat["g"][t].double())
            decayed = (decay[:, :, None] if c["gate_k"] else decay[:, None, None]) * H
            seen = (k[:, :, None] * (decayed if c["decay_first"] else H)).sum(1)
            r = flat["beta"][t].double()[:, None] * (flat["v"][t].double() - seen)
            H = decayed + k[:, :, None] * r[:, None, :]
            o[t] = (q[:, :, None] * H).sum(1)
            if c["per_token"]:
                state[outs[t]] = H
            t += 1
        if not c["per_token"]:
            state[outs[i]] = H
    return {"o": o.view(s["o"].shape), "state": state}
