"""Cases for the operators on the heads of a projection: RMSNorm of queries and keys with the
position rotation in the same pass (forward, and forward with backward), the rotation alone over
one to three axes, a key/value cache quantised as it is written and read back, and the serving
form that norms, rotates and writes the cache in one call.

`own` false: the plain form, elementary torch operations in float32 (angles in float64), rounded
once at the end.  `own` true: the calls of the library.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
QMAX = {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}
EPS = 1e-6
#: about the elements that the largest listed cases move; a drawn case moves half of it at most
MOST_ELEMENTS = 1 << 28


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of one sequence, norms and rotation alone: launch latency
        _case("norm_rope", "bf16", 1, 32, 8, 128, name="norm_rope 1 token"),
        # a long prompt through grouped-query heads cut out of one fused projection of width 4096 + 2*1024
        _case("norm_rope", "bf16", 16384, 32, 8, 128, fused=True, name="norm_rope 16384"),
        # a ragged batch on wide heads with only a quarter of each rotated, neighbouring pairs, one key head
        _case("norm_rope", "f16", 1003, 7, 1, 256, rot=64, pairs="pair", fused=True, name="norm_rope ragged d256"),
        # one training step's share of the same projection: forward, then gradients of both inputs and both weights
        _case("norm_rope_train", "bf16", 16384, 32, 8, 128, fused=True, name="train 16384"),
        # a small float32 model with an odd token count and heads of 80, half of each rotated
        _case("norm_rope_train", "f32", 777, 5, 5, 80, rot=40, name="train f32 odd"),
        # image tokens (128 images of 197 tokens, 12 heads of 64), rows and columns as two axes, forward and backward
        _case("rope_train", "f16", 25216, 12, 12, 64, axes=2, name="rope image"),
        # one video clip of 21 x 30 x 52 patches: time, height and width interleaved over the pairs
        _case("rope_train", "bf16", 32760, 12, 12, 128, axes=3, mixed=True, fused=True, name="rope video"),
        # a long context kept in four bits, written and read back once
        _case("cache", "bf16", 131072, 0, 8, 128, kind="int4", group=32, page=64, name="cache int4 131072"),
        # a few tokens of a small model, heads of 80, pages that the sequence does not fill
        _case("cache", "f16", 37, 0, 3, 80, kind="e4m3", group=80, page=16, name="cache e4m3 37"),
        # decoding, one sequence: one token in, its short context read back for the attention
        _case("serve", "bf16", 1, 32, 8, 128, kind="e4m3", group=128, page=16, context=1000, name="serve 1 token"),
        # decoding, a batch of 250 sequences with a little context each
        _case("serve", "f16", 250, 16, 4, 128, kind="int8", group=128, page=32, context=60, name="serve batch 250"),
        # a chunk of a long prompt, three position axes, written and read back with the part before it
        _case("serve", "bf16", 8192, 32, 8, 128, axes=3, kind="e4m3", group=64, page=64, context=8192, chunk=True,
              fused=True, name="serve chunk 8192"),
    ]


def _case(op, dtype, tokens, hq, hk, d, rot=None, pairs="half", axes=1, mixed=False, fused=False, kind="", group=0,
          page=0, context=0, chunk=False, name=None):
    c = dict(op=op, dtype=dtype, tokens=tokens, hq=hq, hk=hk, d=d, rot=d if rot is None else rot, pairs=pairs,
             axes=axes, mixed=mixed, fused=fused, kind=kind, group=group, page=page, context=context, chunk=chunk)
    if name is not None:
        c["name"] = name
    return c


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_train", "rope_train", "cache", "serve"])
    d = rng.choice([40, 64, 72, 80, 96, 128, 128, 160, 256])
    hk = rng.choice([1, 2, 3, 4, 5, 8, 12])
    hq = 0 if op == "cache" else hk * rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    kind, group, page, context, chunk = "", 0, 0, 0, False
    tokens = _log_uniform(rng, 1, 40000)
    if op in ("cache", "serve"):
        # four bits only where the cache stores the inputs themselves
        kind = rng.choice(["e4m3", "int8", "int4"] if op == "cache" else ["e4m3", "int8"])
        group = d // rng.choice([n for n in (1, 2, 4) if d % (8 * n) == 0])
        page = rng.choice([8, 16, 32, 64, 100])
        tokens = _log_uniform(rng, 1, 130000 if op == "cache" else 8192)
    if op == "serve":
        dtype = "bf16" if dtype == "f32" else dtype  # quantised keys go with 16-bit activations
        chunk = tokens > 256 or rng.random() < 0.3
        context = _log_uniform(rng, 1, 16384 if chunk else max(2, 200000 // tokens))
    axes = rng.choice([1, 1, 2, 3])
    rot = d if rng.random() < 0.6 else rng.choice([d // 2 - d // 2 % 2, d // 4 - d // 4 % 2])
    c = _case(op, dtype, tokens, hq, hk, d, rot, rng.choice(["half", "half", "pair"]),
              axes, axes > 1 and rng.random() < 0.5, rng.random() < 0.5, kind, group, page, context,
              chunk)
    while _elements(c) > MOST_ELEMENTS // 2:
        c["tokens"], c["context"] = max(1, c["tokens"] * 2 // 3), c["context"] * 2 // 3
    return c


def _read_tokens(c):
    """Tokens that the read of a cache case returns: what was written, or each sequence's context too."""
    if c["op"] == "cache":
        return c["tokens"]
    if c["chunk"]:  # a chunk of one prompt and the part before it
        return c["tokens"] + c["context"]
    return c["tokens"] * (c["context"] + 1)  # one token of each sequence and its context


def _elements(c):
    n = c["tokens"] * (c["hq"] + c["hk"]) * c["d"]
    if c["op"] == "cache":
        return 4 * n
    if c["op"] == "serve":
        return 2 * n + 2 * _read_tokens(c) * c["hk"] * c["d"]
    return n * {"norm_rope": 1, "norm_rope_train": 3, "rope_train": 2}[c["op"]]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    t, hq, hk, d, rot = (case[n] for n in ("tokens", "hq", "hk", "d", "rot"))
    n = t * (hq + hk) * d  # elements of q and k
    rows = t * (hq + hk)
    at = 8 * case["axes"] * t + 2 * rot  # positions and frequencies, read once a pass
    spin = t * (hq + hk) * rot * 3  # four products and two sums for each pair
    norm = {"bytes": 2 * n * e + 4 * rows + at + 2 * d * e, "flops": 4 * n + spin}
    if case["op"] == "norm_rope":
        return norm
    if case["op"] == "norm_rope_train":
        # backward: gradients and inputs in, gradients out, the saved statistic, the weights and theirs
        return {"bytes": norm["bytes"] + 3 * n * e + 4 * rows + at + 4 * d * e, "flops": norm["flops"] + spin + 9 * n}
    if case["op"] == "rope_train":
        return {"bytes": 2 * (2 * n * e + at), "flops": 2 * spin}
    bits = 0.5 if case["kind"] == "int4" else 1
    per = bits + 4 / case["group"]  # bytes of a stored element, with its share of the scale
    kv, back = 2 * t * hk * d, 2 * _read_tokens(case) * hk * d
    io = {"bytes": kv * (e + per) + 8 * t + back * (e + per) + 8 * _read_tokens(case), "flops": 4 * kv + back}
    if case["op"] == "cache":
        return io
    q = t * hq * d
    return {"bytes": io["bytes"] + 2 * q * e + at + 2 * d * e, "flops": io["flops"] + 4 * n + spin}


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------

def _axis_map(c):
    """The axis of each pair: sections one after another, or taken in turn."""
    n, a = c["rot"] // 2, c["axes"]
    if c["mixed"]:
        return [p % a for p in range(n)]
    return [min(p * a // max(n, 1), a - 1) for p in range(n)]


def _positions(c, start):
    """[axes, tokens]: places in a sequence, or in a grid of time, height and width."""
    t = torch.arange(c["tokens"], device="cuda")
    if c["axes"] == 1:
        return (t + start)[None]
    w = max(1, round(c["tokens"] ** (1.0 / c["axes"])))
    if c["axes"] == 2:
        return torch.stack([t // w, t % w])
    return torch.stack([t // (w * w) + start, t // w % w, t % w])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[c["dtype"]]
    t, hq, hk, d, rot = (c[n] for n in ("tokens", "hq", "hk", "d", "rot"))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    # projections have a few channels far larger than the rest, keys most of all
    loud = torch.ones(d, device="cuda")
    loud[torch.randint(0, d, (3,), generator=g, device="cuda")] = 6.0
    s = {"case": c}
    if c["fused"]:
        qkv = normal(t, hq + 2 * hk, d)
        qkv[:, hq:hq + hk] *= loud
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:
        s["q"], s["k"], s["v"] = normal(t, hq, d).to(dt), (normal(t, hk, d) * loud).to(dt), normal(t, hk, d).to(dt)
    s["wq"] = (1 + 0.1 * normal(d)).to(dt)
    s["wk"] = (1 + 0.1 * normal(d)).to(dt)
    start = int(torch.randint(0, 200000, (1,), generator=g, device="cuda"))
    s["pos"] = _positions(c, start).contiguous()
    s["inv_freq"] = (10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) / max(rot // 2, 1))).float()
    s["axis_bytes"] = bytes(_axis_map(c)) if c["axes"] > 1 else None  # the form the library takes
    s["axis"] = torch.tensor(_axis_map(c), device="cuda")
    if c["op"].endswith("train"):
        s["dq_out"], s["dk_out"] = normal(t, hq, d).to(dt), normal(t, hk, d).to(dt)
    for name in ("q", "k") if c["op"] != "cache" else ():  # buffers that a program keeps for its results
        s[name + "_out"] = torch.empty_like(s[name], memory_format=torch.contiguous_format)
    if c["op"].endswith("train"):
        s["dq"], s["dk"] = torch.empty_like(s["q_out"]), torch.empty_like(s["k_out"])
    if c["op"].startswith("norm_rope"):
        s["rstd_q"], s["rstd_k"] = torch.empty(t, hq, device="cuda"), torch.empty(t, hk, device="cuda")
    if c["op"] == "norm_rope_train":
        s["dwq"], s["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
        if own:
            import normalization_layernorm_rmsnorm_gb300 as nrm
            s["ws"] = nrm.qk_norm_workspace(s["q"])
    if c["kind"]:
        _prepare_cache(s, c, g)
    return s


def _prepare_cache(s, c, g):
    t, hk, d, page = (c[n] for n in ("tokens", "hk", "d", "page"))
    back = _read_tokens(c)
    pages = -(-back // page) + 3  # the pool is a little larger than what is used
    shape = (pages, page, hk, d)
    for n in ("k", "v"):
        values = torch.randn(shape, generator=g, device="cuda")
        s[n + "_codes"], s[n + "_scales"] = _quantise(values, c)
    order = torch.randperm(pages, generator=g, device="cuda")  # pages are handed out in no order
    at = torch.arange(back, device="cuda")
    slots = order[at // page] * page + at % page
    s["read_slots"] = slots.contiguous()
    if c["op"] == "cache":
        s["slots"] = s["read_slots"]
    elif c["chunk"]:
        s["slots"] = slots[c["context"]:].contiguous()  # the chunk follows the part before it
    else:
        s["slots"] = slots[c["context"]::c["context"] + 1].contiguous()  # the last token of each sequence
    dt = TYPES[c["dtype"]]
    s["k_back"] = torch.empty(back, hk, d, device="cuda", dtype=dt)
    s["v_back"] = torch.empty_like(s["k_back"])
    if own:
        import normalization_layernorm_rmsnorm_gb300 as nrm
        s["cache"] = nrm.kv_cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import normalization_layernorm_rmsnorm_gb300 as nrm
    c = s["case"]
    how = {"axis": s["axis_bytes"], "pairs": c["pairs"]}
    if c["op"] == "norm_rope" or c["op"] == "norm_rope_train":
        nrm.nrm_qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"],
                                 s["rstd_q"], s["rstd_k"], EPS, **how)
        out = {n: s[n] for n in ("q_out", "k_out", "rstd_q", "rstd_k")}
        if c["op"] == "norm_rope_train":
            nrm.nrm_qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["wq"], s["wk"], s["rstd_q"], s["rstd_k"],
                                     s["pos"], s["inv_freq"], s["dq"], s["dk"], s["dwq"], s["dwk"], s["ws"], **how)
            out |= {n: s[n] for n in ("dq", "dk", "dwq", "dwk")}
        return out
    if c["op"] == "rope_train":
        nrm.nrm_rope_fwd(s["q"], s["k"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"], **how)
        nrm.nrm_rope_bwd(s["dq_out"], s["dk_out"], s["pos"], s["inv_freq"], s["dq"], s["dk"], **how)
        return {n: s[n] for n in ("q_out", "k_out", "dq", "dk")}
    out = {}
    if c["op"] == "cache":
        nrm.nrm_kv_cache_write(s["k"], s["v"], s["cache"], s["slots"])
    else:
        nrm.nrm_qk_norm_rope_cache(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["pos"], s["inv_freq"], s["q_out"], None,
                                   s["cache"], s["slots"], EPS, **how)
        out["q_out"] = s["q_out"]
    nrm.nrm_kv_cache_read(s["cache"], s["read_slots"], s["k_back"], s["v_back"])
    return out | {"k_back": s["k_back"], "v_back": s["v_back"]}


def _run_plain(s):
    c = s["case"]
    dt = TYPES[c["dtype"]]
    if c["op"] != "cache":
        # angles of far positions need 64 bits
        angle = s["pos"][s["axis"]].t().double() * s["inv_freq"].double()
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["op"] == "rope_train":
        return {"q_out": _rotate(s["q"].float(), cos, sin, c).to(dt), "k_out": _rotate(s["k"].float(), cos, sin, c).to(dt),
                "dq": _rotate(s["dq_out"].float(), cos, -sin, c).to(dt),
                "dk": _rotate(s["dk_out"].float(), cos, -sin, c).to(dt)}
    if c["op"] == "cache":
        k, v, out = s["k"].float(), s["v"].float(), {}
    else:
        rq, rk = _rstd(s["q"].float()), _rstd(s["k"].float())
        q_out = _rotate(s["q"].float() * rq * s["wq"].float(), cos, sin, c).to(dt)
        k_out = _rotate(s["k"].float() * rk * s["wk"].float(), cos, sin, c).to(dt)
        if c["op"].startswith("norm_rope"):
            out = {"q_out": q_out, "k_out": k_out, "rstd_q": rq[..., 0], "rstd_k": rk[..., 0]}
            if c["op"] == "norm_rope_train":
                out["dq"], out["dwq"] = _norm_rope_grad(s["dq_out"].float(), s["q"].float(), s["wq"].float(), rq, cos, sin, c)
                out["dk"], out["dwk"] = _norm_rope_grad(s["dk_out"].float(), s["k"].float(), s["wk"].float(), rk, cos, sin, c)
                out |= {n: out[n].to(dt) for n in ("dq", "dk", "dwq", "dwk")}
            return out
        # the cache stores the key as the norm and the rotation give it in the activations' type
        k, v, out = k_out.float(), s["v"].float(), {"q_out": q_out}
    for n, x in (("k", k), ("v", v)):
        codes, scales = _quantise(x, c)
        kept, kept_scales = s[n + "_codes"].flatten(0, 1), s[n + "_scales"].flatten(0, 1)
        kept.view(torch.uint8)[s["slots"]] = codes.view(torch.uint8)
        kept_scales[s["slots"]] = scales
        back = kept.view(torch.uint8)[s["read_slots"]].view(kept.dtype)
        out[n + "_back"] = _values(back, kept_scales[s["read_slots"]], c).to(dt)
    return out


def _rstd(x):
    return ((x * x).mean(-1, keepdim=True) + EPS) ** -0.5


def _rotate(x, cos, sin, c):
    rot = c["rot"]
    if c["pairs"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def _norm_rope_grad(dy, x, w, r, cos, sin, c):
    back = _rotate(dy, cos, -sin, c)
    g = back * w
    dx = r * g - x * r ** 3 * ((g * x).sum(-1, keepdim=True) / c["d"])
    return dx, (back * x * r).sum((0, 1))


def _quantise(x, c):
    """Codes and scales of x[..., d] in float32: each group divided by its largest magnitude.
    In 64 bits, where values next to a border between two codes keep their side."""
    q = QMAX[c["kind"]]
    groups = x.unflatten(-1, (-1, c["group"]))
    m = groups.abs().amax(-1, keepdim=True)
    u = (groups.double() * q / torch.where(m == 0, 1.0, m)).flatten(-2)
    scales = (m / q)[..., 0]
    if c["kind"] == "e4m3":
        step = torch.ldexp(torch.ones_like(u), torch.frexp(u.abs().clamp_min(2.0 ** -6)).exponent - 4)
        return ((u / step).round() * step).to(torch.float8_e4m3fn), scales
    codes = u.round().to(torch.int8)
    if c["kind"] == "int8":
        return codes, scales
    low, high = codes[..., 0::2] & 15, codes[..., 1::2] & 15
    return (low | high << 4).view(torch.uint8), scales


def _values(codes, scales, c):
    if c["kind"] == "int4":
        codes = codes.view(torch.int8)
        codes = torch.stack([codes << 4 >> 4, codes >> 4], -1).flatten(-2)
    return (codes.float().unflatten(-1, (-1, c["group"])) * scales[..., None]).flatten(-2)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    dt = TYPES[c["dtype"]]
    out = {}
    if c["op"] != "cache":
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           torch.einsum("pt,p->tp", s["pos"].double()[s["axis"]], s["inv_freq"].double()))[:, None]

    def spin(x, by):
        y = x.clone()
        if c["pairs"] == "half":
            a, b = slice(0, c["rot"] // 2), slice(c["rot"] // 2, c["rot"])
        else:
            a, b = slice(0, c["rot"], 2), slice(1, c["rot"], 2)
        z = torch.complex(x[..., a], x[..., b]) * by
        y[..., a], y[..., b] = z.real, z.imag
        return y

    if c["op"] == "rope_train":
        for x, n, by in (("q", "q_out", turn), ("k", "k_out", turn), ("dq_out", "dq", turn.conj()), ("dk_out", "dk", turn.conj())):
            out[n] = spin(s[x].double(), by)
        return out
    kept = {"k": s["k"].double(), "v": s["v"].double()}
    if c["op"] != "cache":
        for n in ("q", "k"):
            x, w = s[n].double(), s["w" + n].double()
            r = 1 / torch.sqrt(torch.einsum("thi,thi->th", x, x) / c["d"] + EPS)
            y = spin(torch.einsum("thi,th,i->thi", x, r, w), turn)
            if c["op"] == "serve":
                kept[n] = y.to(dt).double()  # rounded to the activations' type: what the cache is defined to store
                if n == "q":
                    out["q_out"] = y
                continue
            out[n + "_out"], out["rstd_" + n] = y, r
            if c["op"] == "norm_rope_train":
                unit = x * r[..., None]  # dx is the part of the gradient orthogonal to the row, in units of 1/rms
                back = spin(s["d" + n + "_out"].double(), turn.conj())
                along = torch.einsum("thi,thi,i->th", back, unit, w) / c["d"]
                out["d" + n] = (back * w - unit * along[..., None]) * r[..., None]
                out["dw" + n] = torch.einsum("thi,thi->i", back, unit)
        if c["op"] != "serve":
            return out
    for n in ("k", "v"):
        table = _decode_all(s[n + "_codes"], s[n + "_scales"], c)
        table[s["slots"]] = _nearest(kept[n], c)
        out[n + "_back"] = table[s["read_slots"]]
    return out


def _nearest(x, c):
    """The stored values that stand for x: the nearest of the format's grid, ties to even, group by group."""
    parts = x.reshape(*x.shape[:-1], -1, c["group"])
    top = parts.abs().max(-1, keepdim=True).values
    u = parts * QMAX[c["kind"]] / torch.where(top > 0, top, torch.ones_like(top))  # the product is exact: ties stay ties
    if c["kind"] == "e4m3":
        step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))) - 3)
        u = (u / step).round() * step
    else:
        u = u.round()
    return (u * top / QMAX[c["kind"]]).reshape(x.shape)


def _decode_all(codes, scales, c):
    codes = codes.flatten(0, 1)
    if c["kind"] == "int4":
        b = codes.to(torch.int64)
        codes = torch.stack([(b + 8) % 16 - 8, (b // 16 + 8) % 16 - 8], -1).reshape(*b.shape[:-1], -1)
    x = codes.to(torch.float32).double()
    return (x.reshape(*x.shape[:-1], -1, c["group"]) * scales.flatten(0, 1).double()[..., None]).reshape(x.shape)
