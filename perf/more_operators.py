"""Cases for what a served layer does around its cache, and a layer of either kind between its blocks:
attention of one new token of each sequence over the paged, quantised key/value cache (with the
attention weight that every position has received so far), eviction from that cache by the weight, and
the norm after a block, its gate and residual scale, and the norm before the next block in one pass
(forward, and forward with backward).

`own` false: the plain form, elementary torch operations in float32, rounded once at the end.
`own` true: the calls of the library.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
QMAX = {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}
EPS = 1e-6
#: about the elements that the largest listed cases move; a drawn case moves half of them at most
MOST_CACHED = 1 << 28
MOST_ROWS = 1 << 26


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # decoding, one sequence with a short context: latency
        _attend("bf16", 1, 1001, 32, 8, 128, "e4m3", 128, 16, ragged=False, name="attend 1 token"),
        # decoding, a large batch of short sequences
        _attend("f16", 250, 120, 16, 4, 128, "int8", 128, 32, name="attend batch 250"),
        # decoding, sequences of very different lengths, with the weights that eviction goes by
        _attend("bf16", 64, 2048, 32, 8, 128, "e4m3", 64, 64, weights=True, name="attend ragged 64"),
        # one long context in four bits
        _attend("bf16", 1, 131072, 32, 8, 128, "int4", 32, 64, ragged=False, name="attend int4 131072"),
        # a small float32 model: a head of keys for each query head, a sliding window, pages of an odd size
        _attend("f32", 9, 3001, 12, 12, 80, "e4m3", 80, 100, weights=True, window=777, name="attend f32 window"),
        # one wide head of keys and values for all queries, long sequences
        _attend("bf16", 16, 16384, 16, 1, 256, "int8", 256, 64, name="attend shared head"),
        # a conversation that has reached its budget
        _evict("bf16", 1, 4096, 8, 128, "e4m3", 128, 16, 1024, 4, 256, ragged=False, name="evict 4096"),
        # half of a long context goes
        _evict("bf16", 1, 131072, 8, 128, "e4m3", 128, 64, 65536, 4, 1000, ragged=False, name="evict 131072"),
        # a ragged batch in four bits, some sequences still under the budget
        _evict("f16", 24, 4000, 8, 128, "int4", 32, 32, 1000, 0, 100, name="evict ragged int4"),
        # decoding, one token between two blocks: launch latency
        _block("bf16", 1, 4096, name="block 1 token"),
        # one training step's share between two blocks of width 4096, a learned scale per channel
        _block("bf16", 16384, 4096, gate=1, alpha=0.5, train=True, name="block train 16384"),
        # image tokens (128 images of 197 tokens) of width 768, each image with its own gate, forward and backward
        _block("f16", 25216, 768, gate=128, train=True, name="block train image"),
    ]


def _attend(dtype, seqs, cap, hq, hk, d, kind, group, page, ragged=True, weights=False, window=0, name=None):
    c = dict(op="attend", dtype=dtype, seqs=seqs, cap=cap, hq=hq, hk=hk, d=d, kind=kind, group=group, page=page,
             ragged=ragged, weights=weights, window=window)
    return c if name is None else dict(c, name=name)


def _evict(dtype, seqs, cap, hk, d, kind, group, page, keep, first, recent, ragged=True, name=None):
    c = dict(op="evict", dtype=dtype, seqs=seqs, cap=cap, hq=hk, hk=hk, d=d, kind=kind, group=group, page=page,
             ragged=ragged, keep=keep, first=first, recent=recent)
    return c if name is None else dict(c, name=name)


def _block(dtype, rows, cols, gate=0, alpha=1.0, post=True, train=False, name=None):
    """gate: 0 none, else the rows of the gate, each for rows / gate rows."""
    c = dict(op="block", dtype=dtype, rows=rows, cols=cols, gate=gate, alpha=alpha, post=post, train=train)
    return c if name is None else dict(c, name=name)


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "evict", "block"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "block":
        step = rng.choice([1, 2, 8, 64])
        cols = max(step, _log_uniform(rng, 64, 12000) // step * step)
        rows = max(1, min(_log_uniform(rng, 1, 40000), MOST_ROWS // 2 // cols))
        gate = rng.choice([0, 1, 1, 2])
        if gate == 2:  # a gate for each sample
            gate = _log_uniform(rng, 1, min(rows, 256))
            rows = max(1, rows // gate) * gate
        return _block(dtype, rows, cols, gate, rng.choice([1.0, 0.5, 0.1]), rng.random() < 0.8, rng.random() < 0.6)
    d = rng.choice([64, 80, 96, 128, 128, 160, 256])
    hk = rng.choice([1, 2, 3, 4, 5, 8, 12])
    kind = rng.choice(["e4m3", "int8", "int4"])
    group = d // rng.choice([n for n in (1, 2, 4) if d % (16 * n) == 0])
    page = rng.choice([8, 16, 32, 64, 100])
    seqs = _log_uniform(rng, 1, 300)
    cap = _log_uniform(rng, 1, max(8, min(131072, MOST_CACHED // 2 // (seqs * hk * d))))
    if op == "attend":
        return _attend(dtype, seqs, cap, hk * rng.choice([1, 2, 3, 4, 6, 8, 16]), hk, d, kind, group, page,
                       rng.random() < 0.7, rng.random() < 0.4, rng.choice([0, 0, _log_uniform(rng, 1, cap)]))
    keep = max(1, cap * rng.randint(10, 90) // 100)
    return _evict(dtype, seqs, cap, hk, d, kind, group, page, keep, rng.randint(0, min(4, keep // 2)),
                  rng.randint(0, keep // 2), rng.random() < 0.7)


def _lengths(c):
    """Each sequence's length: all of the capacity, or anything up to it (an empty one among many)."""
    if not c["ragged"]:
        return [c["cap"]] * c["seqs"]
    # by the golden ratio, so that the cost of a case does not hang on its seed
    n = [1 + int((0.5 + 0.6180339887498949 * i) % 1.0 * c["cap"]) for i in range(c["seqs"])]
    if c["seqs"] > 4:
        n[3] = 0
    return [min(x, c["cap"]) for x in n]


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "block":
        n, gates = c["rows"] * c["cols"], c["gate"] * c["cols"]
        params = (2 if c["post"] else 1) * c["cols"] + gates
        stats = 4 * c["rows"] * (2 if c["post"] else 1)
        fwd = {"bytes": 4 * n * e + params * e + (stats if c["train"] else 0), "flops": 9 * n}
        if not c["train"]:
            return fwd
        return {"bytes": fwd["bytes"] + 6 * n * e + 2 * params * e + stats, "flops": fwd["flops"] + 24 * n}
    bits = 0.5 if c["kind"] == "int4" else 1
    row = 2 * c["hk"] * c["d"] * (bits + 4 / c["group"])  # bytes of a slot's keys and values, with their scales
    if c["op"] == "attend":
        seen = sum(min(n, c["window"] or n) for n in _lengths(c))
        q = c["seqs"] * c["hq"] * c["d"]
        return {"bytes": seen * row + 2 * q * e + 16 * c["seqs"] + 8 * (seen // c["page"] + c["seqs"])
                + (8 * c["hk"] * seen if c["weights"] else 0), "flops": 4 * seen * c["hq"] * c["d"]}
    held = sum(_lengths(c))
    kept = sum(min(n, c["keep"]) for n in _lengths(c))
    # weights read, the kept ones and their positions written, their rows copied; then read back
    return {"bytes": 4 * c["hk"] * held + 12 * c["hk"] * kept + 2 * kept * row + kept * (row + 2 * c["hk"] * c["d"] * e),
            "flops": 2 * kept * c["hk"] * c["d"]}


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_block(c, g) if c["op"] == "block" else _prepare_cache(c, g)


def _prepare_block(c, g):
    dt, rows, cols = TYPES[c["dtype"]], c["rows"], c["cols"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {"case": c}
    # a residual stream has a few channels far larger than the rest
    loud = torch.ones(cols, device="cuda")
    loud[torch.randint(0, cols, (min(3, cols),), generator=g, device="cuda")] = 20.0
    s["x"], s["f"] = (normal(rows, cols) * loud).to(dt), (0.5 * normal(rows, cols)).to(dt)
    s["w_post"] = (0.3 + 0.1 * normal(cols)).to(dt) if c["post"] else None
    s["w_pre"] = (1 + 0.1 * normal(cols)).to(dt)
    s["gate"] = (0.5 * normal(c["gate"], cols)).to(dt) if c["gate"] else None
    for n in ("y", "h"):
        s[n] = torch.empty_like(s["x"])
    s["rstd_post"] = s["rstd_pre"] = s["ws"] = None
    if c["train"]:
        s["dh"], s["dy"] = normal(rows, cols).to(dt), normal(rows, cols).to(dt)
        s["rstd_post"] = torch.empty(rows, device="cuda") if c["post"] else None
        s["rstd_pre"] = torch.empty(rows, device="cuda")
        for n, like in (("dx", "x"), ("df", "x"), ("dgate", "gate"), ("dw_post", "w_post"), ("dw_pre", "w_pre")):
            s[n] = None if s[like] is None else torch.empty_like(s[like])
        if own:
            import normalization_layernorm_rmsnorm_gb300 as nrm
            s["ws"] = nrm.block_norm_workspace(s["x"], s["gate"])
    return s


def _prepare_cache(c, g):
    seqs, cap, hq, hk, d, page = (c[n] for n in ("seqs", "cap", "hq", "hk", "d", "page"))
    dt = TYPES[c["dtype"]]
    width = -(-cap // page)
    new_width = -(-c["keep"] // page) if c["op"] == "evict" else 0
    pages = seqs * (width + new_width) + 3  # the pool is a little larger than what is used
    # pages are handed out in no order
    order = torch.randperm(pages, generator=g, device="cuda")
    s = {"case": c, "table": order[:seqs * width].view(seqs, width).contiguous()}
    s["lengths"] = torch.tensor(_lengths(c), device="cuda")
    loud = torch.ones(d, device="cuda")
    loud[torch.randint(0, d, (3,), generator=g, device="cuda")] = 6.0
    # slots that no token has been written to hold anything
    used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    at = torch.arange(width * page, device="cuda")
    used[s["table"][:, at // page], at % page] = at < s["lengths"][:, None]
    for n in ("k", "v"):
        values = torch.randn((pages, page, hk, d), generator=g, device="cuda")
        s[n + "_codes"], scales = _quantise(values * loud if n == "k" else values, c)
        s[n + "_scales"] = torch.where(used[..., None, None], scales, math.nan).contiguous()
        del values
    if c["op"] == "attend":
        s["q"] = (2 * torch.randn((seqs, hq, d), generator=g, device="cuda")).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["weights"] = torch.rand((seqs, hk, cap), generator=g, device="cuda") if c["weights"] else None
        s["lse"] = torch.empty(seqs, hq, device="cuda") if c["weights"] else None
    else:
        # a few positions have most of the weight; some never had any
        w = torch.exp(2 * torch.randn((seqs, hk, cap), generator=g, device="cuda"))
        s["weights"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, 0.0, w)
        s["new_table"] = order[seqs * width:seqs * (width + new_width)].view(seqs, new_width).contiguous()
        s["new_lengths"] = torch.empty_like(s["lengths"])
        s["new_weights"] = torch.zeros(seqs, hk, c["keep"], device="cuda")
        s["kept"] = torch.empty(seqs, hk, c["keep"], dtype=torch.int64, device="cuda")
        # what is read back afterwards: the rows that stayed
        i = torch.arange(c["keep"], device="cuda")
        slots = s["new_table"][:, i // page] * page + i % page
        s["read_slots"] = torch.where(i < s["lengths"].clamp(max=c["keep"])[:, None], slots, -1).flatten().contiguous()
        s["k_back"] = torch.zeros(seqs * c["keep"], hk, d, device="cuda", dtype=dt)
        s["v_back"] = torch.zeros_like(s["k_back"])
    if own:
        import normalization_layernorm_rmsnorm_gb300 as nrm
        s["cache"] = nrm.kv_cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
        if c["op"] == "attend":
            s["ws"] = nrm.kv_attention_workspace(s["q"], s["cache"], s["table"], weights=c["weights"])
    return s


def _quantise(x, c):
    """Codes and scales of x[..., d]: each group divided by its largest magnitude."""
    groups = x.unflatten(-1, (-1, c["group"]))
    m = groups.abs().amax(-1, keepdim=True)
    u = (groups * (QMAX[c["kind"]] / m)).flatten(-2)
    scales = (m / QMAX[c["kind"]])[..., 0]
    if c["kind"] == "e4m3":
        return u.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scales
    codes = u.round().clamp(-QMAX[c["kind"]], QMAX[c["kind"]]).to(torch.int8)
    if c["kind"] == "int8":
        return codes, scales
    return (codes[..., 0::2] & 15 | (codes[..., 1::2] & 15) << 4).view(torch.uint8), scales


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import normalization_layernorm_rmsnorm_gb300 as nrm
    c = s["case"]
    if c["op"] == "attend":
        nrm.nrm_kv_cache_attention(s["q"], s["cache"], s["table"], s["lengths"], s["out"], c["d"] ** -0.5, s["ws"],
                                   window=c["window"], lse=s["lse"], weights=s["weights"])
        return {n: s[n] for n in ("out", "lse", "weights") if s[n] is not None}
    if c["op"] == "evict":
        nrm.nrm_kv_cache_evict(s["cache"], s["table"], s["lengths"], s["weights"], s["new_table"], s["new_lengths"],
                               s["new_weights"], s["kept"], first=c["first"], recent=c["recent"])
        nrm.nrm_kv_cache_read(s["cache"], s["read_slots"], s["k_back"], s["v_back"])
        return {n: s[n] for n in ("new_lengths", "new_weights", "kept", "k_back", "v_back")}
    nrm.nrm_block_norm_fwd(s["x"], s["f"], s["gate"], s["w_post"], s["w_pre"], s["y"], s["h"], s["rstd_post"],
                           s["rstd_pre"], c["alpha"], EPS, post=c["post"])
    names = ["y", "h"]
    if c["train"]:
        nrm.nrm_block_norm_bwd(s["dh"], s["dy"], s["f"], s["y"], s["gate"], s["w_post"], s["w_pre"], s["rstd_post"],
                               s["rstd_pre"], s["dx"], s["df"], s["dgate"], s["dw_post"], s["dw_pre"], s["ws"],
                               c["alpha"], post=c["post"])
        names += ["dx", "df", "dgate", "dw_post", "dw_pre"]
    return {n: s[n] for n in names if s[n] is not None}


def _run_plain(s):
    return {"attend": _plain_attend, "evict": _plain_evict, "block": _plain_block}[s["case"]["op"]](s)


def _values(codes, scales, c):
    if c["kind"] == "int4":
        codes = codes.view(torch.int8)
        codes = torch.stack([codes << 4 >> 4, codes >> 4], -1).flatten(-2)
    return (codes.float().unflatten(-1, (-1, c["group"])) * scales[..., None]).flatten(-2)


def _rows(s, name, slots):
    """The values in the slots [..., hk, d] (a slot's heads together)."""
    codes, scales = s[name + "_codes"].flatten(0, 1), s[name + "_scales"].flatten(0, 1)
    return _values(codes.view(torch.uint8)[slots].view(codes.dtype), scales[slots], s["case"])


def _plain_attend(s):
    c = s["case"]
    at = torch.arange(c["cap"], device="cuda")
    slots = s["table"][:, at // c["page"]] * c["page"] + at % c["page"]
    n = s["lengths"][:, None]
    seen = at < n
    if c["window"]:
        seen = seen & (at >= n - c["window"])
    k = _rows(s, "k", slots).permute(0, 2, 3, 1)  # [seqs, hk, d, cap]
    q = s["q"].float().unflatten(1, (c["hk"], -1)) * c["d"] ** -0.5
    logits = torch.where(seen[:, None, None], q @ k, -math.inf)  # [seqs, hk, heads of one, cap]
    del k
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    v = torch.where(seen[:, :, None, None], _rows(s, "v", slots), 0.0).transpose(1, 2)  # [seqs, hk, cap, d]
    out = {"out": (p @ v).flatten(1, 2).to(TYPES[c["dtype"]])}
    if c["weights"]:
        out["lse"] = (m + torch.log(total)).flatten(1)
        s["weights"] += p.sum(2)
        out["weights"] = s["weights"]
    return out


def _plain_evict(s):
    c = s["case"]
    page, keep = c["page"], c["keep"]
    at = torch.arange(c["cap"], device="cuda")
    n = s["lengths"][:, None, None]
    always = (at < c["first"]) | (at >= n - c["recent"])
    rank = torch.where(at < n, torch.where(always, math.inf, s["weights"]), -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    new = n.clamp(max=keep)
    i = torch.arange(keep, device="cuda")
    here = (i < new).expand_as(best)
    # the positions that stay, in order; those behind the end after all others
    kept = torch.where(here, best, c["cap"]).sort(-1).values
    kept = torch.where(here, kept, -1)
    place = s["new_table"][:, i // page] * page + i % page
    seq, head, _ = torch.nonzero(here, as_tuple=True)
    old = kept[here]
    src = s["table"][seq, old // page] * page + old % page
    dst = place[:, None].expand_as(best)[here]
    out = {"new_lengths": new[:, 0, 0], "kept": kept}
    s["new_weights"][here] = s["weights"][seq, head, old]
    out["new_weights"] = s["new_weights"]
    for name in ("k", "v"):
        for part in (s[name + "_codes"].view(torch.uint8).flatten(0, 1), s[name + "_scales"].flatten(0, 1)):
            part[dst, head] = part[src, head]
        valid = s["read_slots"] >= 0
        back = s[name + "_back"]
        out[name + "_back"] = torch.where(valid[:, None, None], _rows(s, name, s["read_slots"].clamp(min=0)).to(back.dtype), back)
    return out


def _plain_block(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    f, w_pre = s["f"].float(), s["w_pre"].float()
    r1 = ((f * f).mean(-1, keepdim=True) + EPS) ** -0.5 if c["post"] else None
    w_post = s["w_post"].float() if c["post"] else 1.0
    n = f * r1 * w_post if c["post"] else f
    gate = _spread(s["gate"].float(), c) * c["alpha"] if c["gate"] else c["alpha"]
    # the norm before the next block takes the stream as it is stored
    y = (s["x"].float() + gate * n).to(dt)
    z = y.float()
    r2 = ((z * z).mean(-1, keepdim=True) + EPS) ** -0.5
    out = {"y": y, "h": (z * r2 * w_pre).to(dt)}
    if c["train"]:
        dh = s["dh"].float()
        g = dh * w_pre
        dx = s["dy"].float() + r2 * g - z * r2 ** 3 * ((g * z).sum(-1, keepdim=True) / c["cols"])
        out["dx"], out["dw_pre"] = dx.to(dt), (dh * z * r2).sum(0).to(dt)
        dn = gate * dx
        if c["gate"]:
            out["dgate"] = (c["alpha"] * dx * n).unflatten(0, (c["gate"], -1)).sum(1).to(dt)
        if c["post"]:
            g = dn * w_post
            out["dw_post"] = (dn * f * r1).sum(0).to(dt)
            dn = r1 * g - f * r1 ** 3 * ((g * f).sum(-1, keepdim=True) / c["cols"])
        out["df"] = dn.to(dt)
    return out


def _spread(gate, c):
    """A row of the gate for every row, or one for all."""
    return gate if c["gate"] == 1 else gate.repeat_interleave(c["rows"] // c["gate"], 0)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "evict": _exact_evict, "block": _exact_block}[s["case"]["op"]](s, s["case"])


def _stored(s, name, head, slots, c):
    """Values of one head's rows in the slots, from the codes one by one."""
    codes = s[name + "_codes"][slots // c["page"], slots % c["page"], head]
    if c["kind"] == "int4":
        b = codes.to(torch.int64)
        codes = torch.stack([(b + 8) % 16 - 8, (b // 16 + 8) % 16 - 8], -1).reshape(b.shape[0], -1)
    x = codes.to(torch.float32).double().reshape(codes.shape[0], -1, c["group"])
    return (x * s[name + "_scales"][slots // c["page"], slots % c["page"], head].double()[..., None]).reshape(codes.shape[0], -1)


def _exact_attend(s, c):
    heads = c["hq"] // c["hk"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if c["weights"] else None
    for i, n in enumerate(_lengths(c)):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == first:
            continue
        j = torch.arange(first, n, device="cuda")
        slots = s["table"][i, j // c["page"]] * c["page"] + j % c["page"]
        for h in range(c["hk"]):
            q = s["q"][i, h * heads:(h + 1) * heads].double()
            l = torch.einsum("hd,jd->hj", q, _stored(s, "k", h, slots, c)) / math.sqrt(c["d"])
            lse[i, h * heads:(h + 1) * heads] = torch.logsumexp(l, 1)
            p = torch.softmax(l, 1)
            out[i, h * heads:(h + 1) * heads] = torch.einsum("hj,jd->hd", p, _stored(s, "v", h, slots, c))
            if weights is not None:
                weights[i, h, first:n] += p.sum(0)
    return {"out": out, "lse": lse, "weights": weights} if c["weights"] else {"out": out}


def _exact_evict(s, c):
    kept, weights = torch.full_like(s["kept"], -1), s["new_weights"].double()
    backs = [torch.zeros(s["k_back"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    new = [min(n, c["keep"]) for n in _lengths(c)]
    for i, n in enumerate(_lengths(c)):
        for h in range(c["hk"] if n else 0):
            w = s["weights"][i, h, :n]
            if n > c["keep"]:
                stop = n - c["recent"]
                # descending, and among equals the lowest position first
                order = torch.argsort(-w[c["first"]:stop], stable=True)[:c["keep"] - c["first"] - c["recent"]] + c["first"]
                j = torch.cat([torch.arange(c["first"], device="cuda"), order.sort().values, torch.arange(stop, n, device="cuda")])
            else:
                j = torch.arange(n, device="cuda")
            kept[i, h, :new[i]] = j
            weights[i, h, :new[i]] = w[j].double()
            slots = s["table"][i, j // c["page"]] * c["page"] + j % c["page"]
            for b, name in zip(backs, ("k", "v")):
                b[i * c["keep"]:i * c["keep"] + new[i], h] = _stored(s, name, h, slots, c)
    return {"new_lengths": torch.tensor(new, device="cuda"), "new_weights": weights, "kept": kept, "k_back": backs[0],
            "v_back": backs[1]}


def _exact_block(s, c):
    dt, rows = TYPES[c["dtype"]], c["rows"]
    f, x = s["f"].double(), s["x"].double()
    unit_f, unit = None, f
    if c["post"]:
        r1 = 1 / torch.sqrt(torch.einsum("rc,rc->r", f, f) / c["cols"] + EPS)
        unit_f = f * r1[:, None]
        unit = unit_f * s["w_post"].double()
    which = torch.arange(rows, device="cuda") // max(1, rows // max(1, c["gate"]))
    gate = s["gate"].double()[which] if c["gate"] else torch.ones((), dtype=torch.float64, device="cuda")
    y = torch.addcmul(x, gate.expand_as(x), unit, value=c["alpha"])
    z = y.to(dt).double()  # as the next block finds it
    r2 = 1 / torch.sqrt(torch.einsum("rc,rc->r", z, z) / c["cols"] + EPS)
    unit_z = z * r2[:, None]
    out = {"y": y, "h": unit_z * s["w_pre"].double()}
    if c["train"]:
        # a norm's gradient is what is orthogonal to the row, in units of 1/rms
        dh = s["dh"].double()
        g = dh * s["w_pre"].double()
        along = torch.einsum("rc,rc->r", g, unit_z) / c["cols"]
        dx = s["dy"].double() + (g - unit_z * along[:, None]) * r2[:, None]
        out["dx"], out["dw_pre"] = dx, torch.einsum("rc,rc->c", dh, unit_z)
        if c["gate"]:
            out["dgate"] = torch.zeros(s["gate"].shape, dtype=torch.float64, device="cuda").index_add_(0, which, c["alpha"] * dx * unit)
        dn = c["alpha"] * gate * dx
        if c["post"]:
            out["dw_post"] = torch.einsum("rc,rc->c", dn, unit_f)
            g = dn * s["w_post"].double()
            along = torch.einsum("rc,rc->r", g, unit_f) / c["cols"]
            dn = (g - unit_f * along[:, None]) * r1[:, None]
        out["df"] = dn
    return out
