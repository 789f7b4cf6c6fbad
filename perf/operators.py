"""The operators of the 4-bit key/value cache, as cases to time and to compare.

Three operators work on a cache whose keys and values are held in 4 bits:

* writing rows of keys and values into it (``kv_quantize``),
* reading rows back (``kv_dequantize``),
* the attention of a few, some or many query rows per sequence over all of its
  keys (``partial_attention_quantized``).

The cache's format. Per row (position) and key/value head the head's values are
cut into groups of ``group`` consecutive dims. A group holds a step s and an
offset z in bf16 and a code c in 0..15 per value, and a value reads back as
(16 + c) s + z, rounded once to the storage type. Writing a group x, in float32
steps: lo, hi its extremes, z = lo - 16 ((hi - lo) / 15) rounded down to bf16,
s = (hi - z) / 31 rounded to bf16, c = (x - (16 s + z)) / s rounded to the
nearest whole number (ties to even) and clamped to 0..15. A group with a value
that is not finite reads back as NaN.

Codes: eight dims to a 32-bit word, dim 2i of the eight in bits 4i..4i+3 and dim
2i + 1 in bits 16 + 4i..16 + 4i + 3. Steps and offsets: a pair of bf16 each.

With ``own`` false ``run`` computes the same in elementary torch operations.
"""
import functools
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
_SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)  # of the eight dims of a word


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one query of one short sequence, 16 heads: the smallest call of a step, all latency
        _attend("attend-one", 1, 1, 512, heads=16),
        # the first rows to be kept after a skip point, batch 32: the cache is read once for one row each
        _attend("attend-one-batch32", 32, 1, 1536),
        # one row over a long cache whose heads are shared by eight query heads; sequences of very different lengths
        _attend("attend-one-long-shared", 4, 1, 65536, kv=4, group=128, short=0.7),
        # the current block of 64 positions of 32 sequences, padded to the longest
        _attend("attend-block-ragged", 32, 64, 1536, short=0.6),
        # the selected quarter of one sequence of 768 positions
        _attend("attend-selected", 1, 192, 768),
        # a quarter of 16 sequences of 4096 positions: the largest
        _attend("attend-selected-batch16", 16, 1024, 4096, group=128),
        # a float32 model: head_dim 64, odd sizes, one sequence without any key
        _attend("attend-float32", 3, 33, 1001, heads=12, head_dim=64, group=32, dtype="f32", short=0.5, empty=True),
        # the fresh rows of one sparse step go into the cache of one layer
        _cache("write-selected", "write", 1, 192, 768),
        # a dense refresh: every row of 16 sequences
        _cache("write-refresh", "write", 16, 4096, 4096, every=True),
        # a float32 model, odd sizes, padding rows
        _cache("write-float32", "write", 3, 77, 501, heads=4, head_dim=64, group=32, dtype="f32", padding=0.2),
        # the salient rows of 32 sequences are read back
        _cache("read-selected", "read", 32, 384, 1536, group=32, padding=0.1),
        # a whole cache is read back
        _cache("read-all", "read", 16, 4096, 4096, group=128, every=True),
    ]


def _attend(name, batch, rows, length, heads=32, kv=None, head_dim=128, group=64, dtype="bf16", short=0.0, empty=False):
    return {"name": name, "op": "attend", "batch": batch, "rows": rows, "length": length, "capacity": length,
            "heads": heads, "kv_heads": kv or heads, "head_dim": head_dim, "group": group, "dtype": dtype,
            "short": short, "empty": empty}


def _cache(name, op, batch, rows, length, heads=32, head_dim=128, group=64, dtype="bf16", every=False, padding=0.0):
    return {"name": name, "op": op, "batch": batch, "rows": rows, "length": length, "capacity": length,
            "heads": heads, "kv_heads": heads, "head_dim": head_dim, "group": group, "dtype": dtype,
            "every": every, "padding": padding}


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm, odd ones as often as even ones."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    """A case of the ranges above: every operator, type, head layout and group size, lengths 1 to 65536,
    rows 1 to 1024, padded batches, a cache with more room than the sequences use."""
    op = rng.choice(("attend", "attend", "attend", "attend", "write", "read"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if dtype == "f32":
        head_dim = rng.choice((32, 64, 96, 128))
        heads = rng.choice((1, 2, 4, 6, 12))
        most, longest = 1 << 21, 4096
    else:
        head_dim = 128
        heads = rng.choice((4, 8, 16, 28, 32))
        most, longest = 1 << 23, 65536
    group = rng.choice([g for g in (32, 64, 128) if head_dim % g == 0])
    kv = rng.choice([h for h in (heads, heads, heads // 2, heads // 4, heads // 7) if h >= 1 and heads % h == 0])
    batch = _spread(rng, 1, 32)
    length = _spread(rng, 1, min(longest, max(1, most // (32 * batch))))
    capacity = length + rng.choice((0, 0, 1, 37, 128))
    if op == "attend":
        rows = _spread(rng, 1, min(1024, length))
        while batch * rows * length * heads * head_dim > (1 << 36 if dtype == "bf16" else 1 << 31):
            rows = max(1, rows // 2)
        c = _attend("", batch, rows, length, heads, kv, head_dim, group, dtype,
                    short=rng.choice((0.0, 0.3, 0.9)), empty=batch > 1 and rng.random() < 0.2)
    else:
        c = _cache("", op, batch, _spread(rng, 1, length), length, heads, head_dim, group, dtype,
                   every=rng.random() < 0.3, padding=rng.choice((0.0, 0.0, 0.3)))
        c["kv_heads"] = kv
    c["capacity"] = capacity
    del c["name"]
    return c


def _lengths(case, gen):
    """Keys of each sequence: `length` less up to `short` of it; the last one empty where the case says so."""
    b, n = case["batch"], case["length"]
    lens = (n - torch.floor(torch.rand(b, generator=gen, dtype=torch.float64) * case["short"] * n)).to(torch.int32)
    lens[0] = n
    if case["empty"]:
        lens[b - 1] = 0
    return lens


def _generator(case, seed):
    """The host's draws: whole numbers only."""
    gen = torch.Generator()
    gen.manual_seed(1000003 * seed + 7)
    return gen


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    gen = _generator(case, seed)
    dev = torch.Generator(device="cuda")
    dev.manual_seed(seed)
    dtype = BF16 if case["dtype"] == "bf16" else F32
    b, n, cap, kv, hd, g = (case[k] for k in ("batch", "rows", "capacity", "kv_heads", "head_dim", "group"))
    rand = lambda *shape: torch.randn(*shape, generator=dev, device="cuda", dtype=F32)  # noqa: E731
    # keys have a few strong channels, as trained ones do; values are even
    strong = 1 + 3 * (torch.rand(kv, hd, generator=dev, device="cuda") > 0.95).to(F32)
    state = {"case": case}
    if case["op"] != "write":
        codes = torch.empty(2, b, cap, kv, hd // 8, dtype=torch.int32, device="cuda")
        scales = torch.empty(2, b, cap, kv, hd // g, 2, dtype=BF16, device="cuda")
        for i in range(b):
            for j, by in enumerate((strong, 1.0)):
                codes[j, i], scales[j, i] = _pack(*_quantise((rand(cap, kv, hd) * by).to(dtype), g))
    else:
        codes = torch.zeros(2, b, cap, kv, hd // 8, dtype=torch.int32, device="cuda")
        scales = torch.zeros(2, b, cap, kv, hd // g, 2, dtype=BF16, device="cuda")
        state["k"] = (rand(b * n, kv, hd) * strong).to(dtype)
        state["v"] = rand(b * n, kv, hd).to(dtype)
    state["codes"], state["scales"] = codes, scales
    if case["op"] == "attend":
        h = case["heads"]
        state["q"] = rand(b * n, h * hd).to(dtype)
        state["out"] = torch.empty_like(state["q"])
        lens = _lengths(case, gen)
        state["lens"] = lens.cuda() if case["short"] or case["empty"] else None
    else:
        state["idx"] = None if case["every"] else _positions(case, gen).cuda()
        state["k_out"] = torch.empty(b * n, kv * hd, dtype=dtype, device="cuda")
        state["v_out"] = torch.empty_like(state["k_out"])
    if own:
        state["ctx"], state["cache"] = _handle(case, codes, scales)
    return state


def _positions(case, gen):
    """Sorted positions of the rows in each sequence, -1 in the place of the padding rows (the last ones)."""
    b, n = case["batch"], case["rows"]
    idx = torch.stack([torch.sort(torch.randperm(case["length"], generator=gen)[:n])[0] for _ in range(b)]).to(torch.int32)
    pad = torch.floor(torch.rand(b, 1, generator=gen) * case["padding"] * n).to(torch.int32)
    return torch.where(torch.arange(n)[None] >= n - pad, torch.full_like(idx, -1), idx).contiguous()


@functools.lru_cache(maxsize=1)
def _context(heads, head_dim, dtype, batch, length):
    """A model's context with this head geometry (the operators use no weights: two thin layers)."""
    import token_skipping_sparse_step_b200 as esd
    d, f, v = heads * head_dim, 128, 128
    t = BF16 if dtype == "bf16" else F32
    new = lambda *shape: torch.zeros(*shape, dtype=t, device="cuda")  # noqa: E731
    layer = {"wq": new(d, d), "wk": new(d, d), "wv": new(d, d), "wo": new(d, d), "wg": new(f, d), "wu": new(f, d), "wd": new(d, f)}
    dims = esd.make_dims(2, d, heads, head_dim, f, v, v - 1, dtype=dtype)
    run_cfg = esd.make_run(skip_layer=1, max_batch=batch, max_len=length)
    return esd.Context(dims, {"embed": new(v, d), "w_out": new(v, d), "layers": [layer, layer]}, run_cfg)


def _handle(case, codes, scales):
    import token_skipping_sparse_step_b200 as esd
    ctx = _context(case["heads"], case["head_dim"], case["dtype"], case["batch"], case["length"])
    return ctx, esd.KVQuant(codes[0], codes[1], scales[0], scales[1], case["head_dim"])


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    b, n, cap, kv, hd = (case[k] for k in ("batch", "rows", "capacity", "kv_heads", "head_dim"))
    codes, scales = state["codes"], state["scales"]
    if case["op"] == "attend":
        return _attention(state["q"].view(b, n, -1, hd), codes, scales, state["lens"], case["length"]).view(b * n, -1)
    at, valid = _where(state["idx"], b, n, cap, codes.device)
    if case["op"] == "write":
        for j, x in enumerate((state["k"], state["v"])):
            c, s = _pack(*_quantise(x, case["group"]))
            codes[j].view(b * cap, kv, -1)[at[valid]] = c[valid]
            scales[j].view(b * cap, kv, -1, 2)[at[valid]] = s[valid]
    keep = valid[:, None].to(F32)
    return [(_values(codes[j].view(b * cap, kv, -1)[at], scales[j].view(b * cap, kv, -1, 2)[at]).view(b * n, kv * hd) * keep)
            .to(state["k_out"].dtype) for j in (0, 1)]


def _run_own(case, state):
    ctx, cache = state["ctx"], state["cache"]
    b, n = case["batch"], case["rows"]
    if case["op"] == "attend":
        ctx.partial_attention_quantized(state["q"], cache, b, case["length"], n, state["out"], lens=state["lens"])
        return state["out"]
    if case["op"] == "write":
        ctx.kv_quantize(state["k"], state["v"], state["idx"], b, n, cache)
    ctx.kv_dequantize(cache, state["idx"], b, n, state["k_out"], state["v_out"])
    return [state["k_out"], state["v_out"]]


# --------------------------------------------------------------------------
# the plain form
# --------------------------------------------------------------------------
def _where(idx, b, n, cap, device):
    """Rows of the cache [b * cap] of the call's rows, and which of them are no padding."""
    pos = torch.arange(n, device=device).expand(b, n) if idx is None else idx.long()
    at = pos.clamp(min=0) + torch.arange(b, device=device)[:, None] * cap
    return at.reshape(-1), (pos >= 0).reshape(-1)


def _bf16_down(x):
    """x rounded down to bf16."""
    r = x.to(BF16)
    bits = r.view(torch.int16).to(torch.int32)
    below = torch.where(r == 0, torch.full_like(bits, -32767), torch.where(bits < 0, bits + 1, bits - 1)).to(torch.int16).view(BF16)
    return torch.where(r.to(F32) > x, below, r)


def _quantise(x, group):
    """Codes [..., hd] and steps, offsets [..., hd / group] of x [..., hd]."""
    x = x.to(F32).unflatten(-1, (-1, group))
    lo, hi = x.amin(-1), x.amax(-1)
    # (a quotient by a number is taken in 64 bits: in 32 the library multiplies by the reciprocal)
    z = _bf16_down(lo - ((hi - lo).double() / 15).to(F32) * 16)
    s = ((hi - z.to(F32)).double() / 31).to(F32).to(BF16)
    fine = torch.isfinite(s.to(F32)) & torch.isfinite(z.to(F32))
    nan = torch.full_like(s, math.nan)
    s32 = s.to(F32)[..., None]
    d = x - (s32 * 16 + z.to(F32)[..., None])
    # the nearest whole number of the quotient itself: 64 bits next to a border
    c = torch.round(d.double() / s32.double()).clamp(0, 15)
    c = torch.where((s32 > 0) & fine[..., None], c, torch.zeros_like(c)).to(torch.int32)
    return c.flatten(-2), torch.where(fine, s, nan), torch.where(fine, z, nan)


def _pack(c, s, z):
    shifts = torch.tensor(_SHIFTS, dtype=torch.int64, device=c.device)
    words = (c.unflatten(-1, (-1, 8)).long() << shifts).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words)
    return words.to(torch.int32), torch.stack([s, z], -1)


def _values(words, scales):
    """The values of codes [..., hd / 8] and scales [..., hd / group, 2], in float32 before their rounding."""
    shifts = torch.tensor(_SHIFTS, dtype=torch.int32, device=words.device)
    c = ((words[..., None] >> shifts) & 15).flatten(-2).to(F32)
    s, z = scales[..., 0].to(F32)[..., None], scales[..., 1].to(F32)[..., None]
    return ((c.unflatten(-1, (scales.shape[-2], -1)) + 16) * s + z).flatten(-2)


def _attention(q, codes, scales, lens, length):
    """q [b, n, heads, hd] over the cache's first `length` rows, of which a sequence's own are the first lens[b]."""
    b, n, h, hd = q.shape
    out = torch.empty_like(q)
    for i in range(b):
        k, v = (_values(codes[j, i, :length], scales[j, i, :length]).to(q.dtype).to(F32).transpose(0, 1) for j in (0, 1))  # [kv, length, hd]
        qi = q[i].to(F32).unflatten(1, (k.shape[0], -1)).permute(1, 0, 2, 3).flatten(1, 2)  # [kv, n * heads / kv, hd]
        s = qi @ k.transpose(1, 2) / math.sqrt(hd)
        if lens is not None:
            s = s.masked_fill(torch.arange(length, device=s.device) >= lens[i], -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-3e38))
        o = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
        out[i] = o.unflatten(1, (n, -1)).permute(1, 0, 2, 3).flatten(1, 2).to(q.dtype)
    return out


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    """The outputs from the definition: the format's own roundings where it has them, all else in 64 bits."""
    state = prepare(case, seed)
    b, n, cap, kv, hd, g = (case[k] for k in ("batch", "rows", "capacity", "kv_heads", "head_dim", "group"))
    if case["op"] == "attend":
        if b * n * case["length"] * case["heads"] > 1 << 33:
            return None
        q, scale = state["q"].double().view(b, n, kv, -1, hd), hd ** -0.5
        out = torch.zeros(b, n, kv, case["heads"] // kv, hd, dtype=torch.float64, device="cuda")
        for i in range(b):
            own_keys = case["length"] if state["lens"] is None else int(state["lens"][i])
            if not own_keys:
                continue
            for m in range(kv):
                keys, vals = (_exact_values(state["codes"][j, i, :own_keys, m], state["scales"][j, i, :own_keys, m], state["q"].dtype) for j in (0, 1))
                logits = torch.einsum("nhd,ld->nhl", q[i, :, m], keys) * scale
                out[i, :, m] = torch.softmax(logits, -1) @ vals
        return out.view(b * n, -1)
    rows = _where(state["idx"], b, n, cap, "cuda")[0]
    real = torch.ones(b * n, 1, dtype=torch.float64, device="cuda") if state["idx"] is None else (state["idx"].view(-1, 1) >= 0).double()
    result = []
    for j, name in enumerate(("k", "v")):
        if case["op"] == "write":
            parts = [_exact_round_trip(x, g) for x in state[name].split(1 << 12)]
        else:
            words, pairs = state["codes"][j].view(b * cap, kv, -1), state["scales"][j].view(b * cap, kv, -1, 2)
            parts = [_exact_values(words[r], pairs[r], state["k_out"].dtype) for r in rows.split(1 << 12)]
        result.append(torch.cat([p.reshape(p.shape[0], -1) for p in parts]) * real)
    return result


def _exact_values(words, pairs, dtype):
    hd = words.shape[-1] * 8
    c = torch.zeros(*words.shape[:-1], hd, dtype=torch.float64, device=words.device)
    bits = words.long() & 0xFFFFFFFF
    for dim in range(8):
        c[..., dim::8] = ((bits >> (4 * (dim // 2) + 16 * (dim % 2))) % 16).double()
    each = hd // pairs.shape[-2]
    s, z = pairs.double().repeat_interleave(each, dim=-2).unbind(-1)
    return ((16 + c) * s + z).to(dtype).double()


def _exact_round_trip(x, group):
    """What x [rows, heads, hd] reads back as, written and read in 64 bits with the format's roundings made one by one."""
    f32 = lambda t: t.to(F32).double()  # noqa: E731
    v = x.double().unflatten(-1, (-1, group))
    lo, hi = v.min(-1, keepdim=True)[0], v.max(-1, keepdim=True)[0]
    z = f32(lo - 16 * f32(f32(hi - lo) / 15))
    # down to bf16: the low half of the float32's bits goes, away from zero for the negative ones
    bits = z.to(F32).view(torch.int32).long() & 0xFFFFFFFF
    bits = torch.where((bits >= 1 << 31) & (bits % (1 << 16) != 0), bits + (1 << 16), bits) >> 16 << 16
    z = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).view(F32).double()
    s = f32(f32(hi - z) / 31).to(BF16).double()
    t = f32(v - f32(16 * s + z)) / torch.where(s > 0, s, torch.ones_like(s))
    low = torch.floor(t)
    c = low + ((t - low > 0.5) | ((t - low == 0.5) & (low % 2 == 1)))
    c = torch.where(s > 0, c.clamp(0, 15), torch.zeros_like(c))
    return ((16 + c) * s + z).to(x.dtype).double().flatten(-2)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    b, n, kv, hd = (case[k] for k in ("batch", "rows", "kv_heads", "head_dim"))
    row = 2 * kv * (hd // 2 + 4 * hd // case["group"])  # bytes of one position: codes, steps and offsets of K and V
    if case["op"] == "attend":
        keys = b * case["length"] * (1 - case["short"] / 2)
        io = 2 * b * n * case["heads"] * hd * esz
        return {"bytes": keys * row + io, "flops": 4.0 * n * keys * case["heads"] * hd}
    values = b * n * 2 * kv * hd
    if case["op"] == "read":
        return {"bytes": b * n * row + values * esz, "flops": 2.0 * values}
    # a write: the rows are read, their codes written, then read back to return the values they stand for
    return {"bytes": 2 * b * n * row + 2 * values * esz, "flops": 12.0 * values}
