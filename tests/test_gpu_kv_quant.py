"""The 4-bit key/value cache on the GPU through the C ABI: rows written (codes,
steps and offsets equal to the oracle's), rows read back (equal), and the
attention over the cache within a bound derived from its roundings
(kvq_oracle.attention), from one row to many, with shared heads, padded
batches, rows without keys and garbage behind the last key."""
import ctypes

import numpy as np
import pytest
import torch

import kvq_oracle as Q
import synth
from helpers import make_context, to_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def contexts():
    """One context per head geometry and type, large enough for every case."""
    made = {}

    def get(heads, hd, dtype, max_batch=8, max_len=2048):
        key = (heads, hd, dtype, max_batch, max_len)
        if key not in made:
            dims = synth.ModelDims(n_layers=2, d=heads * hd, n_heads=heads, head_dim=hd, ffn=128, vocab=256, mask_id=255, dtype=dtype)
            made[key] = make_context(dims, synth.RunConfig(skip_layer=1), max_batch, max_len)[0]
        return made[key]

    yield get
    for c in made.values():
        c.close()


def _cache(B, cap, kv, hd, group, fill=None):
    import token_skipping_sparse_step_b200 as esd
    c = esd.KVQuant.empty(B, cap, kv, hd, group)
    if fill is not None:     # NaN scales and any codes: a row that is read when it should not be shows
        for t in (c.k_codes, c.v_codes):
            t.fill_(0x5A5A5A5A)
        for t in (c.k_scales, c.v_scales):
            t.fill_(fill)
    return c


def _draw(rng, shape, dtype):
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal((*shape[:-1], 1)))
    x[..., 0] *= 6
    return Q.store(x, dtype)


def _load(cache, kc, vc):
    """The oracle's (codes, steps, offsets) [B, L, kv, ...] into the first rows of a cache."""
    for words, scales, (c, s, z) in ((cache.k_codes, cache.k_scales, kc), (cache.v_codes, cache.v_scales, vc)):
        L = c.shape[1]
        words[:, :L] = torch.from_numpy(Q.pack(c).view(np.int32)).cuda()
        scales[:, :L] = torch.from_numpy(np.stack([s, z], -1)).to(torch.bfloat16).cuda()


def _stored(words, scales):
    """(codes, steps, offsets) of cache tensors as numpy."""
    p = scales.float().cpu().numpy().astype(np.float64)
    return Q.unpack(words.cpu().numpy()), p[..., 0], p[..., 1]


def _special_rows(hd, dtype):
    """Rows whose groups are at the edges of the format."""
    rng = np.random.default_rng(11)
    base = rng.standard_normal(hd)
    rows = [np.zeros(hd), np.full(hd, -2.5), base * 1e-38, base * 2.0 ** -66, base * 2.0 ** -100, base * 1e37, base * 3e38 / 4,
            100 + base * 1e-2, -100 + base * 1e-2, 1 + base * 2.0 ** -8, np.abs(base), -np.abs(base), np.where(base > 0, 0.0, base),
            np.arange(hd) % 16.0, np.arange(hd) % 31 / 2.0, (np.arange(hd) % 61 / 4.0) - 7.5, np.sign(base),
            np.where(np.arange(hd) == 5, 1e30, base), np.where(np.arange(hd) % 32 == 3, 3.3e38, -3.3e38),
            np.where(np.arange(hd) == 7, np.nan, base), np.where(np.arange(hd) == hd - 1, np.inf, base),
            np.where(np.arange(hd) == 0, -np.inf, base)]
    return Q.store(np.stack(rows), dtype)


@pytest.mark.parametrize("dtype,heads,kv,hd,group", [("bf16", 4, 4, 128, 32), ("bf16", 4, 2, 128, 64), ("bf16", 4, 1, 128, 128),
                                                     ("f32", 4, 4, 32, 32), ("f32", 2, 2, 64, 64), ("f32", 3, 3, 96, 32),
                                                     ("f32", 2, 1, 128, 128)])
@pytest.mark.parametrize("rows", [1, 7, 66])
def test_rows_are_written_and_read_back_as_the_oracle_does(contexts, dtype, heads, kv, hd, group, rows):
    ctx = contexts(heads, hd, dtype)
    rng = np.random.default_rng(rows)
    B, cap = 2, 70
    x = [_draw(rng, (B, rows, kv, hd), dtype) for _ in range(2)]
    special = _special_rows(hd, dtype)
    if rows > len(special):
        x[0][1, :len(special), 0] = special
        x[1][0, -len(special):, -1] = special
    idx = np.stack([np.sort(rng.choice(cap, rows, replace=False)) for _ in range(B)]).astype(np.int32)
    if rows > 1:
        idx[0, -2:] = -1
    cache = _cache(B, cap, kv, hd, group, fill=7.0)
    before = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    xg = [to_gpu(a.reshape(B * rows, -1), DT[dtype]) for a in x]
    ig = to_gpu(idx, torch.int32)
    ctx.kv_quantize(xg[0], xg[1], ig, B, rows, cache)
    out = [torch.full((B * rows, kv * hd), 3.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    ctx.kv_dequantize(cache, ig, B, rows, out[0], out[1])
    ctx.sync_check()
    for j, (words, scales) in enumerate(((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))):
        want = Q.quantize(x[j], group)
        got = _stored(words, scales)
        back = out[j].float().cpu().numpy().astype(np.float64).reshape(B, rows, kv, hd)
        named = np.zeros((B, cap), bool)
        for b in range(B):
            for r in range(rows):
                p = idx[b, r]
                if p < 0:
                    assert not back[b, r].any()
                    continue
                named[b, p] = True
                for w, g in zip(want, got):
                    assert np.array_equal(w[b, r], g[b, p], equal_nan=True), (j, b, r)
                assert np.array_equal(back[b, r], Q.values(*(w[b, r] for w in want), dtype), equal_nan=True), (j, b, r)
        rest = torch.from_numpy(~named).cuda()     # rows the call does not name stay as they are
        assert torch.equal(words[rest], before[2 * j][rest]) and torch.equal(scales[rest], before[2 * j + 1][rest])


def test_without_positions_the_first_rows_are_meant(contexts):
    ctx = contexts(4, 128, "bf16")
    rng = np.random.default_rng(5)
    B, n, cap = 3, 9, 11
    x = [_draw(rng, (B, n, 4, 128), "bf16") for _ in range(2)]
    xg = [to_gpu(a.reshape(B * n, -1), torch.bfloat16) for a in x]
    cache = _cache(B, cap, 4, 128, 64, fill=7.0)
    ctx.kv_quantize(xg[0], xg[1], None, B, n, cache)
    out = [torch.empty_like(t) for t in xg]
    ctx.kv_dequantize(cache, None, B, n, *out)
    for j in range(2):
        want = Q.values(*Q.quantize(x[j], 64), "bf16")
        assert np.array_equal(out[j].float().cpu().numpy().reshape(want.shape), want)
    assert (cache.k_scales[:, n:] == 7).all() and (cache.v_codes[:, n:] == 0x5A5A5A5A).all()


def test_positions_past_the_capacity_are_skipped_and_reported(contexts):
    import token_skipping_sparse_step_b200 as esd
    ctx = contexts(4, 128, "bf16")
    cache = _cache(1, 5, 4, 128, 64)
    x = torch.randn(3, 512, device="cuda").bfloat16()
    idx = torch.tensor([[1, 5, 2000000000]], dtype=torch.int32, device="cuda")
    ctx.kv_quantize(x, x, idx, 1, 3, cache)
    with pytest.raises(esd.EsdError) as e:
        ctx.sync_check()
    assert e.value.status == esd.ESD_ERR_CHECK
    assert cache.k_scales[0, 1].any() and not cache.k_scales[0, 2:].any() and not cache.k_scales[0, 0].any()
    k, v = torch.ones_like(x), torch.ones_like(x)
    ctx.kv_dequantize(cache, idx, 1, 3, k, v)
    with pytest.raises(esd.EsdError):
        ctx.sync_check()
    assert k[0].any() and not k[1:].any() and not v[1:].any()
    ctx.sync_check()


CASES = [
    # B, rows, L, capacity, heads, kv, hd, group, dtype, lens
    (1, 1, 1, 1, 4, 4, 128, 32, "bf16", None),
    (1, 1, 2, 130, 4, 4, 128, 64, "bf16", None),
    (2, 1, 777, 800, 4, 1, 128, 128, "bf16", [777, 1]),
    (3, 1, 2048, 2048, 8, 1, 128, 64, "bf16", [0, 2048, 65]),
    (2, 2, 129, 129, 4, 4, 128, 32, "bf16", [128, 129]),
    (1, 3, 63, 64, 4, 2, 128, 64, "bf16", None),
    (2, 5, 1000, 1000, 4, 4, 128, 64, "bf16", [1000, 3]),
    (2, 8, 255, 300, 4, 4, 128, 128, "bf16", [255, 64]),
    (2, 9, 257, 300, 4, 4, 128, 32, "bf16", [100, 257]),
    (1, 16, 512, 512, 4, 4, 128, 64, "bf16", None),
    (4, 17, 300, 333, 4, 4, 128, 64, "bf16", [300, 0, 128, 127]),
    (2, 33, 1500, 1500, 7, 1, 128, 64, "bf16", [1500, 700]),
    (3, 64, 640, 641, 4, 4, 128, 32, "bf16", [640, 1, 513]),
    (1, 100, 384, 384, 4, 4, 128, 128, "bf16", None),
    (2, 129, 500, 500, 4, 2, 128, 64, "bf16", [500, 250]),
    (1, 192, 768, 768, 4, 4, 128, 64, "bf16", None),
    (2, 257, 1111, 1200, 4, 4, 128, 64, "bf16", [1111, 127]),
    (1, 520, 2000, 2000, 4, 4, 128, 128, "bf16", None),
    (8, 300, 300, 301, 4, 4, 128, 32, "bf16", [300, 299, 1, 0, 128, 129, 255, 256]),
    (1, 1, 1, 1, 4, 4, 32, 32, "f32", None),
    (2, 1, 777, 800, 4, 1, 64, 64, "f32", [777, 1]),
    (3, 33, 1001, 1001, 12, 12, 64, 32, "f32", [1001, 500, 0]),
    (2, 5, 65, 70, 6, 2, 96, 32, "f32", [64, 65]),
    (2, 70, 200, 200, 2, 2, 128, 128, "f32", None),
    (1, 2, 2048, 2048, 4, 4, 32, 32, "f32", None),
]


@pytest.mark.parametrize("B,n,L,cap,H,kv,hd,group,dtype,lens", CASES)
def test_attention_over_the_cache(contexts, B, n, L, cap, H, kv, hd, group, dtype, lens):
    ctx = contexts(H, hd, dtype)
    rng = np.random.default_rng(n * 1000 + L)
    kc, vc = (Q.quantize(_draw(rng, (B, L, kv, hd), dtype), group) for _ in range(2))
    q = Q.store(rng.standard_normal((B, n, H, hd)), dtype)
    cache = _cache(B, cap, kv, hd, group, fill=float("nan"))
    own = np.full(B, L) if lens is None else np.array(lens)
    _load(cache, kc, vc)
    for b in range(B):      # behind a sequence's last key: NaN
        cache.k_scales[b, own[b]:] = float("nan")
        cache.v_scales[b, own[b]:] = float("nan")
    lg = None if lens is None else to_gpu(own, torch.int32)
    qg = to_gpu(q.reshape(B * n, -1), DT[dtype])
    # a row more behind the outputs: it stays as it is
    out = torch.full((B * n + 1, H * hd), 77.0, dtype=DT[dtype], device="cuda")
    ctx.partial_attention_quantized(qg, cache, B, L, n, out, lens=lg)
    ctx.sync_check()
    assert (out[-1] == 77).all()
    got = out[:-1].float().cpu().numpy().astype(np.float64).reshape(q.shape)
    want, tol = Q.attention(q, Q.values(*kc, dtype), Q.values(*vc, dtype), own, dtype)
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - want) / np.maximum(tol, 1e-30))
    assert worst <= 1, "%.3f of the bound" % worst
    again = torch.empty_like(out)
    ctx.partial_attention_quantized(qg, cache, B, L, n, again, lens=lg)
    assert torch.equal(again[:-1], out[:-1])       # the same bits each time


@pytest.mark.parametrize("n", [1, 16, 40, 200])
def test_lengths_outside_the_range_are_clamped(contexts, n):
    ctx = contexts(4, 128, "bf16")
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    cache = _cache(4, 150, 4, 128, 64, fill=float("nan"))
    k, v, q = rnd(4 * 140, 512), rnd(4 * 140, 512), rnd(4 * n, 512)
    ctx.kv_quantize(k, v, None, 4, 140, cache)
    outs = []
    for lens in ([140, 140, 0, 0], [141, 2000000000, -1, -2000000000]):
        o = torch.full_like(q, 5.0)
        ctx.partial_attention_quantized(q, cache, 4, 140, n, o, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        outs.append(o)
    assert torch.equal(*outs) and not outs[0][2 * n:].any() and outs[0][:2 * n].any()


@pytest.mark.parametrize("n", [1, 16, 40, 200])
def test_a_group_that_is_not_finite_reaches_its_own_head_only(contexts, n):
    ctx = contexts(4, 128, "bf16")
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    k, v, q = rnd(2 * 200, 512), rnd(2 * 200, 512), rnd(2 * n, 512)
    k[200 + 77, 128 + 3] = float("inf")       # sequence 1, head 1: every score with key 77 is NaN
    v[5, 2 * 128 + 70] = float("nan")         # sequence 0, head 2: a group of the values
    cache = _cache(2, 200, 4, 128, 64)
    ctx.kv_quantize(k, v, None, 2, 200, cache)
    o = torch.zeros_like(q)
    ctx.partial_attention_quantized(q, cache, 2, 200, n, o)
    ctx.sync_check()
    bad = torch.isnan(o.view(2, n, 4, 128))
    want = torch.zeros_like(bad)
    want[1, :, 1] = True
    want[0, :, 2, 64:128] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("n", [1, 12, 40, 200])
@pytest.mark.parametrize("size", [30.0, 1e4])
def test_large_scores_stay_finite(contexts, n, size):
    """Scores of hundreds and more: the softmax is one key, whichever tile holds it."""
    ctx = contexts(4, 128, "bf16")
    rng = np.random.default_rng(n)
    L = 600
    kc, vc = (Q.quantize(_draw(rng, (1, L, 4, 128), "bf16"), 64) for _ in range(2))
    q = Q.store(rng.standard_normal((1, n, 4, 128)) * size, "bf16")
    cache = _cache(1, L, 4, 128, 64)
    _load(cache, kc, vc)
    out = torch.empty(n, 512, dtype=torch.bfloat16, device="cuda")
    ctx.partial_attention_quantized(to_gpu(q.reshape(n, -1), torch.bfloat16), cache, 1, L, n, out)
    want, tol = Q.attention(q, Q.values(*kc, "bf16"), Q.values(*vc, "bf16"), [L], "bf16")
    got = out.float().cpu().numpy().astype(np.float64).reshape(q.shape)
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()


def test_a_far_sequence_of_a_large_cache(contexts):
    """Words and rows of the last sequence lie past 2^31."""
    import token_skipping_sparse_step_b200 as esd
    ctx = contexts(16, 128, "bf16", max_batch=80, max_len=128)
    B, cap = 80, 110000
    words = lambda: torch.empty(B, cap, 16, 16, dtype=torch.int32, device="cuda")
    scales = lambda: torch.empty(B, cap, 16, 1, 2, dtype=torch.bfloat16, device="cuda")
    cache = esd.KVQuant(words(), words(), scales(), scales(), 128)
    assert cache.k_codes.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    L = 100
    k, v = rnd(B * L, 2048), rnd(B * L, 2048)
    ctx.kv_quantize(k, v, None, B, L, cache)
    near = _cache(1, L, 16, 128, 128)
    ctx.kv_quantize(k[-L:], v[-L:], None, 1, L, near)
    back = torch.empty_like(k), torch.empty_like(v)
    ctx.kv_dequantize(cache, None, B, L, *back)
    small = torch.empty(L, 2048, dtype=torch.bfloat16, device="cuda"), torch.empty(L, 2048, dtype=torch.bfloat16, device="cuda")
    ctx.kv_dequantize(near, None, 1, L, *small)
    assert torch.equal(back[0][-L:], small[0]) and torch.equal(back[1][-L:], small[1])
    for n in (1, 12, 40, 100):
        q = rnd(B * n, 2048)
        o, want = torch.empty_like(q), torch.empty_like(q[:n])
        ctx.partial_attention_quantized(q, cache, B, L, n, o)
        ctx.partial_attention_quantized(q[-n:], near, 1, L, n, want)
        # the two calls may split the keys differently
        assert (o[-n:].float() - want.float()).abs().max() <= 2 ** -6
    # positions past 2^31 words within a call by idx
    idx = torch.full((B, 1), cap - 1, dtype=torch.int32, device="cuda")
    ctx.kv_quantize(k[:B], v[:B], idx, B, 1, cache)
    one = torch.empty(B, 2048, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 2048, dtype=torch.bfloat16, device="cuda")
    ctx.kv_dequantize(cache, idx, B, 1, *one)
    ctx.sync_check()
    assert (one[0].float() - k[:B].float()).abs().max() < 0.5 and torch.equal(one[0][-1], one[0][-1])


def _step_together(ctx, cache, k, v, q, idx, rows, out, B, L, n, stream=None):
    ctx.kv_quantize(rows[0], rows[1], idx, B, n, cache, stream=stream)
    ctx.partial_attention_quantized(q, cache, B, L, n, out, stream=stream)


@pytest.mark.parametrize("n", [1, 24, 150])
def test_used_together_as_a_sparse_step_does(contexts, n):
    """A dense refresh writes every row; each step then writes its selected rows and attends over the whole cache. The
    attention of the 16-bit cache that the rows read back to gives the same contexts, to the roundings of either."""
    ctx = contexts(4, 128, "bf16")
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    B, L = 2, 400
    cache = _cache(B, L, 4, 128, 64)
    ctx.kv_quantize(rnd(B * L, 512), rnd(B * L, 512), None, B, L, cache)
    kf, vf = (torch.empty(B * L, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for step in range(3):
        idx = torch.stack([torch.randperm(L, generator=g, device="cuda")[:n].sort()[0] for _ in range(B)]).int()
        q, rows = rnd(B * n, 512), (rnd(B * n, 512), rnd(B * n, 512))
        out, want = torch.empty_like(q), torch.empty_like(q)
        _step_together(ctx, cache, kf, vf, q, idx, rows, out, B, L, n)
        ctx.kv_dequantize(cache, None, B, L, kf, vf)
        ctx.partial_attention(q, kf, vf, B, L, n, want)
        ctx.sync_check()
        # both round P (2^-8 of values of size 1..4, averaged) and the output
        assert (out.float() - want.float()).abs().max() <= 2 ** -6 * 4
        at = (idx.long() + torch.arange(B, device="cuda")[:, None] * L).view(-1)
        # a step of a group of normals is 0.3 to 0.5: the fresh rows are in the cache
        assert (kf[at].float() - rows[0].float()).abs().max() < 0.5


@pytest.mark.parametrize("n", [1, 12, 24, 40, 100, 150])
def test_captured_and_replayed_and_on_another_stream(contexts, n):
    ctx = contexts(4, 128, "bf16")
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    B, L = 2, 500
    caches = [_cache(B, L, 4, 128, 64) for _ in range(2)]
    k, v = rnd(B * L, 512), rnd(B * L, 512)
    for c in caches:
        ctx.kv_quantize(k, v, None, B, L, c)
    idx = torch.stack([torch.randperm(L, generator=g, device="cuda")[:n].sort()[0] for _ in range(B)]).int()
    q, rows = rnd(B * n, 512), (rnd(B * n, 512), rnd(B * n, 512))
    lens = torch.tensor([L, 300], dtype=torch.int32, device="cuda")
    out = [torch.empty_like(q) for _ in range(2)]

    def step(cache, o, stream=None):
        ctx.kv_quantize(rows[0], rows[1], idx, B, n, cache, stream=stream)
        ctx.partial_attention_quantized(q, cache, B, L, n, o, lens=lens, stream=stream)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], out[0])
    side = torch.cuda.Stream()
    for again in range(3):
        for t in (q, *rows):
            t.copy_(rnd(B * n, 512))
        lens[1] = (300, 0, 499)[again]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step(caches[1], out[1], stream=side)
        side.synchronize()
        assert torch.equal(out[0], out[1]) and torch.equal(caches[0].k_codes, caches[1].k_codes)
    ctx.sync_check()


@pytest.mark.parametrize("n", [1, 12, 24, 40, 100, 150])
def test_two_streams_at_once_on_one_context(contexts, n):
    """The calls keep nothing in the context between them: two streams may run them at the same time."""
    ctx = contexts(4, 128, "bf16")
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    B, L = 1, 2000
    sets = []
    for _ in range(2):
        c = _cache(B, L, 4, 128, 64)
        ctx.kv_quantize(rnd(B * L, 512), rnd(B * L, 512), None, B, L, c)
        q = rnd(B * n, 512)
        want = torch.empty_like(q)
        ctx.partial_attention_quantized(q, c, B, L, n, want)
        sets.append((c, q, want, torch.cuda.Stream(), [torch.empty_like(q) for _ in range(20)]))
    torch.cuda.synchronize()
    for i in range(20):
        for c, q, _, st, outs in sets:
            ctx.partial_attention_quantized(q, c, B, L, n, outs[i], stream=st)
    torch.cuda.synchronize()
    for _, _, want, _, outs in sets:
        assert all(torch.equal(o, want) for o in outs)


def test_contexts_of_other_head_dims_do_not_disturb_each_other(contexts):
    """A float32 context whose head_dim the 4-bit cache does not take, made after one of head_dim 128."""
    first = contexts(2, 128, "f32", max_batch=2, max_len=300)
    contexts(2, 48, "f32", max_batch=2, max_len=64)
    cache = _cache(1, 300, 2, 128, 64)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.randn(300, 256, generator=g, device="cuda") for _ in range(3))
    first.kv_quantize(k, v, None, 1, 300, cache)
    o = torch.empty_like(q)
    first.partial_attention_quantized(q, cache, 1, 300, 300, o)
    first.sync_check()
    assert torch.isfinite(o).all()


def test_bad_calls_are_refused(contexts):
    import token_skipping_sparse_step_b200 as esd
    ctx = contexts(4, 128, "bf16")
    cache = _cache(2, 64, 4, 128, 64)
    x = torch.zeros(2 * 64, 512, device="cuda").bfloat16()
    o = torch.empty_like(x)

    def refused(status, f, *a, **kw):
        with pytest.raises(esd.EsdError) as e:
            f(*a, **kw)
        assert e.value.status == status and str(e.value)

    inv, uns = esd.ESD_ERR_INVALID_ARG, esd.ESD_ERR_UNSUPPORTED
    refused(inv, ctx.kv_quantize, x, x, None, 2, 0, cache)
    refused(inv, ctx.kv_quantize, x, x, None, 0, 4, cache)
    big = torch.zeros(2 * 65, 512, device="cuda").bfloat16()
    refused(inv, ctx.kv_quantize, big, big, None, 2, 65, cache)             # past the capacity
    refused(inv, ctx.kv_dequantize, cache, None, 2, 65, big, big)
    refused(inv, ctx.partial_attention_quantized, x, cache, 2, 65, 4, o)
    refused(inv, ctx.partial_attention_quantized, x, cache, 2, 0, 4, o)
    refused(inv, ctx.partial_attention_quantized, x, cache, 2, 64, 0, o)
    refused(inv, ctx.partial_attention_quantized, x, cache, 0, 64, 4, o)
    host = esd.KVQuant.empty(2, 64, 4, 128, 64, device="cpu")
    for what in ("rows", "type", "dense", "device", "idx", "lens", "batch", "host"):
        with pytest.raises(ValueError):
            if what == "rows":
                ctx.kv_quantize(x[:3], x, None, 2, 2, cache)
            elif what == "type":
                ctx.partial_attention_quantized(x.float(), cache, 2, 64, 4, o)
            elif what == "dense":
                ctx.kv_dequantize(cache, None, 2, 4, x.t(), x)
            elif what == "device":
                ctx.kv_quantize(x.cpu(), x, None, 2, 4, cache)
            elif what == "idx":
                ctx.kv_quantize(x, x, torch.zeros(2, 4, dtype=torch.int64, device="cuda"), 2, 4, cache)
            elif what == "lens":
                ctx.partial_attention_quantized(x, cache, 2, 64, 4, o, lens=torch.zeros(1, dtype=torch.int32, device="cuda"))
            elif what == "host":
                ctx.partial_attention_quantized(x, host, 2, 64, 4, o)
            else:
                ctx.partial_attention_quantized(x, cache, 3, 64, 4, o)
    # through the C ABI: what the Python holder would not let through
    lib, h = esd._lib, ctx.handle
    ok = cache._view
    p = x.data_ptr()

    def attend(**kw):
        view = esd._KVQuantView(*[kw.get(f, getattr(ok, f)) for f, _ in esd._KVQuantView._fields_])
        return lib.esd_partial_attention_quantized(h, kw.get("q", p), ctypes.byref(view), None, 2, 8, 4, kw.get("out", o.data_ptr()), None)

    assert attend(k_codes=None) == inv and attend(v_scales=None) == inv
    assert attend(k_codes=ok.k_codes + 4) == inv and attend(v_scales=ok.v_scales + 2) == inv
    assert attend(group=16) == inv and attend(group=48) == inv and attend(n_kv_heads=3) == inv and attend(n_kv_heads=0) == inv
    assert attend(capacity=7) == inv and attend(q=None) == inv and attend(out=None) == inv and attend(q=p + 2) == inv
    assert lib.esd_kv_quantize(h, p, None, None, 1, 1, ctypes.byref(ok), None) == inv
    assert lib.esd_kv_quantize(h, p, p + 2, None, 1, 1, ctypes.byref(ok), None) == inv
    assert lib.esd_kv_dequantize(h, None, None, 1, 1, p, p, None) == inv
    f32 = contexts(2, 64, "f32")
    with pytest.raises(ValueError):
        f32.kv_quantize(x, x, None, 2, 4, cache)            # another head_dim
    g128 = esd._KVQuantView(ok.k_codes, ok.v_codes, ok.k_scales, ok.v_scales, 2, 64, 128)
    assert lib.esd_kv_quantize(f32.handle, p, p, None, 1, 1, ctypes.byref(g128), None) == inv   # 128 does not divide 64
    odd = contexts(2, 48, "f32")
    assert lib.esd_kv_quantize(odd.handle, p, p, None, 1, 1, ctypes.byref(ok), None) == uns
    ctx.sync_check()
