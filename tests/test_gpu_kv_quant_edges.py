"""Edges of the 4-bit key/value cache on the GPU: groups whose grid float32 cannot
resolve, scores that are infinite, calls on one stream without a wait between
them, and the few-row kernel with several heads to a CTA."""
import os
import subprocess
import sys

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
    made = {}

    def get(heads, hd, dtype, max_batch=8, max_len=1024):
        key = (heads, hd, dtype, max_batch, max_len)
        if key not in made:
            dims = synth.ModelDims(n_layers=2, d=heads * hd, n_heads=heads, head_dim=hd, ffn=128, vocab=256, mask_id=255, dtype=dtype)
            made[key] = make_context(dims, synth.RunConfig(skip_layer=1), max_batch, max_len)[0]
        return made[key]

    yield get
    for c in made.values():
        c.close()


def _cache(B, cap, kv, hd, group):
    import token_skipping_sparse_step_b200 as esd
    return esd.KVQuant.empty(B, cap, kv, hd, group)


def _close_groups(hd, group):
    """float32 rows of groups that span a few units in the last place (u) just above a number of 8 bits, where
    16 s + z itself is rounded by several steps: [rows, hd]."""
    rng = np.random.default_rng(group)
    rows = []
    for base in (1.0, -1.0, 1.5, 2.0 ** 20, -(2.0 ** -30), 2.0 ** -55, 3 * 2.0 ** 90):
        u = 2.0 ** (np.floor(np.log2(abs(base))) - 23)
        one = lambda k: base + np.asarray(k) * u
        for k in (*range(0, 36), 63, 64, 255, 4097):
            rows.append(np.full(hd, one(k)))
        rows.append(one(1 + np.arange(hd) % 2))                        # 1, 2, 1, 2 units
        rows.append(one(np.where(np.arange(hd) % group == 5, 32, 23)))  # one value over the top
        for spread in (2, 3, 9, 40, 200):
            for _ in range(12):
                rows.append(one(rng.integers(0, spread, hd) + rng.integers(0, 40)))
    x = np.stack(rows)
    return x.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("hd,group", [(32, 32), (64, 64), (128, 32), (128, 128)])
def test_groups_of_a_few_units_in_the_last_place(contexts, hd, group):
    """float32 rows whose quotients pass 15 (or fall below 0) are clamped, and do not reach their neighbours' codes."""
    ctx = contexts(2, hd, "f32", max_batch=1)
    x = _close_groups(hd, group)
    rows = len(x)
    k, v = np.stack([x, x[::-1]], 1), np.stack([x[::-1], x], 1)       # two heads
    cache = _cache(1, rows, 2, hd, group)
    out = [torch.empty(rows, 2 * hd, device="cuda") for _ in range(2)]
    ctx.kv_quantize(to_gpu(k.reshape(rows, -1), torch.float32), to_gpu(v.reshape(rows, -1), torch.float32), None, 1, rows, cache)
    ctx.kv_dequantize(cache, None, 1, rows, *out)
    ctx.sync_check()
    for x, words, scales, back in ((k, cache.k_codes, cache.k_scales, out[0]), (v, cache.v_codes, cache.v_scales, out[1])):
        c, s, z = Q.quantize(x, group)
        p = scales[0].float().cpu().numpy().astype(np.float64)
        assert np.array_equal(p[..., 0], s) and np.array_equal(p[..., 1], z)
        got = Q.unpack(words[0].cpu().numpy())
        bad = np.flatnonzero((got != c).any((1, 2)))
        assert bad.size == 0, "%d of %d rows, the first: %s for %s" % (bad.size, rows, got[bad[0], 0], c[bad[0], 0])
        assert np.array_equal(back.cpu().numpy().astype(np.float64).reshape(x.shape), Q.values(c, s, z, "f32"))


def _draw(rng, shape, dtype):
    return Q.store(rng.standard_normal(shape) * np.exp(rng.standard_normal((*shape[:-1], 1))), dtype)


def _load(cache, kc, vc):
    """The oracle's (codes, steps, offsets) [B, L, kv, ...] into the first rows of a cache."""
    for words, scales, (c, s, z) in ((cache.k_codes, cache.k_scales, kc), (cache.v_codes, cache.v_scales, vc)):
        L = c.shape[1]
        words[:, :L] = torch.from_numpy(Q.pack(c).view(np.int32)).cuda()
        scales[:, :L] = torch.from_numpy(np.stack([s, z], -1)).to(torch.bfloat16).cuda()


def _attend(ctx, q, cache, L, lens, dtype):
    B, n = q.shape[:2]
    out = torch.full((B * n, q.shape[2] * q.shape[3]), 77.0, dtype=DT[dtype], device="cuda")
    ctx.partial_attention_quantized(to_gpu(q.reshape(B * n, -1), DT[dtype]), cache, B, L, n, out,
                                    lens=None if lens is None else to_gpu(np.asarray(lens), torch.int32))
    ctx.sync_check()
    return out.float().cpu().numpy().astype(np.float64).reshape(q.shape)


@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("bf16", 12), ("bf16", 24), ("bf16", 40), ("bf16", 100), ("bf16", 150),
                                     ("bf16", 300), ("f32", 3), ("f32", 40)])
def test_a_row_whose_scores_are_all_minus_infinity_is_nan(contexts, dtype, n):
    """An infinite query against keys of one sign: the softmax is not defined, and the row must not read as if its
    sequence had no keys (zeros). The other rows and heads are as ever."""
    ctx = contexts(4, 128, dtype)
    rng = np.random.default_rng(n)
    B, L, lens = 3, 600, [600, 130, 0]
    k, v = _draw(rng, (B, L, 4, 128), dtype), _draw(rng, (B, L, 4, 128), dtype)
    k[..., 7] = -np.abs(k[..., 7]) - 16 * np.abs(k).max(-1)     # far below: it reads back negative
    kc, vc = Q.quantize(Q.store(k, dtype), 64), Q.quantize(v, 64)
    kk, vv = Q.values(*kc, dtype), Q.values(*vc, dtype)
    assert (kk[..., 7] < 0).all()
    q = Q.store(rng.standard_normal((B, n, 4, 128)), dtype)
    hit = np.zeros((B, n, 4), bool)
    hit[:, ::3, 1] = hit[:, n - 1, 2] = True
    q[..., 7] = np.where(hit, np.inf, q[..., 7] / 16)
    cache = _cache(B, L, 4, 128, 64)
    _load(cache, kc, vc)
    got = _attend(ctx, q, cache, L, lens, dtype)
    want, tol = Q.attention(np.where(hit[..., None], 0.0, q), kk, vv, lens, dtype)
    assert not got[2].any()                                     # no keys: zeros, whatever the query
    hit[2] = False
    assert np.array_equal(np.isnan(got), np.broadcast_to(hit[..., None], got.shape))
    assert (np.abs(got - want) <= tol)[~hit].all()


@pytest.mark.parametrize("n", [1, 12, 24, 40, 100, 150])
def test_calls_that_feed_each_other_without_a_wait_between_them(contexts, n):
    """Rows written, attended over, the outputs written over the same rows, read back, and attended with: each call may
    start while the one before it ends. The same calls with a wait after each give the same bits."""
    ctx = contexts(4, 128, "bf16")
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    B, L = 1, 500
    first, rows = (rnd(L, 512), rnd(L, 512)), [(rnd(n, 512), rnd(n, 512), rnd(n, 512)) for _ in range(8)]
    idx = torch.arange(0, n, device="cuda", dtype=torch.int32)[None] * (L // n)
    results = []
    for wait in (True, False):
        cache = _cache(B, L, 4, 128, 64)
        outs = [[torch.empty_like(rows[0][0]) for _ in range(4)] for _ in range(40)]
        torch.cuda.synchronize()
        ctx.kv_quantize(*first, None, B, L, cache)
        for i, (o, p, k, v) in enumerate(outs):
            a, b, q = rows[i % 8]
            for call in (lambda: ctx.kv_quantize(a, b, idx, B, n, cache),
                         lambda: ctx.partial_attention_quantized(q, cache, B, L, n, o),
                         lambda: ctx.kv_quantize(o, q, idx, B, n, cache),
                         lambda: ctx.kv_dequantize(cache, idx, B, n, k, v),
                         lambda: ctx.partial_attention_quantized(v, cache, B, L, n, p)):
                call()
                if wait:
                    torch.cuda.synchronize()
        ctx.sync_check()
        results.append((outs, cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales))
    for one, two in zip(results[0][0], results[1][0]):
        assert all(torch.equal(x, y) for x, y in zip(one, two))
    assert all(torch.equal(x, y) for x, y in zip(results[0][1:], results[1][1:]))
    assert not torch.equal(results[0][0][0][0], results[0][0][1][0])    # the rows that were written are attended over


@pytest.mark.parametrize("B,heads,kv,n,group", [(40, 8, 8, 1, 64), (40, 16, 8, 6, 32), (40, 8, 8, 9, 128),      # 2 heads to a CTA
                                                (80, 8, 8, 1, 32), (80, 16, 8, 1, 128), (80, 8, 8, 12, 64),     # 4
                                                (80, 16, 8, 4, 64), (75, 8, 8, 16, 32)])
def test_few_rows_of_many_heads(contexts, B, heads, kv, n, group):
    """From two heads per SM on a CTA of the few-row kernel takes several heads, and fewer slices of the keys."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert B * kv >= 2 * sms
    ctx = contexts(heads, 128, "bf16", max_batch=80, max_len=256)
    rng = np.random.default_rng(B + n)
    L = 200
    lens = rng.integers(0, L + 1, B)
    lens[:6] = [L, 0, 1, 32, 33, 127]
    kc, vc = (Q.quantize(_draw(rng, (B, L, kv, 128), "bf16"), group) for _ in range(2))
    q = Q.store(rng.standard_normal((B, n, heads, 128)), "bf16")
    cache = _cache(B, L + 3, kv, 128, group)
    _load(cache, kc, vc)
    for b in range(B):
        cache.k_scales[b, lens[b]:] = float("nan")
        cache.v_scales[b, lens[b]:] = float("nan")
    got = _attend(ctx, q, cache, L, lens, "bf16")
    want, tol = Q.attention(q, Q.values(*kc, "bf16"), Q.values(*vc, "bf16"), lens, "bf16")
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("heads,hd,group", [(2, 128, 128), (2, 96, 32), (4, 64, 64)])
def test_float32_attention_of_many_rows_over_many_keys(contexts, heads, hd, group):
    """After a float32 context whose head_dim the cache does not take was made."""
    ctx = contexts(heads, hd, "f32")
    contexts(2, 48, "f32", max_batch=2, max_len=64)
    rng = np.random.default_rng(hd)
    B, n, L, lens = 2, 301, 1000, [1000, 897]
    kc, vc = (Q.quantize(_draw(rng, (B, L, heads, hd), "f32"), group) for _ in range(2))
    q = Q.store(rng.standard_normal((B, n, heads, hd)), "f32")
    cache = _cache(B, L, heads, hd, group)
    _load(cache, kc, vc)
    got = _attend(ctx, q, cache, L, lens, "f32")
    want, tol = Q.attention(q, Q.values(*kc, "f32"), Q.values(*vc, "f32"), lens, "f32")
    assert (np.abs(got - want) <= tol).all()


def test_rows_past_2_31_words_are_the_rows_of_a_small_cache(contexts):
    import token_skipping_sparse_step_b200 as esd
    ctx = contexts(16, 128, "bf16", max_batch=80, max_len=128)
    B, cap = 80, 110000
    words = lambda: torch.empty(B, cap, 16, 16, dtype=torch.int32, device="cuda")
    scales = lambda: torch.empty(B, cap, 16, 1, 2, dtype=torch.bfloat16, device="cuda")
    cache, near = esd.KVQuant(words(), words(), scales(), scales(), 128), _cache(B, 1, 16, 128, 128)
    assert cache.k_codes[:-1].numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(B, 2048, generator=g, device="cuda").bfloat16() for _ in range(2))
    ctx.kv_quantize(k, v, torch.full((B, 1), cap - 1, dtype=torch.int32, device="cuda"), B, 1, cache)
    ctx.kv_quantize(k, v, None, B, 1, near)
    for a, b in ((cache.k_codes, near.k_codes), (cache.v_codes, near.v_codes), (cache.k_scales, near.k_scales), (cache.v_scales, near.v_scales)):
        assert torch.equal(a[:, -1], b[:, 0])
    out = [torch.empty(B, 2048, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    ctx.kv_dequantize(cache, torch.full((B, 1), cap - 1, dtype=torch.int32, device="cuda"), B, 1, *out[:2])
    ctx.kv_dequantize(near, None, B, 1, *out[2:])
    ctx.sync_check()
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3]) and not torch.equal(out[0], out[1])


@pytest.mark.parametrize("dtype,n", [("bf16", 4), ("bf16", 12), ("bf16", 24), ("bf16", 40), ("bf16", 100), ("bf16", 300), ("f32", 40)])
def test_query_rows_that_are_not_finite_stay_to_themselves(contexts, dtype, n):
    """NaN in a row, and infinite scores of both signs (softmax of +infinity: NaN); more rows than keys, too."""
    ctx = contexts(4, 128, dtype)
    rng = np.random.default_rng(n)
    B, L, lens = 2, 200, [200, 33]
    kc, vc = (Q.quantize(_draw(rng, (B, L, 4, 128), dtype), 64) for _ in range(2))
    kk, vv = Q.values(*kc, dtype), Q.values(*vc, dtype)
    for b in range(B):
        for h in range(4):
            assert (kk[b, :lens[b], h, 9] > 0).any() and (kk[b, :lens[b], h, 9] < 0).any()
    q = Q.store(rng.standard_normal((B, n, 4, 128)), dtype)
    hit = np.zeros((B, n, 4), bool)
    hit[0, 1, 2] = hit[1, n - 1, 0] = True
    q[0, 1, 2, 100], q[1, n - 1, 0, 9] = np.nan, np.inf
    cache = _cache(B, L, 4, 128, 64)
    _load(cache, kc, vc)
    got = _attend(ctx, q, cache, L, lens, dtype)
    want, tol = Q.attention(np.where(hit[..., None], 0.0, q), kk, vv, lens, dtype)
    assert np.array_equal(np.isnan(got), np.broadcast_to(hit[..., None], got.shape))
    assert (np.abs(got - want) <= tol)[~hit].all()


@pytest.mark.parametrize("dtype,heads,hd,group", [("bf16", 4, 128, 32), ("bf16", 4, 128, 128), ("f32", 2, 64, 64)])
def test_a_position_given_twice_leaves_the_others_right(contexts, dtype, heads, hd, group):
    """What that position itself holds is not said: its codes and steps may come from either row."""
    ctx = contexts(heads, hd, dtype)
    rng = np.random.default_rng(hd)
    n, cap = 300, 400
    k, v = (_draw(rng, (1, n, heads, hd), dtype) for _ in range(2))
    idx = rng.permutation(cap)[:n].astype(np.int32)
    twice = [int(idx[i]) for i in (0, 7, 290)]
    idx[[150, 8, 299]] = twice
    cache = _cache(1, cap, heads, hd, group)
    ctx.kv_quantize(*(to_gpu(x.reshape(n, -1), DT[dtype]) for x in (k, v)), to_gpu(idx[None], torch.int32), 1, n, cache)
    out = [torch.empty(n, heads * hd, dtype=DT[dtype], device="cuda") for _ in range(2)]
    ctx.kv_dequantize(cache, to_gpu(idx[None], torch.int32), 1, n, *out)
    ctx.sync_check()
    alone = ~np.isin(idx, twice)
    assert alone.sum() == n - 6
    for x, o in ((k, out[0]), (v, out[1])):
        back = o.float().cpu().numpy().astype(np.float64).reshape(n, heads, hd)
        assert np.array_equal(back[alone], Q.values(*Q.quantize(x, group), dtype)[0][alone]) and np.isfinite(back).all()
    named = torch.zeros(cap, dtype=torch.bool)
    named[torch.from_numpy(idx).long()] = True
    assert not cache.k_scales[0][~named.cuda()].any() and not cache.v_codes[0][~named.cuda()].any()


FIRST = r"""
import sys
sys.path.insert(0, %r)
import torch
import token_skipping_sparse_step_b200 as esd
n, share = int(sys.argv[1]), int(sys.argv[2])
B, L, kv, group, d = 2, 3239, 28 // share, 32, 28 * 128
new = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
layer = {"wq": new(d, d), "wk": new(d, d), "wv": new(d, d), "wo": new(d, d), "wg": new(128, d), "wu": new(128, d), "wd": new(d, 128)}
ctx = esd.Context(esd.make_dims(2, d, 28, 128, 128, 128, 127, dtype="bf16"), {"embed": new(128, d), "w_out": new(128, d), "layers": [layer, layer]},
                  esd.make_run(skip_layer=1, max_batch=B, max_len=L))
g = torch.Generator(device="cuda").manual_seed(n)
rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
cache = esd.KVQuant.empty(B, L, kv, 128, group)
k, v, q = rnd(B * L, kv * 128), rnd(B * L, kv * 128), rnd(B * n, 28 * 128)
ctx.kv_quantize(k * 2, v, None, B, L, cache)
ctx.kv_dequantize(cache, None, B, L, k, v)
lens = torch.tensor([L, 2744], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
outs = [torch.empty_like(q) for _ in range(6)]
for o in outs:              # the first of them is the kernel's first launch in this process
    ctx.partial_attention_quantized(q, cache, B, L, n, o, lens=lens)
ctx.sync_check()
assert all(torch.equal(outs[0], o) for o in outs[1:]), "not the same bits each time"
# bf16: P and the output are rounded, 2^-8 each; float32 sums as in kvq_oracle.attention
u, e = 2.0 ** -8, 2.0 ** -24
for b in range(B):
    for h in range(28):
        m = int(lens[b])
        kk = k.view(B, L, kv, 128)[b, :m, h // share].double()
        vv = v.view(B, L, kv, 128)[b, :m, h // share].double()
        qq = q.view(B, n, 28, 128)[b, :, h].double()
        p = torch.softmax(qq @ kk.T / 128 ** 0.5, -1)
        want, a = p @ vv, p @ vv.abs()
        size = 1 + (qq.abs() @ kk.abs().T / 128 ** 0.5).amax(-1, keepdim=True)
        tol = u * want.abs() + u * a + 2 * (136 * size + m + 16) * e * a
        assert ((outs[0].view(B, n, 28, 128)[b, :, h].double() - want).abs() <= tol).all(), (b, h)
"""


@pytest.mark.parametrize("n,share", [(88, 1), (40, 1), (24, 1), (200, 1), (9, 1)])
def test_the_first_launch_of_a_process(n, share):
    """Caches of instructions, addresses and data are cold, and warps and copies come at other times than ever after."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % root, str(n), str(share)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype,heads,hd,group", [("bf16", 1, 128, 128), ("bf16", 3, 128, 64), ("bf16", 3, 128, 32), ("f32", 3, 32, 32),
                                                  ("f32", 1, 96, 32), ("f32", 3, 128, 64)])
def test_a_layer_of_one_array_over_all_layers(contexts, dtype, heads, hd, group):
    """Views whose steps and offsets start at a head's pairs, not at 16 bytes: the bits of a cache of its own."""
    import token_skipping_sparse_step_b200 as esd
    ctx = contexts(heads, hd, dtype)
    g = torch.Generator(device="cuda").manual_seed(hd)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[dtype])
    B, cap, L = 1, 331, 317
    codes = torch.zeros(2, 4, B, cap, heads, hd // 8, dtype=torch.int32, device="cuda")
    scales = torch.zeros(2, 4, B, cap, heads, hd // group, 2, dtype=torch.bfloat16, device="cuda")
    assert (hd, group) == (128, 32) or any(t.data_ptr() % 16 for t in scales.flatten(0, 1))
    k, v, idx = rnd(L, heads * hd), rnd(L, heads * hd), torch.arange(L, device="cuda", dtype=torch.int32)[None].contiguous()
    q = rnd(200, heads * hd)
    want = None
    for layer in (None, 0, 1, 2, 3):
        cache = _cache(B, cap, heads, hd, group) if layer is None else esd.KVQuant(codes[0, layer], codes[1, layer], scales[0, layer], scales[1, layer], hd)
        ctx.kv_quantize(k, v, idx, B, L, cache)
        back = [torch.empty_like(k) for _ in range(2)]
        ctx.kv_dequantize(cache, idx, B, L, *back)
        outs = []
        for n in (1, 12, 24, 50, 100, 200):
            outs.append(torch.empty_like(q[:n]))
            ctx.partial_attention_quantized(q[:n], cache, B, L, n, outs[-1])
        ctx.sync_check()
        got = [cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, *back, *outs]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.isfinite(want[-1]).all() and want[-1].any()


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("seed", [0, 1])
def test_calls_in_any_order_without_a_wait(contexts, dtype, hd, seed):
    """Writes, reads, and attention of one to many rows over long and short sequences, on one stream, two caches and
    shared outputs: the bits of the same calls with a wait after each."""
    ctx = contexts(4, hd, dtype, max_batch=2, max_len=3000)
    d = 4 * hd
    results = []
    for wait in (True, False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[dtype])
        rng = np.random.default_rng(seed)
        B, cap = 2, 3000
        caches = [_cache(B, cap, kv, hd, 32) for kv in (4, 2)]
        pool = [rnd(B * cap, d) for _ in range(3)]
        kept = []
        torch.cuda.synchronize()
        for c in caches:
            ctx.kv_quantize(pool[0], pool[1], None, B, cap, c)
        for _ in range(60):
            c = caches[rng.integers(2)]
            n = int(rng.choice([1, 2, 9, 24, 40, 88, 128, 150, 300]))
            idx = to_gpu(np.stack([rng.permutation(cap)[:n] for _ in range(B)]).astype(np.int32), torch.int32)
            lens = to_gpu(rng.integers(0, cap + 1, B).astype(np.int32), torch.int32)
            a, b, o = (pool[i] for i in rng.permutation(3))
            kind = rng.integers(4)
            if kind == 0:
                ctx.kv_quantize(a, b, idx, B, n, c)
            elif kind == 1:
                ctx.kv_dequantize(c, idx, B, n, a, b)
            else:
                ctx.partial_attention_quantized(a, c, B, cap, n, o, lens=None if kind == 2 else lens)
                kept.append(o[:B * n].clone())
            if wait:
                torch.cuda.synchronize()
        ctx.sync_check()
        results.append([*kept, *pool, *(t for c in caches for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales))])
    assert len(kept) > 15
    for x, y in zip(*results):
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))
