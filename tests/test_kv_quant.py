"""The 4-bit key/value cache without a device: the cache holder's checks, and
the oracle of the GPU tests (kvq_oracle) against hand-evaluated groups."""
import ctypes

import numpy as np
import pytest
import torch

import kvq_oracle as Q


def test_calls_without_a_context_are_rejected():
    import token_skipping_sparse_step_b200 as esd
    lib, kv = esd._lib, esd._KVQuantView()
    assert lib.esd_kv_quantize(None, None, None, None, 1, 1, ctypes.byref(kv), None) == 1
    assert lib.esd_kv_dequantize(None, ctypes.byref(kv), None, 1, 1, None, None, None) == 1
    assert lib.esd_partial_attention_quantized(None, None, ctypes.byref(kv), None, 1, 1, 1, None, None) == 1


def test_struct_layout_matches_c(tmp_path):
    import os
    import subprocess

    import token_skipping_sparse_step_b200 as esd
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "sz.c"
    src.write_text('#include "esd.h"\n#include <stdio.h>\n#include <stddef.h>\n'
                   'int main(void){printf("%zu %zu %zu\\n", sizeof(esd_kv_quant), offsetof(esd_kv_quant, n_kv_heads),'
                   ' offsetof(esd_kv_quant, group));return 0;}\n')
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    v = esd._KVQuantView
    assert got == [ctypes.sizeof(v), v.n_kv_heads.offset, v.group.offset]


def _parts(b=2, cap=5, kv=3, hd=64, groups=2):
    return (torch.zeros(b, cap, kv, hd // 8, dtype=torch.int32), torch.zeros(b, cap, kv, hd // 8, dtype=torch.int32),
            torch.zeros(b, cap, kv, groups, 2, dtype=torch.bfloat16), torch.zeros(b, cap, kv, groups, 2, dtype=torch.bfloat16))


def test_the_holder_checks_its_tensors():
    import token_skipping_sparse_step_b200 as esd
    c = esd.KVQuant(*_parts(), 64)
    assert (c.batch, c.capacity, c.n_kv_heads, c.head_dim, c.group) == (2, 5, 3, 64, 32)
    bad = []
    kc, vc, ks, vs = _parts()
    bad.append((kc, vc, ks, vs, 32))                                     # head_dim of other codes
    bad.append((kc.long(), vc, ks, vs, 64))                              # types
    bad.append((kc, vc, ks.float(), vs, 64))
    bad.append((kc, vc, ks, vs[:, :4].contiguous(), 64))                 # shapes
    bad.append((kc, vc[:, :, :2].contiguous(), ks, vs, 64))
    bad.append((kc, vc.transpose(0, 1).contiguous().transpose(0, 1), ks, vs, 64))   # not contiguous
    bad.append((*_parts(hd=64, groups=4)[:2], *_parts(groups=4)[2:], 64))            # groups of 16
    bad.append((kc[0], vc[0], ks[0], vs[0], 64))                         # no batch
    for args in bad:
        with pytest.raises(ValueError):
            esd.KVQuant(*args)
    with pytest.raises(ValueError):
        esd.KVQuant.empty(1, 1, 1, 64, group=48, device="cpu")
    with pytest.raises(ValueError):
        esd.KVQuant.empty(1, 1, 1, 96, group=64, device="cpu")
    e = esd.KVQuant.empty(1, 2, 1, 96, group=32, device="cpu")
    assert e.k_scales.shape == (1, 2, 1, 3, 2) and e.k_codes.shape == (1, 2, 1, 12)


def test_oracle_on_hand_evaluated_groups():
    # 0..15 in steps of one, twice: t = 1, z = -16, s = 31 / 31 = 1: every value is its own code
    x = np.tile(np.arange(16.0), 2)[None, None]
    c, s, z = Q.quantize(x, 32)
    assert s[0, 0, 0] == 1 and z[0, 0, 0] == -16 and np.array_equal(c[0, 0], x[0, 0])
    assert np.array_equal(Q.values(c, s, z, "f32"), x)
    # a tie goes to the even code: 0.5 -> 0, 1.5 -> 2, 2.5 -> 2
    x[0, 0, 16:19] = [0.5, 1.5, 2.5]
    assert list(Q.quantize(x, 32)[0][0, 0, 16:19]) == [0, 2, 2]
    # equal values: s = 0 and z the value
    c, s, z = Q.quantize(np.full((1, 1, 32), -3.25), 32)
    assert s[0, 0, 0] == 0 and z[0, 0, 0] == -3.25 and not c.any()
    # one value that is not finite spoils its group only
    x = np.tile(np.arange(16.0), 4)[None, None]
    x[0, 0, 40] = np.inf
    c, s, z = Q.quantize(x, 32)
    assert np.isnan(s[0, 0, 1]) and np.isnan(z[0, 0, 1]) and s[0, 0, 0] == 1
    # the word layout: dim 2i in bits 4i, dim 2i + 1 in bits 16 + 4i
    assert Q.pack(np.arange(8)[None, None])[0, 0, 0] == 0x7531_6420


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_oracle_error_is_at_most_about_half_a_step(dtype, group):
    """|x - value| <= (1/2 + 1/8) s + the storage rounding: half a step within the grid; at its ends the roundings of
    s (2^-9 of up to 31 steps, 0.06) and of the storage type add less than an eighth."""
    rng = np.random.default_rng(3)
    x = Q.store(rng.standard_normal((50, 2, 128)) * np.exp(rng.standard_normal((50, 2, 1)) * 3) + rng.standard_normal((50, 1, 1)), dtype)
    c, s, z = Q.quantize(x, group)
    v = Q.values(c, s, z, dtype)
    step = np.repeat(s, group, axis=-1)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert (np.abs(x - v) <= 0.625 * step + half * np.abs(v)).all()
