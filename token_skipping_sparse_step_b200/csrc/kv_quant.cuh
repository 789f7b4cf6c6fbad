// The 4-bit key/value cache: rows of keys and values written into it and read
// back.
//
// Format. Row (b, i) of the cache is position i of sequence b, b * capacity + i
// of a sequence stride of `capacity` rows. A row holds, per key/value head,
// head_dim codes of 4 bits (codes [rows, n_kv, head_dim / 8] 32-bit words) and,
// per group of `group` consecutive dims, a step s and an offset z in bf16
// (scales [rows, n_kv, head_dim / group] pairs, s in the low half). A value
// reads back as
//     (16 + c) s + z,   c in 0..15,
// rounded once to the storage type. 16 + c instead of c costs nothing in the
// grid it spans and drops straight into a bf16 number: 0x4180 | c << 3 is
// 16 + c, so two values take one mask-and-or (the codes of a dim pair lie 16
// bits apart in the word) and one packed multiply-add, with no bias to subtract.
//
// Writing a group (float32 steps, fl = rounding to nearest): lo, hi its
// extremes, t = fl(fl(hi - lo) / 15), z = bf16 below fl(lo - 16 t),
// s = bf16(fl(fl(hi - z) / 31)). z lies at or below lo - 16 t, so the step that
// takes 31 s + z to hi takes 16 s + z to lo or below: the sixteen values span
// the group. c is the whole number nearest to (x - m) / s, m = fl(16 s + z), with
// the difference in float32 and the quotient exact (ties to even), clamped to
// 0..15. A group of equal values has s = 0 and z their value. A group with a NaN
// or an infinity, or whose span overflows, reads back as NaN.
#pragma once

#include "common.cuh"

namespace esd {

struct KvQuant {
  uint32_t* kc;  // codes of the keys and the values
  uint32_t* vc;
  uint32_t* ks;  // their (step, offset) pairs
  uint32_t* vs;
  int n_kv;
  int capacity;
  int group_log2;  // 5, 6 or 7
};

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// bits of the code of dim j (0..7) of a word
__host__ __device__ constexpr int kv_shift(int j) { return 4 * (j >> 1) + 16 * (j & 1); }

__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// the codes of dims 2i and 2i + 1 of a word as the bf16 numbers 16 + c
__device__ __forceinline__ uint32_t kv_code_pair(uint32_t w, int i) {
  const uint32_t x = i == 0 ? w << 3 : w >> (4 * i - 3);
  uint32_t r;
  // one mask-and-or (written out, or the two constants become two operations)
  asm("lop3.b32 %0, %1, 0x00780078, 0x41804180, 0xEA;" : "=r"(r) : "r"(x));
  return r;
}

// The eight values of a word. ss, zz: the step and the offset in both halves
// (bf16), or as float32.
__device__ __forceinline__ void kv_word_bf16(uint32_t w, uint32_t ss, uint32_t zz, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = bf16x2_fma(kv_code_pair(w, i), ss, zz);
}
__device__ __forceinline__ void kv_word_f32(uint32_t w, float s, float z, float (&o)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = fmaf((float)(16u + ((w >> kv_shift(j)) & 15u)), s, z);
}
__device__ __forceinline__ float pair_step(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float pair_offset(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

// The cache row of row j of sequence b of a call with n rows per sequence: its
// position is idx[b n + j], or j without idx. -1 for a padding row (negative
// position), and, with the error flag raised, for a position past the cache.
__device__ __forceinline__ long long kv_cache_row(const int32_t* __restrict__ idx, int r, int n, int capacity,
                                                  int* flag) {
  const int b = r / n;
  const int pos = idx ? idx[r] : r - b * n;
  if (pos < 0) return -1;
  if (pos >= capacity) {
    raise_flag(flag, kFlagCheck);
    return -1;
  }
  return (long long)b * capacity + pos;
}

// ---------------------------------------------------------------------------
// Rows k, v [B n, n_kv hd] (storage type) into the cache. blockIdx.y: keys or
// values. A thread takes 16 consecutive values (its eight bytes of codes), so a
// group is 2, 4 or 8 neighbouring lanes.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
kv_quantize_kernel(const T* __restrict__ k, const T* __restrict__ v, const int32_t* __restrict__ idx, long long total,
                   int n, int per_row, KvQuant cache, int* flag) {
  const long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const bool live = t < total;
  const long long tc = live ? t : total - 1;  // idle lanes repeat the last one: every lane takes part in the shuffles
  const int r = (int)(tc / per_row), c = (int)(tc - (long long)r * per_row);
  const T* src = (blockIdx.y ? v : k) + (size_t)tc * 16;
  float x[16];
  {
    float a[8], b[8];
    load8_stream(src, a);
    load8_stream(src + 8, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = a[i];
      x[8 + i] = b[i];
    }
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
  const int lanes = 1 << (cache.group_log2 - 4);
  for (int o = 1; o < lanes; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float span15 = __fdiv_rn(__fsub_rn(hi, lo), 15.0f);
  const __nv_bfloat16 zb = __float2bfloat16_rd(fmaf(-16.0f, span15, lo));  // 16 t is exact: one rounding
  const float z = __bfloat162float(zb);
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, z), 31.0f));
  const float s = __bfloat162float(sb);
  // |s| and |z| finite, without a NaN (a NaN among the values is one in lo and hi)
  const bool fine = fabsf(s) < INFINITY && fabsf(z) < INFINITY;
  uint32_t pair = 0x7FFF7FFFu;
  uint32_t words[2] = {0, 0};
  if (fine) {
    pair = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(zb) << 16);
    if (s > 0.0f) {
      const float m = fmaf(16.0f, s, z);  // 16 s is exact: one rounding
      // steps near the bottom of the range are scaled up (exactly) so that their reciprocal is finite
      const float up = s < 0x1p-60f ? 0x1p64f : 1.0f;
      const float su = s * up, inv = __frcp_rn(su), half = 0.5f * su;
      // just below half a step: an odd code gives a tie away, an even one keeps it
      const float half_odd = __uint_as_float(__float_as_uint(half) - 1u);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float d = __fsub_rn(x[i], m) * up;
        // the nearest whole number up to the error of the reciprocal, in the low bits of 1.5 2^23 + c
        const float u = fmaf(d, inv, 12582912.0f);
        const float cf = u - 12582912.0f;
        int code = __float_as_int(u) - 0x4B400000;
        // the remainder is exact (c s has 12 bits, and cancels d): it says whether a neighbour is nearer
        const float rem = fmaf(-cf, su, d);
        const float lim = (code & 1) ? half_odd : half;
        code += (rem > lim) - (rem < -lim);
        code = min(max(code, 0), 15);
        words[i >> 3] |= (uint32_t)code << kv_shift(i & 7);
      }
    }
  }
  if (!live) return;
  const long long row = kv_cache_row(idx, r, n, cache.capacity, flag);
  if (row < 0) return;
  // c: which 16 values of the row
  uint32_t* codes = (blockIdx.y ? cache.vc : cache.kc) + ((size_t)row * per_row + c) * 2;
  *reinterpret_cast<uint2*>(codes) = make_uint2(words[0], words[1]);
  if ((c & (lanes - 1)) == 0) {
    uint32_t* sc = blockIdx.y ? cache.vs : cache.ks;
    sc[((size_t)row * per_row + c) >> (cache.group_log2 - 4)] = pair;
  }
}

// ---------------------------------------------------------------------------
// Rows of the cache back into k_out, v_out [B n, n_kv hd] (storage type); zeros
// for a padding row. A thread takes one word (8 values).
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
kv_dequantize_kernel(KvQuant cache, const int32_t* __restrict__ idx, long long total, int n, int per_row,
                     T* __restrict__ k_out, T* __restrict__ v_out, int* flag) {
  const long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= total) return;
  const int r = (int)(t / per_row), c = (int)(t - (long long)r * per_row);
  T* dst = (blockIdx.y ? v_out : k_out) + (size_t)t * 8;
  const long long row = kv_cache_row(idx, r, n, cache.capacity, flag);
  uint32_t w = 0, p = 0;  // s = z = 0: zeros
  if (row >= 0) {
    w = __ldcs((blockIdx.y ? cache.vc : cache.kc) + (size_t)row * per_row + c);
    p = __ldg((blockIdx.y ? cache.vs : cache.ks) + (((size_t)row * per_row + c) >> (cache.group_log2 - 3)));
  }
  if constexpr (sizeof(T) == 2) {
    uint32_t o[4];
    kv_word_bf16(w, __byte_perm(p, p, 0x1010), __byte_perm(p, p, 0x3232), o);
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    float o[8];
    kv_word_f32(w, pair_step(p), pair_offset(p), o);
    Storage<float>::store8(dst, o);
  }
}

}  // namespace esd
