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
// the group, but for the rounding of s (2^-9 of up to 31 steps, 0.06 s). c is the
// whole number nearest to (x - m) / s, m = fl(16 s + z), with the difference in
// float32 and the quotient exact (ties to even), clamped to 0..15: float32 groups of
// a few units in the last place have steps below the rounding of m, and quotients up
// to 16. A group of equal values has s = 0 and z their value where that is a bf16
// number. A group with a NaN or an infinity, or with an offset that bf16 does not
// hold (a span of 2.4e38 can do), reads back as NaN.
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

// packed pairs of float32
__device__ __forceinline__ uint64_t pack_f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack_f2(uint64_t a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// The cache row of row r = b n + j of a call with n rows per sequence: its
// position is idx[r], or j without idx. -1 for a padding row (negative position),
// and, with the error flag raised, for a position past the cache.
__device__ __forceinline__ long long kv_cache_row(const int32_t* idx, int r, int n, int capacity,
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

// Both kernels below: a block takes `rpb` whole rows of the call, cut into items
// (16 values to write, 8 to read back) in the order of memory. Which row an item is
// in takes one high product: i < 2^16 and per_row <= 2^16 make it exact.
//
// These kernels and the attention kernels over the cache may start before the kernel
// ahead of them ends, which may be the one that writes what they read. They wait for
// it, and read by plain loads (or asynchronous copies) alone: the read-only path
// (__ldg, or const __restrict__ parameters) is for data that nobody writes while the
// kernel lives. It costs nothing but 1% of the shortest (192 rows x 768 keys attended
// over: 18.5 -> 18.7 us).
constexpr int kKvThreads = 256, kKvItems = 2048;  // items of a block, unless a row alone has more
__device__ __forceinline__ int kv_row_of(int i, uint32_t magic) { return (int)__umulhi((uint32_t)i, magic); }

// ---------------------------------------------------------------------------
// Rows k, v [B n, n_kv hd] (storage type) into the cache. blockIdx.y: keys or
// values. An item is 16 consecutive values (eight bytes of codes), so a group is
// 2, 4 or 8 neighbouring lanes.
//
// Per value the quotient is taken as a product with the reciprocal, rounded by
// adding 1.5 2^23, and then set right by its exact remainder x - m - c s (c s has 12
// bits and cancels): more than half a step away, or half a step from an odd code,
// the neighbour on that side is the nearest. Of bf16 values m is exact (their span is
// at least a unit of their 8 bits, and so is 16 s + z within 24 bits) and the quotients
// stay within 0..15 by themselves; float32 values need the clamp, and so do steps near
// the bottom of the range, whose own rounding is coarse (and which are scaled to keep
// their reciprocal finite). What bounds it is the
// instructions, about 20 a value at 3.3 of the 4 that an SM can issue: 16 x 4096 rows
// of 32 heads take 338 us (1.38 GB, 4.1 TB/s). Two values to an instruction where
// there is one for a pair took 605 to 561 us with the reading back. float32 rows are
// bound by their bytes: 8 x 2048 rows of 16 heads 51.6 us (5.9 TB/s), 0.7 of it the
// clamp.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void kv_load16(const T* p, float (&x)[16], float& lo, float& hi) {
  if constexpr (sizeof(T) == 2) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p)), b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
    __nv_bfloat162 mn = h[0], mx = h[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      mn = __hmin2_nan(mn, h[i]);
      mx = __hmax2_nan(mx, h[i]);
    }
    lo = min_nan(__low2float(mn), __high2float(mn));
    hi = max_nan(__low2float(mx), __high2float(mx));
  } else {
    float a[8], b[8];
    load8_stream(p, a);
    load8_stream(p + 8, b);
    lo = hi = a[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = a[i];
      x[8 + i] = b[i];
      lo = min_nan(lo, min_nan(a[i], b[i]));
      hi = max_nan(hi, max_nan(a[i], b[i]));
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kKvThreads)
kv_quantize_kernel(const T* k, const T* v, const int32_t* idx, int rows, int n,
                   int per_row, int rpb, uint32_t magic, KvQuant cache, int* flag) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int r0 = blockIdx.x * rpb, items = min(rpb, rows - r0) * per_row;
  const T* src = (blockIdx.y ? v : k) + (size_t)r0 * per_row * 16;
  uint32_t* codes = blockIdx.y ? cache.vc : cache.kc;
  uint32_t* scales = blockIdx.y ? cache.vs : cache.ks;
  const int lanes = 1 << (cache.group_log2 - 4);
  for (int i0 = 0; i0 < items; i0 += kKvThreads) {
    const bool live = i0 + (int)threadIdx.x < items;
    const int i = live ? i0 + (int)threadIdx.x : items - 1;  // idle lanes repeat the last one: every lane takes part in the shuffles
    const int rr = kv_row_of(i, magic), c = i - rr * per_row;
    float x[16], lo, hi;
    kv_load16(src + (size_t)i * 16, x, lo, hi);
    const long long row = kv_cache_row(idx, r0 + rr, n, cache.capacity, flag);
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
    const uint32_t pair =
        fine ? (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(zb) << 16) : 0x7FFF7FFFu;
    const float m = fmaf(16.0f, s, z);  // 16 s is exact: one rounding
    uint32_t words[2] = {0, 0};
    if (fine && s >= 0x1p-60f) {
      const float inv = __frcp_rn(s);
      const int half = __float_as_int(0.5f * s);
      const uint64_t m2 = pack_f2(-m, -m), inv2 = pack_f2(inv, inv), s2 = pack_f2(-s, -s), radix = pack_f2(16.0f, 16.0f);
      const uint64_t round2 = pack_f2(12582912.0f, 12582912.0f), unround2 = pack_f2(-12582912.0f, -12582912.0f);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint64_t sum = 0;  // the codes of the even and of the odd dims as digits of 4 bits
#pragma unroll
        for (int j = 6; j >= 0; j -= 2) {
          const uint64_t d = add_f2(pack_f2(x[8 * w + j], x[8 * w + j + 1]), m2);
          const uint64_t u = fma_f2(d, inv2, round2), c = add_f2(u, unround2);
          const uint64_t rem = fma_f2(c, s2, d);
          float uu[2], cc[2], rr[2];
          unpack_f2(u, uu[0], uu[1]);
          unpack_f2(c, cc[0], cc[1]);
          unpack_f2(rem, rr[0], rr[1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // half a step, or the next number below it where the code is odd (the low bit of u)
            const float lim = __int_as_float(half - (__float_as_int(uu[e]) & 1));
            if (fabsf(rr[e]) > lim) cc[e] += copysignf(1.0f, rr[e]);
            // before it is a digit: a 16 would carry into the next dim's code
            if constexpr (sizeof(T) == 4) cc[e] = fminf(fmaxf(cc[e], 0.0f), 15.0f);
          }
          sum = fma_f2(sum, radix, pack_f2(cc[0], cc[1]));
        }
        float even, odd;
        unpack_f2(sum, even, odd);
        words[w] = (uint32_t)even | ((uint32_t)odd << 16);
      }
    } else if (fine && s > 0.0f) {
      const float su = s * 0x1p64f, inv = __frcp_rn(su), half = 0.5f * su;
      const float half_odd = __uint_as_float(__float_as_uint(half) - 1u);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float d = __fsub_rn(x[j], m) * 0x1p64f;
        const float u = fmaf(fminf(fmaxf(d, -su), 16.0f * su), inv, 12582912.0f), cf = u - 12582912.0f;
        int code = __float_as_int(u) - 0x4B400000;
        const float rem = fmaf(-cf, su, d), lim = (code & 1) ? half_odd : half;
        code = min(max(code + (rem > lim) - (rem < -lim), 0), 15);
        words[j >> 3] |= (uint32_t)code << kv_shift(j & 7);
      }
    }
    if (live && row >= 0) {
      const size_t at = (size_t)row * per_row + c;
      *reinterpret_cast<uint2*>(codes + at * 2) = make_uint2(words[0], words[1]);
      if ((c & (lanes - 1)) == 0) scales[at >> (cache.group_log2 - 4)] = pair;
    }
  }
}

// ---------------------------------------------------------------------------
// Rows of the cache back into k_out, v_out [B n, n_kv hd] (storage type); zeros
// for a padding row. An item is one word (8 values); a thread has four in flight (one
// at a time: 356 us for 222). Bound by the bytes, most of them written: 16 x 4096
// rows of 32 heads, groups of 128, 222 us, 6.1 TB/s; 8 x 2048 float32 rows of 16
// heads 63.5 us, 4.8 TB/s.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kKvThreads)
kv_dequantize_kernel(KvQuant cache, const int32_t* idx, int rows, int n, int per_row, int rpb,
                     uint32_t magic, T* __restrict__ k_out, T* __restrict__ v_out, int* flag) {
  grid_launch_dependents();
  grid_dependency_wait();
  constexpr int kFly = 4;
  const int r0 = blockIdx.x * rpb, items = min(rpb, rows - r0) * per_row;
  T* dst = (blockIdx.y ? v_out : k_out) + (size_t)r0 * per_row * 8;
  const uint32_t* codes = blockIdx.y ? cache.vc : cache.kc;
  const uint32_t* scales = blockIdx.y ? cache.vs : cache.ks;
  for (int i0 = threadIdx.x; i0 < items; i0 += kFly * kKvThreads) {
    uint32_t w[kFly], p[kFly];
#pragma unroll
    for (int e = 0; e < kFly; ++e) {
      const int i = i0 + e * kKvThreads;
      w[e] = p[e] = 0;  // s = z = 0: zeros
      if (i < items) {
        const int rr = kv_row_of(i, magic);
        const long long row = kv_cache_row(idx, r0 + rr, n, cache.capacity, flag);
        if (row >= 0) {
          const size_t at = (size_t)row * per_row + (i - rr * per_row);
          w[e] = __ldcs(codes + at);
          p[e] = scales[at >> (cache.group_log2 - 3)];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kFly; ++e) {
      const int i = i0 + e * kKvThreads;
      if (i >= items) break;
      if constexpr (sizeof(T) == 2) {
        uint32_t o[4];
        kv_word_bf16(w[e], __byte_perm(p[e], p[e], 0x1010), __byte_perm(p[e], p[e], 0x3232), o);
        __stcs(reinterpret_cast<uint4*>(dst + (size_t)i * 8), make_uint4(o[0], o[1], o[2], o[3]));
      } else {
        float o[8];
        kv_word_f32(w[e], pair_step(p[e]), pair_offset(p[e]), o);
        Storage<float>::store8(dst + (size_t)i * 8, o);
      }
    }
  }
}

}  // namespace esd
