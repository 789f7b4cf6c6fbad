// Partial attention over the 4-bit key/value cache for few query rows, bf16,
// head_dim 128: at most 16 rows per key/value head (rows of the call times the
// query heads that share it). With so few rows the cache is read for little
// arithmetic, and what counts besides its bytes is how few instructions turn
// codes into operands: every value is expanded once, in the registers of the
// thread that loaded it, straight into an mma.sync fragment.
//
// One warp walks blocks of 32 keys of one head: S^T = K Q^T takes the keys as the
// MMA's 16 rows and the query rows as its 8 columns, O^T += V^T P^T the dims as
// rows. The fragments' index permutations are free, as long as both operands of a
// product agree, so the thread (g, t) of a fragment (g = lane / 4, t = lane % 4)
// takes
//   keys g and g + 8 of a tile of 16, dims 32 t .. 32 t + 31: 16 bytes of codes
//     each, all of one group; the product's steps walk the 8 words' pairs, and Q
//     is kept in that order;
//   dims 16 g .. 16 g + 15 of keys 2t, 2t + 1, 2t + 8, 2t + 9: 8 bytes each; two
//     byte permutes pair the codes of two keys, whose steps and offsets ride in
//     the two halves of the packed multiply-add.
// P goes from the score layout (key, query pair) to the operand layout (query,
// key pair) by an 8x8 transpose between the lanes (movmatrix). The running
// maximum moves only when a score passes it by more than 2^8 (the result O / l is
// the same; how often O is scaled changes), which one vote per block decides.
// Scores, maxima, sums, O and the merge are float32. P alone is rounded to bf16: both
// operands of the product have one type, V's values are bf16 already (their range
// leaves no other type of 16 bits), and P kept to more bits would take a second
// product per tile. It moves an output by at most 2^-8 of sum p |v|, the size of its
// own rounding; measured 0.0019 to 0.0024 from 64 bits, where float32 P has 0.0017.
//
// Each warp copies its own blocks (cp.async, no other thread waits on them)
// through a ring of its own in shared memory; two rows of codes share a 128-byte
// line whose 16-byte chunks are permuted by the line, so that both access shapes
// above are free of bank conflicts. Copying through registers instead (a block
// ahead) took 78 us where this takes 61 to 66: its addresses and its registers
// cost the occupancy that hides the latency.
//
// What bounds it: 32 sequences x 1536 keys x 32 heads, groups of 64, one row: 67 us,
// 3.4 TB/s of the 226 MB (a bare copy of those codes in one launch, 64 bytes a row
// and head, reaches 4.5 TB/s). The bit operations of the expansion (two per pair of
// values, at half the issue rate) keep their pipe at 55%; shifts taken as products,
// and a line of blocks cut evenly over all warps of the machine, were no faster.
//
// The warps of a CTA take neighbouring heads (the steps and offsets of 2 to 8
// heads share a 32-byte sector, which they so fetch once) or, when there are too
// few CTAs, slices of the keys; the CTAs of a cluster take slices of the keys.
// Every warp leaves (m, l, O) in shared memory, and the CTAs of the cluster merge
// a share of the outputs each, in (CTA, warp) order.
#pragma once

#include <initializer_list>

#include "attention_mma.cuh"   // mma_bf16
#include "attention_pair.cuh"  // ex2_ftz, distributed shared memory
#include "kv_quant.cuh"

namespace esd {

constexpr int kArWarps = 4, kArKeys = 32, kArHd = 128, kArMaxSplits = 16, kArStages = 3;
constexpr int kArLd = kArHd + 4;
constexpr float kArLazy = 8.0f;

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// asynchronous copy of BYTES (4, 8 or 16) into shared memory, zeros if !valid
template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? BYTES : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

// bytes of a warp's stage: codes of 32 keys and of 32 values, their steps and offsets
template <int GPH>
constexpr int ar_stage() {
  return 2 * kArKeys * 64 + 2 * kArKeys * GPH * 4;
}
template <int NT, int GPH>
constexpr int ar_smem() {
  const int ring = kArWarps * kArStages * ar_stage<GPH>(), merge = kArWarps * 8 * NT * kArLd * 4;
  return ring > merge ? ring : merge;
}

// NT tiles of 8 query rows, GPH groups per head. Grid (splits, B * heads / wh),
// cluster (splits, 1, 1); wh: heads per CTA (1, 2 or 4).
template <int NT, int GPH>
__global__ void __launch_bounds__(kArWarps * 32, NT == 1 ? 4 : 2)
quant_attention_rows_kernel(const __nv_bfloat16* Q, KvQuant cache, const int32_t* lens,
                            __nv_bfloat16* __restrict__ O, int n, int L, int share, int splits, int wh,
                            float scale_log2) {
  constexpr int kRows = 8 * NT, kStage = ar_stage<GPH>(), kGlog = GPH == 4 ? 5 : GPH == 2 ? 6 : 7;
  constexpr int kV = kArKeys * 64, kKs = 2 * kArKeys * 64, kVs = kKs + kArKeys * GPH * 4;
  extern __shared__ __align__(128) uint8_t sm_ar[];
  __shared__ float s_m[kArWarps][kRows], s_l[kArWarps][kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  grid_launch_dependents();
  grid_dependency_wait();
  const int hgroups = cache.n_kv / wh;
  const int split = blockIdx.x, b = blockIdx.y / hgroups, hslot = warp & (wh - 1), kslot = warp / wh;
  const int h0 = (blockIdx.y % hgroups) * wh, kvh = h0 + hslot, per_head = kArWarps / wh;
  const int H = cache.n_kv * share, rows = n * share;
  const int len = lens ? min(L, max(0, lens[b])) : L;
  const int blocks = (len + kArKeys - 1) / kArKeys, workers = splits * per_head;

  // the copies of a lane: 16-byte chunk lane % 4 of rows lane / 4 + 8 u, the steps and offsets of row `lane`
  const size_t first = (size_t)b * cache.capacity * cache.n_kv + kvh;  // (row, head) index of key 0
  const uint32_t* kc = cache.kc + first * 16 + 4 * t;
  const uint32_t* vc = cache.vc + first * 16 + 4 * t;
  const uint32_t* ks = cache.ks + first * GPH;
  const uint32_t* vs = cache.vs + first * GPH;
  const uint32_t cstep = (uint32_t)cache.n_kv * 16, sstep = (uint32_t)cache.n_kv * GPH;
  const uint32_t ring = smem_u32(sm_ar) + (uint32_t)(warp * kArStages * kStage);
  // rows g + 8 u lie in lines g / 2 + 4 u, whose permutation is that of line g / 2
  const uint32_t put = (uint32_t)((g >> 1) * 128 + ((((g & 1) << 2 | t) ^ ((g >> 1) << 1)) << 4));
  auto load = [&](int blk, int stage) {
    const uint32_t st = ring + (uint32_t)(stage * kStage);
    const int key0 = blk * kArKeys;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int key = key0 + g + 8 * u;
      const uint64_t at = (uint64_t)(uint32_t)min(key, len - 1) * cstep;
      cp_async16(st + put + u * 512, kc + at, key < len);
      cp_async16(st + kV + put + u * 512, vc + at, key < len);
    }
    const int key = key0 + lane;
    const uint64_t at = (uint64_t)(uint32_t)min(key, len - 1) * sstep;
    cp_async_small<GPH * 4>(st + kKs + lane * GPH * 4, ks + at, key < len);
    cp_async_small<GPH * 4>(st + kVs + lane * GPH * 4, vs + at, key < len);
  };
  int next = split * per_head + kslot;  // the next block to copy
#pragma unroll
  for (int i = 0; i < kArStages - 1; ++i) {
    if (next < blocks) load(next, i);
    next += workers;
    cp_async_commit();
  }

  // the query rows in the order in which the product walks a thread's 32 dims
  uint32_t q[NT][16];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int row = 8 * i + g;
    if (row < rows) {
      const uint4* src = reinterpret_cast<const uint4*>(
          Q + (((size_t)b * n + row / share) * H + kvh * share + row % share) * kArHd + 32 * t);
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(&q[i][4 * j]) = src[j];
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) q[i][j] = 0;
    }
  }
  float o[8][NT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    m[i][0] = m[i][1] = -INFINITY;
    l[i][0] = l[i][1] = 0.0f;
#pragma unroll
    for (int d = 0; d < 8; ++d) o[d][i][0] = o[d][i][1] = o[d][i][2] = o[d][i][3] = 0.0f;
  }

  const uint8_t* mine = sm_ar + warp * kArStages * kStage;
  // V: 8 bytes g of rows 2t, 2t + 1 (+ 8): lines t, t + 4, even and odd row
  const int get_v0 = t * 128 + (((g >> 1) ^ (t << 1)) << 4) + (g & 1) * 8;
  const int get_v1 = t * 128 + ((4 | (g >> 1)) ^ (t << 1)) * 16 + (g & 1) * 8;
  const int get_ks = (g * GPH + ((32 * t) >> kGlog)) * 4, get_vs = (2 * t * GPH + ((16 * g) >> kGlog)) * 4;
  int stage = 0;
  for (int blk = split * per_head + kslot; blk < blocks; blk += workers) {
    cp_async_wait<kArStages - 2>();
    __syncwarp();  // every lane's copies of this block have landed; every lane has read the stage refilled next
    {
      const int fill = stage == 0 ? kArStages - 1 : stage - 1;
      if (next < blocks) load(next, fill);
      next += workers;
      cp_async_commit();
    }
    const uint8_t* st = mine + stage * kStage;
    stage = stage == kArStages - 1 ? 0 : stage + 1;
    const int key0 = blk * kArKeys;

    float s[2][NT][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < NT; ++i) s[u][i][0] = s[u][i][1] = s[u][i][2] = s[u][i][3] = 0.0f;
      const uint32_t p0 = *reinterpret_cast<const uint32_t*>(st + kKs + get_ks + u * 64 * GPH);
      const uint32_t p1 = *reinterpret_cast<const uint32_t*>(st + kKs + get_ks + u * 64 * GPH + 32 * GPH);
      const uint32_t s0 = __byte_perm(p0, p0, 0x1010), z0 = __byte_perm(p0, p0, 0x3232);
      const uint32_t s1 = __byte_perm(p1, p1, 0x1010), z1 = __byte_perm(p1, p1, 0x3232);
      const uint4 c0 = *reinterpret_cast<const uint4*>(st + put + u * 1024);
      const uint4 c1 = *reinterpret_cast<const uint4*>(st + put + u * 1024 + 512);
      const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t x[4], y[4];
        kv_word_bf16(w0[w], s0, z0, x);
        kv_word_bf16(w1[w], s1, z1, y);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          mma_bf16(s[u][i], x[0], y[0], x[1], y[1], q[i][4 * w], q[i][4 * w + 1]);
          mma_bf16(s[u][i], x[2], y[2], x[3], y[3], q[i][4 * w + 2], q[i][4 * w + 3]);
        }
      }
    }
    if (key0 + kArKeys > len) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if (key0 + 16 * u + g >= len) s[u][i][0] = s[u][i][1] = -INFINITY;
          if (key0 + 16 * u + 8 + g >= len) s[u][i][2] = s[u][i][3] = -INFINITY;
        }
    }
    float mx[NT][2];
    bool need = false;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[i][e] = fmaxf(fmaxf(s[0][i][e], s[0][i][e + 2]), fmaxf(s[1][i][e], s[1][i][e + 2])) * scale_log2;
        need |= mx[i][e] > m[i][e] + kArLazy;
      }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = mx[i][e];
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sh));
          x = fmaxf(x, m[i][e]);
          const float f = x == m[i][e] ? 1.0f : exp2f(m[i][e] - x);  // -inf stays -inf until a score is seen
          m[i][e] = x;
          l[i][e] *= f;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            o[d][i][e] *= f;
            o[d][i][e + 2] *= f;
          }
        }
    }
    uint32_t p[2][NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float sub[2] = {m[i][0] == -INFINITY ? 0.0f : m[i][0], m[i][1] == -INFINITY ? 0.0f : m[i][1]};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pv[e] = ex2_ftz(fmaf(s[u][i][e], scale_log2, -sub[e & 1]));
          l[i][e & 1] += pv[e];
        }
        p[u][i][0] = movmatrix_trans(pack_bf16(pv[0], pv[1]));
        p[u][i][1] = movmatrix_trans(pack_bf16(pv[2], pv[3]));
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* sv = st + kVs + get_vs + u * 64 * GPH;
      const uint32_t v0 = *reinterpret_cast<const uint32_t*>(sv), v1 = *reinterpret_cast<const uint32_t*>(sv + 4 * GPH);
      const uint32_t v2 = *reinterpret_cast<const uint32_t*>(sv + 32 * GPH);
      const uint32_t v3 = *reinterpret_cast<const uint32_t*>(sv + 36 * GPH);
      const uint32_t sa = __byte_perm(v0, v1, 0x5410), za = __byte_perm(v0, v1, 0x7632);
      const uint32_t sb = __byte_perm(v2, v3, 0x5410), zb = __byte_perm(v2, v3, 0x7632);
      const uint2 x0 = *reinterpret_cast<const uint2*>(st + kV + get_v0 + u * 1024);
      const uint2 x1 = *reinterpret_cast<const uint2*>(st + kV + get_v1 + u * 1024);
      const uint2 x2 = *reinterpret_cast<const uint2*>(st + kV + get_v0 + u * 1024 + 512);
      const uint2 x3 = *reinterpret_cast<const uint2*>(st + kV + get_v1 + u * 1024 + 512);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t c0 = w ? x0.y : x0.x, c1 = w ? x1.y : x1.x, c2 = w ? x2.y : x2.x, c3 = w ? x3.y : x3.x;
        uint32_t e0[4], e1[4], e2[4], e3[4];  // even dims of keys 2t, 2t + 1; odd ones; the same of 2t + 8, 2t + 9
        kv_word_bf16(__byte_perm(c0, c1, 0x5410), sa, za, e0);
        kv_word_bf16(__byte_perm(c0, c1, 0x7632), sa, za, e1);
        kv_word_bf16(__byte_perm(c2, c3, 0x5410), sb, zb, e2);
        kv_word_bf16(__byte_perm(c2, c3, 0x7632), sb, zb, e3);
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int i = 0; i < NT; ++i)
            mma_bf16(o[4 * w + d][i], e0[d], e1[d], e2[d], e3[d], p[u][i][0], p[u][i][1]);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // the rings are done with: their memory holds the merge from here on

  // this warp's (m, l, O): thread (g, t) holds dims 16 g + 2 d, + 1 of rows 2t, 2t + 1 (of each 8)
  float* s_o = reinterpret_cast<float*>(sm_ar);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], sh);
      const int row = 8 * i + 2 * t + e;
      if (g == 0) {
        s_m[warp][row] = m[i][e];
        s_l[warp][row] = l[i][e];
      }
#pragma unroll
      for (int d = 0; d < 8; ++d)
        *reinterpret_cast<float2*>(s_o + (warp * kRows + row) * kArLd + 16 * g + 2 * d) =
            make_float2(o[d][i][e], o[d][i][e + 2]);
    }
  __syncthreads();
  if (splits > 1) cluster_sync_all();
  // a warp merges a row: source k of head slot j is warp (k % per_head) wh + j of CTA k / per_head, lane k % 32
  // holds its weight (at most 64 sources)
  for (int i = split * kArWarps + warp; i < wh * rows; i += splits * kArWarps) {
    const int j = i / rows, row = i % rows;
    float mk[2], wk[2], ms = -INFINITY, ls = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = lane + 32 * e;
      mk[e] = -INFINITY;
      if (k < workers) mk[e] = ld_dsmem_f32(mapa_shared(smem_u32(&s_m[(k % per_head) * wh + j][row]), k / per_head));
      ms = fmaxf(ms, mk[e]);
    }
    ms = warp_max(ms);
    const float sub = ms == -INFINITY ? 0.0f : ms;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = lane + 32 * e;
      wk[e] = exp2f(mk[e] - sub);
      if (k < workers)
        ls += wk[e] * ld_dsmem_f32(mapa_shared(smem_u32(&s_l[(k % per_head) * wh + j][row]), k / per_head));
    }
    ls = warp_sum(ls);
    const float inv = len == 0 ? 0.0f : 1.0f / ls;  // no key: zeros (all scores -inf: NaN)
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll 8
      for (int k = 32 * e; k < min(workers, 32 * e + 32); ++k) {
        const float f = __shfl_sync(0xffffffffu, wk[e], k & 31);
        const float4 x = ld_dsmem_f4(
            mapa_shared(smem_u32(s_o + (((k % per_head) * wh + j) * kRows + row) * kArLd + 4 * lane), k / per_head));
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
      }
    uint2 u;
    u.x = pack_bf16(acc.x * inv, acc.y * inv);
    u.y = pack_bf16(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(O + (((size_t)b * n + row / share) * H + (h0 + j) * share + row % share) * kArHd +
                              4 * lane) = u;
  }
  __syncwarp();
  if (splits > 1) cluster_sync_all();  // no CTA leaves while another reads its memory
}

template <int NT, int GPH>
cudaError_t quant_attention_rows_setup_one() {
  auto* k = quant_attention_rows_kernel<NT, GPH>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ar_smem<NT, GPH>());
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}
inline cudaError_t quant_attention_rows_setup() {
  cudaError_t e = cudaSuccess;
  for (cudaError_t x : {quant_attention_rows_setup_one<1, 1>(), quant_attention_rows_setup_one<1, 2>(),
                        quant_attention_rows_setup_one<1, 4>(), quant_attention_rows_setup_one<2, 1>(),
                        quant_attention_rows_setup_one<2, 2>(), quant_attention_rows_setup_one<2, 4>()})
    if (e == cudaSuccess) e = x;
  return e;
}

template <int NT, int GPH>
cudaError_t quant_attention_rows_launch(const void* Q, const KvQuant& kv, const int32_t* lens, void* O, int B, int n,
                                        int L, int share, int num_sms, cudaStream_t st) {
  const int units = B * kv.n_kv, blocks = (L + kArKeys - 1) / kArKeys, resident = num_sms * (NT == 1 ? 3 : 2);
  // the most heads per CTA that still fill the SMs (32 x 32 heads x 1536 keys: 66 us with four, 70 with one); then
  // slices while they are all resident and none is empty (16 heads x 512 keys: 5.7 us in four, 6.5 in one; 16 heads
  // x 65536 keys: 53 us in sixteen, 95 in four). CTAs of eight warps, for twice the warps in sixteen slices, took
  // 78 us there: half as many clusters of sixteen are resident at once.
  int wh = 1;
  while (wh < 4 && kv.n_kv % (2 * wh) == 0 && units / (2 * wh) >= num_sms) wh *= 2;
  int splits = 1;
  while (splits < kArMaxSplits && splits * 2 * (kArWarps / wh) <= blocks && units / wh * splits * 2 <= resident)
    splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(splits, units / wh, 1);
  cfg.blockDim = dim3(kArWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = ar_smem<NT, GPH>();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  // Started while the kernel before ends only with a CTA per SM at most (16 heads x 512 keys: 8.2 -> 6.8 us a call):
  // more would wait on the SMs that free first and leave the others idle (32 x 32 heads x 1536 keys: 68 -> 124 us)
  cfg.numAttrs = units / wh * splits <= num_sms ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, quant_attention_rows_kernel<NT, GPH>, (const __nv_bfloat16*)Q, kv, lens,
                            (__nv_bfloat16*)O, n, L, share, splits, wh, 1.4426950408889634f / sqrtf((float)kArHd));
}

inline cudaError_t quant_attention_rows(const void* Q, const KvQuant& kv, const int32_t* lens, void* O, int B, int n,
                                        int L, int share, int num_sms, cudaStream_t st) {
  const bool one = n * share <= 8;
  if (kv.group_log2 == 5)
    return one ? quant_attention_rows_launch<1, 4>(Q, kv, lens, O, B, n, L, share, num_sms, st)
               : quant_attention_rows_launch<2, 4>(Q, kv, lens, O, B, n, L, share, num_sms, st);
  if (kv.group_log2 == 6)
    return one ? quant_attention_rows_launch<1, 2>(Q, kv, lens, O, B, n, L, share, num_sms, st)
               : quant_attention_rows_launch<2, 2>(Q, kv, lens, O, B, n, L, share, num_sms, st);
  return one ? quant_attention_rows_launch<1, 1>(Q, kv, lens, O, B, n, L, share, num_sms, st)
             : quant_attention_rows_launch<2, 1>(Q, kv, lens, O, B, n, L, share, num_sms, st);
}

}  // namespace esd
