// Partial attention over the 4-bit key/value cache for the float32 models, on the
// CUDA cores:
// out = softmax(q K^T / sqrt(hd)) V per head over the first len keys of each
// sequence, K and V the values that the cache reads back as (kv_quant.cuh), all
// sums and softmax statistics in float32.
//
// A key/value head's query rows are the n rows of the call times the `share`
// query heads that use it: row i is query i / share, head kvh share + i % share.
// One CTA takes 32 of them and a slice of the keys; each tile of 64 keys is
// expanded into shared memory once for all 32 rows. Thread (ty, tx) of 16 x 16
// holds rows 2 ty, 2 ty + 1: the scores of keys tx, tx + 16, tx + 32, tx + 48 and
// the outputs of dims 4 (tx + 16 j) .. + 3. The slices of one row tile are the
// CTAs of a cluster, which merge their maxima, sums and unnormalised outputs
// through distributed shared memory in slice order.
#pragma once

#include "kv_quant.cuh"
#include "tc_gemm2.cuh"  // cluster helpers
#include "attention_pair.cuh"  // distributed shared memory loads

namespace esd {

constexpr int kAqRows = 32, kAqKeys = 64, kAqMaxHd = 128;
constexpr int kAqMaxSplits = 8;

// floats of shared memory: Q, K and V tiles (rows padded by 4), scores, row statistics
constexpr int aq_smem_floats(int hd) {
  return (kAqRows + 2 * kAqKeys) * (hd + 4) + kAqRows * (kAqKeys + 4) + 2 * kAqRows;
}

template <int HD>
__global__ void __launch_bounds__(256)
quant_attention_simt_kernel(const float* __restrict__ Q, KvQuant cache, const int32_t* __restrict__ lens, float* __restrict__ O,
                            int n, int L, int share, int splits, float scale_log2) {
  constexpr int LD = HD + 4, LDP = kAqKeys + 4, WPR = HD / 8;
  constexpr int NJ = (HD + 63) / 64;  // dim quads per thread
  extern __shared__ __align__(16) float sm_aq[];
  float* sQ = sm_aq;
  float* sK = sQ + kAqRows * LD;
  float* sV = sK + kAqKeys * LD;
  float* sP = sV + kAqKeys * LD;
  float* sM = sP + kAqRows * LDP;  // merge: row maxima, sums
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int split = blockIdx.x % splits, tile = blockIdx.x / splits;
  const int b = blockIdx.y / cache.n_kv, kvh = blockIdx.y % cache.n_kv;
  const int H = cache.n_kv * share, rows = n * share, r0 = tile * kAqRows;
  const int len = lens ? min(L, max(0, lens[b])) : L;
  const int tiles = (len + kAqKeys - 1) / kAqKeys, per = (tiles + splits - 1) / splits;
  const int t0 = min(tiles, split * per), t1 = min(tiles, t0 + per);

  for (int i = tid; i < kAqRows * (HD / 8); i += 256) {
    const int r = i / (HD / 8), c = (i % (HD / 8)) * 8, row = r0 + r;
    float q[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (row < rows)
      Storage<float>::load8(Q + (((size_t)b * n + row / share) * H + kvh * share + row % share) * HD + c, q);
    Storage<float>::store8(sQ + r * LD + c, q);
  }
  float o[2][NJ * 4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < NJ * 4; ++i) o[0][i] = o[1][i] = 0.0f;

  // a thread's words of a tile (K, then V) and their steps and offsets, a tile ahead
  constexpr int kWords = kAqKeys * WPR * 2 / 256;
  uint32_t cw[kWords], cp[kWords];
  auto load = [&](int t) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const int i = tid + j * 256;
      const bool is_v = i >= kAqKeys * WPR;
      const int w = is_v ? i - kAqKeys * WPR : i, key = w / WPR, pos = t * kAqKeys + key;
      const size_t at = (((size_t)b * cache.capacity + min(pos, len - 1)) * cache.n_kv + kvh) * WPR + w % WPR;
      cw[j] = __ldg((is_v ? cache.vc : cache.kc) + at);
      cp[j] = __ldg((is_v ? cache.vs : cache.ks) + (at >> (cache.group_log2 - 3)));
    }
  };
  if (t0 < t1) load(t0);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();  // the previous tile is read; Q is written
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const int i = tid + j * 256;
      const bool is_v = i >= kAqKeys * WPR;
      const int w = is_v ? i - kAqKeys * WPR : i, key = w / WPR, wd = w % WPR;
      // keys past the end read as zeros whatever the cache holds there
      const uint32_t pr = t * kAqKeys + key < len ? cp[j] : 0u;
      float x[8];
      kv_word_f32(cw[j], pair_step(pr), pair_offset(pr), x);
      Storage<float>::store8((is_v ? sV : sK) + key * LD + wd * 8, x);
    }
    if (t + 1 < t1) load(t + 1);
    __syncthreads();
    float s[2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = 0.0f;
#pragma unroll 4
    for (int c = 0; c < HD; c += 4) {
      const float4 q0 = *reinterpret_cast<const float4*>(sQ + (2 * ty) * LD + c);
      const float4 q1 = *reinterpret_cast<const float4*>(sQ + (2 * ty + 1) * LD + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 kk = *reinterpret_cast<const float4*>(sK + (tx + 16 * e) * LD + c);
        s[0][e] = fmaf(q0.x, kk.x, fmaf(q0.y, kk.y, fmaf(q0.z, kk.z, fmaf(q0.w, kk.w, s[0][e]))));
        s[1][e] = fmaf(q1.x, kk.x, fmaf(q1.y, kk.y, fmaf(q1.z, kk.z, fmaf(q1.w, kk.w, s[1][e]))));
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = t * kAqKeys + tx + 16 * e < len ? s[i][e] * scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[i][e]);
      }
#pragma unroll
      for (int sh = 8; sh > 0; sh >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
      const float mn = fmaxf(m[i], mx);
      // all scores NaN: the maximum stays -inf, and so that the NaNs reach the sum no shift is taken
      const float sub = mn == -INFINITY ? 0.0f : mn;
      const float f = exp2f(m[i] - sub);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = exp2f(s[i][e] - sub);
        sP[(2 * ty + i) * LDP + tx + 16 * e] = p;
        sum += p;
      }
      l[i] = l[i] * f + sum;
      m[i] = mn;
#pragma unroll
      for (int j = 0; j < NJ * 4; ++j) o[i][j] *= f;
    }
    __syncwarp();  // a row's scores are written and read by one warp
#pragma unroll 2
    for (int key = 0; key < kAqKeys; key += 4) {
      const float4 p0 = *reinterpret_cast<const float4*>(sP + (2 * ty) * LDP + key);
      const float4 p1 = *reinterpret_cast<const float4*>(sP + (2 * ty + 1) * LDP + key);
      const float a0[4] = {p0.x, p0.y, p0.z, p0.w}, a1[4] = {p1.x, p1.y, p1.z, p1.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int c = 4 * (tx + 16 * j);
          if (HD % 64 == 0 || c < HD) {
            const float4 vv = *reinterpret_cast<const float4*>(sV + (key + u) * LD + c);
            o[0][4 * j] = fmaf(a0[u], vv.x, o[0][4 * j]);
            o[0][4 * j + 1] = fmaf(a0[u], vv.y, o[0][4 * j + 1]);
            o[0][4 * j + 2] = fmaf(a0[u], vv.z, o[0][4 * j + 2]);
            o[0][4 * j + 3] = fmaf(a0[u], vv.w, o[0][4 * j + 3]);
            o[1][4 * j] = fmaf(a1[u], vv.x, o[1][4 * j]);
            o[1][4 * j + 1] = fmaf(a1[u], vv.y, o[1][4 * j + 1]);
            o[1][4 * j + 2] = fmaf(a1[u], vv.z, o[1][4 * j + 2]);
            o[1][4 * j + 3] = fmaf(a1[u], vv.w, o[1][4 * j + 3]);
          }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int sh = 8; sh > 0; sh >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], sh);

  // the slice's result into shared memory (over the K tile), then each CTA of
  // the cluster merges the rows r with r % splits == split
  __syncthreads();
  float* sO = sK;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * ty + i;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int c = 4 * (tx + 16 * j);
      if (HD % 64 == 0 || c < HD)
        *reinterpret_cast<float4*>(sO + r * LD + c) =
            make_float4(o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]);
    }
    if (tx == 0) {
      sM[r] = m[i];
      sM[kAqRows + r] = l[i];
    }
  }
  __syncwarp();
  cluster_sync_all();
  for (int i = tid; i < kAqRows * (HD / 8); i += 256) {
    const int r = i / (HD / 8), c = (i % (HD / 8)) * 8, row = r0 + r;
    if (r % splits != split || row >= rows) continue;
    float ms = -INFINITY, ls = 0.0f, acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int q = 0; q < splits; ++q) ms = fmaxf(ms, ld_dsmem_f32(mapa_shared(smem_u32(sM + r), q)));
    const float sub = ms == -INFINITY ? 0.0f : ms;
    for (int q = 0; q < splits; ++q) {
      const float w = exp2f(ld_dsmem_f32(mapa_shared(smem_u32(sM + r), q)) - sub);
      ls += w * ld_dsmem_f32(mapa_shared(smem_u32(sM + kAqRows + r), q));
      const uint32_t at = mapa_shared(smem_u32(sO + r * LD + c), q);
      const float4 x = ld_dsmem_f4(at), y = ld_dsmem_f4(at + 16);
      const float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += w * z[j];
    }
    const float inv = len == 0 ? 0.0f : 1.0f / ls;  // no key: zeros (all scores -inf: NaN)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] *= inv;
    Storage<float>::store8(O + (((size_t)b * n + row / share) * H + kvh * share + row % share) * HD + c, acc);
  }
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while another reads its memory
}

// Shared-memory opt-in of the kernel for head_dim hd.
inline cudaError_t quant_attention_simt_setup(int hd) {
  if (hd % 32) return cudaSuccess;  // refused by the calls; the opt-in of another head_dim's kernel stays as it is
  const int smem = aq_smem_floats(hd) * (int)sizeof(float);
  const void* k = hd == 32   ? (const void*)quant_attention_simt_kernel<32>
                  : hd == 64 ? (const void*)quant_attention_simt_kernel<64>
                  : hd == 96 ? (const void*)quant_attention_simt_kernel<96>
                             : (const void*)quant_attention_simt_kernel<128>;
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

inline cudaError_t quant_attention_simt(const void* Q, const KvQuant& kv, const int32_t* lens, void* O, int B, int n, int L,
                                 int share, int hd, int num_sms, cudaStream_t st) {
  const long long tiles = ((long long)n * share + kAqRows - 1) / kAqRows, units = tiles * B * kv.n_kv;
  const int key_tiles = (L + kAqKeys - 1) / kAqKeys;
  int splits = 1;
  while (splits < kAqMaxSplits && splits * 2 <= key_tiles && units * splits * 2 <= 3LL * num_sms) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * splits), (unsigned)(B * kv.n_kv), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = aq_smem_floats(hd) * sizeof(float);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* k = hd == 32   ? quant_attention_simt_kernel<32>
            : hd == 64 ? quant_attention_simt_kernel<64>
            : hd == 96 ? quant_attention_simt_kernel<96>
                       : quant_attention_simt_kernel<128>;
  return cudaLaunchKernelEx(&cfg, k, (const float*)Q, kv, lens, (float*)O, n, L, share, splits,
                            1.4426950408889634f / sqrtf((float)hd));
}

}  // namespace esd
