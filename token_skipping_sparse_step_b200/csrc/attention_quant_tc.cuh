// Partial attention over the 4-bit key/value cache for many query rows, bf16,
// head_dim 128, on the tensor cores (tcgen05): the codes of a chunk of 128 keys
// are expanded once, in shared memory, for up to 256 query rows.
//
// A CTA takes one key/value head of one sequence, a slice of its keys, and query
// rows (row i: query i / share, head kvh share + i % share) in two streams of 128
// rows, TMEM lane = row. More than 128 rows: the streams are two row tiles, and
// each chunk serves both. Up to 128: the streams are the even and the odd chunks of
// the same rows, each with sums and an accumulator of its own, merged at the end;
// up to 64 rows the odd stream's rows lie in lanes 64 and up, so that the softmax
// of the two streams runs on different schedulers. Two streams keep the tensor
// cores at work: while one stream's scores go through the softmax, the other's
// products run.
//
// Warps: 0..3 and 4..7 the softmax of streams 0 and 1 (thread = row: no exchange
// between threads); 8..15 expand codes: the next chunk's codes, steps and offsets
// are in registers while the current one becomes bf16 K and V tiles, [128 keys][64
// dims] x 2 in the 128-byte swizzle that TMA would write (K: K-major operand, V:
// MN-major); a warp's lanes are laid out so that its 16-byte stores are free of
// bank conflicts. 16 issues the MMAs: per stream S = Q K^T (M 128, N 128 keys, K
// 128 dims) into TMEM, then O += P V with P (bf16) read from TMEM, where the
// softmax wrote it over the scores that it came from. S of a stream's next chunk is
// issued once its P V is done.
//
// The running maximum moves only when a chunk's exceeds it by more than 2^8 (O is
// then scaled in TMEM; the result O / l is the same). P is rounded to bf16 for its
// product, everything else is float32. Keys at or past the sequence's length are
// masked, and read as zeros. The slices of a row tile are the CTAs of a cluster,
// merged through distributed shared memory in slice order. Every mbarrier wait is
// bounded (error flag); every CTA reaches every cluster barrier.
#pragma once

#include "attention_pair.cuh"
#include "kv_quant.cuh"

namespace esd {

constexpr int kAtRows = 128, kAtKeys = 128, kAtHd = 128;
constexpr int kAtBox = 128 * 64 * 2;              // 128 rows x 64 dims
constexpr int kAtTile = 2 * kAtBox;               // Q of a stream, K or V of a chunk
constexpr int kAtConv = 256, kAtThreads = 256 + kAtConv + 32;
constexpr int kAtLd = kAtHd + 4;                  // floats of a merge row
constexpr int kAtMain = 2 * kAtTile + 4 * kAtTile;  // Q, K ring, V ring
constexpr int kAtStats = 2 * 2 * kAtRows * 4;     // merge: row maxima and sums of both streams
constexpr int kAtSmem = kAtMain + kAtStats + 256 + 1024;
constexpr int kAtMaxSplits = 8;
static_assert(2 * kAtRows * kAtLd * 4 <= kAtMain, "the merge rows lie over the tiles");

__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// D (+)= A B with A in tensor memory (lane = row, two bf16 per column)
__device__ __forceinline__ void tc_mma_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x 32 bit, 32 consecutive columns per thread
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// A thread's share of a chunk: rows r and r + 64 of K and of V, 32 dims each.
struct AtRaw {
  uint4 k[2], v[2];
  uint32_t ks[2], vs[2];
};

// Grid (tiles * splits, B * n_kv), cluster (splits). TWO: two row tiles per CTA;
// else one (rows <= 128).
template <bool TWO>
__global__ void __launch_bounds__(kAtThreads, 1)
quant_attention_tc_kernel(const __nv_bfloat16* __restrict__ Q, KvQuant cache, const int32_t* __restrict__ lens,
                          __nv_bfloat16* __restrict__ O, int n, int L, int share, int splits, float scale_log2,
                          int* flag) {
  extern __shared__ __align__(1024) uint8_t smem_at_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_at_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;                  // [stream][dims 0-63 | 64-127][128 rows]
  uint8_t* sK = sQ + 2 * kAtTile;      // [stage][...][128 keys]
  uint8_t* sV = sK + 2 * kAtTile;
  float* s_m = reinterpret_cast<float*>(sV + 2 * kAtTile);  // [stream][128]
  float* s_l = s_m + 2 * kAtRows;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_l + 2 * kAtRows);
  uint64_t* qfull = bars;         // Q written
  uint64_t* kfull = bars + 1;     // [2] K of a chunk written
  uint64_t* vfull = bars + 3;     // [2]
  uint64_t* kempty = bars + 5;    // [2] the scores that read it are done
  uint64_t* vempty = bars + 7;    // [2]
  uint64_t* sfull = bars + 9;     // [2] a stream's scores in TMEM
  uint64_t* pready = bars + 11;   // [2] a stream's P written, its O scaled
  uint64_t* pvdone = bars + 13;   // [2] a stream's P V accumulated
  uint64_t* drain = bars + 15;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % splits, tile = blockIdx.x / splits;
  const int b = blockIdx.y / cache.n_kv, kvh = blockIdx.y % cache.n_kv;
  const int H = cache.n_kv * share, r0 = tile * (TWO ? 256 : 128);
  const int rows = min(n * share - r0, TWO ? 256 : 128);  // rows of this CTA
  const int shift = !TWO && rows <= 64 ? 64 : 0;          // lanes between a row of the two streams
  const int len = lens ? min(L, max(0, lens[b])) : L;
  const int chunks = (len + kAtKeys - 1) / kAtKeys;
  const int c0 = (int)((long long)chunks * split / splits), nc = (int)((long long)chunks * (split + 1) / splits) - c0;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(qfull), kAtConv / 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&kfull[i]), kAtConv / 32);
      mbar_init(smem_u32(&vfull[i]), kAtConv / 32);
      mbar_init(smem_u32(&kempty[i]), 1);
      mbar_init(smem_u32(&vempty[i]), 1);
      mbar_init(smem_u32(&sfull[i]), 1);
      mbar_init(smem_u32(&pready[i]), 4);
      mbar_init(smem_u32(&pvdone[i]), 1);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto row_at = [&](int i) {  // of Q and O
    const int row = r0 + i;
    return (((size_t)b * n + row / share) * H + kvh * share + row % share) * kAtHd;
  };
  // steps of stream s, and the chunk of its step i
  auto steps = [&](int s) { return TWO ? nc : (nc - s + 1) >> 1; };

  if (warp >= 8 && warp < 16) {
    // ---------------- codes to tiles. Lane bits: 0 and 3 the 32 dims, 1, 2 and 4 the row of eight: a store's
    // 8 lanes cover 4 rows x 2 halves of their 128 bytes, which the swizzle spreads over all banks.
    const int p = (lane & 1) | ((lane >> 2) & 2), r = (warp - 8) * 8 + ((lane >> 1) & 3) + ((lane >> 4) << 2);
    const size_t first = (size_t)b * cache.capacity * cache.n_kv + kvh;
    const int gk = 7 - cache.group_log2, gp = (32 * p) >> cache.group_log2;
    const uint32_t* kc = cache.kc + first * 16 + 4 * p;
    const uint32_t* vc = cache.vc + first * 16 + 4 * p;
    const uint32_t* ks = cache.ks + (first << gk) + gp;
    const uint32_t* vs = cache.vs + (first << gk) + gp;
    const uint32_t cstep = (uint32_t)cache.n_kv * 16, sstep = (uint32_t)cache.n_kv << gk;
    auto load = [&](AtRaw& a, int j) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int key = (c0 + j) * kAtKeys + r + 64 * u;
        const uint32_t at = (uint32_t)min(key, len - 1);
        a.k[u] = __ldg(reinterpret_cast<const uint4*>(kc + (uint64_t)at * cstep));
        a.v[u] = __ldg(reinterpret_cast<const uint4*>(vc + (uint64_t)at * cstep));
        const uint32_t sk = __ldg(ks + (uint64_t)at * sstep), sv = __ldg(vs + (uint64_t)at * sstep);
        a.ks[u] = key < len ? sk : 0u;  // past the end: zeros, whatever the codes
        a.vs[u] = key < len ? sv : 0u;
      }
    };
    const int box = (p >> 1) * kAtBox, half = (p & 1) * 4;
    auto expand = [&](uint8_t* dst, const uint4 (&c)[2], const uint32_t (&sc)[2]) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t ss = __byte_perm(sc[u], sc[u], 0x1010), zz = __byte_perm(sc[u], sc[u], 0x3232);
        const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
        uint8_t* row = dst + box + (r + 64 * u) * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
          kv_word_bf16(w[i], ss, zz, o);
          *reinterpret_cast<uint4*>(row + (((half + i) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    bool ok = true;
    auto chunk = [&](const AtRaw& a, int j) {
      const int st = j & 1;
      const uint32_t par = (uint32_t)(((j >> 1) - 1) & 1);
      if (j >= 2) ok = ok && warp_wait(smem_u32(&kempty[st]), par, abort_flag, flag);
      if (!ok) return;
      expand(sK + st * kAtTile, a.k, a.ks);
      if (lane == 0) mbar_arrive(smem_u32(&kfull[st]));
      if (j >= 2) ok = ok && warp_wait(smem_u32(&vempty[st]), par, abort_flag, flag);
      if (!ok) return;
      expand(sV + st * kAtTile, a.v, a.vs);
      if (lane == 0) mbar_arrive(smem_u32(&vfull[st]));
    };
    AtRaw a0, a1;
    if (nc > 0) load(a0, 0);
    // Q, zeros past the last row
    for (int i = threadIdx.x - 256; i < 2 * kAtRows * 16 && nc > 0; i += kAtConv) {
      const int s = i >> 11, lrow = (i >> 4) & 127, c = i & 15;
      const int row = TWO ? s * 128 + lrow : (lrow - s * shift) & 127;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row < rows) x = *reinterpret_cast<const uint4*>(Q + row_at(row) + c * 8);
      *reinterpret_cast<uint4*>(sQ + s * kAtTile + (c >> 3) * kAtBox + lrow * 128 + (((c & 7) ^ (lrow & 7)) << 4)) = x;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(qfull));
    for (int j = 0; j < nc && ok; j += 2) {
      if (j + 1 < nc) load(a1, j + 1);
      chunk(a0, j);
      if (j + 1 >= nc || !ok) break;
      if (j + 2 < nc) load(a0, j + 2);
      chunk(a1, j + 1);
    }
  } else if (warp == 16) {
    if (lane == 0 && nc > 0) {
      // ---------------- MMA issuer: whichever product can go
      constexpr uint32_t id_s = idesc_bf16_b(128, 128, 0), id_o = idesc_bf16_b(128, 128, 1);
      const bool ok = mbar_wait(smem_u32(qfull), 0u, abort_flag, flag);
      const int total[2] = {steps(0), steps(1)};
      int si[2] = {0, 0}, pi[2] = {0, 0};  // the stream's next S, its next P V
      int kused = 0, vused = 0;            // bit s + 2 stage: stream s has issued its product with the stage's chunk
      uint32_t idle = 0;
      bool issued = false;
      while (ok && (pi[0] < total[0] || pi[1] < total[1])) {
        bool progress = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (si[s] < total[s] && si[s] == pi[s]) {
            const int j = TWO ? si[s] : 2 * si[s] + s, st = j & 1;
            if ((si[s] == 0 || mbar_test_wait(smem_u32(&pvdone[s]), (uint32_t)((si[s] - 1) & 1))) &&
                mbar_test_wait(smem_u32(&kfull[st]), (uint32_t)((j >> 1) & 1))) {
              tc_fence_after();
              const uint32_t qa = smem_u32(sQ + s * kAtTile), ka = smem_u32(sK + st * kAtTile);
#pragma unroll
              for (int kk = 0; kk < kAtHd / 16; ++kk) {
                const uint32_t off = (uint32_t)((kk >> 2) * kAtBox + (kk & 3) * 32);
                tc_mma(tmem + (uint32_t)(s * 128), smem_desc_sw128(qa + off), smem_desc_sw128(ka + off), id_s,
                       kk != 0 ? 1u : 0u);
              }
              tc_commit(smem_u32(&sfull[s]));
              kused |= 1 << (s + 2 * st);
              if (!TWO || ((kused >> (2 * st)) & 3) == 3) {
                tc_commit(smem_u32(&kempty[st]));
                kused &= ~(3 << (2 * st));
              }
              ++si[s];
              issued = true;
              progress = true;
            }
          }
          if (pi[s] < si[s]) {
            const int j = TWO ? pi[s] : 2 * pi[s] + s, st = j & 1;
            if (mbar_test_wait(smem_u32(&pready[s]), (uint32_t)(pi[s] & 1)) &&
                mbar_test_wait(smem_u32(&vfull[st]), (uint32_t)((j >> 1) & 1))) {
              tc_fence_after();
              const uint32_t va = smem_u32(sV + st * kAtTile);
#pragma unroll
              for (int kk = 0; kk < kAtKeys / 16; ++kk)
                tc_mma_ta(tmem + 256u + (uint32_t)(s * 128), tmem + (uint32_t)(s * 128 + kk * 8),
                          smem_desc_sw128_mn(va + (uint32_t)(kk * 16 * 128), kAtBox), id_o, (pi[s] | kk) != 0 ? 1u : 0u);
              tc_commit(smem_u32(&pvdone[s]));
              vused |= 1 << (s + 2 * st);
              if (!TWO || ((vused >> (2 * st)) & 3) == 3) {
                tc_commit(smem_u32(&vempty[st]));
                vused &= ~(3 << (2 * st));
              }
              ++pi[s];
              progress = true;
            }
          }
        }
        if (progress) {
          idle = 0;
        } else if (++idle >= kWaitLimit) {
          *abort_flag = 1;
          raise_flag(flag, kFlagTimeout);
          break;
        } else if ((idle & 255u) == 255u && *abort_flag) {
          break;
        }
      }
      if (issued) {  // nothing in flight when the memory is given back
        tc_commit(smem_u32(drain));
        for (uint32_t it = 0; it < kWaitLimit; ++it)
          if (mbar_try_wait(smem_u32(drain), 0u)) break;
      }
    }
  } else {
    // ---------------- softmax of stream s: TMEM lane = row
    const int s = warp >> 2, lrow = (warp & 3) * 32 + lane, ns = steps(s);
    const int row = TWO ? s * 128 + lrow : (lrow - s * shift) & 127;  // of this CTA
    // a warp without a row only keeps the barriers going
    const bool work = __any_sync(0xffffffffu, row < rows);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + (uint32_t)(s * 128), tO = tmem + lane_off + 256u + (uint32_t)(s * 128);
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int i = 0; i < ns; ++i) {
      ok = warp_wait(smem_u32(&sfull[s]), (uint32_t)(i & 1), abort_flag, flag);
      if (!ok) break;
      if (work) {
        tc_fence_after();
        const int left = len - (c0 + (TWO ? i : 2 * i + s)) * kAtKeys;  // keys from the chunk's first on
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < kAtKeys; c += 32) {
          float v[32];
          tmem_ld32(tS + (uint32_t)c, v);
          tmem_ld_wait();
          if (left < kAtKeys) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e >= left) v[e] = -INFINITY;
          }
          float x4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int e = 4; e < 32; ++e) x4[e & 3] = fmaxf(x4[e & 3], v[e]);
          mx = fmaxf(mx, fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])));
        }
        mx *= scale_log2;
        const bool need = mx > m + kApLazy;
        if (__any_sync(0xffffffffu, need)) {
          // the stream's earlier products are in O (its scores were issued after them)
          const float f = need ? exp2f(m - mx) : 1.0f;
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < kAtHd; c += 16) {
              float v[16];
              tmem_ld16(tO + (uint32_t)c, v);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] *= f;
              tmem_st16(tO + (uint32_t)c, v);
            }
          }
          if (need) {
            l *= f;
            m = mx;
          }
        }
        const float sub = m == -INFINITY ? 0.0f : m;
        float rs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kAtKeys; c += 32) {
          float v[32];
          tmem_ld32(tS + (uint32_t)c, v);
          tmem_ld_wait();
          if (left < kAtKeys) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e >= left) v[e] = -INFINITY;
          }
          float pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float x = ex2_ftz(fmaf(v[e], scale_log2, -sub)), y = ex2_ftz(fmaf(v[e + 1], scale_log2, -sub));
            rs[(e >> 1) & 3] += x + y;
            pk[e >> 1] = __uint_as_float(pack_bf16_tc(x, y));
          }
          tmem_st16(tS + (uint32_t)(c >> 1), pk);  // P lies over scores that have been read
        }
        l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(smem_u32(&pready[s]));
    }
    if (ok && ns > 0) ok = warp_wait(smem_u32(&pvdone[s]), (uint32_t)((ns - 1) & 1), abort_flag, flag);
    tc_fence_after();
    const bool have = ok && ns > 0 && work;  // whole warp
    if (TWO && splits == 1) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no key: zeros
      if (work) {
#pragma unroll
        for (int c = 0; c < kAtHd; c += 16) {
          float v[16];
          if (have) {
            tmem_ld16(tO + (uint32_t)c, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= inv;
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.0f;
          }
          if (row < rows) store16_bf16(O + row_at(row) + c, v);
        }
      }
    } else {
      asm volatile("bar.sync 2, 256;" ::: "memory");  // both streams' products are done with the tiles
      float* dst = reinterpret_cast<float*>(smem) + (size_t)(s * kAtRows + (TWO ? lrow : row)) * kAtLd;
      if (work) {
#pragma unroll
        for (int c = 0; c < kAtHd; c += 16) {
          float v[16];
          if (have) {
            tmem_ld16(tO + (uint32_t)c, v);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.0f;
          }
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(dst + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        s_m[s * kAtRows + (TWO ? lrow : row)] = m;
        s_l[s * kAtRows + (TWO ? lrow : row)] = l;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, 512);
  if (!TWO || splits > 1) {
    if (splits > 1) cluster_sync_all();
    // a warp merges a row: source k is CTA k (TWO), or stream k % 2 of CTA k / 2
    const int src = TWO ? splits : 2 * splits, warps = kAtThreads / 32;
    for (int i = split * warps + warp; i < rows; i += splits * warps) {
      const int at = TWO ? i : i + (lane & 1) * kAtRows;  // the row's place in source `lane`
      const uint32_t cta = TWO ? lane : lane >> 1;
      const float mk = lane < src ? ld_dsmem_f32(mapa_shared(smem_u32(s_m + at), cta)) : -INFINITY;
      const float ms = warp_max(mk), sub = ms == -INFINITY ? 0.0f : ms;
      const float wk = exp2f(mk - sub);
      const float ls = warp_sum(lane < src ? wk * ld_dsmem_f32(mapa_shared(smem_u32(s_l + at), cta)) : 0.0f);
      const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int k = 0; k < src; ++k) {
        const float f = __shfl_sync(0xffffffffu, wk, k);
        const int place = TWO ? i : i + (k & 1) * kAtRows;
        const float4 x = ld_dsmem_f4(mapa_shared(
            smem_u32(reinterpret_cast<float*>(smem) + (size_t)place * kAtLd + 4 * lane), TWO ? k : k >> 1));
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
      }
      uint2 u;
      u.x = pack_bf16_tc(acc.x * inv, acc.y * inv);
      u.y = pack_bf16_tc(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(O + row_at(i) + 4 * lane) = u;
    }
    __syncwarp();
    if (splits > 1) cluster_sync_all();  // no CTA leaves while another reads its memory
  }
}

inline cudaError_t quant_attention_tc_setup() {
  cudaError_t e =
      cudaFuncSetAttribute(quant_attention_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAtSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(quant_attention_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAtSmem);
  return e;
}

inline cudaError_t quant_attention_tc(const void* Q, const KvQuant& kv, const int32_t* lens, void* O, int B, int n,
                                      int L, int share, int num_sms, int* flag, cudaStream_t st) {
  const long long R = (long long)n * share;
  const bool two = R > 128;
  const long long tiles = two ? (R + 255) / 256 : 1, units = tiles * B * kv.n_kv;
  const int chunks = (L + kAtKeys - 1) / kAtKeys;
  int splits = 1;
  while (splits < kAtMaxSplits && splits < chunks && units * (splits + 1) <= num_sms) ++splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * splits), (unsigned)(B * kv.n_kv), 1);
  cfg.blockDim = dim3(kAtThreads, 1, 1);
  cfg.dynamicSmemBytes = kAtSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, two ? quant_attention_tc_kernel<true> : quant_attention_tc_kernel<false>,
                            (const __nv_bfloat16*)Q, kv, lens, (__nv_bfloat16*)O, n, L, share, splits,
                            1.4426950408889634f / sqrtf((float)kAtHd), flag);
}

}  // namespace esd
