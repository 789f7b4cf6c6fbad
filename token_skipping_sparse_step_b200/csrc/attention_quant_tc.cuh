// Partial attention over the 4-bit key/value cache for many query rows, bf16,
// head_dim 128, on the tensor cores (tcgen05): the codes of a chunk of 128 keys
// are expanded once, in shared memory, for up to 256 query rows.
//
// A CTA takes one key/value head of one sequence, a slice of its keys, and query
// rows (row i: query i / share, head kvh share + i % share) in two streams of 128
// lanes (TMEM lane = row). More than 128 rows: the streams are two row tiles, and
// each chunk serves both. Up to 128: the streams are the even and the odd chunks of
// the same rows, each with sums and an accumulator of its own. Two streams keep the
// tensor cores at work: while one's scores go through the softmax, the other's
// products run. Up to 64 (32) rows, 2 (4) copies of a row lie in the 128 lanes, and
// each copy takes a half (quarter) of every chunk's keys, with P zero at the
// others: the products cost the same, the softmax is spread over all its warps.
// Streams and copies are merged at the end.
//
// Warps: 0..3 and 4..7 the softmax of streams 0 and 1 (thread = lane: no exchange
// between threads, a row's scores in registers). A stream is a chain: S = Q K^T (M
// 128, N 128 keys, K 128 dims) into TMEM, softmax, P (bf16) into TMEM over the
// scores that it came from, O += P V with P read from there, the next S. So its
// first warp issues its MMAs too, in the time in which it would wait for them (one
// thread that issues for both and polls for what can go took 1.4x the time: it
// stands still while an MMA is queued). 8..15 expand codes, each the same 16 rows of
// K and of V in every chunk, the next chunk's K before a V that may have to wait for
// its stage: they copy codes by TMA through rings of their own (no other warp waits
// on them; registers as the ring kept too few bytes in flight: 1.65 us a chunk for
// 1.42), steps and offsets up to three chunks ahead into registers, and write bf16
// tiles [128 keys][64 dims] x 2 in the 128-byte swizzle that TMA would write (K:
// K-major operand, V: MN-major); a warp's lanes are laid out so that its 16-byte
// stores are free of bank conflicts. Without copies the softmax warps take registers
// from these (setmaxnreg).
//
// What bounds it: that chain. 16 x 1024 rows x 4096 keys x 32 heads take 1549 us (710
// TFLOP/s), 15% less without exponentials, 22% less without products, the same
// without the expansion (the tensor pipe is active 32% of the cycles); 32 x 64 rows x
// 6144 keys 1.4 us per 128 keys and CTA, 1.15 with every load, expansion and product
// taken out. A CTA's start and merge cost about 7 us, which shows where each has few
// chunks (32 x 64 rows x up to 1536 keys: 135 us).
//
// The running maximum moves only when a chunk's exceeds it by more than 2^8 (O is
// then scaled in TMEM; the result O / l is the same). P is rounded to bf16 for its
// product, everything else is float32: both operands of an MMA have one type, V's
// values are bf16 (their range leaves no other type of 16 bits), and P in two parts
// would double the product; it moves an output by at most 2^-8 of sum p |v|, the size
// of the output's own rounding. Keys at or past the sequence's length are
// masked, and read as zeros. The slices of a row tile are the CTAs of a cluster,
// merged through distributed shared memory in slice order. Every mbarrier wait is
// bounded (error flag); every CTA reaches every cluster barrier.
#pragma once

#include "attention_pair.cuh"
#include "copy_window.h"
#include "kv_quant.cuh"

namespace esd {

constexpr int kAtRows = 128, kAtKeys = 128, kAtHd = 128;
constexpr int kAtBox = 128 * 64 * 2;              // 128 rows x 64 dims
constexpr int kAtTile = 2 * kAtBox;               // Q of a stream, K or V of a chunk
// registers a thread: at launch, then (without copies: a copy's share of a row's scores leaves room as it is)
constexpr int kAtRegs = 128, kAtSoftRegs = 176, kAtOtherRegs = 80;
static_assert(kAtSoftRegs + kAtOtherRegs <= 2 * kAtRegs, "half of the threads each");
constexpr int kAtLd = kAtHd + 4;                  // floats of a merge row
constexpr int kAtConv = 8, kAtThreads = 512;  // expanding warps
constexpr int kAtRaw = kAtConv * 2 * 16 * 64;       // a chunk's codes: per warp 16 rows of K, 16 of V
constexpr int kAtStats = 2 * 2 * kAtRows * 4;     // merge: row maxima and sums of both streams (over the raw ring)
// Q, the K and V stages, the raw ring
constexpr int at_stages(bool two) { return two ? 2 : 3; }
constexpr int at_main(bool two) { return ((two ? 2 : 1) + 4) * kAtTile; }
constexpr int at_smem(bool two) { return at_main(two) + at_stages(two) * kAtRaw + 512 + 1024; }
constexpr int kAtMaxSplits = 8;
static_assert(2 * kAtRows * kAtLd * 4 <= at_main(false), "the merge rows lie over the tiles");
static_assert(kAtStats <= 2 * kAtRaw, "the merge statistics lie over the raw ring");
static_assert(at_smem(true) <= 232448 && at_smem(false) <= 232448, "227 KB");

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

__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts_f4(uint32_t addr, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

// Grid (tiles * splits, B * n_kv), cluster (splits). TWO: two row tiles per CTA
// (NSUB 1); else one of at most 128 / NSUB rows, in NSUB copies.
template <bool TWO, int NSUB>
__global__ void __launch_bounds__(kAtThreads, 1)
quant_attention_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __nv_bfloat16* Q, KvQuant cache, const int32_t* lens,
                          __nv_bfloat16* __restrict__ O, int n, int L, int share, int splits, float scale_log2,
                          int* flag) {
  static_assert(!TWO || NSUB == 1, "copies only of one tile");
  constexpr bool kTurns = NSUB == 1;
  constexpr bool kSplitRegs = NSUB == 1;
  constexpr int kStages = at_stages(TWO);
  constexpr int kPad = kAtRows / NSUB, kPer = kAtKeys / NSUB;  // lanes of a copy, its keys of a chunk
  extern __shared__ __align__(1024) uint8_t smem_at_raw[];
  grid_launch_dependents();
  grid_dependency_wait();  // from here on what the kernels before wrote is read
  const uint32_t base = (smem_u32(smem_at_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_at_raw + (base - smem_u32(smem_at_raw));
  const uint32_t aQ = base;                 // [stream (TWO)][dims 0-63 | 64-127][128 rows]
  const uint32_t aK = aQ + (TWO ? 2 : 1) * kAtTile;  // [stage][...][128 keys]
  const uint32_t aV = aK + 2 * kAtTile;
  const uint32_t aRaw = base + at_main(TWO);         // [warp][stage][16 rows of K | of V]
  float* s_m = reinterpret_cast<float*>(smem + at_main(TWO));  // [stream][128], over the ring
  float* s_l = s_m + 2 * kAtRows;
  const uint32_t bars = aRaw + kStages * kAtRaw;
  const uint32_t qfull = bars;          // Q written
  const uint32_t kfull = bars + 8;      // [2] K of a chunk written
  const uint32_t vfull = bars + 24;     // [2]
  const uint32_t kempty = bars + 40;    // [2] the scores that read it are done
  const uint32_t vempty = bars + 56;    // [2]
  const uint32_t sfull = bars + 72;     // [2] a stream's scores in TMEM
  const uint32_t pready = bars + 88;    // [2] a stream's P written, its O scaled
  const uint32_t pvdone = bars + 104;   // [2] a stream's P V accumulated
  const uint32_t drain = bars + 120;    // [2] a stream's MMAs, all of them
  const uint32_t turn = bars + 136;     // [2] the stream may take its exponentials
  const uint32_t rawfull = bars + 152;  // [warp][stage] a warp's codes have landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (bars - base) + 152 + kAtConv * kStages * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % splits, tile = blockIdx.x / splits;
  const int b = blockIdx.y / cache.n_kv, kvh = blockIdx.y % cache.n_kv;
  const int H = cache.n_kv * share, r0 = tile * 256;
  const int rows = min(n * share - r0, TWO ? 256 : kPad);  // rows of this CTA
  const int streams = TWO && rows <= kAtRows ? 1 : 2;

  const int len = lens ? min(L, max(0, lens[b])) : L;
  const int chunks = (len + kAtKeys - 1) / kAtKeys;
  const int c0 = chunks * split / splits, nc = chunks * (split + 1) / splits - c0;

  // 16 rows of codes of chunk j into the warp's stage j % kStages
  CopyWindow copies;  // started: lane 0's
  auto copy = [&](int j) {
    copies.start(j);
    const int w = warp - 8, st = j % kStages, row = b * cache.capacity + (c0 + j) * kAtKeys + 16 * w;
    const uint32_t bar = rawfull + (w * kStages + st) * 8, dst = aRaw + (w * kStages + st) * 2048;
    mbar_expect_tx(bar, 2048);
    const uint64_t policy = TWO ? policy_evict_last() : policy_evict_first();  // other row tiles read them too, or nobody
    tma_load_2d(dst, &tmK, bar, kvh * 16, row, policy);
    tma_load_2d(dst + 1024, &tmV, bar, kvh * 16, row, policy);
  };
  if (warp >= 8 && lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(rawfull + ((warp - 8) * kStages + i) * 8, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // the copies, which no barrier of the block follows first, see them too
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    for (int j = 0; j < min(kStages, nc); ++j) copy(j);
  }
  auto row_at = [&](int i) {  // of Q and O
    const int row = r0 + i, q = share == 1 ? row : row / share;
    return (((size_t)b * n + q) * H + kvh * share + row - q * share) * kAtHd;
  };
  // the expanding warps' share of Q: 16 lanes a row, eight loads in flight, zeros past the last row
  auto load_q = [&](uint4 (&x)[8], int i0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int lrow = i0 + (e * kAtConv + warp - 8) * 2 + (lane >> 4), row = TWO ? lrow : lrow % kPad;
      x[e] = row < rows ? *reinterpret_cast<const uint4*>(Q + row_at(row) + (lane & 15) * 8) : make_uint4(0, 0, 0, 0);
    }
  };
  uint4 xq[8];
  if (warp >= 8 && nc > 0) load_q(xq, 0);  // lands while the barriers are set up
  if (threadIdx.x == 0) {
    mbar_init(qfull, kAtConv);
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + 8 * i, kAtConv);
      mbar_init(vfull + 8 * i, kAtConv);
      mbar_init(kempty + 8 * i, TWO ? streams : 1);
      mbar_init(vempty + 8 * i, TWO ? streams : 1);
      mbar_init(sfull + 8 * i, 1);
      mbar_init(pready + 8 * i, 4);
      mbar_init(pvdone + 8 * i, 1);
      mbar_init(drain + 8 * i, 1);
      mbar_init(turn + 8 * i, 4);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // steps of stream s (the chunk of its step i: i, or 2 i + s)
  auto steps = [&](int s) { return TWO ? (s < streams ? nc : 0) : (nc - s + 1) >> 1; };

  if (warp >= 8) {
    if (kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtOtherRegs));
    // ---------------- codes to tiles: rows 16 w + 8 u + r of every chunk.
    // Lane bits 0 and 3: 32 dims; 1, 2 and 4: the row. A store's 8 lanes cover 4 rows x 2 halves of their 128
    // bytes, which the swizzle spreads over all banks.
    const int w = warp - 8, p = (lane & 1) | ((lane >> 2) & 2), r = ((lane >> 1) & 3) + ((lane >> 4) << 2);
    const size_t first = (size_t)b * cache.capacity * cache.n_kv + kvh;
    const int gk = 7 - cache.group_log2, gp = (32 * p) >> cache.group_log2;
    const uint32_t* ks = cache.ks + (first << gk) + gp;
    const uint32_t* vs = cache.vs + (first << gk) + gp;
    const uint32_t sstep = (uint32_t)cache.n_kv << gk;
    struct Scales {  // of the two rows
      uint32_t k[2], v[2];
    };
    auto load = [&](Scales& a, int j) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint64_t at = (uint64_t)(uint32_t)min((c0 + j) * kAtKeys + 16 * w + 8 * u + r, len - 1) * sstep;
        a.k[u] = ks[at];
        a.v[u] = vs[at];
      }
    };
    const uint32_t put = (uint32_t)((p >> 1) * kAtBox + (16 * w + r) * 128), half = (p & 1) * 4;
    auto expand = [&](uint32_t dst, const uint4 (&c)[2], const uint32_t (&sc)[2], int left) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // past the end: zeros, whatever the codes (decided here: next to its load it would wait for it)
        const uint32_t y = 16 * w + 8 * u + r < left ? sc[u] : 0u;
        const uint32_t ss = __byte_perm(y, y, 0x1010), zz = __byte_perm(y, y, 0x3232);
        const uint32_t word[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t o[4];
          kv_word_bf16(word[e], ss, zz, o);
          sts128(dst + put + u * 1024 + (((half + e) ^ r) << 4), o);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    bool ok = true;
    // K of chunk j + 1, then V of chunk j: a V stage that is not free yet does not hold back the next scores
    auto step = [&](const Scales& ak, const Scales& av, int j) {
      const uint32_t src = aRaw + w * kStages * 2048 + r * 64 + p * 16;
      const int jk = j + 1;
      if (jk < nc) {
        const int rs = jk % kStages, st = jk & 1;
        ok = warp_wait(rawfull + (w * kStages + rs) * 8, (uint32_t)((jk / kStages) & 1), abort_flag, flag);
        if (!ok) return;
        copies.land(jk);
        const uint4 c[2] = {lds128(src + rs * 2048), lds128(src + rs * 2048 + 512)};
        if (jk >= 2) ok = warp_wait(kempty + 8 * st, (uint32_t)(((jk >> 1) - 1) & 1), abort_flag, flag);
        if (!ok) return;
        expand(aK + st * kAtTile, c, ak.k, len - (c0 + jk) * kAtKeys);
        if (lane == 0) mbar_arrive(kfull + 8 * st);
      }
      if (j >= 0) {
        const int rs = j % kStages, st = j & 1;
        const uint4 c[2] = {lds128(src + rs * 2048 + 1024), lds128(src + rs * 2048 + 1536)};
        if (j >= 2) ok = warp_wait(vempty + 8 * st, (uint32_t)(((j >> 1) - 1) & 1), abort_flag, flag);
        if (!ok) return;
        expand(aV + st * kAtTile, c, av.v, len - (c0 + j) * kAtKeys);
        if (lane == 0) {
          mbar_arrive(vfull + 8 * st);
          // Only here has the stage been read: the tiles hold what the loads above brought, behind the fence that ends
          // expand(). A copy does not queue behind loads that are on their way, and could overtake them: issued before
          // the wait, it gave some keys of a head the values of a later chunk in 2 of 3 first launches of a process
          // (88 rows x 3239 keys). Nor is it late here (16 x 1024 rows x 4096 keys: 1567 -> 1549 us, the others the same)
          if (j + kStages < nc) copy(j + kStages);
        }
      }
    };
    constexpr int kSc = 4;  // chunks of steps and offsets in registers
    Scales sc[kSc];
#pragma unroll
    for (int i = 0; i < kSc - 1; ++i)
      if (i < nc) load(sc[i], i);
    if (nc > 0) {
#pragma unroll
      for (int i0 = 0; i0 < (TWO ? 2 : 1) * kAtRows; i0 += 8 * 2 * kAtConv) {
        if (i0 > 0) load_q(xq, i0);
        const int c = lane & 15;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int lrow = i0 + (e * kAtConv + w) * 2 + (lane >> 4);
          const uint32_t v[4] = {xq[e].x, xq[e].y, xq[e].z, xq[e].w};
          sts128(aQ + (lrow >> 7) * kAtTile + (c >> 3) * kAtBox + (lrow & 127) * 128 + (((c & 7) ^ (lrow & 7)) << 4), v);
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(qfull);
    if (nc > 0) step(sc[0], sc[0], -1);
    for (int j0 = 0; j0 < nc && ok; j0 += kSc) {
#pragma unroll
      for (int i = 0; i < kSc; ++i) {
        const int j = j0 + i;
        if (j + kSc - 1 < nc) load(sc[(i + kSc - 1) % kSc], j + kSc - 1);
        if (j < nc && ok) step(sc[(i + 1) % kSc], sc[i], j);
      }
    }
    // a walk that gave up: its copies land before the memory is given back
    if (!ok && lane == 0)
      copies.drain([&](int j) {
        for (uint32_t it = 0; it < kWaitLimit; ++it)
          if (mbar_try_wait(rawfull + (w * kStages + j % kStages) * 8, (uint32_t)((j / kStages) & 1))) break;
      });
  } else {
    if (kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtSoftRegs));
    // ---------------- stream s, TMEM lane lrow = copy sub of a row
    const int s = warp >> 2, lrow = (warp & 3) * 32 + lane, ns = steps(s);
    const int sub = lrow / kPad, row = TWO ? s * 128 + lrow : lrow % kPad;  // of this CTA
    // a warp without a row only keeps the barriers going
    const bool work = __any_sync(0xffffffffu, row < rows);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + (uint32_t)(s * 128), tO = tmem + lane_off + 256u + (uint32_t)(s * 128);
    const bool issuer = (warp & 3) == 0 && lane == 0;
    bool issued = false;
    auto issue_s = [&](int i) {  // S of step i, once the products of the step before are done with its P
      const int j = TWO ? i : 2 * i + s, st = j & 1;
      if (i == 0 && !mbar_wait(qfull, 0u, abort_flag, flag)) return false;
      if (i > 0 && !mbar_wait(pvdone + 8 * s, (uint32_t)((i - 1) & 1), abort_flag, flag)) return false;
      if (!mbar_wait(kfull + 8 * st, (uint32_t)((j >> 1) & 1), abort_flag, flag)) return false;
      tc_fence_after();
      const uint32_t qa = aQ + (TWO ? s * kAtTile : 0), ka = aK + st * kAtTile;
#pragma unroll
      for (int kk = 0; kk < kAtHd / 16; ++kk) {
        const uint32_t off = (uint32_t)((kk >> 2) * kAtBox + (kk & 3) * 32);
        tc_mma(tmem + (uint32_t)(s * 128), smem_desc_sw128(qa + off), smem_desc_sw128(ka + off),
               idesc_bf16_b(128, 128, 0), kk != 0 ? 1u : 0u);
      }
      tc_commit(sfull + 8 * s);
      tc_commit(kempty + 8 * st);
      issued = true;
      return true;
    };
    auto issue_pv = [&](int i) {
      const int j = TWO ? i : 2 * i + s, st = j & 1;
      if (!mbar_wait(pready + 8 * s, (uint32_t)(i & 1), abort_flag, flag)) return false;
      if (!mbar_wait(vfull + 8 * st, (uint32_t)((j >> 1) & 1), abort_flag, flag)) return false;
      tc_fence_after();
      const uint32_t va = aV + st * kAtTile;
#pragma unroll
      for (int kk = 0; kk < kAtKeys / 16; ++kk)
        tc_mma_ta(tmem + 256u + (uint32_t)(s * 128), tmem + (uint32_t)(s * 128 + kk * 8),
                  smem_desc_sw128_mn(va + (uint32_t)(kk * 16 * 128), kAtBox), idesc_bf16_b(128, 128, 1),
                  (i | kk) != 0 ? 1u : 0u);
      tc_commit(pvdone + 8 * s);
      tc_commit(vempty + 8 * st);
      return true;
    };
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    if (issuer && ns > 0) issue_s(0);  // a wait that gives up has set the flag that ends the others
    __syncwarp();
    for (int i = 0; i < ns; ++i) {
      ok = warp_wait(sfull + 8 * s, (uint32_t)(i & 1), abort_flag, flag);
      if (!ok) break;
      if (work) {
        tc_fence_after();
        float v[kPer];
#pragma unroll
        for (int c = 0; c < kPer; c += 32) tmem_ld32(tS + (uint32_t)(sub * kPer + c), *reinterpret_cast<float(*)[32]>(v + c));
        tmem_ld_wait();
        // the copy's keys that exist
        const int left = len - (c0 + (TWO ? i : 2 * i + s)) * kAtKeys - sub * kPer;
        if (left < kPer) {
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if (e >= left) v[e] = -INFINITY;
        }
        float x4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int e = 4; e < kPer; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x4[k] = e + 4 + k < kPer ? fmaxf(x4[k], fmaxf(v[e + k], v[e + 4 + k])) : fmaxf(x4[k], v[e + k]);
        const float mx = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * scale_log2;
        const bool need = mx > m + kApLazy;
        if (__any_sync(0xffffffffu, need)) {
          // the stream's earlier products are in O (its scores were issued after them)
          const float f = need ? exp2f(m - mx) : 1.0f;
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < kAtHd; c += 16) {
              float u[16];
              tmem_ld16(tO + (uint32_t)c, u);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] *= f;
              tmem_st16(tO + (uint32_t)c, u);
            }
          }
          if (need) {
            l *= f;
            m = mx;
          }
        }
        // the two streams take their exponentials in turn: at once, each would take twice as long, and the tensor
        // cores would wait for both
        if (kTurns && streams == 2 && (s == 1 || i > 0)) {
          ok = warp_wait(turn + 8 * s, (uint32_t)((s == 1 ? i : i - 1) & 1), abort_flag, flag);
          if (!ok) break;
        }
        const float sub_m = m == -INFINITY ? 0.0f : -m;
        const uint64_t sc2 = pack_f2(scale_log2, scale_log2), m2 = pack_f2(sub_m, sub_m);
        uint64_t rs[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < kPer; c += 32) {
          float pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x, y;
            unpack_f2(fma_f2(pack_f2(v[c + e], v[c + e + 1]), sc2, m2), x, y);
            x = ex2_ftz(x);
            y = ex2_ftz(y);
            rs[(e >> 1) & 1] = add_f2(rs[(e >> 1) & 1], pack_f2(x, y));
            pk[e >> 1] = __uint_as_float(pack_bf16_tc(x, y));
          }
          tmem_st16(tS + (uint32_t)((sub * kPer + c) >> 1), pk);  // P lies over scores that have been read
        }
        if (NSUB > 1) {  // the other copies' keys
          float zero[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) zero[e] = 0.0f;
#pragma unroll
          for (int c = 0; c < kAtKeys - kPer; c += 32)
            tmem_st16(tS + (uint32_t)(((sub * kPer + kPer + c) % kAtKeys) >> 1), zero);
        }
        if (kTurns && lane == 0) mbar_arrive(turn + 8 * (1 - s));
        float a0, a1;
        unpack_f2(add_f2(rs[0], rs[1]), a0, a1);
        l += a0 + a1;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
      }
      if (kTurns && !work && lane == 0) mbar_arrive(turn + 8 * (1 - s));
      if (lane == 0) mbar_arrive(pready + 8 * s);
      if (issuer && issue_pv(i) && i + 1 < ns) issue_s(i + 1);
      __syncwarp();
    }
    if (issuer && issued) {  // nothing in flight when the memory is given back
      tc_commit(drain + 8 * s);
      for (uint32_t it = 0; it < kWaitLimit; ++it)
        if (mbar_try_wait(drain + 8 * s, 0u)) break;
    }
    __syncwarp();
    if (ok && ns > 0) ok = warp_wait(pvdone + 8 * s, (uint32_t)((ns - 1) & 1), abort_flag, flag);
    tc_fence_after();
    const bool have = ok && ns > 0 && work;  // whole warp
    const bool direct = TWO && splits == 1;
    if (!direct) asm volatile("bar.sync 2, 256;" ::: "memory");  // both streams' products are done with the tiles
    if (work) {
      const float inv = direct ? 1.0f / l : 1.0f;  // all scores -inf: NaN (no key: zeros below)
      const uint32_t dst = base + (uint32_t)((s * kAtRows + lrow) * kAtLd * 4);
#pragma unroll
      for (int c = 0; c < kAtHd; c += 16) {
        float u[16];
        if (have) {
          tmem_ld16(tO + (uint32_t)c, u);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] *= inv;
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] = 0.0f;
        }
        if (!direct) {
#pragma unroll
          for (int e = 0; e < 16; e += 4) sts_f4(dst + (c + e) * 4, u[e], u[e + 1], u[e + 2], u[e + 3]);
        } else if (row < rows) {
          store16_bf16(O + row_at(row) + c, u);
        }
      }
      s_m[s * kAtRows + lrow] = m;
      s_l[s * kAtRows + lrow] = l;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (!TWO && splits == 1) {
    // the streams and copies of this CTA alone: eight threads a row
    for (int i = threadIdx.x; i < rows * 8; i += kAtThreads) {
      const int r = i >> 3, part = i & 7;
      float w[2 * NSUB], ms = -INFINITY, ls = 0.0f;
#pragma unroll
      for (int k = 0; k < 2 * NSUB; ++k) ms = fmaxf(ms, w[k] = s_m[r + k * kPad]);
      const float sub = ms == -INFINITY ? 0.0f : ms;
#pragma unroll
      for (int k = 0; k < 2 * NSUB; ++k) {
        w[k] = exp2f(w[k] - sub);
        ls += w[k] * s_l[r + k * kPad];
      }
      const float inv = len == 0 ? 0.0f : 1.0f / ls;  // no key: zeros
      __nv_bfloat16* dst = O + row_at(r);
      const float* src = reinterpret_cast<const float*>(smem) + r * kAtLd;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 4 * (part + 8 * e);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < 2 * NSUB; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(src + k * kPad * kAtLd + c);
          acc.x = fmaf(w[k], x.x, acc.x);
          acc.y = fmaf(w[k], x.y, acc.y);
          acc.z = fmaf(w[k], x.z, acc.z);
          acc.w = fmaf(w[k], x.w, acc.w);
        }
        uint2 u;
        u.x = pack_bf16_tc(acc.x * inv, acc.y * inv);
        u.y = pack_bf16_tc(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(dst + c) = u;
      }
    }
  } else if (splits > 1) {
    cluster_sync_all();
    // a warp merges a row: source k is CTA k (TWO), or stream and copy k % (2 NSUB) of CTA k / (2 NSUB); lane k % 32
    // holds its weight (at most 64 sources)
    constexpr int kOf = TWO ? 1 : 2 * NSUB, kStep = TWO ? 0 : kPad;
    const int src = kOf * splits;
    for (int i = split * (kAtThreads / 32) + warp; i < rows; i += splits * (kAtThreads / 32)) {
      float mk[2], wk[2], ms = -INFINITY, ls = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = lane + 32 * e;
        mk[e] = k < src ? ld_dsmem_f32(mapa_shared(smem_u32(s_m + i + k % kOf * kStep), k / kOf)) : -INFINITY;
        ms = fmaxf(ms, mk[e]);
      }
      ms = warp_max(ms);
      const float sub = ms == -INFINITY ? 0.0f : ms;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = lane + 32 * e;
        wk[e] = exp2f(mk[e] - sub);
        if (k < src) ls += wk[e] * ld_dsmem_f32(mapa_shared(smem_u32(s_l + i + k % kOf * kStep), k / kOf));
      }
      ls = warp_sum(ls);
      const float inv = len == 0 ? 0.0f : 1.0f / ls;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll 4
        for (int k = 32 * e; k < min(src, 32 * e + 32); ++k) {
          const float f = __shfl_sync(0xffffffffu, wk[e], k & 31);
          const float4 x = ld_dsmem_f4(
              mapa_shared(base + (uint32_t)((i + k % kOf * kStep) * kAtLd * 4 + 16 * lane), k / kOf));
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
    cluster_sync_all();  // no CTA leaves while another reads its memory
  }
}

using AtKernel = void (*)(const CUtensorMap, const CUtensorMap, const __nv_bfloat16*, KvQuant, const int32_t*, __nv_bfloat16*, int, int, int, int, float, int*);

// Shared-memory opt-in. The register split of the first two kernels adds up only if
// they were built with kAtRegs: a launch with fewer would wait for registers for
// good. Then *usable stays false, and the calls that need them are refused.
inline cudaError_t quant_attention_tc_setup(bool* usable) {
  *usable = true;
  const AtKernel all[] = {quant_attention_tc_kernel<true, 1>, quant_attention_tc_kernel<false, 1>,
                          quant_attention_tc_kernel<false, 2>, quant_attention_tc_kernel<false, 4>};
  for (int i = 0; i < 4; ++i) {
    AtKernel k = all[i];
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, k);
    if (e == cudaSuccess && i < 2 && a.numRegs < kAtRegs) *usable = false;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, at_smem(i == 0));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Codes [rows][n_kv * 16] words, boxes of one head's 16 words x 16 rows.
inline bool at_encode(const TcPlan& pl, CUtensorMap* m, const void* codes, const KvQuant& kv, int B) {
  const cuuint64_t dim[2] = {(cuuint64_t)kv.n_kv * 16, (cuuint64_t)B * kv.capacity}, stride[1] = {(cuuint64_t)kv.n_kv * 64};
  const cuuint32_t box[2] = {16, 16}, one[2] = {1, 1};
  return pl.encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(codes), dim, stride, box, one,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline cudaError_t quant_attention_tc(const TcPlan& pl, const void* Q, const KvQuant& kv, const int32_t* lens, void* O, int B, int n,
                                      int L, int share, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!at_encode(pl, &mk, kv.kc, kv, B) || !at_encode(pl, &mv, kv.vc, kv, B)) return cudaErrorInvalidValue;
  const long long R = (long long)n * share;
  const long long tiles = R > 128 ? (R + 255) / 256 : 1, units = tiles * B * kv.n_kv;
  const int chunks = (L + kAtKeys - 1) / kAtKeys;
  // Slices of the keys while every CTA has an SM of its own, as many as pay: a step of a stream takes about 3.5 us (two
  // row tiles; 2.8 us for one, two chunks), a merge of s CTAs about 2 + 1.5 s (32 heads, 192 rows x 768 keys: 26.6,
  // 22.0, 18.5 and 19.2 us in 1 to 4 slices; 64 rows: 14.4, 15.0, 14.7 and 16.6; 192 rows x 4096 keys: 112, 64, 48
  // and 39). More CTAs than SMs lose in any case (64 rows x 2048 keys x 96 heads: 28.6 us in one, 41 in two).
  int splits = 1;
  float best = 1e30f;
  for (int k = 1; k <= kAtMaxSplits && k <= chunks && (k == 1 || units * k <= pl.num_sms); ++k) {
    const int per = (chunks + k - 1) / k;
    const float t = R > 128 ? 3.5f * per : 2.8f * ((per + 1) / 2);
    const float all = t + (k > 1 ? 2.0f + 1.5f * k : 0.0f);
    if (all < best) {
      best = all;
      splits = k;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * splits), (unsigned)(B * kv.n_kv), 1);
  cfg.blockDim = dim3(kAtThreads, 1, 1);
  cfg.dynamicSmemBytes = at_smem(R > 128);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  // started while the kernel before ends only where every CTA is resident at once (192 rows x 768 keys: 20.5 -> 19.2
  // us a call; 16 x 1024 rows x 4096 keys lose 3%)
  cfg.numAttrs = units * splits <= pl.num_sms ? 2 : 1;
  const AtKernel k = R > 128  ? quant_attention_tc_kernel<true, 1>
                     : R > 64 ? quant_attention_tc_kernel<false, 1>
                     : R > 32 ? quant_attention_tc_kernel<false, 2>
                              : quant_attention_tc_kernel<false, 4>;
  return cudaLaunchKernelEx(&cfg, k, mk, mv, (const __nv_bfloat16*)Q, kv, lens, (__nv_bfloat16*)O, n, L, share, splits,
                            1.4426950408889634f / sqrtf((float)kAtHd), pl.flag);
}

}  // namespace esd
