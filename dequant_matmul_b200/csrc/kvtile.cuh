#pragma once
// Attention over the paged Q3 KV cache for many rows per kv head (chunks of new
// tokens): 128 (token, head) rows x 64 keys at a time on the tcgen05 tensor
// cores (sm_100a).  The mathematics, the sharing of the work and the join are
// those of kvattn.cuh.
//
// A CTA works on one row tile at a time.  Tensor memory: O [128 x 256] fp32 in
// columns 0..255, the rotated rows Q [128 x 256] binary16 in 256..383, two score
// tiles S [128 x 64] fp32 in 384..511, each overwritten by its P (binary16, 32
// columns).  Q and P are the A operands (so shared memory carries only what is
// decoded); K [64 keys][256 dims] and V^T [256 dims][64 keys] are the B operands,
// both K-major with the 128-byte swizzle, decoded there from the 3-bit codes.
//
// Roles (18 warps):
//   0..7   softmax: two threads per row (warps q and q + 4 of tensor-memory quarter
//          q), half the columns each.  They put Q into tensor memory (rotated in
//          two passes over the columns of O, which are free then), turn S(j) into
//          P(j), rescale O when a row's reference rises (seldom, as in the few-row
//          kernel; one reducing barrier of the two warps finds out), rotate O back
//          and write the rows.
//   8..15  decode: code pairs -> binary16 pairs through the 64-entry table (one
//          copy per lane) -> 16-byte stores into the K and V^T tiles; window
//          tiles are copied (K) and transposed (V) as they are, bf16.
//   16     issues the MMAs: S(j + 1), then O += P(j) V(j).
//   17     fetches codes and norms, 16 keys (never two pages) per bulk copy.
//
// Keys stand in the tiles in an order that keeps every shared-memory access of
// the decoders free of bank conflicts: row n = 8 w + g of the K tile is key
// 16 (g & 3) + 2 (g >> 2) + f(w), f = 0 1 4 5 8 9 12 13, and place 8 g + w of V^T's
// rows is the same key; P's columns follow by picking registers.  The 16-key
// groups of a stage are 16 bytes further apart than their contents for the same reason.
//
// Fewer than 32 bits: as in the few-row kernel (query and p n 11 bits, centroids about
// 14).  A second part of the query has no room: O, Q and the two S tiles fill the tensor
// memory, and of shared memory 42 of the 64 KB that it takes are free.
//
// What bounds it, per tile of 64 keys (about 2900 cycles; the matrix work is 1024):
// the softmax warps, busy for some 2500 cycles from S(j) to P(j) (tensor-memory
// reads, norms and their logarithms, 8192 exponentials at 16 per cycle, packing; the
// logarithms, which let the reference follow p n, are 2 % of the time), close to the decoders' 2250
// and to shared memory, whose 128 bytes per cycle are busy four fifths of the time
// (table reads and tile stores 1000 cycles, staging and norms 300, the MMAs' B
// operands 512).  Tried and slower: four threads per row (1.07 times the time),
// tiles taken in turn by two sets of softmax warps (1.2; the two S tiles that
// tensor memory has room for then wait for each other), one issuing thread per product
// (1.07), pairs of CTAs that decode half each for 256 rows (1.02 to 1.07).
//
// Every wait is bounded (wait_limit_ns from its own beginning), after which the
// kernel raises HLWQ_DEVERR_TIMEOUT, drains its copies and MMAs and frees its
// tensor memory.

#include <type_traits>

#include "gemm_tc.cuh"
#include "kvattn.cuh"

namespace hlwq {

namespace {

constexpr int kAtRows = 128;
constexpr int kAtWarps = 18, kAtThreads = 32 * kAtWarps;
constexpr int kAtDec0 = 8, kAtMma = 16;
constexpr int kAtWinUnit = 64;
constexpr int kAtItemCost = 8;                       // units: an item takes about 12 us besides its tiles of 1.5 us
constexpr int kGrp = 1536 + 16;                      // 16 keys' codes, and the gap
constexpr int kCodeStage = 12800;                    // K codes, V codes, norms [2][64] binary16, mask
constexpr int kCodeStages = 3;
constexpr int kNormOff = 2 * 4 * kGrp;               // 12416
constexpr int kMaskOff = kNormOff + 256;
constexpr int kKvTile = 64 * 256 * 2;                // one K or V^T tile
constexpr int kNrmSlot = 192 * 4 + 16;               // K norms, V norms (kNvScale times), log2_above of V's, mask
constexpr int kSlotMask = 192 * 4;
constexpr float kMinQm = 1e-36f;                     // encoded scores of less are 0; log2_above / kMinQm is finite
constexpr int kPasses = 3;                           // of a tile while rows' shifts move: the third finds them exact
constexpr uint32_t kColO = 0, kColQ = 256, kColS = 384;
constexpr int kAtSmem = 8192 /*align*/ + 8192 /*table*/ + 4 * kKvTile + kCodeStages * kCodeStage + 4 * kNrmSlot + 512 +
                        2 * kAtRows * 4 /*row exchange*/;
static_assert(kMaskOff + 4 <= kCodeStage, "code stage");
static_assert(kAtSmem <= 227 * 1024, "shared memory");

// Offset of key n of a tile (its row in the K tile, its score column).
__host__ __device__ constexpr int at_key(int n) {
  return 16 * (n & 3) + 2 * ((n >> 2) & 1) + ((n >> 3) & 1) + 4 * (n >> 4);
}

// Instruction descriptor: kind::f16 with binary16 or bfloat16 operands, K-major, D fp32, M = 128.
__host__ __device__ constexpr uint32_t idesc_16(int n, bool bf16) {
  return idesc_f16(n) | (bf16 ? (1u << 7) | (1u << 10) : 0u);
}

// Bounded wait whose limit starts when it has to wait.
__device__ __forceinline__ bool at_wait(uint32_t bar, uint32_t parity) {
  uint64_t deadline = 0;
  for (uint32_t n = 1;; ++n) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((n & 63u) == 0u) {
      const uint64_t t = globaltimer_ns();
      if (deadline == 0) deadline = t + wait_limit_ns();
      else if (t > deadline) return false;
    }
  }
}

// MMAs and commits are issued by one elected lane, but in warp-uniform control flow:
// descriptors and addresses then stay in uniform registers.  Inside a branch of
// one lane every MMA took about 90 cycles to issue, here 50.
__device__ __forceinline__ void at_mma(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The MMAs issued so far arrive at this barrier when they are done.
__device__ __forceinline__ void at_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// The same for a whole warp: all lanes or none.
__device__ __forceinline__ bool at_wait_warp(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, at_wait(bar, parity));
}

// No MMA may be under way when the tensor memory is freed: an issuing warp that
// gives up waits for the ones it has issued, on a barrier of its own.
__device__ __forceinline__ void drain_mma(uint32_t bar, int lane) {
  if (lane == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  __syncwarp();
  at_commit(bar);
  at_wait_warp(bar, 0);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ void tc_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ void tc_ld4(uint32_t taddr, uint32_t (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(taddr)
               : "memory");
}

__device__ __forceinline__ float2 fma2_up(float2 a, float2 b, float2 c) {  // rounded upwards
  float2 r;
  asm("{ .reg .b64 pa, pb, pc, pd; mov.b64 pa, {%2, %3}; mov.b64 pb, {%4, %5}; mov.b64 pc, {%6, %7};\n\t"
      "fma.rp.f32x2 pd, pa, pb, pc; mov.b64 {%0, %1}, pd; }"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// 64 columns of this warp's rows <-> registers.
__device__ __forceinline__ void tc_ld64(uint32_t taddr, float (&v)[64]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t x[16];
    tc_ld16(taddr + 16 * c, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[16 * c + i] = __uint_as_float(x[i]);
  }
  tc_wait_ld();
}

__device__ __forceinline__ void tc_st64(uint32_t taddr, const float (&v)[64]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(v[16 * c + i]);
    tc_st16(taddr + 16 * c, x);
  }
}

__device__ __forceinline__ void fwht64(float (&v)[64]) {
#pragma unroll
  for (int h = 1; h < 64; h <<= 1)
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if ((i & h) == 0) {
        const float a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
}

// The two warps of a tensor-memory quarter: barrier 1 + quarter, 64 threads.
__device__ __forceinline__ void pair_sync(int quarter) {
  tc_fence_before();
  asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
  tc_fence_after();
}

// Whether x holds for any thread of the two warps (a barrier for both).  A warp whose
// wait ran out tells the other one here before it gives up, so that
// neither is left at a barrier.
__device__ __forceinline__ bool pair_any(int quarter, bool x) {
  uint32_t y;
  tc_fence_before();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"(x ? 1u : 0u), "r"(1 + quarter)
      : "memory");
  tc_fence_after();
  return y != 0u;
}

// The 64-column blocks 2 half, 2 half + 1 of the 256-point transform of a row in O's columns.
__device__ __forceinline__ void within_blocks(uint32_t row, int half) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    float v[64];
    tc_ld64(row + kColO + 128 * half + 64 * c, v);
    fwht64(v);
    tc_st64(row + kColO + 128 * half + 64 * c, v);
  }
  tc_wait_st();
}

// Then across the blocks: four values 64 columns apart at a time, 16 columns per
// step, columns 32 half .. + 31 of each block; f(c, v) takes column c + 64 k + i
// as v[16 k + i].
template <class F>
__device__ __forceinline__ void across_blocks(uint32_t row, int half, F&& f) {
#pragma unroll 1
  for (int c = 32 * half; c < 32 * half + 32; c += 16) {
    float v[64];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t x[16];
      tc_ld16(row + kColO + 64 * k + c, x);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[16 * k + i] = __uint_as_float(x[i]);
    }
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float p = v[i] + v[16 + i], q = v[i] - v[16 + i], r = v[32 + i] + v[48 + i], s = v[32 + i] - v[48 + i];
      v[i] = p + r;
      v[16 + i] = q + s;
      v[32 + i] = p - r;
      v[48 + i] = q - s;
    }
    f(c, v);
  }
  tc_wait_st();
}

__global__ void __launch_bounds__(kAtThreads, 1)
kv_attn_tile_kernel(const KvAttn a, int tiles, float* __restrict__ parts, KvCut* __restrict__ cuts) {
  extern __shared__ __align__(16) uint8_t asm_raw[];
  __shared__ int64_t warp_sums[kAtWarps], found[2];
  __shared__ uint32_t best_scale[kAtWarps];
  __shared__ float back;
  pdl_trigger();
  const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(asm_raw));
  const uint32_t tab0 = (raw + 8191u) & ~8191u;
  uint8_t* g0 = asm_raw + (tab0 - raw);
  const uint32_t k_tiles = tab0 + 8192, v_tiles = k_tiles + 2 * kKvTile, codes = v_tiles + 2 * kKvTile;
  const uint32_t nrm = codes + kCodeStages * kCodeStage, bars = nrm + 4 * kNrmSlot;
  const uint32_t c_full = bars, c_empty = c_full + 8 * kCodeStages, k_full = c_empty + 8 * kCodeStages, k_empty = k_full + 16,
                 v_full = k_empty + 16, v_empty = v_full + 16, s_full = v_empty + 16, p_full = s_full + 16,
                 q_full = p_full + 16, misc = q_full + 8;
  volatile uint32_t* misc_g = reinterpret_cast<volatile uint32_t*>(g0 + (misc - tab0));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) cuts[blockIdx.x] = {0, 0, 0, 0};
  choose_centroid_scale<kAtThreads>(a.codebook, best_scale);
  int64_t mine0;
  const int64_t U = kv_total_cost<kAtRows, kAtWinUnit, kAtItemCost, kAtThreads>(a, tiles, warp_sums, mine0);
  const KvShares share(U, blockIdx.x, gridDim.x);
  if (share.i >= share.ctas) return;  // before any barrier or tensor memory
  kv_find<kAtRows, kAtWinUnit, kAtItemCost, kAtThreads>(a, tiles, mine0, share(share.i), found);
  KvWalk<kAtRows, kAtWinUnit, kAtItemCost> w;
  w.begin(a, tiles, share, found);

  kv_check_codebook(a.codebook);
  fill_centroid_table<kAtThreads>(a.codebook, best_scale, reinterpret_cast<uint32_t*>(g0), &back);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kCodeStages; ++s) {
      mbar_init(c_full + 8 * s, 1);
      mbar_init(c_empty + 8 * s, 8);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full + 8 * s, 8);
      mbar_init(k_empty + 8 * s, 1);
      mbar_init(v_full + 8 * s, 8);
      mbar_init(v_empty + 8 * s, 1);
      mbar_init(s_full + 8 * s, 1);
      mbar_init(p_full + 8 * s, 8);
    }
    mbar_init(q_full, 8);
    fence_barrier_init();
  }
  if (warp == kAtMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(misc), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc_g[0];
  bool ok = true;

  // Tiles are numbered through the CTA's whole share: gt, and ce for encoded ones.
  // Ring slot and parity of tile j: j % 2 and (j / 2) & 1.
  if (warp < kAtDec0) {
    // ------------------------------------------------------------ softmax
    const int half = warp >> 2, quarter = warp & 3, r = 32 * quarter + lane;  // r: row of the tile
    const uint32_t row = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const float sgn = a.scale < 0.0f ? -1.0f : a.scale > 0.0f ? 1.0f : 0.0f;  // a zero scale: Q is 0, qm is not
    float* mine = reinterpret_cast<float*>(g0 + (bars + 512 - tab0)) + half * kAtRows + r;       // exchange with the
    const float* other = reinterpret_cast<float*>(g0 + (bars + 512 - tab0)) + (half ^ 1) * kAtRows + r;  // row's other thread
    uint32_t gt = 0;
    // the product of tile j has been added to O (tile j - 2's was before S(j) came)
    auto pv_done = [&](uint32_t j) { return at_wait_warp(v_empty + 8 * (j & 1u), (j >> 1) & 1u); };
    while (ok && w.next(a, tiles)) {
      const KvItem& it = w.it;
      const bool on = r < it.nrows;
      const int tr = it.row0 + (on ? r : 0), tok = tr / a.G, head = w.h * a.G + (tr - tok * a.G);
      const uint16_t* qrow = a.q + static_cast<int64_t>(it.c0 + tok) * a.ldq + head * kKvDim;
      const int lim = on ? it.p + tok + 1 : 0;
      if (threadIdx.x == 0) {
        KvCut cut;
        if (w.note(share, cut)) cuts[blockIdx.x] = cut;
      }
      // m: the row's reference, which follows its largest p n as in the few-row
      // kernel; l: this thread's share of the row's sum
      float m = kMinM, l = 0.0f, qm = 0.0f, inv_qm = 0.0f;
      float shift = 0.0f;    // what is taken off the row's scores first, where they are large
      bool far = false;      // any row of the two warps has one
      float q_inv = 0.0f;    // what takes the row's power of two back (0: not looked for yet)
      bool started = false;  // O holds something

      // One tile: S(gt) -> P(gt).  win: window keys, p in two bf16 parts.  This
      // thread's score columns are 8 i + 4 half + k (i < 8, k < 4), v[i][k].
      auto tile = [&](auto win, int k0, int end) -> bool {
        constexpr bool kWin = decltype(win)::value;
        const uint32_t s = gt & 1u, par = (gt >> 1) & 1u;
        const uint32_t sc = row + kColS + 64 * s, nb = nrm + (gt & 3u) * kNrmSlot + 16 * half;
        const bool got = at_wait_warp(s_full + 8 * s, par);
        tc_fence_after();
        float2 v[8][2];
        for (int pass = 0;; ++pass) {  // again where a row's shift moves
          uint32_t x[8][4];
#pragma unroll
          for (int i = 0; i < 8; ++i) tc_ld4(sc + 8 * i + 4 * half, x[i]);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[i][0] = make_float2(__uint_as_float(x[i][0]), __uint_as_float(x[i][1]));
            v[i][1] = make_float2(__uint_as_float(x[i][2]), __uint_as_float(x[i][3]));
          }
          if constexpr (!kWin) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 x = lds_f4(nb + 32 * i);
              v[i][0] = mul2(v[i][0], make_float2(x.x, x.y));
              v[i][1] = mul2(v[i][1], make_float2(x.z, x.w));
            }
          }
          if (far) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int k = 0; k < 2; ++k) v[i][k] = make_float2(__fsub_rn(v[i][k].x, shift), __fsub_rn(v[i][k].y, shift));
          }
          const uint32_t there = kWin ? 15u : lds32(nb - 16 * half + kSlotMask);  // 16-key groups whose page is there
          const int see = min(lim, end) - k0;
          if (__any_sync(0xffffffffu, see < 64) || there != 15u) {
            const int sh = see - 2 * half;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int f = at_key(8 * i);
              if (f >= sh || !(there & 1u)) v[i][0].x = -INFINITY;
              if (f + 16 >= sh || !(there & 2u)) v[i][0].y = -INFINITY;
              if (f + 32 >= sh || !(there & 4u)) v[i][1].x = -INFINITY;
              if (f + 48 >= sh || !(there & 8u)) v[i][1].y = -INFINITY;
            }
          }
          // the largest score + log2 norm, rounded so that p n never passes 2^8
          float mx = -INFINITY, my = -INFINITY;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float2 x = v[i][0], y = v[i][1];
            if constexpr (!kWin) {
              const float4 z = lds_f4(nb + 512 + 32 * i);
              x = fma2_up(make_float2(z.x, z.y), make_float2(inv_qm, inv_qm), x);
              y = fma2_up(make_float2(z.z, z.w), make_float2(inv_qm, inv_qm), y);
            }
            mx = fmaxf(fmaxf(x.x, x.y), mx);
            my = fmaxf(fmaxf(y.x, y.y), my);
          }
          mx = __fmul_ru(fmaxf(mx, my), qm);
          if constexpr (kWin) mx = __fadd_ru(mx, kWinSize);
          // also: both halves of S have been read, P may take its place
          if (!pair_any(quarter, !got || mx > __fadd_rd(m, 8.0f))) break;  // nearly always
          if (pair_any(quarter, !got)) return false;
          *mine = mx;
          pair_sync(quarter);
          const float nm = fmaxf(m, fmaxf(mx, *other));
          pair_sync(quarter);
          const bool big = nm > m && fabsf(nm) > (far ? kFarNext : kFar);
          if (pass < kPasses && __any_sync(0xffffffffu, big)) {  // the other warp has the same rows
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fmaxf(v[i][0].x, v[i][0].y), fmaxf(v[i][1].x, v[i][1].y)));
            *mine = top;
            pair_sync(quarter);
            if (big) {
              const float to = shift + fmaxf(top, *other);
              if (m != kMinM) m = fmaf(shift - to, qm, m);
              shift = to;
            }
            far = true;
            pair_sync(quarter);
            continue;
          }
          const float corr = ex2(m - nm);
          m = nm;
          l *= corr;
          if (started) {  // rescale O once the product before has been added
            if (pair_any(quarter, !pv_done(gt - 1))) return false;
#pragma unroll 1
            for (int c = 128 * half; c < 128 * half + 128; c += 16) {
              uint32_t x[16];
              tc_ld16(row + kColO + c, x);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * corr);
              tc_st16(row + kColO + c, x);
            }
          }
          break;
        }
        // p = 2^(s qm - m), and its sum
        const float2 q2 = make_float2(qm, qm), b2 = make_float2(-m, -m);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 x = fma2(v[i][k], q2, b2);
            v[i][k] = make_float2(ex2(x.x), ex2(x.y));
            sum[k] = add2(sum[k], v[i][k]);
          }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        // place 8 g + i of V's rows is the key of score column 8 i + g; word (g, i / 2)
        if constexpr (!kWin) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 x = lds_f4(nb + 256 + 32 * i);
            v[i][0] = mul2(v[i][0], make_float2(x.x, x.y));
            v[i][1] = mul2(v[i][1], make_float2(x.z, x.w));
          }
          uint32_t x[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = pack_half2(v[2 * i][0].x, v[2 * i + 1][0].x);
            x[4 + i] = pack_half2(v[2 * i][0].y, v[2 * i + 1][0].y);
            x[8 + i] = pack_half2(v[2 * i][1].x, v[2 * i + 1][1].x);
            x[12 + i] = pack_half2(v[2 * i][1].y, v[2 * i + 1][1].y);
          }
          tc_st16(sc + 16 * half, x);
        } else {
          uint32_t hi[16], lo[16];
          auto split = [&](int j, float x, float y) {
            hi[j] = pack_bf162(x, y);
            lo[j] = pack_bf162(x - bf16x2_lo(hi[j]), y - bf16x2_hi(hi[j]));
          };
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            split(i, v[2 * i][0].x, v[2 * i + 1][0].x);
            split(4 + i, v[2 * i][0].y, v[2 * i + 1][0].y);
            split(8 + i, v[2 * i][1].x, v[2 * i + 1][1].x);
            split(12 + i, v[2 * i][1].y, v[2 * i + 1][1].y);
          }
          tc_st16(sc + 16 * half, hi);
          tc_st16(sc + 32 + 16 * half, lo);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * s);
        started = true;
        ++gt;
        return true;
      };

      if (w.ta < w.e_tb) {
        // Q, rotated: this thread's two blocks of 64 dims, then its columns across
        // the blocks, into binary16
        float mx = 0.0f;
#pragma unroll 1
        for (int c = 2 * half; c < 2 * half + 2; ++c) {
          float v[64];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (on) x = __ldg(reinterpret_cast<const uint4*>(qrow + 64 * c) + i);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) v[8 * i + 2 * k] = bf16x2_lo(xs[k]), v[8 * i + 2 * k + 1] = bf16x2_hi(xs[k]);
          }
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            mx = fmaxf(mx, fabsf(v[i]));
            v[i] *= 1.0f / 512.0f;  // no sum of 256 values overflows
          }
          fwht64(v);
          tc_st64(row + kColO + 64 * c, v);
        }
        tc_wait_st();
        *mine = mx;
        pair_sync(quarter);
        const float sc = sgn * 512.0f * pow2_scale(fmaxf(mx, *other), q_inv);
        qm = sgn == 0.0f ? 1.0f : fmaxf(fabsf(a.scale) * q_inv * (kLog2e / 256.0f) * back, kMinQm);
        inv_qm = 1.0f / qm;
        across_blocks(row, half, [&](int c, const float(&v)[64]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = pack_half2(v[16 * k + 2 * i] * sc, v[16 * k + 2 * i + 1] * sc);
            tc_st8(row + kColQ + 32 * k + (c >> 1), x);
          }
        });
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        for (int t = w.ta; ok && t < w.e_tb; ++t) ok = tile(std::false_type{}, t * kUnit, it.e_lim);
        if (!ok || pair_any(quarter, !pv_done(gt - 1))) {
          ok = false;
          break;
        }
        // O out of the rotated domain
        within_blocks(row, half);
        pair_sync(quarter);
        const float nm = m + kWinSize, corr = ex2(m - nm);  // the window's reference, at once
        const float f = corr * back / (256.0f * kNvScale);
        l *= corr;
        m = nm;
        across_blocks(row, half, [&](int c, const float(&v)[64]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(v[16 * k + i] * f);
            tc_st16(row + kColO + 64 * k + c, x);
          }
        });
        pair_sync(quarter);
      }
      if (w.e_tb < w.tb) {
        // window units: Q not rotated, its bf16 bits with another exponent
        if (q_inv == 0.0f) {
          __nv_bfloat162 mx = __float2bfloat162_rn(0.0f);
#pragma unroll 4
          for (int i = 0; i < 16; ++i) {
            uint4 y = make_uint4(0u, 0u, 0u, 0u);
            if (on) y = __ldg(reinterpret_cast<const uint4*>(qrow + 128 * half) + i);
            const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
            for (int k = 0; k < 4; ++k) mx = __hmax2(mx, __habs2(p[k]));
          }
          const float2 f = __bfloat1622float2(mx);
          *mine = fmaxf(f.x, f.y);
          pair_sync(quarter);
          pow2_scale(fmaxf(fmaxf(f.x, f.y), *other), q_inv);
        }
        const __nv_bfloat162 sc = __float2bfloat162_rn(sgn / q_inv);
#pragma unroll 1
        for (int c = 4 * half; c < 4 * half + 4; ++c) {
          uint32_t x[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 y = make_uint4(0u, 0u, 0u, 0u);
            if (on) y = __ldg(reinterpret_cast<const uint4*>(qrow + 32 * c) + i);
            const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 z = __hmul2(__hmul2(p[k], sc), __float2bfloat162_rn(kWinScale));
              x[4 * i + k] = *reinterpret_cast<const uint32_t*>(&z);
            }
          }
          tc_st16(row + kColQ + 16 * c, x);
        }
        tc_wait_st();
        const float was = qm;
        qm = sgn == 0.0f ? 1.0f : fmaxf(window_qm(fabsf(a.scale) * q_inv * (kLog2e / kWinScale)), kMinQm);
        if (far) shift *= was / qm;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        for (int t = w.e_tb; ok && t < w.tb; ++t) ok = tile(std::true_type{}, it.e_lim + (t - it.e_units) * kAtWinUnit, it.w_lim);
        if (!ok || pair_any(quarter, !pv_done(gt - 1))) {
          ok = false;
          break;
        }
      }
      // the rows, or their part: this thread's half of the columns
      *mine = l;
      pair_sync(quarter);
      l = half ? *other + l : l + *other;
      const bool whole = w.ta == 0 && w.tb == it.units;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      float fold = 1.0f;
      if (far && shift != 0.0f) {  // one number for the reference again, the rest of it in the part
        fold = ex2(m - kFarEnd);
        l *= fold;
        m = fmaf(shift, qm, kFarEnd);
      }
      uint16_t* orow = a.out + static_cast<int64_t>(it.c0 + tok) * a.ldo + head * kKvDim;
      float* part = parts + static_cast<int64_t>(2 * blockIdx.x + (w.ta == 0 ? 1 : 0)) * (kAtRows * (kKvDim + 2));
#pragma unroll 1
      for (int c = 128 * half; c < 128 * half + 128; c += 16) {
        uint32_t x[16];
        tc_ld16(row + kColO + c, x);
        tc_wait_ld();
        if (on && whole) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              y[i] = pack_bf162(__uint_as_float(x[8 * k + 2 * i]) * inv, __uint_as_float(x[8 * k + 2 * i + 1]) * inv);
            reinterpret_cast<uint4*>(orow + c)[k] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else if (on) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * fold);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // [256 columns / 4][row][4]: a warp writes 512 bytes at a time
            reinterpret_cast<uint4*>(part)[(c / 4 + k) * kAtRows + r] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        }
        __syncwarp();
      }
      if (!whole && on && half == 0) {
        part[kAtRows * kKvDim + r] = m;
        part[kAtRows * (kKvDim + 1) + r] = l;
      }
      pair_sync(quarter);  // O, Q and the exchange words are free for the next segment
    }
  } else if (warp < kAtMma) {
    // ------------------------------------------------------------ decode
    const int dw = warp - kAtDec0, g = lane & 7, t4 = lane >> 3, tid = threadIdx.x - 32 * kAtDec0;
    const uint32_t tab = tab0 + 4 * lane;
    uint32_t gt = 0, ce = 0;
    while (ok && w.next(a, tiles)) {
      for (int t = w.ta; ok && t < w.e_tb; ++t, ++gt, ++ce) {
        const uint32_t cs = ce % kCodeStages, st = codes + cs * kCodeStage, s = gt & 1u, par = (gt >> 1) & 1u;
        ok = at_wait_warp(c_full + 8 * cs, (ce / kCodeStages) & 1u) && at_wait_warp(k_empty + 8 * s, par ^ 1u);
        if (!ok) break;
        const uint32_t there = lds32(st + kMaskOff);
        const int left = w.it.e_lim - t * kUnit;  // keys from here to the end
        if (tid < 128) {
          const int n = tid & 63, key = at_key(n);
          const uint16_t hv = lds16(st + kNormOff + 128 + 2 * key);
          const float nk = lds_half(st + kNormOff + 2 * key), nv = half_bits_to_float(hv);
          // A value's norm that is not finite goes into its key's: the rows that see it
          // come out NaN, and 0 * inf does not reach those that do not.
          float x = tid < 64 ? (isfinite(nv) ? nk : NAN) : (isfinite(nv) ? nv * kNvScale : 0.0f);
          if (key >= left || !((there >> (key >> 4)) & 1u)) x = 0.0f;
          const uint32_t slot = nrm + (gt & 3u) * kNrmSlot;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(slot + 4 * tid), "f"(x) : "memory");
          if (tid >= 64) asm volatile("st.shared.f32 [%0], %1;" ::"r"(slot + 256 + 4 * tid), "f"(log2_above(hv)) : "memory");
          if (tid == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(slot + kSlotMask), "r"(there) : "memory");
        }
        {  // K: key of row 8 dw + g, dims 64 t4 .. + 63
          const uint32_t src = st + (g & 3) * kGrp + (2 * (g >> 2) + (dw & 1) + 4 * (dw >> 1)) * kKvBytes + 24 * t4;
          uint32_t x[6];
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const uint2 y = lds64(src + 8 * i);
            x[2 * i] = y.x, x[2 * i + 1] = y.y;
          }
          const uint32_t dst = k_tiles + s * kKvTile + 8192 * t4 + (8 * dw + g) * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int bit = 24 * c + 6 * k, wi = bit >> 5, sh = bit & 31;
              uint32_t y;
              if (sh > 26) y = __funnelshift_r(x[wi], x[wi + 1], sh - 7);
              else if (sh >= 7) y = x[wi] >> (sh - 7);
              else y = x[wi] << (7 - sh);
              h[k] = lds32((y & 0x1f80u) | tab);
            }
            sts128(dst + ((c ^ g) << 4), h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(k_full + 8 * s);
        }
        ok = at_wait_warp(v_empty + 8 * s, par ^ 1u);
        if (!ok) break;
        {  // V^T: places 8 g .. + 7, dims 8 (4 dw + t4) .. + 7: 24 bits of each of eight keys
          const uint32_t src = st + 4 * kGrp + (g & 3) * kGrp + 2 * (g >> 2) * kKvBytes + 12 * dw + 4 * ((24 * t4) >> 5);
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t at = src + ((i & 1) + 4 * (i >> 1)) * kKvBytes;
            x[i] = __funnelshift_r(lds32(at), lds32(at + 4), (24 * t4) & 31);
          }
          const uint32_t dst = v_tiles + s * kKvTile + 8 * (4 * dw + t4) * 128;
          constexpr uint32_t kEven = 0x1c71c7u;
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // even and odd codes of two keys side by side
            const uint32_t p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = (p & kEven) | ((q << 3) & ~kEven);
            x[2 * i + 1] = ((p >> 3) & kEven) | (q & ~kEven);
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t y = x[2 * i + (c & 1)];
              const int sh = 6 * (c >> 1);
              h[i] = lds32(((sh >= 7 ? y >> (sh - 7) : y << (7 - sh)) & 0x1f80u) | tab);
            }
            sts128(dst + c * 128 + ((g ^ c) << 4), h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_full + 8 * s);
        }
        if (lane == 0) mbar_arrive(c_empty + 8 * cs);
      }
      if (!ok) break;
      const int R = static_cast<int>(a.R);
      const int64_t ring = (static_cast<int64_t>(w.it.b) * a.H + w.h) * R;
      for (int t = w.e_tb; ok && t < w.tb; ++t, ++gt) {
        const uint32_t s = gt & 1u, par = (gt >> 1) & 1u;
        const int k0 = w.it.e_lim + (t - w.it.e_units) * kAtWinUnit, end = w.it.w_lim;
        // some rows see this tile in part: a value that is not finite is carried by its
        // key, as an encoded one's norm is
        const bool part = min(k0 + kAtWinUnit, end) > w.it.p + w.it.row0 / a.G + 1;
        ok = at_wait_warp(k_empty + 8 * s, par ^ 1u);
        if (!ok) break;
        {
          const int key = k0 + at_key(8 * dw + g);
          uint32_t bad = 0;
          if (part) {
            if (key < end) {
              const uint4* src = reinterpret_cast<const uint4*>(a.vwin + (ring + key % R) * kKvDim + 64 * t4);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint4 x = __ldg(src + c);
                bad |= not_finite_bf162(x.x) | not_finite_bf162(x.y) | not_finite_bf162(x.z) | not_finite_bf162(x.w);
              }
            }
            bad |= __shfl_xor_sync(0xffffffffu, bad, 8);
            bad |= __shfl_xor_sync(0xffffffffu, bad, 16);
            if (bad) bad = 0x7fff7fffu;  // NaN, or-ed into the key
          }
          const uint4* src = reinterpret_cast<const uint4*>(a.kwin + (ring + (key < end ? key % R : 0)) * kKvDim + 64 * t4);
          const uint32_t dst = k_tiles + s * kKvTile + 8192 * t4 + (8 * dw + g) * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (key < end) x = __ldg(src + c);
            sts128(dst + ((c ^ g) << 4), x.x | bad, x.y | bad, x.z | bad, x.w | bad);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(k_full + 8 * s);
        }
        ok = at_wait_warp(v_empty + 8 * s, par ^ 1u);
        if (!ok) break;
        {
          uint32_t x[8][4];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int key = k0 + at_key(8 * i + g);
            uint4 y = make_uint4(0u, 0u, 0u, 0u);
            if (key < end) y = __ldg(reinterpret_cast<const uint4*>(a.vwin + (ring + key % R) * kKvDim + 8 * (4 * dw + t4)));
            x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
            if (part)
#pragma unroll
              for (int k = 0; k < 4; ++k) x[i][k] &= ~((not_finite_bf162(x[i][k]) >> 15) * 0xffffu);
          }
          const uint32_t dst = v_tiles + s * kKvTile + 8 * (4 * dw + t4) * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __byte_perm(x[2 * i][c >> 1], x[2 * i + 1][c >> 1], (c & 1) ? 0x7632 : 0x5410);
            sts128(dst + c * 128 + ((g ^ c) << 4), h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_full + 8 * s);
        }
      }
    }
    if (ok) {  // the last commits' arrivals land before the CTA ends
      const uint32_t s = (gt - 1) & 1u, par = ((gt - 1) >> 1) & 1u;
      ok = at_wait_warp(k_empty + 8 * s, par) && at_wait_warp(v_empty + 8 * s, par);
    }
  } else if (warp == kAtMma) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t gt = 0, nq = 0;
    // O (+)= P(j) V(j)
    auto pv = [&](uint32_t j, bool win, bool first) -> bool {
      const uint32_t s = j & 1u, par = (j >> 1) & 1u;
      if (!at_wait_warp(v_full + 8 * s, par) || !at_wait_warp(p_full + 8 * s, par)) return false;
      tc_fence_after();
      const uint64_t desc = smem_desc_sw128(v_tiles + s * kKvTile);
      const uint32_t id = idesc_16(256, win);
      for (int part = 0; part < (win ? 2 : 1); ++part)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          at_mma(tmem + kColO, tmem + kColS + 64 * s + 32 * part + 8 * k, desc + static_cast<uint64_t>(2 * k), id,
                        first && part == 0 && k == 0 ? 0u : 1u);
      at_commit(v_empty + 8 * s);
      return true;
    };
    while (ok && w.next(a, tiles)) {
      bool first = true;
      for (int phase = 0; ok && phase < 2; ++phase) {
        const bool win = phase == 1;
        const int n = win ? w.tb - w.e_tb : w.e_tb - w.ta;
        if (n == 0) continue;
        ok = at_wait_warp(q_full, nq & 1u);
        ++nq;
        const uint32_t id = idesc_16(64, win);
        for (int t = 0; ok && t < n; ++t, ++gt) {
          const uint32_t s = gt & 1u, par = (gt >> 1) & 1u;
          ok = at_wait_warp(k_full + 8 * s, par);
          if (!ok) break;
          tc_fence_after();
          // S(gt)'s columns were P(gt - 2): its product was issued before, and MMAs run in order
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint64_t desc = smem_desc_sw128(k_tiles + s * kKvTile + 8192 * c);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              at_mma(tmem + kColS + 64 * s, tmem + kColQ + 32 * c + 8 * k, desc + static_cast<uint64_t>(2 * k), id,
                            c || k ? 1u : 0u);
          }
          at_commit(k_empty + 8 * s);
          at_commit(s_full + 8 * s);
          if (t > 0) {
            ok = pv(gt - 1, win, first);
            first = false;
          }
        }
        if (ok) {
          ok = pv(gt - 1, win, first);
          first = false;
        }
      }
    }
    if (!ok) drain_mma(misc + 16, lane);
  } else {
    // ------------------------------------------------------------ loader
    uint32_t ce = 0;
    while (ok && w.next(a, tiles)) {
      for (int t = w.ta; ok && t < w.e_tb; ++t) {
        const uint32_t cs = ce % kCodeStages, st = codes + cs * kCodeStage, bar = c_full + 8 * cs;
        ok = at_wait_warp(c_empty + 8 * cs, ((ce / kCodeStages) & 1u) ^ 1u);
        if (!ok) break;
        if (fault_skip_tma()) {
          ++ce;
          continue;
        }
        // lane = 4 kind + group: codes of K, codes of V, norms of K, norms of V
        const int grp = lane & 3, kind = lane >> 2, key = t * kUnit + 16 * grp;
        bool there = false;
        int64_t row_ = 0;
        if (lane < 16 && key < w.it.e_lim) {
          const int kp = key / static_cast<int>(a.P);
          const int page = kp < a.max_pages ? __ldg(a.table + w.it.b * a.max_pages + kp) : -1;
          there = page >= 0 && page < a.num_pages;
          if (!there) raise_device_error(HLWQ_DEVERR_KV_RANGE);
          row_ = (static_cast<int64_t>(page) * a.H + w.h) * a.P + (key - kp * static_cast<int>(a.P));
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, there);
        if (lane == 0) {
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(st + kMaskOff), "r"(mask & 15u) : "memory");
          mbar_arrive_expect_tx(bar, __popc(mask & 15u) * 2 * (1536 + 32));
        }
        __syncwarp();
        if (there) {
          if (kind == 0) bulk_load(st + grp * kGrp, a.kp + row_ * kKvBytes, 1536, bar);
          else if (kind == 1) bulk_load(st + 4 * kGrp + grp * kGrp, a.vp + row_ * kKvBytes, 1536, bar);
          else if (kind == 2) bulk_load(st + kNormOff + 32 * grp, a.kn + row_, 32, bar);
          else bulk_load(st + kNormOff + 128 + 32 * grp, a.vn + row_, 32, bar);
        }
        ++ce;
      }
    }
    // no copy may be landing when the CTA ends: the last ones issued into each stage
    if (!fault_skip_tma())
      for (uint32_t j = ce > kCodeStages ? ce - kCodeStages : 0; j < ce; ++j)
        at_wait_warp(c_full + 8 * (j % kCodeStages), (j / kCodeStages) & 1u);
  }
  if (!ok && lane == 0) raise_device_error(HLWQ_DEVERR_TIMEOUT);

  tc_fence_before();
  __syncthreads();
  if (warp == kAtMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

int launch_tiles(const KvAttn& a, int ctas, int tiles, float* parts, KvCut* cuts, cudaStream_t stream) {
  static PerDeviceOnce attr;
  if (const int st = attr([&] {
        return cudaFuncSetAttribute(kv_attn_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAtSmem) ==
               cudaSuccess;
      }))
    return st;
  kv_attn_tile_kernel<<<ctas, kAtThreads, kAtSmem, stream>>>(a, tiles, parts, cuts);
  if (cudaGetLastError() != cudaSuccess) return HLWQ_ECUDA;
  return launch_join<kAtRows>(a, ctas, parts, cuts, stream);
}

// Rows per tile, CTAs, and row tiles of a request for max_new new tokens: the
// few-row kernel up to 16 rows per kv head, the tensor-core tiles above.  Measured, us
// for 16 requests of 100 to 7000 tokens and 8 kv heads / one of 60000 tokens and 4:
//   rows              8           12           16           18           24           32           48
//   tiles of 8     58 / 42     95 / 52      94 / 53     125 / 67     126 / 67     154 / 82     218 / 111
//   tiles of 16    78 / 51     81 / 51      83 / 53     153 / 68     154 / 69     158 / 69     208 / 97
//   tiles of 128  106 / 79    108 / 80     108 / 81     109 / 81     109 / 81     109 / 81     111 / 81
// (One request alone would do better on two tiles of 16 up to 32 rows; batches would not.)
struct KvGrid {
  int rows, ctas;
  int64_t tiles;
};
inline KvGrid kv_grid(int64_t max_new, int64_t G) {
  const int64_t n = max_new * G;
  const int rows = n <= 8 ? 8 : n <= 16 ? 16 : kAtRows;
  return {rows, sm_count() * (rows == 8 ? RowCfg<1>::kCtas : rows == 16 ? RowCfg<2>::kCtas : 1), ceil_div(n, rows)};
}

}  // namespace

// Workspace: two partial results per CTA, then a note per CTA for the join.
size_t kv_attention_workspace_bytes(int64_t, int64_t max_new, int64_t, int64_t Hq, int64_t H) {
  const KvGrid gr = kv_grid(max_new, Hq / H);
  return static_cast<size_t>(gr.ctas) * (2 * gr.rows * (kKvDim + 2) * sizeof(float) + sizeof(KvCut));
}

int launch_kv_attention(const KvAttn& a, void* workspace, size_t, cudaStream_t stream) {
  const KvGrid gr = kv_grid(a.max_new, a.G);
  if (gr.tiles * a.B > INT32_MAX) return HLWQ_EUNSUPPORTED;
  const int tiles = static_cast<int>(gr.tiles);
  float* parts = static_cast<float*>(workspace);
  KvCut* cuts = reinterpret_cast<KvCut*>(parts + static_cast<int64_t>(2) * gr.ctas * gr.rows * (kKvDim + 2));
  switch (gr.rows) {
    case 8: return launch_rows<1>(a, gr.ctas, tiles, parts, cuts, stream);
    case 16: return launch_rows<2>(a, gr.ctas, tiles, parts, cuts, stream);
    default: return launch_tiles(a, gr.ctas, tiles, parts, cuts, stream);
  }
}

}  // namespace hlwq
