#pragma once
// Attention of new tokens over the paged Q3 KV cache (sm_100a): the sharing of the
// work, the kernel for few rows per kv head, the join of split results.  The
// kernel for chunks is kvtile.cuh.
//
// Query i of a request with p cached and n new tokens sees keys j <= p + i:
//   s_j = scale * q . k_j,  o = sum_j softmax(s)_j v_j,
// keys and values below n_enc(p + n) decoded from their pages, the rest exact
// from the window.  With H = H256 (symmetric, H H = 256 I), an encoded key is
// n / 256 c[code] H: q . k = (n / 256) (q H) . c[code], and the encoded values add up to
// (1 / 256) (sum_j p_j n_j c[code_j]) H.  The query is rotated once, the sum once,
// and the cached vectors never; what is multiplied are the 8 centroids.

#include "kvpage.cuh"
#include "sm100.cuh"

namespace hlwq {

namespace {

// What a kernel needs to know about the cache and the step.
struct KvAttn {
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq, ldo, T, max_new;
  const int32_t* cu;
  const int32_t* n_past;
  int B, Hq, H, G;
  float scale;
  const float* codebook;
  const uint8_t* kp;
  const uint16_t* kn;
  const uint8_t* vp;
  const uint16_t* vn;
  int64_t num_pages, P;
  const int32_t* table;
  int64_t max_pages;
  const uint16_t* kwin;
  const uint16_t* vwin;
  int64_t R;
};

// ---------------------------------------------------------------- the work, shared out
//
// An item is (request, row tile, kv head): a row tile is kRows consecutive
// (token, query head) rows of a request, row = token * G + g.  An item's keys are
// cut into units (64 encoded tokens, or kWinUnit window tokens).  An item costs its units
// and what beginning and ending it takes (rotations, the row's output), counted in
// units.  All items' costs in order, 0 .. U - 1, are shared out evenly over the
// grid's CTAs in contiguous ranges, whatever the requests' lengths are: one long
// request is split over the machine, many short ones are not split.  Where a boundary
// between two CTAs falls inside an item, its parts go to the workspace and
// kv_attn_join_kernel adds them up.  Everything follows from cu and n_past, so every CTA
// works its share out for itself: no plan is made beforehand and the host needs
// no lengths.  A CTA that begins inside an item leaves a note for the join.

constexpr int kUnit = 64;  // encoded tokens per unit

constexpr int64_t kMaxKeys = INT32_MAX - 4096;  // key positions are 32-bit below

struct KvItem {
  int b;         // request
  int c0, n;     // its first row of Q and its new tokens
  int p;         // cached tokens before the step
  int row0;      // first row of the tile
  int nrows;     // rows of the tile
  int e_lim;     // encoded tokens that the tile's last row sees
  int w_lim;     // tokens that it sees, window included
  int e_units, units;
  int64_t cost;  // of all the kv heads' items of this pair; an item's own cost is cost / H
};

// The pair (request, row tile) number `pair`; units = 0 where it has no rows.
// (T * q_heads and key positions are below 2^31: checked by the host and here.)
template <int kRows, int kWinUnit, int kItemCost>
__device__ __forceinline__ KvItem kv_item(const KvAttn& a, int pair, int tiles, bool& bad) {
  KvItem it;
  it.b = tiles == 1 ? pair : pair / tiles;
  const int rt = pair - it.b * tiles;
  it.c0 = __ldg(a.cu + it.b);
  it.p = __ldg(a.n_past + it.b);
  const int64_t n = static_cast<int64_t>(__ldg(a.cu + it.b + 1)) - it.c0;
  it.n = static_cast<int>(n);
  it.units = it.e_units = 0;
  it.cost = 0;
  if (it.c0 < 0 || n < 0 || it.c0 + n > a.T || it.p < 0 || it.p + n > kMaxKeys) {
    bad = true;
    return it;
  }
  const int rows = it.n * a.G;
  if (n > a.max_new) bad = true;  // (the rows past the last tile have no item)
  it.row0 = rt * kRows;
  it.nrows = min(kRows, rows - it.row0);
  if (it.nrows <= 0) return it;
  const int sees = it.p + (it.row0 + it.nrows - 1) / a.G + 1;  // keys of the tile's last token
  it.e_lim = min(max(0, it.p + it.n - static_cast<int>(a.R)), sees);
  it.w_lim = sees;
  it.e_units = (it.e_lim + kUnit - 1) / kUnit;
  it.units = it.e_units + (it.w_lim - it.e_lim + kWinUnit - 1) / kWinUnit;
  it.cost = static_cast<int64_t>(it.units + kItemCost) * a.H;
  return it;
}

// The pair to look at after `pair`: a request without rows left in it has none further
// on, so at most one of them is looked at (a request may have far fewer rows than
// max_new's tiles, which only bound them).
__device__ __forceinline__ int kv_after(const KvItem& it, int pair, int tiles) {
  return it.cost ? pair + 1 : (it.b + 1) * tiles;
}

// The pairs [first, last) of this thread of kThreads.
template <int kThreads>
__device__ __forceinline__ void kv_mine(const KvAttn& a, int tiles, int& first, int& last) {
  const int64_t pairs = static_cast<int64_t>(a.B) * tiles, per = (pairs + kThreads - 1) / kThreads;
  first = static_cast<int>(min(threadIdx.x * per, pairs));
  last = static_cast<int>(min(first + per, pairs));
}

// The total of all costs; `mine0` = the cost before this thread's pairs.  Called
// by all kThreads threads of the CTA.
template <int kRows, int kWinUnit, int kItemCost, int kThreads>
__device__ __forceinline__ int64_t kv_total_cost(const KvAttn& a, int tiles, int64_t* warp_sums, int64_t& mine0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int pair, last;
  kv_mine<kThreads>(a, tiles, pair, last);
  int64_t sum = 0;
  bool bad = false;
#pragma unroll 1
  while (pair < last) {
    const KvItem it = kv_item<kRows, kWinUnit, kItemCost>(a, pair, tiles, bad);
    sum += it.cost;
    pair = kv_after(it, pair, tiles);
  }
  if (bad) raise_device_error(HLWQ_DEVERR_KV_RANGE);
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  mine0 = before + inc - sum;
  return total;
}

// After kv_total_cost: the pair holding cost `want`, found by the thread whose
// pairs contain it and published in found[0] (pair) and found[1] (where its cost begins).
template <int kRows, int kWinUnit, int kItemCost, int kThreads>
__device__ __forceinline__ void kv_find(const KvAttn& a, int tiles, int64_t mine0, int64_t want, int64_t* found) {
  int pair, last;
  kv_mine<kThreads>(a, tiles, pair, last);
  int64_t u = mine0;
  bool bad = false;
  if (u <= want) {
#pragma unroll 1
    while (pair < last) {
      const KvItem it = kv_item<kRows, kWinUnit, kItemCost>(a, pair, tiles, bad);
      if (want < u + it.cost) {
        found[0] = pair;
        found[1] = u;
        break;
      }
      u += it.cost;
      pair = kv_after(it, pair, tiles);
    }
  }
  __syncthreads();
}

// What the CTA after a cut tells the join: the item whose first cut this is, and
// how many CTAs' parts it has (0: no item is first cut here).
struct KvCut {
  int count, b, h, row0;
};

// The shares of the cost U of n CTAs, this one being number i: each
// that has one has a cost of at least 1.
struct KvShares {
  int64_t U;
  int i, ctas;
  __device__ __forceinline__ KvShares(int64_t total, int me, int n) : U(total), i(me) {
    ctas = static_cast<int>(min(U, static_cast<int64_t>(n)));
  }
  __device__ __forceinline__ int64_t operator()(int c) const { return U * c / ctas; }  // where CTA c's share begins
  // the number of CTAs whose share begins before cost u
  __device__ __forceinline__ int before(int64_t u) const {
    return static_cast<int>(min((u * ctas + U - 1) / U, static_cast<int64_t>(ctas)));
  }
};

// One after another, the segments (item, range of its units) of a CTA's share
// [u0, u1) of the cost.  An item's first kItemCost are its beginning and end, then
// comes a unit at each step: a boundary among the first ones cuts nothing.
template <int kRows, int kWinUnit, int kItemCost>
struct KvWalk {
  int64_t u0, u, u1, at;  // share, where the walk is, where the pair's cost begins
  int pair;
  KvItem it;
  int h, ta, tb, e_tb;    // the segment: kv head, units [ta, tb), encoded ones [ta, e_tb)

  __device__ __forceinline__ void begin(const KvAttn& a, int tiles, const KvShares& share, const int64_t* found) {
    u = u0 = share(share.i);
    u1 = share(share.i + 1);
    pair = static_cast<int>(found[0]);
    at = found[1];
    bool bad = false;
    it = kv_item<kRows, kWinUnit, kItemCost>(a, pair, tiles, bad);
  }
  __device__ __forceinline__ bool next(const KvAttn& a, int tiles) {
    bool bad = false;
    while (u < u1) {
      while (u >= at + it.cost) {
        at += it.cost;
        pair = kv_after(it, pair, tiles);
        it = kv_item<kRows, kWinUnit, kItemCost>(a, pair, tiles, bad);
      }
      const int each = it.units + kItemCost;
      h = static_cast<int>((u - at) / each);
      const int o = static_cast<int>(u - at - static_cast<int64_t>(h) * each);
      const int n = static_cast<int>(min(static_cast<int64_t>(each - o), u1 - u));
      u += n;
      ta = max(0, o - kItemCost);
      tb = max(0, o + n - kItemCost);
      e_tb = max(ta, min(tb, it.e_units));
      if (tb > ta) return true;
    }
    return false;
  }
  // The note for the join when this is the share's first segment and begins
  // inside its item: whether the boundary before this CTA is the item's first cut.
  __device__ __forceinline__ bool note(const KvShares& share, KvCut& cut) const {
    const int each = it.units + kItemCost;
    const int64_t s0 = at + static_cast<int64_t>(h) * each, s1 = s0 + each;
    if (ta == 0 || u0 <= s0) return false;
    if (share(share.i - 1) > s0 + kItemCost) return false;
    // parts: the CTA before this one, this one, and those that begin before the item's end
    cut = {1 + share.before(s1) - share.i, it.b, h, it.row0};
    return true;
  }
};

// ---------------------------------------------------------------- building blocks

// 2^k that brings the largest magnitude mx of a row of Q into [64, 128), so that no
// coordinate of the rotated row passes 128 * 256 = 2^15; 1 for a zero row.  (The power of
// the smallest rows stays below 2^118: 512 times it is finite.)
__device__ __forceinline__ float pow2_scale(float mx, float& inv) {
  const int e = static_cast<int>(__float_as_uint(mx) >> 23);
  const int k = e == 0 ? 0 : max(-126, min(117, 133 - e));
  inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}

// On top of it for the window's products, so that 256 of them with any finite keys
// stay finite: Q below 2^-9 in magnitude.
constexpr float kWinScale = 1.0f / 65536.0f;
// The factor that takes it back, with the query's own, passes fp32 for the largest
// queries.  It stops at the largest finite number: their scores are beyond 2^100 and stay
// as far apart as weights tell.
constexpr float kMaxFinite = 3.402823466e38f;
__device__ __forceinline__ float window_qm(float x) { return fminf(fmaxf(x, -kMaxFinite), kMaxFinite); }
// And the size that window values count with in their row's reference: p stays below
// 2^-24, so that the sum of up to 2^20 finite values is finite.  (p is above 2^-32 for the
// row's largest score: values below 2^-94 are multiplied as fp32 subnormals.)
constexpr float kWinSize = 32.0f;

// A row's reference is one number m, score + log2 norm, while its magnitude is at most
// kFar (steps of 2^-7).  Beyond it rounding the sum would take the row's largest weight
// away (from 2^27 on p n is 0 in binary16): the row's scores then count from one of them,
// its shift, and m is a small number again, at most kFarNext (beyond it the shift
// follows) and the window's size.  A result that is joined with others has
// shift + kFarEnd in one number, its weights brought to that.
constexpr float kFar = 65536.0f, kFarNext = 64.0f, kFarEnd = kFarNext + kWinSize;

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The centroids as binary16: c times a scale of kCentroidScales between two powers of two
// (the largest |c| goes to [2^7, 2^9)), the one under which the 8 roundings agree best
// with one common factor.  That factor goes back into the scores and the outputs
// in fp32.  The roundings come the same way at every use of a code and do not
// average out: under a power of two the Lloyd-Max centroids are off by up to
// 0.8 of 2^-12, under the best scale by 0.09.  Values below 1/64 of the largest count
// by their absolute error (they are left out of the choice).
constexpr int kCentroidScales = 256;

struct Centroids {
  float c[kKvLevels], inv[kKvLevels];  // inv 0: not counted
  float unit;                          // scale number 0
  __device__ __forceinline__ explicit Centroids(const float* codebook) {
    float mx = 0.0f;
#pragma unroll
    for (int k = 0; k < kKvLevels; ++k) {
      c[k] = __ldg(codebook + k);
      mx = fmaxf(mx, fabsf(c[k]));
    }
    const int e = max(7, static_cast<int>(__float_as_uint(mx) >> 23));
    unit = __uint_as_float(static_cast<uint32_t>(261 - min(e, 254)) << 23);
#pragma unroll
    for (int k = 0; k < kKvLevels; ++k) inv[k] = 64.0f * fabsf(c[k]) < mx || mx == 0.0f ? 0.0f : __fdividef(1.0f, c[k] * unit);
  }
  __device__ __forceinline__ float step(int i) const { return 1.0f + static_cast<float>(i) * (1.0f / kCentroidScales); }
  __device__ __forceinline__ float scale(int i) const { return unit * step(i); }
  // What the rounded centroids are of `unit` times them, on average; the return value is
  // how far they are apart.
  __device__ __forceinline__ float spread(int i, float& ratio) const {
    const float s = scale(i);
    float hi = 0.0f, lo = 4.0f;
#pragma unroll
    for (int k = 0; k < kKvLevels; ++k) {
      const float r = __half2float(__float2half_rn(c[k] * s)) * inv[k];
      hi = fmaxf(hi, r);
      lo = fminf(lo, inv[k] == 0.0f ? lo : r);
    }
    ratio = 0.5f * (hi + lo);
    return (hi - lo) * __fdividef(1.0f, step(i));
  }
};

// The choice: one key per warp, the smallest of which (after a barrier) is it.
template <int kThreads>
__device__ __forceinline__ void choose_centroid_scale(const float* codebook, uint32_t* best) {
  uint32_t key = 0xffffffffu;
  if (threadIdx.x < kCentroidScales) {
    const Centroids cs(codebook);
    for (int i = threadIdx.x; i < kCentroidScales; i += kThreads) {
      float ratio;
      key = min(key, (__float_as_uint(fabsf(cs.spread(i, ratio))) & ~(kCentroidScales - 1u)) | static_cast<uint32_t>(i));
    }
  }
  key = __reduce_min_sync(0xffffffffu, key);
  if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = key;
}

// The table of binary16 pairs for two codes (one copy per lane), and in *back
// the factor that takes a sum of its entries back; a barrier must follow.
template <int kThreads>
__device__ __forceinline__ void fill_centroid_table(const float* codebook, const uint32_t* best, uint32_t* table, float* back) {
  uint32_t key = best[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) key = min(key, best[w]);
  const Centroids cs(codebook);
  const int n = static_cast<int>(key & (kCentroidScales - 1u));
  const float scale = cs.scale(n);
  if (threadIdx.x == 0) {
    float ratio;
    cs.spread(n, ratio);
    *back = 1.0f / (ratio * cs.unit);
  }
  for (int i = threadIdx.x; i < 64 * 32; i += kThreads)
    table[i] = pack_half2(__ldg(codebook + ((i >> 5) & 7)) * scale, __ldg(codebook + (i >> 8)) * scale);
}

// 2^x, one instruction (relative error below 2^-22; results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float oct_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
}

__device__ __forceinline__ void load_bf16x32(float (&v)[32], const uint16_t* src, bool on) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (on) u = __ldg(reinterpret_cast<const uint4*>(src) + c);
    const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[8 * c + 2 * k] = bf16x2_lo(wd[k]);
      v[8 * c + 2 * k + 1] = bf16x2_hi(wd[k]);
    }
  }
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Of two bf16 values, the sign bits of those that are not finite (exponent all ones).
__device__ __forceinline__ uint32_t not_finite_bf162(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ uint16_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ float lds_half(uint32_t a) { return half_bits_to_float(lds16(a)); }

// The least power of two above a binary16 norm, as an exponent: -14 (below 2^-14)
// to 16; 17 when it is not finite.
__device__ __forceinline__ float log2_above(uint16_t h) {
  return __uint_as_float(0x43000000u | ((h & 0x7c00u) << 6)) - 142.0f;  // 128 + exponent field, less its bias
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// ---------------------------------------------------------------- few rows per kv head
//
// At most 16 (token, head) rows per kv head: single tokens, a few drafted ones.
// The codes are decoded into the registers of matrix instructions and nowhere else.
//
// S^T = K q^T with m16n8k16: A = 16 keys x 16 dims, B = 8 rows of q.  The
// contraction's dims may come in any order, so lane (g, t) = (lane / 4, lane % 4)
// takes dims 64 t + 4 s .. + 3 of keys g and g + 8 in step s: 24 contiguous bytes of each
// key.  O^T = V^T P^T: A = 16 dims x 16 keys; its pairs run along keys 2t, 2t + 1
// (and + 8), its rows are dims 32 g + 2 m and 32 g + 2 m + 1 of tile m, so a lane
// takes 12 contiguous bytes of four keys.  Two 3-bit codes index a table of 64
// binary16 pairs, one copy per lane (its own bank): two neighbouring codes of a
// key, or the same code of two keys (the even and odd 3-bit fields of two words
// are brought together with one select).  That is one table load and two integer
// instructions for two values.
//
// P^T comes out of S^T's registers by two 8 x 8 transposes; row sums
// stay in the lane until the end.  A value's norm rides on p, and a row's running
// reference m follows its largest score + log2 norm, the size of the term p n: it is
// raised only when one exceeds it by 8 (in powers of two), so most steps need no exchange
// between lanes.  Then p n < 2^8 (p itself, at most 2^22, is summed in fp32), and kNvScale
// brings it to where binary16 has 11 bits for it down to 2^-20 of the row's largest
// term (of a norm from 2^-14 up) and steps of 2^-30 of that term below, whatever the
// norms of keys are that the row does not see or gives no weight.  O^T's registers hold 32 consecutive dims of two
// rows: the rotation back is five in-register and three shuffle stages.  The window's
// keys come after it and are multiplied as they are, un-rotated bf16 with the
// query's own bits (times a power of two).
//
// Fewer than 32 bits: the rotated query has 11 per coordinate (the query came with 8), p n
// has 11, the centroids about 14 (above).  Their products are exact and are summed in
// fp32.  With scores of up to 65 over 4000 keys the query's part moves the output by
// 0.1 in a thousand in the median and by up to 3 in a thousand, the other two by up to
// 0.3; half a step of the bf16 output is 2 to 4 in a thousand.  The query in two binary16 parts (22 bits)
// was built: 64 requests 214 us instead of 165, one of 131071 tokens 78 instead of 65.
//
// Bound: HBM by its bytes (196 per token and kv head); in fact integer instructions
// and shared-memory reads, one warp instruction in five a table read.  64 requests
// of 64 to 16384 tokens, 4 kv heads of 6 rows (438 MB): 167 us, 2.6 TB/s, DRAM
// traffic equal to the bytes, 730 warp instructions per 16 keys at 2.3 per cycle
// (ALU pipe 58 %, shared memory 56 %).  A tcgen05 kernel would have to write the decoded
// tiles to shared memory first, as much traffic again as the table reads; the
// legacy instruction takes them from registers, and with 8 or 16 rows its
// rate is no limit (tensor pipe 20 %).

constexpr int kRowWarps = 4;
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kStageNorms = 2 * 16 * kKvBytes;  // 16 keys: K codes, V codes,
constexpr int kStage = kStageNorms + 64;        // K norms, V norms
constexpr int kStages = 4;
// An item's beginning and end (rotations, joining the warps) take about 6 us where a
// unit takes 1.3; a window tile of 16 about as long as a unit.
constexpr int kRowItemCost = 5;
constexpr int kRowWinUnit = 16;
constexpr int kTabBytes = 64 * 128;
constexpr float kMinM = -kMaxFinite;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNvScale = 128.0f;  // on the norms of values: p n kNvScale < 2^15

template <int NT>
struct RowCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kQFrag = NT * 16 * 32 * 8;
  static constexpr int kBuf = kStages * kStage;                  // per warp: ring, window tile, or 32 NT x 64 partial sums
  static constexpr int kMerge = NT * 32 * 32 * 8;                // bytes of a warp's O
  static constexpr int kWarpBytes = kBuf > kMerge ? kBuf : kMerge;
  static constexpr int kSmem = 8192 /*align*/ + kTabBytes + 2 * kQFrag + kRowWarps * kWarpBytes;
  static constexpr int kPart = kRows * (kKvDim + 2);             // floats of one partial result
  static constexpr int kCtas = NT == 1 ? 3 : 2;                  // resident per SM
};

// Adds 16 keys' values to O: codes of four keys in w[4][3].
template <int NT>
__device__ __forceinline__ void rows_pv(float (&o)[NT][16][4], const uint32_t (&w)[4][3], uint32_t tab,
                                        const uint32_t (&b)[NT][2]) {
  constexpr uint32_t kEven = 0x071c71c7u;  // bits 6f .. 6f + 2
#pragma unroll
  for (int c = 0; c < 4; ++c) {            // ten codes at a time, the last two
    uint32_t x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = c == 0 ? w[k][0] : c == 1 ? __funnelshift_r(w[k][0], w[k][1], 30)
                                       : c == 2 ? __funnelshift_r(w[k][1], w[k][2], 28) : w[k][2] >> 26;
    uint32_t pr[2][2];  // [key pair][even / odd code]
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      pr[k][0] = (x[2 * k] & kEven) | ((x[2 * k + 1] << 3) & ~kEven);
      pr[k][1] = ((x[2 * k] >> 3) & kEven) | (x[2 * k + 1] & ~kEven);
    }
#pragma unroll
    for (int f = 0; f < (c == 3 ? 1 : 5); ++f) {
      uint32_t a[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // a0, a1: even and odd dim of the first key pair; a2, a3 of the second
        // one right shift serves two fields (the lower one is a multiplication further)
        const uint32_t v = pr[k >> 1][k & 1];
        const uint32_t i = f == 0 ? v * 128u : f == 1 ? (v >> 5) * 64u : f == 2 ? v >> 5 : f == 3 ? (v >> 17) * 64u : v >> 17;
        a[k] = lds32((i & 0x1f80u) | tab);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][5 * c + f], a[0], a[1], a[2], a[3], b[nt][0], b[nt][1]);
    }
  }
}

template <int NT>
__global__ void __launch_bounds__(kRowThreads, RowCfg<NT>::kCtas)
kv_attn_rows_kernel(const KvAttn a, int tiles, float* __restrict__ parts, KvCut* __restrict__ cuts) {
  using C = RowCfg<NT>;
  extern __shared__ __align__(16) uint8_t rsm_raw[];
  __shared__ int64_t warp_sums[kRowWarps], found[2];
  __shared__ uint32_t best_scale[kRowWarps];
  __shared__ float back;
  __shared__ float qmul[C::kRows];
  __shared__ float mstat[kRowWarps][C::kRows], lstat[kRowWarps][C::kRows];
  pdl_trigger();  // the join may be set up; it waits for this grid's results
  const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(rsm_raw));
  const uint32_t tab0 = (raw + 8191u) & ~8191u;  // 8 KB aligned: indices are or-ed in
  uint8_t* gtab = rsm_raw + (tab0 - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3, l8 = lane & 7;
  const uint32_t qfrag = tab0 + kTabBytes, wbuf = qfrag + 2 * C::kQFrag + warp * C::kWarpBytes;
  uint8_t* gbuf = gtab + (wbuf - tab0);
  const uint32_t tab = tab0 + 4 * lane;
  const int page_size = static_cast<int>(a.P);

  kv_check_codebook(a.codebook);
  choose_centroid_scale<kRowThreads>(a.codebook, best_scale);
  int64_t mine0;
  const int64_t U = kv_total_cost<C::kRows, kRowWinUnit, kRowItemCost, kRowThreads>(a, tiles, warp_sums, mine0);
  if (threadIdx.x == 0) cuts[blockIdx.x] = {0, 0, 0, 0};
  const KvShares share(U, blockIdx.x, gridDim.x);
  if (share.i >= share.ctas) return;
  kv_find<C::kRows, kRowWinUnit, kRowItemCost, kRowThreads>(a, tiles, mine0, share(share.i), found);
  KvWalk<C::kRows, kRowWinUnit, kRowItemCost> w;
  w.begin(a, tiles, share, found);
  fill_centroid_table<kRowThreads>(a.codebook, best_scale, reinterpret_cast<uint32_t*>(gtab), &back);

  while (w.next(a, tiles)) {
    const KvItem& it = w.it;
    const int h = w.h, ta = w.ta, tb = w.tb, nrows = it.nrows;
    if (threadIdx.x == 0) {
      KvCut cut;
      if (w.note(share, cut)) cuts[blockIdx.x] = cut;
    }

    // rotate the tile's rows into matrix-instruction order
    for (int r0 = warp * 4; r0 < C::kRows; r0 += kRowWarps * 4) {
      const int r = r0 + (lane >> 3);
      const bool on = r < nrows;
      const int row = it.row0 + (on ? r : 0), tok = row / a.G;
      float v[32];
      load_bf16x32(v, a.q + static_cast<int64_t>(it.c0 + tok) * a.ldq + (h * a.G + (row - tok * a.G)) * kKvDim + 32 * l8, on);
      const uint32_t dst = qfrag + ((r >> 3) * 16 * 32 + (r & 7) * 4 + (l8 >> 1)) * 8 + (l8 & 1) * 8 * 256;
      float mx = 0.0f, inv;
#pragma unroll
      for (int e = 0; e < 32; ++e) mx = fmaxf(mx, fabsf(v[e]));
      const float sc = pow2_scale(oct_max(mx), inv);
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] *= sc * kWinScale;
      // not rotated (for the window's keys): its bf16 bits, another exponent
#pragma unroll
      for (int s = 0; s < 8; ++s)
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst + C::kQFrag + s * 256),
                     "r"(__byte_perm(__float_as_uint(v[4 * s]), __float_as_uint(v[4 * s + 1]), 0x7632)),
                     "r"(__byte_perm(__float_as_uint(v[4 * s + 2]), __float_as_uint(v[4 * s + 3]), 0x7632))
                     : "memory");
      kv_fwht(v, lane);
      if (l8 == 0) qmul[r] = inv * a.scale * (kLog2e / 256.0f);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst + s * 256),
                     "r"(pack_half2(v[4 * s] / kWinScale, v[4 * s + 1] / kWinScale)),
                     "r"(pack_half2(v[4 * s + 2] / kWinScale, v[4 * s + 3] / kWinScale))
                     : "memory");
    }
    __syncthreads();

    float o[NT][16][4], m[NT][2], shift[NT][2], l[NT][2], qm[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 8 * nt + 2 * t4 + k;
        m[nt][k] = kMinM;
        shift[nt][k] = l[nt][k] = 0.0f;
        qm[nt][k] = qmul[r] * back;
        lim[nt][k] = r < nrows ? it.p + (it.row0 + r) / a.G + 1 : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[nt][i][k] = o[nt][i][2 + k] = 0.0f;
      }

    // scores of M tiles of 16 keys, times their factors f[.][0] (this lane's first
    // key, index key[.]) and f[.][1] (8 further), with the log2 of their values' size
    // in size[.][.]; keys from end[.] on are not there.  The rows' references follow;
    // d becomes p = exp2(s - shift - m)
    auto score = [&](auto& d, const auto& f, const auto& size, const auto& key, const auto& end) {
      constexpr int M = sizeof(key) / sizeof(key[0]);
      // the largest score less shift + size, of two rows
      auto largest = [&](int nt) -> float2 {
        float2 x = make_float2(-INFINITY, -INFINITY);
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 t = add2(add2(make_float2(d[i][nt][2 * j], d[i][nt][2 * j + 1]), make_float2(-shift[nt][0], -shift[nt][1])),
                                  make_float2(size[i][j], size[i][j]));
            x.x = fmaxf(x.x, t.x);
            x.y = fmaxf(x.y, t.y);
          }
        return x;
      };
      auto row_max = [](float x) {
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
      };
      float2 x[NT];
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // rounded here: the selection keeps it from being fused with the shift's subtraction,
            // where the score that a shift was taken from has to come out 0
            const float2 s = mul2(make_float2(d[i][nt][2 * j], d[i][nt][2 * j + 1]),
                                  mul2(make_float2(f[i][j], f[i][j]), make_float2(qm[nt][0], qm[nt][1])));
            d[i][nt][2 * j] = key[i] + 8 * j < min(lim[nt][0], end[i]) ? s.x : -INFINITY;
            d[i][nt][2 * j + 1] = key[i] + 8 * j < min(lim[nt][1], end[i]) ? s.y : -INFINITY;
          }
        x[nt] = largest(nt);
        over |= x[nt].x > m[nt][0] + 8.0f || x[nt].y > m[nt][1] + 8.0f;
      }
      if (__any_sync(0xffffffffu, over)) {
        float nm[NT][2];
        bool big = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            nm[nt][k] = fmaxf(m[nt][k], row_max(k ? x[nt].y : x[nt].x));
            big |= nm[nt][k] > m[nt][k] && fabsf(nm[nt][k]) > (shift[nt][k] == 0.0f ? kFar : kFarNext);
          }
        if (__any_sync(0xffffffffu, big)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float s = -INFINITY;
#pragma unroll
              for (int i = 0; i < M; ++i) s = fmaxf(s, fmaxf(d[i][nt][k], d[i][nt][2 + k]));
              s = row_max(s);
              if (nm[nt][k] > m[nt][k] && fabsf(nm[nt][k]) > (shift[nt][k] == 0.0f ? kFar : kFarNext)) {
                if (m[nt][k] != kMinM) m[nt][k] += __fsub_rn(shift[nt][k], s);
                shift[nt][k] = s;
              }
            }
            const float2 y = largest(nt);
            nm[nt][0] = fmaxf(m[nt][0], row_max(y.x));
            nm[nt][1] = fmaxf(m[nt][1], row_max(y.y));
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float c = ex2(m[nt][k] - nm[nt][k]);
            m[nt][k] = nm[nt][k];
            l[nt][k] *= c;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              o[nt][i][k] *= c;
              o[nt][i][2 + k] *= c;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float2 sum = make_float2(l[nt][0], l[nt][1]);
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 t = add2(add2(make_float2(d[i][nt][2 * j], d[i][nt][2 * j + 1]), make_float2(-shift[nt][0], -shift[nt][1])),
                                  make_float2(-m[nt][0], -m[nt][1]));
            d[i][nt][2 * j] = ex2(t.x);
            d[i][nt][2 * j + 1] = ex2(t.y);
            sum = add2(sum, make_float2(d[i][nt][2 * j], d[i][nt][2 * j + 1]));
          }
        l[nt][0] = sum.x;
        l[nt][1] = sum.y;
      }
    };

    // ---- encoded keys: each warp a contiguous part of the segment's tiles of 16,
    // two tiles per step, the next step's two under way meanwhile
    const int e_tb = w.e_tb;
    if (ta < e_tb) {
      const int s_end = min(e_tb * kUnit, it.e_lim), n16 = (s_end - ta * kUnit + 15) >> 4;
      const int k_first = ta * kUnit + 16 * (n16 * warp / kRowWarps);
      const int k_end = min(s_end, ta * kUnit + 16 * (n16 * (warp + 1) / kRowWarps));
      // the page that the next tile to be requested lies in, the one after it, tiles left in it
      const int32_t* tab_row = a.table + it.b * a.max_pages;
      int kp = k_first / page_size, left = (page_size - (k_first - kp * page_size)) >> 4;
      int page = k_first < k_end && kp < a.max_pages ? __ldg(tab_row + kp) : -1;
      int page2 = k_first + 16 * left < k_end && kp + 1 < a.max_pages ? __ldg(tab_row + kp + 1) : -1;
      int64_t row = (static_cast<int64_t>(page) * a.H + h) * page_size + (k_first - kp * page_size);
      int k_ask = k_first;
      auto request = [&](uint32_t dst) -> uint32_t {  // two tiles; bit i: tile i's page is there
        uint32_t there = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i, dst += kStage, k_ask += 16) {
          if (k_ask >= k_end) continue;
          if (left == 0) {
            page = page2;
            ++kp;
            left = page_size >> 4;
            row = (static_cast<int64_t>(page) * a.H + h) * page_size;
            page2 = k_ask + page_size < k_end && kp + 1 < a.max_pages ? __ldg(tab_row + kp + 1) : -1;
          }
          --left;
          if (page < 0 || page >= a.num_pages) {
            if (lane == 0) raise_device_error(HLWQ_DEVERR_KV_RANGE);
          } else {
            there |= 1u << i;
            const uint8_t* ks = a.kp + row * kKvBytes + 16 * lane;
            const uint8_t* vs = a.vp + row * kKvBytes + 16 * lane;
#pragma unroll
            for (int c = 0; c < 3; ++c) {
              cp_async16(dst + 16 * lane + 512 * c, ks + 512 * c);
              cp_async16(dst + 1536 + 16 * lane + 512 * c, vs + 512 * c);
            }
            if (lane < 16) cp_async4(dst + kStageNorms + 4 * lane, (lane < 8 ? a.kn : a.vn) + row + 2 * (lane & 7));
          }
          row += 16;
        }
        cp_async_commit();
        return there;
      };
      // row r of a tile's matrix operands is key r ^ (r >> 2 & 1): both operands are then
      // read from the tile's 96-byte rows without bank conflicts
      const int key_g = g ^ (g >> 2);
      uint32_t there = request(wbuf), stage = 0;
      for (int k0 = k_first; k0 < k_end; k0 += 32) {
        __syncwarp();  // every lane has read the stage that is refilled
        const uint32_t there2 = request(wbuf + (stage ^ 1u) * 2 * kStage);
        cp_async_wait<1>();
        __syncwarp();
        const uint32_t st = wbuf + stage * 2 * kStage;
        float d[2][NT][4], nk[2][2], nv[2][2], size[2][2];
        const int key[2] = {k0 + key_g, k0 + 16 + key_g};
        const int end[2] = {there & 1u ? k_end : 0, there & 2u ? k_end : 0};
        {
          uint32_t x[2][2][6];  // [tile][key g, g + 8]: 64 codes
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t src = st + i * kStage + (key_g + 8 * k) * kKvBytes + 24 * t4;
#pragma unroll
              for (int c = 0; c < 3; ++c) {
                const uint2 y = lds64(src + 8 * c);
                x[i][k][2 * c] = y.x, x[i][k][2 * c + 1] = y.y;
              }
              nk[i][k] = lds_half(st + i * kStage + kStageNorms + 2 * (key_g + 8 * k));
            }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 4; ++k) d[i][nt][k] = 0.0f;
#pragma unroll
          for (int s = 0; s < 16; ++s) {
            uint2 q[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) q[nt] = lds64(qfrag + ((nt * 16 + s) * 32 + lane) * 8);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t af[4];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                // codes 4 s .. + 3: the second pair's index at bit 7, the first one's at bit 1
                const int bit = 12 * s - 1, wi = bit >> 5, sh = bit & 31;
                const uint32_t y = s == 0           ? x[i][k][0] * 2u
                                   : sh + 12 <= 31 || wi == 5 ? x[i][k][wi] >> sh
                                                    : __funnelshift_r(x[i][k][wi], x[i][k][wi + 1], sh);
                af[k] = lds32(((y * 64u) & 0x1f80u) | tab);
                af[2 + k] = lds32((y & 0x1f80u) | tab);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816(d[i][nt], af[0], af[1], af[2], af[3], q[nt].x, q[nt].y);
            }
          }
        }
        uint16_t hv[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            hv[i][k] = lds16(st + i * kStage + kStageNorms + 32 + 2 * (key_g + 8 * k));
            size[i][k] = log2_above(hv[i][k]);
          }
        score(d, nk, size, key, end);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) nv[i][k] = half_bits_to_float(hv[i][k]) * kNvScale;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t b[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // a key that is masked out has no say, whatever its norm is (NaN stays NaN)
            float p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = d[i][nt][k] == 0.0f ? 0.0f : d[i][nt][k] * nv[i][k >> 1];
            b[nt][0] = transpose_8x8(pack_half2(p[0], p[1]));
            b[nt][1] = transpose_8x8(pack_half2(p[2], p[3]));
          }
          uint32_t vw[4][3];
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int c = 0; c < 3; ++c)
              vw[k][c] = lds32(st + i * kStage + 1536 + (((2 * t4 + (k & 1)) ^ (t4 >> 1)) + 8 * (k >> 1)) * kKvBytes + 12 * g + 4 * c);
          rows_pv<NT>(o, vw, tab, b);
        }
        there = there2;
        stage ^= 1u;
      }
      cp_async_wait<0>();
      __syncwarp();
    }

    // ---- out of the rotated domain: O^T <- H O^T / (256 kNvScale), in registers
    if (ta < e_tb) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float nm = m[nt][k] + kWinSize, c = ex2(m[nt][k] - nm);  // the window's reference, at once
          const float f = c * back / (256.0f * kNvScale);
          l[nt][k] *= c;
          m[nt][k] = nm;
          float v[32];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[2 * i] = o[nt][i][k] * f, v[2 * i + 1] = o[nt][i][2 + k] * f;
          kv_stage<float, 1>(v);
          kv_stage<float, 2>(v);
          kv_stage<float, 4>(v);
          kv_stage<float, 8>(v);
          kv_stage<float, 16>(v);
          kv_stage_x<float, 4>(v, lane);
          kv_stage_x<float, 8>(v, lane);
          kv_stage_x<float, 16>(v, lane);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[nt][i][k] = v[2 * i], o[nt][i][2 + k] = v[2 * i + 1];
        }
    }

    // ---- window keys, 16 at a time and as they are: bf16 operands, scores exact to
    // fp32, p in two bf16 parts (16 bits).  In a tile that some rows see in part, a value
    // that is not finite is carried by the sums of the rows that see it (they come out
    // NaN), and 0 * inf does not reach those that do not.
    const int w_first = it.e_lim + (max(ta, it.e_units) - it.e_units) * kRowWinUnit;
    const int w_end = min(it.e_lim + (tb - it.e_units) * kRowWinUnit, it.w_lim);
    if (w_first < w_end) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) qm[nt][k] = window_qm(256.0f / kWinScale * qmul[8 * nt + 2 * t4 + k]);
    }
#pragma unroll 1
    for (int k0 = w_first + 16 * warp; k0 < w_end; k0 += 16 * kRowWarps) {
      const int R = static_cast<int>(a.R);
      const int64_t ring = (static_cast<int64_t>(it.b) * a.H + h) * R;
      float d[1][NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) d[0][nt][0] = d[0][nt][1] = d[0][nt][2] = d[0][nt][3] = 0.0f;
      {
        const bool on0 = k0 + g < w_end, on1 = k0 + g + 8 < w_end;
        const uint16_t* s0 = a.kwin + (ring + (on0 ? (k0 + g) % R : 0)) * kKvDim + 64 * t4;
        const uint16_t* s1 = a.kwin + (ring + (on1 ? (k0 + g + 8) % R : 0)) * kKvDim + 64 * t4;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
          if (on0) x = __ldg(reinterpret_cast<const uint4*>(s0) + s);
          if (on1) y = __ldg(reinterpret_cast<const uint4*>(s1) + s);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 q0 = lds64(qfrag + C::kQFrag + ((nt * 16 + 2 * s) * 32 + lane) * 8);
            const uint2 q1 = lds64(qfrag + C::kQFrag + ((nt * 16 + 2 * s + 1) * 32 + lane) * 8);
            mma_16816_bf16(d[0][nt], x.x, y.x, x.y, y.y, q0.x, q0.y);
            mma_16816_bf16(d[0][nt], x.z, y.z, x.w, y.w, q1.x, q1.y);
          }
        }
      }
      const float one[1][2] = {{1.0f, 1.0f}}, size[1][2] = {{kWinSize, kWinSize}};
      const int key[1] = {k0 + g}, end[1] = {w_end};
      score(d, one, size, key, end);
      uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t hi = pack_bf162(d[0][nt][2 * k], d[0][nt][2 * k + 1]);
          bh[nt][k] = transpose_8x8(hi);
          bl[nt][k] = transpose_8x8(pack_bf162(d[0][nt][2 * k] - bf16x2_lo(hi), d[0][nt][2 * k + 1] - bf16x2_hi(hi)));
        }
      const uint16_t* sv[4];
      bool on[4];
      const bool part = min(k0 + 16, w_end) > it.p + it.row0 / a.G + 1;
      uint32_t bad = 0;  // bit i: key k0 + i
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = k0 + 2 * t4 + (k & 1) + 8 * (k >> 1);
        on[k] = key < w_end;
        sv[k] = a.vwin + (ring + (on[k] ? key % R : 0)) * kKvDim + 32 * g;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t x[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint4 u = make_uint4(0u, 0u, 0u, 0u);
          if (on[k]) u = __ldg(reinterpret_cast<const uint4*>(sv[k]) + c);
          x[k][0] = u.x, x[k][1] = u.y, x[k][2] = u.z, x[k][3] = u.w;
        }
        if (part) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (not_finite_bf162(x[k][0]) | not_finite_bf162(x[k][1]) | not_finite_bf162(x[k][2]) | not_finite_bf162(x[k][3])) {
              bad |= 1u << (2 * t4 + (k & 1) + 8 * (k >> 1));
#pragma unroll
              for (int i = 0; i < 4; ++i) x[k][i] &= ~((not_finite_bf162(x[k][i]) >> 15) * 0xffffu);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = __byte_perm(x[0][i], x[1][i], 0x5410), a1 = __byte_perm(x[0][i], x[1][i], 0x7632);
          const uint32_t a2 = __byte_perm(x[2][i], x[3][i], 0x5410), a3 = __byte_perm(x[2][i], x[3][i], 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816_bf16(o[nt][4 * c + i], a0, a1, a2, a3, bh[nt][0], bh[nt][1]);
            mma_16816_bf16(o[nt][4 * c + i], a0, a1, a2, a3, bl[nt][0], bl[nt][1]);
          }
        }
      }
      if (part) {
        bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (bad & ((1u << max(0, min(16, lim[nt][k] - k0))) - 1u)) l[nt][k] = NAN;
      }
    }

    // ---- the four warps' results: common maximum, sums, and O
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (shift[nt][k] != 0.0f) {
          const float c = ex2(m[nt][k] - kFarEnd);
          m[nt][k] = shift[nt][k] + kFarEnd;
          l[nt][k] *= c;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[nt][i][k] *= c;
            o[nt][i][2 + k] *= c;
          }
        }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], 4);
        l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], 8);
        l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], 16);
        if (g == 0) {
          mstat[warp][8 * nt + 2 * t4 + k] = m[nt][k];
          lstat[warp][8 * nt + 2 * t4 + k] = l[nt][k];
        }
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 8 * nt + 2 * t4 + k;
        float x = mstat[0][r];
#pragma unroll
        for (int w = 1; w < kRowWarps; ++w) x = fmaxf(x, mstat[w][r]);
        const float f = ex2(m[nt][k] - x);
        // [row tile][row parity][tile m, dim parity][lane]
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float* dst = reinterpret_cast<float*>(gbuf) + ((nt * 2 + k) * 32 + 2 * i) * 32 + lane;
          dst[0] = o[nt][i][k] * f;
          dst[32] = o[nt][i][2 + k] * f;
        }
      }
    __syncthreads();
    if (warp < 2 * NT) {
      // this warp: rows 8 nt + 2 t + k of its (nt, k) = (warp / 2, warp % 2)
      const int r = 8 * (warp >> 1) + 2 * t4 + (warp & 1);
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        const float* src = reinterpret_cast<const float*>(gtab + (qfrag + 2 * C::kQFrag - tab0) + w * C::kWarpBytes) + warp * 1024 + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += src[32 * i];
      }
      float mx = mstat[0][r], sum = 0.0f;
#pragma unroll
      for (int w = 1; w < kRowWarps; ++w) mx = fmaxf(mx, mstat[w][r]);
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) sum += lstat[w][r] * ex2(mstat[w][r] - mx);
      if (ta == 0 && tb == it.units) {
        if (r < nrows) {
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          const int row = it.row0 + r, tok = row / a.G;
          uint4* dst = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(it.c0 + tok) * a.ldo + (h * a.G + (row - tok * a.G)) * kKvDim + 32 * g);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4 x;
            x.x = float_to_bf16_bits(v[8 * c] * inv) | (float_to_bf16_bits(v[8 * c + 1] * inv) << 16);
            x.y = float_to_bf16_bits(v[8 * c + 2] * inv) | (float_to_bf16_bits(v[8 * c + 3] * inv) << 16);
            x.z = float_to_bf16_bits(v[8 * c + 4] * inv) | (float_to_bf16_bits(v[8 * c + 5] * inv) << 16);
            x.w = float_to_bf16_bits(v[8 * c + 6] * inv) | (float_to_bf16_bits(v[8 * c + 7] * inv) << 16);
            dst[c] = x;
          }
        }
      } else {
        float* part = parts + static_cast<int64_t>(2 * blockIdx.x + (ta == 0 ? 1 : 0)) * C::kPart;
        float4* dst = reinterpret_cast<float4*>(part + r * kKvDim + 32 * g);
#pragma unroll
        for (int c = 0; c < 8; ++c) dst[c] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        if (g == 0) {
          part[C::kRows * kKvDim + r] = mx;
          part[C::kRows * (kKvDim + 1) + r] = sum;
        }
      }
    }
    __syncthreads();  // the buffers and the statistics are free for the next item
  }
}

// Adds the parts of the items that boundaries between CTAs cut.  CTA (c, y)
// takes rows of the item that attention CTA c + 1 noted as first cut at its
// beginning: part 0 is CTA c's last one, part j > 0 CTA c + j's first one.
// Few-row tiles have many parts: one row per CTA, eight warps take its parts in
// turn.  128-row tiles have few: a warp per row.  A lane holds eight dims.
constexpr int kJoinThreads = 256;
template <int kRows>
struct JoinCfg {
  static constexpr int kSplit = kRows == 128 ? 1 : 8;              // warps per row
  static constexpr int kPerCta = kJoinThreads / 32 / kSplit;       // rows per CTA
  static constexpr int kPart = kRows * (kKvDim + 2);
  // float4 c of row r: row after row, or (128 rows) column after column
  static __device__ __forceinline__ int at(int r, int c) { return kRows == 128 ? c * kRows + r : r * (kKvDim / 4) + c; }
};

template <int kRows>
__global__ void __launch_bounds__(kJoinThreads)
kv_attn_join_kernel(const KvAttn a, const float* __restrict__ parts, const KvCut* __restrict__ cuts) {
  using J = JoinCfg<kRows>;
  __shared__ float acc[J::kSplit][kKvDim], ms[J::kSplit], ls[J::kSplit];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
  const int r = blockIdx.y * J::kPerCta + (J::kSplit == 1 ? warp : 0), first = J::kSplit == 1 ? 0 : warp;
  pdl_wait();  // in every CTA: the join has not ended before the attention has
  const KvCut cut = cuts[c + 1];
  if (cut.count == 0) return;
  const int c0 = __ldg(a.cu + cut.b), row = cut.row0 + r;
  if (row >= (__ldg(a.cu + cut.b + 1) - c0) * a.G) return;  // the same for all warps of a row
  float v[8];
  float m = kMinM, l = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  auto add = [&](float pm, float pl, const float (&x)[8]) {
    const float nm = fmaxf(m, pm), fo = ex2(m - nm), fn = ex2(pm - nm);
    m = nm;
    l = l * fo + pl * fn;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * fo + x[i] * fn;
  };
#pragma unroll 4
  for (int j = first; j < cut.count; j += J::kSplit) {
    const float* part = parts + static_cast<int64_t>(2 * (c + j) + (j == 0 ? 1 : 0)) * J::kPart;
    const float4 x = reinterpret_cast<const float4*>(part)[J::at(r, 2 * lane)];
    const float4 y = reinterpret_cast<const float4*>(part)[J::at(r, 2 * lane + 1)];
    add(part[kRows * kKvDim + r], part[kRows * (kKvDim + 1) + r], {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w});
  }
  if constexpr (J::kSplit > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[warp][8 * lane + i] = v[i];
    if (lane == 0) ms[warp] = m, ls[warp] = l;
    __syncthreads();
    if (warp) return;
    const int warps = min(J::kSplit, cut.count);
    for (int w = 1; w < warps; ++w) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = acc[w][8 * lane + i];
      add(ms[w], ls[w], x);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int tok = row / a.G;
  uint4 x;
  x.x = float_to_bf16_bits(v[0] * inv) | (float_to_bf16_bits(v[1] * inv) << 16);
  x.y = float_to_bf16_bits(v[2] * inv) | (float_to_bf16_bits(v[3] * inv) << 16);
  x.z = float_to_bf16_bits(v[4] * inv) | (float_to_bf16_bits(v[5] * inv) << 16);
  x.w = float_to_bf16_bits(v[6] * inv) | (float_to_bf16_bits(v[7] * inv) << 16);
  reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(c0 + tok) * a.ldo + (cut.h * a.G + (row - tok * a.G)) * kKvDim)[lane] = x;
}

template <int kRows>
int launch_join(const KvAttn& a, int ctas, const float* parts, const KvCut* cuts, cudaStream_t stream) {
  if (ctas < 2) return HLWQ_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas - 1, kRows / JoinCfg<kRows>::kPerCta);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<kRows>, a, parts, cuts) == cudaSuccess ? HLWQ_OK : HLWQ_ECUDA;
}

template <int NT>
int launch_rows(const KvAttn& a, int ctas, int tiles, float* parts, KvCut* cuts, cudaStream_t stream) {
  using C = RowCfg<NT>;
  static PerDeviceOnce attr;
  if (const int st = attr([&] {
        return cudaFuncSetAttribute(kv_attn_rows_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) ==
               cudaSuccess;
      }))
    return st;
  kv_attn_rows_kernel<NT><<<ctas, kRowThreads, C::kSmem, stream>>>(a, tiles, parts, cuts);
  if (cudaGetLastError() != cudaSuccess) return HLWQ_ECUDA;
  return launch_join<C::kRows>(a, ctas, parts, cuts, stream);
}

}  // namespace

}  // namespace hlwq
