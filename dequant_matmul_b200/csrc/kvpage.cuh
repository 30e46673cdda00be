#pragma once
// The paged Q3 KV cache (sm_100a): block tables and slot maps from request
// lengths, and the append that encodes the tokens leaving the exact window.
//
// Of a request's N tokens the last min(N, R) are exact (bf16 ring of R slots,
// token i in slot i % R); the n_enc(N) = max(0, N - R) before them are encoded
// (the vector encoding of kv.cuh) in pages of P tokens.  With p tokens cached
// and n new ones, new token j (0 <= j < n) makes token i = p + j - R leave the
// window; its slot is page * P + i % P, or -1 when i < 0.
//
// Page arrays: packed [num_pages][kv_heads][P][96], norms [num_pages][kv_heads][P],
// so that one head's tokens of a page are contiguous (what attention streams).

#include "kv.cuh"

namespace hlwq {

namespace {

constexpr int kKvMaxRequests = 8192;  // prefix sums of all requests in shared memory
constexpr int kTabThreads = 1024;
constexpr int kAppThreads = 128;
constexpr int kAppVector = 512 + 64;  // bytes from vector to vector of a stage: reads of 8 bytes hit all banks
constexpr int kAppStage = 4 * kAppVector, kAppStages = 3;

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 pa, pb, pd; mov.b64 pa, {%2, %3}; mov.b64 pb, {%4, %5};\n\t"
      "mul.rn.f32x2 pd, pa, pb; mov.b64 {%0, %1}, pd; }"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// cp.async: copies into shared memory that arrive in groups, in order.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Pages of the encoded tokens among n (R slots of window, P tokens to a page).
__device__ __forceinline__ uint32_t kv_pages(uint32_t n, uint32_t R, uint32_t P) { return n > R ? (n - R - 1) / P + 1 : 0u; }

constexpr uint32_t kTabCap = 0x3fffffffu;  // sums saturate here: two of them still add in 32 bits

// Exclusive prefix sums over the CTA of two values per thread (kTabThreads
// threads, sums saturating at kTabCap), and their totals.
__device__ __forceinline__ void tab_scan(uint32_t& a, uint32_t& b, uint32_t& ta, uint32_t& tb, uint2* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) ia = min(ia + x, kTabCap), ib = min(ib + y, kTabCap);
  }
  if (lane == 31) sums[warp] = make_uint2(ia, ib);
  uint32_t ea = __shfl_up_sync(0xffffffffu, ia, 1), eb = __shfl_up_sync(0xffffffffu, ib, 1);
  if (lane == 0) ea = eb = 0u;
  __syncthreads();
  uint32_t x = sums[lane].x, y = sums[lane].y;  // 32 warps: every warp scans their sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x = min(x + u, kTabCap), y = min(y + v, kTabCap);
  }
  ta = __shfl_sync(0xffffffffu, x, 31);
  tb = __shfl_sync(0xffffffffu, y, 31);
  const uint32_t px = __shfl_sync(0xffffffffu, x, (warp + 31) & 31), py = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
  a = min(ea + (warp ? px : 0u), kTabCap);
  b = min(eb + (warp ? py : 0u), kTabCap);
  __syncthreads();
}

// The last i in [0, n) with v[i] <= x (v[0] <= x, ascending).
__device__ __forceinline__ int tab_last(const uint32_t* v, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (v[m] <= x) lo = m;
    else hi = m;
  }
  return lo;
}

// Every CTA scans all requests (B <= 8192: a few KB from L2) and keeps
// cu[b] (new tokens before request b) and first[b] (pages taken before b) in shared
// memory; then the CTAs share the new pages and the T slots in strides, each
// finding its request by bisection.  A slot's page is read from the table where
// the table had it before this call, and from the free stack otherwise, so no
// CTA reads what another one writes and one launch does it all.  Bound by
// latency: a decode step of 8 requests takes 4 us, one of 512 5 us, 139 thousand
// slots of 32 prompts 4 us (launch included).
__global__ void __launch_bounds__(kTabThreads)
kv_tables_kernel(const int32_t* __restrict__ n_past, const int32_t* __restrict__ n_new, int B, uint32_t R, uint32_t P,
                 const int32_t* __restrict__ free_pages, int64_t free_cap, const int32_t* __restrict__ n_free,
                 int32_t* __restrict__ n_free_out, int32_t* __restrict__ table, uint32_t max_pages,
                 int32_t* __restrict__ cu_new, int64_t* __restrict__ slot_map, uint32_t T) {
  extern __shared__ __align__(16) uint32_t tsm[];
  uint32_t* cu = tsm;             // [B + 1]
  uint32_t* first = tsm + B + 1;  // [B + 1]
  __shared__ uint2 sums[32];
  const int have0 = __ldg(n_free);
  bool bad = have0 < 0 || have0 > free_cap, full = false;
  const int64_t have = have0 < 0 ? 0 : min(static_cast<int64_t>(have0), free_cap);
  uint32_t ca = 0, cb = 0;
  for (int b0 = 0; b0 < B; b0 += kTabThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    uint32_t n = 0, need = 0;
    if (b < B) {  // negative lengths count as 0
      const int p = __ldg(n_past + b), m = __ldg(n_new + b);
      const uint32_t up = max(p, 0), un = max(m, 0);
      bad |= p < 0 || m < 0 || up + un > static_cast<uint32_t>(INT32_MAX);
      const uint32_t old = kv_pages(up, R, P), want = kv_pages(up + un, R, P);
      full |= want > max_pages;
      need = min(min(want, max_pages) - min(old, max_pages), kTabCap);
      n = min(un, kTabCap);
    }
    uint32_t ta, tb;
    tab_scan(n, need, ta, tb, sums);
    if (b < B) {
      cu[b] = min(ca + n, kTabCap);
      first[b] = min(cb + need, kTabCap);
    }
    ca = min(ca + ta, kTabCap);
    cb = min(cb + tb, kTabCap);
  }
  bad |= ca > T;
  full |= cb > have;
  if (threadIdx.x == 0) {
    cu[B] = ca;
    first[B] = cb;
    if (blockIdx.x == 0) *n_free_out = static_cast<int32_t>(cb > have ? 0 : have - cb);
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= B; b += kTabThreads) cu_new[b] = static_cast<int32_t>(cu[b]);

  const uint32_t me = blockIdx.x * kTabThreads + threadIdx.x, all = gridDim.x * kTabThreads;
  for (uint32_t q = me; q < cb; q += all) {  // page q of this call
    const int b = tab_last(first, B, q);
    const uint32_t k = min(kv_pages(max(__ldg(n_past + b), 0), R, P), max_pages) + (q - first[b]);
    if (k < max_pages)  // (always, below the sums' cap)
      table[static_cast<int64_t>(b) * max_pages + k] = q < have ? __ldg(free_pages + (have - 1 - q)) : -1;
  }
  for (uint32_t t = me; t < T; t += all) {
    int64_t slot = -1;
    if (t < ca) {
      const int b = tab_last(cu, B, t);
      const uint32_t p = max(__ldg(n_past + b), 0), in = p + (t - cu[b]);
      if (in >= R) {  // token in - R leaves
        const uint32_t i = in - R, k = i / P, old = min(kv_pages(p, R, P), max_pages);
        int page = -1;
        if (k < old) page = table[static_cast<int64_t>(b) * max_pages + k];
        else if (k < max_pages) {
          const int64_t q = static_cast<int64_t>(first[b]) + (k - old);
          if (q < have) page = __ldg(free_pages + (have - 1 - q));
        }
        if (page >= 0) slot = static_cast<int64_t>(page) * P + (i - k * P);
      }
    }
    slot_map[t] = slot;
  }
  if (bad) raise_device_error(HLWQ_DEVERR_KV_RANGE);
  if (full) raise_device_error(HLWQ_DEVERR_KV_PAGES);
}

// The request of token t < cu[B]: the last one that begins at or before t
// (requests without tokens are passed over), found by the whole warp, 32
// probes at a time.
__device__ __forceinline__ int kv_request_of(const int32_t* __restrict__ cu, int B, int64_t t, int lane) {
  int lo = 0, n = B;  // it is among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) >> 5, i = lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, i < n && __ldg(cu + lo + i) <= t);
    const int k = le ? 31 - __clz(le) : 0;  // probe 0 counts as <= t
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// binary16 norm and codes of one vector in fp64, by the whole warp (lane: eight
// values): the definition itself, for vectors that fp32 cannot decide.
__device__ __noinline__ void kv_encode_exact(const uint16_t* src, const double* mid, uint8_t* dst, uint16_t* nrm_out,
                                             int lane) {
  const uint4 u = *reinterpret_cast<const uint4*>(src + 8 * lane);
  const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
  double v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = static_cast<double>(bf16x2_lo(wd[k]));
    v[2 * k + 1] = static_cast<double>(bf16x2_hi(wd[k]));
  }
  double ss = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fma(v[e], v[e], ss);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const double nrm = sqrt(ss);
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & h) == 0) {
        const double a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double p = __shfl_xor_sync(0xffffffffu, v[i], o);
      v[i] = (lane & o) ? p - v[i] : v[i] + p;
    }
  uint32_t bits = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double y = nrm > 0.0 ? v[e] / nrm : 0.0;
    uint32_t code = 0u;
    for (int k = 0; k < kKvLevels - 1; ++k) code += y > mid[k] ? 1u : 0u;
    bits |= code << (3 * e);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) dst[3 * lane + k] = static_cast<uint8_t>(bits >> (8 * k));
  if (lane == 0) *nrm_out = static_cast<uint16_t>(f16_rne_from_f64(nrm));
}

// Eight lanes per vector, four vectors per warp.  A token has 2 H vectors (head,
// key or value); a warp takes four of them (all it has of two tokens when H = 1)
// and goes through a contiguous range of tokens, so that requests and
// ring slots are followed from one token to the next instead of being searched for.
//
// The vector's lanes copy the token that leaves into shared memory (from the ring or,
// when the chunk is longer than the window, from the chunk; two tokens ahead, by
// cp.async), encode it, and then write the ring slot's new content: slot (p + j) % R
// of new token j < R ends up with the chunk's last token of that residue, so one group
// of lanes reads and overwrites a slot and no other touches it.
//
// Rotation: a lane first holds four values of each block of 32 and adds across the
// blocks, then the vector goes through shared memory once and a lane holds a whole
// block (whose codes are 12 consecutive bytes); as shuffles the three stages across
// lanes were 96 instructions instead of 32.
//
// Bound: HBM by its bytes (512 read, 98 written per vector); in fact the
// instructions of the rotation (8 butterfly stages) and of 256 decisions.  The
// definition asks for fp64: y_j = (x H)_j / |x| against the midpoints, |x| to the
// nearest binary16.  fp32 decides nearly always.  With u = 2^-24 and n = |x|:
//   - a butterfly value is off by at most ((1 + u)^8 - 1) sum |x_i| <= 8.01 u 16 n;
//   - the squares are exact, a path through their sum has 8 additions: n is off by
//     less than 6 u n, a border mid n (|mid| < 3) by less than 9 u 3 n;
// so a value farther than e = 160 u n > 156 u n from every border is decided, and a norm
// farther than 8 u n = 2^-21 n from every binary16 rounding border (its product with
// 1 +- 2^-21 is rounded once more).  Distances are tested in pairs: if one of a and b
// is at most e, and they differ by w, then |a b| <= e (w + e); the pairs 0, t2 and t1, t3
// have the same slope at both ends, so the test is no wider than single ones.  About one
// vector in a hundred is not decided, and is encoded by the whole warp in fp64
// (kv_encode_exact).
// 18917 tokens of 4 heads (98 MB): 49 us, 2.0 TB/s, 830 warp instructions per four
// vectors at 2.4 per cycle and SM (five CTAs per SM or 64 threads per CTA: slower); with
// everything in fp64 129 us; loads and bookkeeping alone 21 us.
//
// The decision uses the codebook's symmetry (mid[6 - k] = -mid[k], as Lloyd-Max
// gives it): three borders for |v|; another codebook goes to fp64 throughout.
__global__ void __launch_bounds__(kAppThreads, 4)
kv_append_kernel(const uint16_t* __restrict__ K, int64_t ldk, const uint16_t* __restrict__ V, int64_t ldv, int64_t T,
                 int H, const int64_t* __restrict__ slot_map, const int32_t* __restrict__ cu,
                 const int32_t* __restrict__ n_past, int B, const float* __restrict__ codebook,
                 uint8_t* __restrict__ kp, uint16_t* __restrict__ kn, uint8_t* __restrict__ vp,
                 uint16_t* __restrict__ vn, int64_t num_slots, int P, uint16_t* kwin, uint16_t* vwin, int R) {
  __shared__ double mid[kKvLevels - 1];
  __shared__ __align__(16) uint8_t swaps[kAppThreads / 32][4 * 4 * kKvDim];      // rotated vectors
  __shared__ __align__(16) uint8_t stages[kAppThreads / 32][kAppStages * kAppStage];  // vectors under way
  // every request's rows and length, by all threads (those with nothing to append would
  // not be looked at otherwise)
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kAppThreads + threadIdx.x; r < B;
       r += static_cast<int64_t>(gridDim.x) * kAppThreads) {
    const int from_row = __ldg(cu + r), to_row = __ldg(cu + r + 1), past = __ldg(n_past + r);
    if (from_row < 0 || to_row < from_row || to_row > T || past < 0) raise_device_error(HLWQ_DEVERR_KV_RANGE);
  }
  kv_check_codebook(codebook);
  if (threadIdx.x < kKvLevels - 1)
    mid[threadIdx.x] = 0.5 * (static_cast<double>(__ldg(codebook + threadIdx.x)) +
                              static_cast<double>(__ldg(codebook + threadIdx.x + 1)));
  __syncthreads();
  const bool plain = mid[3] == 0.0 && mid[4] == -mid[2] && mid[5] == -mid[1] && mid[6] == -mid[0] && mid[6] < 3.0;
  const float b1 = static_cast<float>(mid[4]), b2 = static_cast<float>(mid[5]), b3 = static_cast<float>(mid[6]);
  const int lane = threadIdx.x & 31, l8 = lane & 7;
  uint8_t* swap = swaps[threadIdx.x >> 5] + (lane >> 3) * 4 * kKvDim;
  const uint8_t* from = stages[threadIdx.x >> 5] + (lane >> 3) * kAppVector + 8 * l8;
  const uint32_t into = static_cast<uint32_t>(__cvta_generic_to_shared(from)) + 8 * l8;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kAppThreads + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (kAppThreads / 32);
  const int64_t end = min(T, static_cast<int64_t>(__ldg(cu + B)));
  const int toks = H == 1 ? 2 : 1, groups = H == 1 ? 1 : (H + 1) / 2;  // tokens of a step, warps side by side
  const int lanes = static_cast<int>(nwarps / groups);                 // warps along the tokens
  const int group = static_cast<int>(warp % groups);
  const int64_t each = ((end + lanes - 1) / lanes + toks - 1) / toks * toks;
  const int64_t tb = warp / groups * each, te = min(end, tb + each);
  if (warp / groups >= lanes || tb >= te) return;
  const int rem = H == 1 ? (lane >> 3) & 1 : 4 * group + (lane >> 3), h = rem >> 1;
  const bool is_v = rem & 1, has = rem < 2 * H;
  const uint16_t* X = (is_v ? V : K) + (has ? h : 0) * kKvDim + 32 * l8;
  const int64_t ldx = is_v ? ldv : ldk;
  uint16_t* win = (is_v ? vwin : kwin) + 32 * l8;
  int64_t t = tb + (H == 1 ? lane >> 4 : 0);  // this lane's token
  int b = kv_request_of(cu, B, tb, lane);
  const uint32_t inv_P = static_cast<uint32_t>((uint64_t(1) << 32) / static_cast<uint32_t>(P));
  int64_t next = -1;                          // the first token behind request b's
  int c0 = 0, p = 0, n = 0, at = 0;           // its first token, lengths, ring slot of token t
  int last = 0;                               // the last multiple of R below n
  bool live = false;
  // looked up two tokens ahead: whether a token leaves as it enters, from where (its
  // copy into a stage begins at once) and to which slot; its own ring slot and
  // what goes there
  struct Token {
    bool leaves, ring;
    int64_t slot;
    uint16_t* rs;
    const uint16_t *src, *fresh;
  };
  Token a1, a2;
  auto look = [&](Token& a, uint32_t stage) {
    a.leaves = false;
    a.ring = false;
    if (!has || t >= te) return;
    if (t >= next) {  // another request
      while (b + 1 < B && __ldg(cu + b + 1) <= t) ++b;
      c0 = __ldg(cu + b);
      next = __ldg(cu + b + 1);
      p = __ldg(n_past + b);
      live = c0 >= 0 && t >= c0 && t < next && next <= T && p >= 0;
      if (!live) {  // (reported above, unless t is ahead of the first request)
        raise_device_error(HLWQ_DEVERR_KV_RANGE);
        next = t + 1;
      }
      n = static_cast<int>(next - c0);
      last = R ? (n - 1) / R * R : 0;
      at = R ? static_cast<int>((static_cast<uint32_t>(p) + static_cast<uint32_t>(t - c0)) % static_cast<uint32_t>(R)) : 0;
    } else {
      at += toks;
      while (at >= R && R) at -= R;
    }
    if (!live) return;
    const int j = static_cast<int>(t - c0);
    a.ring = j < R;  // this group owns a ring slot
    a.rs = win + ((static_cast<int64_t>(b) * H + h) * R + at) * kKvDim;
    a.src = a.ring ? a.rs : X + (t - R) * ldx;
    a.fresh = X + (c0 + static_cast<int64_t>(last + j < n ? last + j : last - R + j)) * ldx;  // (of a ring token)
    if (p >= R || j >= R - p) {  // token p + j - R leaves
      a.leaves = true;
      a.slot = __ldg(slot_map + t);
#pragma unroll
      for (int c = 0; c < 4; ++c) cp_async16(into + stage * kAppStage + 128 * c, a.src - 24 * l8 + 64 * c);
    }
  };
  look(a1, 0);
  cp_async_commit();
  t += toks;
  look(a2, 1);
  cp_async_commit();
  uint32_t stage = 0;
  for (int64_t step = tb; step < te; step += toks) {
    cp_async_wait<1>();
    __syncwarp();  // this token's values are there; the stage of the one before is free
    const Token a = a1;
    a1 = a2;
    t += toks;
    look(a2, stage == 0 ? kAppStages - 1 : stage - 1);  // (its ring slot, if it has one, is another one than this token's)
    cp_async_commit();
    int64_t slot = -1;
    if (a.leaves) {
      slot = a.slot;
      if (slot < 0 || slot >= num_slots) {
        raise_device_error(HLWQ_DEVERR_KV_RANGE);
        slot = -1;
      }
    }
    float2 v[16];  // values 32 c + 4 l8 .. + 3 in v[2 c], v[2 c + 1] (anything without a slot)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint2 u = *reinterpret_cast<const uint2*>(from + stage * kAppStage + 64 * c);
      v[2 * c] = make_float2(bf16x2_lo(u.x), bf16x2_hi(u.x));
      v[2 * c + 1] = make_float2(bf16x2_lo(u.y), bf16x2_hi(u.y));
    }
    stage = stage == kAppStages - 1 ? 0 : stage + 1;
    if (__any_sync(0xffffffffu, slot >= 0)) {
      // sum of squares: a tree of 5 + 3 additions
      float2 sq[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) sq[k] = add2(mul2(v[k], v[k]), mul2(v[k + 8], v[k + 8]));
#pragma unroll
      for (int o = 4; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < o; ++k) sq[k] = add2(sq[k], sq[k + o]);
      const float ss = oct_sum(sq[0].x + sq[0].y);
      // rotation: across the blocks of 32 values, then (a lane taking a block, pieces of
      // 16 bytes exchanged without bank conflicts) within them
      auto over = [&](int o) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if ((k & o) == 0) {
            const float2 x = v[k], y = v[k + o];
            v[k] = add2(x, y);
            v[k + o] = sub2(x, y);
          }
      };
      over(2);
      over(4);
      over(8);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<float4*>(swap + c * 128 + ((l8 ^ c) << 4)) = make_float4(v[2 * c].x, v[2 * c].y, v[2 * c + 1].x, v[2 * c + 1].y);
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float4 x = *reinterpret_cast<const float4*>(swap + l8 * 128 + ((l8 ^ c) << 4));
        v[2 * c] = make_float2(x.x, x.y);
        v[2 * c + 1] = make_float2(x.z, x.w);
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = make_float2(v[k].x + v[k].y, v[k].x - v[k].y);
      over(1);
      over(2);
      over(4);
      over(8);
      const float nrm = sqrtf(ss);
      const float t1 = b1 * nrm, t2 = b2 * nrm, t3 = b3 * nrm;
      const float2 m1 = make_float2(t1, t1), m2 = make_float2(t2, t2), m3 = make_float2(t3, t3);
      // |x| lies between borders m and m + 1 (m = 0 .. 3): code 4 + m, or 3 - m for a
      // negative x.  A value shifts three sign bits into its word, code bits 2, 1, 0
      // but for inversions: of x, of |x| - t2 (m < 2), and of the product of
      // |x|'s distances from t1, t2 and t3 (m even)
      uint32_t q[4];
      float near1 = INFINITY, near2 = INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t acc = 0u;
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          const float2 x = v[4 * c + e], ax = make_float2(fabsf(x.x), fabsf(x.y));
          const float2 d1 = sub2(ax, m1), d2 = sub2(ax, m2), d3 = sub2(ax, m3);
          const float2 f = mul2(d1, d3), g = mul2(x, d2), d = mul2(f, d2);
          near1 = fminf(fminf(near1, fabsf(f.x)), fabsf(f.y));
          near2 = fminf(fminf(near2, fabsf(g.x)), fabsf(g.y));
          acc = __funnelshift_l(__float_as_uint(x.y), acc, 1);
          acc = __funnelshift_l(__float_as_uint(d2.y), acc, 1);
          acc = __funnelshift_l(__float_as_uint(d.y), acc, 1);
          acc = __funnelshift_l(__float_as_uint(x.x), acc, 1);
          acc = __funnelshift_l(__float_as_uint(d2.x), acc, 1);
          acc = __funnelshift_l(__float_as_uint(d.x), acc, 1);
        }
        const uint32_t neg = acc & 0x924924u;
        q[c] = (acc ^ (neg >> 1) ^ (neg >> 2)) ^ 0xffffffu;
      }
      // every |x| is farther than e from 0 and t2, and from t1 and t3
      const float e = nrm * 0x5p-19f;
      bool sure = near2 > e * (t2 + e) && near1 > e * (t3 - t1 + e);
      sure = (__ballot_sync(0xffffffffu, sure) >> (lane & 24) & 0xffu) == 0xffu;
      // the norm's rounding to binary16: both ends of its interval agree
      const uint32_t h0 = __half_as_ushort(__float2half_rn(nrm * (1.0f - 0x1p-21f)));
      const uint32_t h1 = __half_as_ushort(__float2half_rn(nrm * (1.0f + 0x1p-21f)));
      sure = sure && plain && ss > 0x1p-100f && ss < 0x1p100f && h0 == h1;
      // page and place in it: below 2^32 by the reciprocal, which is at most 1 short
      uint32_t page = __umulhi(static_cast<uint32_t>(slot), inv_P), place = static_cast<uint32_t>(slot) - page * P;
      if (place >= static_cast<uint32_t>(P)) ++page, place -= P;
      if (slot >> 32 > 0) page = static_cast<uint32_t>(slot / P), place = static_cast<uint32_t>(slot % P);
      const int64_t row = static_cast<int64_t>(page) * (H * P) + (h * P + place);
      uint8_t* out = (is_v ? vp : kp) + row * kKvBytes;
      uint16_t* out_n = (is_v ? vn : kn) + row;
      if (slot >= 0 && sure) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(out + 12 * l8);
        dst[0] = q[0] | (q[1] << 24);
        dst[1] = (q[1] >> 8) | (q[2] << 16);
        dst[2] = (q[2] >> 16) | (q[3] << 8);
        if (l8 == 0) *out_n = static_cast<uint16_t>(h0);
      }
      uint32_t again = __ballot_sync(0xffffffffu, slot >= 0 && !sure && l8 == 0);
      while (again) {
        const int src_lane = __ffs(static_cast<int>(again)) - 1;
        again &= again - 1;
        kv_encode_exact(reinterpret_cast<const uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(a.src), src_lane)),
                        mid,
                        reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), src_lane)),
                        reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out_n), src_lane)),
                        lane);
      }
      __syncwarp();  // the ring has been read by every lane
    }
    if (a.ring) {
#pragma unroll
      for (int c = 0; c < 4; ++c) reinterpret_cast<uint4*>(a.rs)[c] = __ldg(reinterpret_cast<const uint4*>(a.fresh) + c);
    }
  }
}

}  // namespace

int launch_kv_tables(const int32_t* n_past, const int32_t* n_new, int B, int64_t R, int64_t P,
                     const int32_t* free_pages, int64_t free_cap, const int32_t* n_free, int32_t* n_free_out,
                     int32_t* table, int64_t max_pages, int32_t* cu_new, int64_t* slot_map, int64_t T,
                     cudaStream_t stream) {
  static PerDeviceOnce attr;
  if (const int st = attr([&] {
        return cudaFuncSetAttribute(kv_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (2 * kKvMaxRequests + 2) * 4) == cudaSuccess;
      }))
    return st;
  const int grid = static_cast<int>(std::min<int64_t>(sm_count(), ceil_div(T, kTabThreads)));
  kv_tables_kernel<<<grid, kTabThreads, (2 * B + 2) * 4, stream>>>(
      n_past, n_new, B, static_cast<uint32_t>(R), static_cast<uint32_t>(P), free_pages, free_cap, n_free, n_free_out, table,
      static_cast<uint32_t>(max_pages), cu_new, slot_map, static_cast<uint32_t>(T));
  return cudaGetLastError() == cudaSuccess ? HLWQ_OK : HLWQ_ECUDA;
}

int launch_kv_append(const uint16_t* K, int64_t ldk, const uint16_t* V, int64_t ldv, int64_t T, int H,
                     const int64_t* slot_map, const int32_t* cu, const int32_t* n_past, int B, const float* codebook,
                     uint8_t* kp, uint16_t* kn, uint8_t* vp, uint16_t* vn, int64_t num_pages, int64_t P,
                     uint16_t* kwin, uint16_t* vwin, int64_t R, cudaStream_t stream) {
  // four CTAs per SM; a few tokens get a warp per step, and enough warps for every group of vectors
  const int64_t groups = H == 1 ? 1 : (H + 1) / 2, warps = std::max<int64_t>(groups, T * groups);
  const int grid = static_cast<int>(std::min<int64_t>(std::max<int64_t>(static_cast<int64_t>(sm_count()) * 4,
                                                                        ceil_div(groups, kAppThreads / 32)),
                                                      ceil_div(warps, kAppThreads / 32)));
  kv_append_kernel<<<grid, kAppThreads, 0, stream>>>(K, ldk, V, ldv, T, H, slot_map, cu, n_past, B, codebook, kp, kn, vp,
                                                     vn, num_pages * P, static_cast<int>(P), kwin, vwin,
                                                     static_cast<int>(R));
  return cudaGetLastError() == cudaSuccess ? HLWQ_OK : HLWQ_ECUDA;
}

}  // namespace hlwq
