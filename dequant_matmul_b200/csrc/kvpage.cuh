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
constexpr int kAppThreads = 256;

// Encoded tokens among n (R slots of window).
__host__ __device__ inline int64_t kv_enc(int64_t n, int64_t R) { return n > R ? n - R : 0; }

// One request's lengths, checked: negative ones count as 0.
__device__ __forceinline__ int kv_len(int v, bool& bad) {
  if (v < 0) bad = true;
  return v < 0 ? 0 : v;
}

// Exclusive prefix sums over the CTA of two values per thread (kTabThreads
// threads), and their totals.
__device__ __forceinline__ void tab_scan(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb, int64_t (*sums)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t a0 = a, b0 = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += x, b += y;
  }
  if (lane == 31) sums[warp][0] = a, sums[warp][1] = b;
  __syncthreads();
  int64_t x = sums[lane][0], y = sums[lane][1];  // 32 warps: every warp scans their sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += u, y += v;
  }
  ta = __shfl_sync(0xffffffffu, x, 31);
  tb = __shfl_sync(0xffffffffu, y, 31);
  const int64_t px = __shfl_sync(0xffffffffu, x, (warp + 31) & 31), py = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
  a += (warp ? px : 0) - a0;
  b += (warp ? py : 0) - b0;
  __syncthreads();
}

// Every CTA scans all requests (B <= 8192: a few KB from L2) and keeps
// cu[b] (new tokens before request b) and first[b] (pages allocated before b)
// in shared memory; then the CTAs share the work: requests round-robin, a warp
// each, for the new table entries, and T in strides for the slot map.  A slot's
// page is read from the table where the table had it before this call, and
// from the free stack otherwise, so no CTA reads what another one writes.
__global__ void __launch_bounds__(kTabThreads)
kv_tables_kernel(const int32_t* __restrict__ n_past, const int32_t* __restrict__ n_new, int B, int64_t R, int64_t P,
                 const int32_t* __restrict__ free_pages, int64_t free_cap, const int32_t* __restrict__ n_free,
                 int32_t* __restrict__ n_free_out, int32_t* __restrict__ table, int64_t max_pages,
                 int32_t* __restrict__ cu_new, int64_t* __restrict__ slot_map, int64_t T) {
  extern __shared__ __align__(16) int32_t tsm[];
  int32_t* cu = tsm;                // [B + 1]
  int32_t* first = tsm + B + 1;     // [B]
  __shared__ int64_t sums[32][2];
  bool bad = false, full = false;
  int64_t ca = 0, cb = 0;
  for (int b0 = 0; b0 < B; b0 += kTabThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int64_t n = 0, need = 0;
    if (b < B) {
      const int64_t p = kv_len(__ldg(n_past + b), bad);
      n = kv_len(__ldg(n_new + b), bad);
      const int64_t old = ceil_div(kv_enc(p, R), P), want = ceil_div(kv_enc(p + n, R), P);
      if (want > max_pages) full = true;
      need = min(want, max_pages) - min(old, max_pages);
    }
    int64_t a = n, c = need, ta, tb;
    tab_scan(a, c, ta, tb, sums);
    if (b < B) {
      cu[b] = static_cast<int32_t>(min(ca + a, static_cast<int64_t>(INT32_MAX)));
      first[b] = static_cast<int32_t>(min(cb + c, static_cast<int64_t>(INT32_MAX)));
    }
    ca += ta;
    cb += tb;
  }
  int64_t have = __ldg(n_free);
  if (have < 0 || have > free_cap) {
    bad = true;
    have = have < 0 ? 0 : free_cap;
  }
  if (ca > T) bad = true;
  if (threadIdx.x == 0) {
    cu[B] = static_cast<int32_t>(min(ca, static_cast<int64_t>(INT32_MAX)));
    if (blockIdx.x == 0) {
      if (cb > have) full = true;
      *n_free_out = static_cast<int32_t>(cb > have ? 0 : have - cb);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= B; b += kTabThreads) cu_new[b] = cu[b];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = blockIdx.x * (kTabThreads / 32) + warp; b < B; b += gridDim.x * (kTabThreads / 32)) {
    bool x = false;
    const int64_t p = kv_len(__ldg(n_past + b), x), n = cu[b + 1] - cu[b];
    const int64_t old = min(ceil_div(kv_enc(p, R), P), max_pages), want = min(ceil_div(kv_enc(p + n, R), P), max_pages);
    for (int64_t k = old + lane; k < want; k += 32) {
      const int64_t at = have - 1 - (first[b] + k - old);
      table[b * max_pages + k] = at >= 0 ? __ldg(free_pages + at) : -1;
    }
  }
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTabThreads + threadIdx.x; t < T;
       t += static_cast<int64_t>(gridDim.x) * kTabThreads) {
    int64_t slot = -1;
    if (t < cu[B]) {
      int lo = 0, hi = B;  // the last request that begins at or before t
      while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (cu[m] <= t) lo = m;
        else hi = m;
      }
      bool x = false;
      const int64_t p = kv_len(__ldg(n_past + lo), x), i = p + (t - cu[lo]) - R;
      if (i >= 0) {
        const int64_t k = i / P, old = min(ceil_div(kv_enc(p, R), P), max_pages);
        int64_t page = -1;
        if (k < old) page = table[lo * max_pages + k];
        else if (k < max_pages) {
          const int64_t at = have - 1 - (first[lo] + k - old);
          if (at >= 0) page = __ldg(free_pages + at);
        }
        if (page >= 0) slot = page * P + i % P;
      }
    }
    slot_map[t] = slot;
  }
  if (bad) raise_device_error(HLWQ_DEVERR_KV_RANGE);
  if (full) raise_device_error(HLWQ_DEVERR_KV_PAGES);
}

// The request of token t: the last one that begins at or before t (requests
// without tokens are passed over); -1 when t is behind the last token or the
// offsets are not usable.
__device__ __forceinline__ int kv_request_of(const int32_t* __restrict__ cu, int B, int64_t t) {
  if (t >= __ldg(cu + B)) return -1;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (__ldg(cu + m) <= t) lo = m;
    else hi = m;
  }
  return lo;
}

// Eight lanes per vector, four vectors per warp; vector v = (token t, head h,
// key or value).  The vector's lanes read the token that leaves (from the ring
// or, when the chunk is longer than the window, from the chunk), encode it, and
// then write the ring slot's new content: slot (p + j) % R of new token j < R
// ends up with the chunk's last token of that residue, so one group of lanes
// reads and overwrites a slot and no other touches it.
__global__ void __launch_bounds__(kAppThreads)
kv_append_kernel(const uint16_t* __restrict__ K, int64_t ldk, const uint16_t* __restrict__ V, int64_t ldv, int64_t T,
                 int H, const int64_t* __restrict__ slot_map, const int32_t* __restrict__ cu,
                 const int32_t* __restrict__ n_past, int B, const float* __restrict__ codebook,
                 uint8_t* __restrict__ kp, uint16_t* __restrict__ kn, uint8_t* __restrict__ vp,
                 uint16_t* __restrict__ vn, int64_t num_slots, int64_t P, uint16_t* kwin, uint16_t* vwin, int64_t R) {
  __shared__ double mid[kKvLevels - 1];
  kv_check_codebook(codebook);
  if (threadIdx.x < kKvLevels - 1)
    mid[threadIdx.x] = 0.5 * (static_cast<double>(__ldg(codebook + threadIdx.x)) +
                              static_cast<double>(__ldg(codebook + threadIdx.x + 1)));
  __syncthreads();
  const int lane = threadIdx.x & 31, l8 = lane & 7;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kAppThreads + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (kAppThreads / 32);
  const int64_t nvec = T * H * 2;
  for (int64_t v0 = warp * 4; v0 < nvec; v0 += nwarps * 4) {
    const int64_t vi = v0 + (lane >> 3);
    const int64_t t = vi / (2 * H);
    const int rem = static_cast<int>(vi - t * 2 * H), h = rem >> 1;
    const bool is_v = rem & 1;
    const uint16_t* X = is_v ? V : K;
    const int64_t ldx = is_v ? ldv : ldk;
    uint16_t* win = is_v ? vwin : kwin;
    int b = -1;
    int64_t c0 = 0, j = 0, p = 0, n = 0;
    if (vi < nvec) {
      b = kv_request_of(cu, B, t);
      if (b >= 0) {
        c0 = __ldg(cu + b);
        n = __ldg(cu + b + 1) - c0;
        j = t - c0;
        p = __ldg(n_past + b);
        if (c0 < 0 || j < 0 || j >= n || c0 + n > T || p < 0) {
          raise_device_error(HLWQ_DEVERR_KV_RANGE);
          b = -1;
        }
      }
    }
    const int64_t i = p + j - R;  // the token that leaves
    int64_t slot = -1;
    if (b >= 0 && i >= 0) {
      slot = __ldg(slot_map + t);
      if (slot < 0 || slot >= num_slots) {
        raise_device_error(HLWQ_DEVERR_KV_RANGE);
        slot = -1;
      }
    }
    const bool ring = b >= 0 && j < R;  // this group owns a ring slot
    uint16_t* rs = win + ((static_cast<int64_t>(b) * H + h) * R + (ring ? (p + j) % R : 0)) * kKvDim + 32 * l8;
    const uint4* src = slot < 0 ? nullptr
                       : ring   ? reinterpret_cast<const uint4*>(rs)
                                : reinterpret_cast<const uint4*>(X + (t - R) * ldx + h * kKvDim + 32 * l8);
    double v[32];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (src) u = src[c];
      const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[8 * c + 2 * k] = static_cast<double>(bf16x2_lo(wd[k]));
        v[8 * c + 2 * k + 1] = static_cast<double>(bf16x2_hi(wd[k]));
      }
    }
    if (ring) {
      const int64_t jf = j + (n - 1 - j) / R * R;
      const uint4* xs = reinterpret_cast<const uint4*>(X + (c0 + jf) * ldx + h * kKvDim + 32 * l8);
#pragma unroll
      for (int c = 0; c < 4; ++c) reinterpret_cast<uint4*>(rs)[c] = __ldg(xs + c);
    }
    if (!__any_sync(0xffffffffu, slot >= 0)) continue;
    double ss = 0.0;
#pragma unroll
    for (int e = 0; e < 32; ++e) ss = fma(v[e], v[e], ss);
    ss = oct_sum(ss);
    const double nrm = sqrt(ss);
    kv_fwht(v, lane);
    uint32_t w[3] = {0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const double y = nrm > 0.0 ? v[e] / nrm : 0.0;
      uint32_t code = 0u;
#pragma unroll
      for (int k = 0; k < kKvLevels - 1; ++k) code += y > mid[k] ? 1u : 0u;
      const int bit = 3 * e, k = bit >> 5, sh = bit & 31;
      w[k] |= code << sh;
      if (sh > 29) w[k + 1] |= code >> (32 - sh);
    }
    if (slot >= 0) {
      const int64_t row = (slot / P * H + h) * P + slot % P;
      uint32_t* dst = reinterpret_cast<uint32_t*>((is_v ? vp : kp) + row * kKvBytes + 12 * l8);
      dst[0] = w[0];
      dst[1] = w[1];
      dst[2] = w[2];
      if (l8 == 0) (is_v ? vn : kn)[row] = static_cast<uint16_t>(f16_rne_from_f64(nrm));
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
                                    (2 * kKvMaxRequests + 1) * 4) == cudaSuccess;
      }))
    return st;
  const int grid = static_cast<int>(std::min<int64_t>(sm_count(), std::max<int64_t>(1, ceil_div(T, kTabThreads))));
  kv_tables_kernel<<<grid, kTabThreads, (2 * B + 1) * 4, stream>>>(n_past, n_new, B, R, P, free_pages, free_cap, n_free,
                                                                   n_free_out, table, max_pages, cu_new, slot_map, T);
  return cudaGetLastError() == cudaSuccess ? HLWQ_OK : HLWQ_ECUDA;
}

int launch_kv_append(const uint16_t* K, int64_t ldk, const uint16_t* V, int64_t ldv, int64_t T, int H,
                     const int64_t* slot_map, const int32_t* cu, const int32_t* n_past, int B, const float* codebook,
                     uint8_t* kp, uint16_t* kn, uint8_t* vp, uint16_t* vn, int64_t num_pages, int64_t P,
                     uint16_t* kwin, uint16_t* vwin, int64_t R, cudaStream_t stream) {
  const int64_t max_ctas = static_cast<int64_t>(sm_count()) * 4;
  const int grid = static_cast<int>(std::min<int64_t>(max_ctas, ceil_div(T * H * 2, kAppThreads / 8)));
  kv_append_kernel<<<grid, kAppThreads, 0, stream>>>(K, ldk, V, ldv, T, H, slot_map, cu, n_past, B, codebook, kp, kn, vp,
                                                     vn, num_pages * P, P, kwin, vwin, R);
  return cudaGetLastError() == cudaSuccess ? HLWQ_OK : HLWQ_ECUDA;
}

}  // namespace hlwq
