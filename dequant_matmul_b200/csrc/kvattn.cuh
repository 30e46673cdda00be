#pragma once
// Attention of new tokens over the paged Q3 KV cache (sm_100a).
//
// Query i of a request with p cached and n new tokens sees keys j <= p + i:
//   s_j = scale * q . k_j,  o = sum_j softmax(s)_j v_j,
// keys and values below n_enc(p + n) decoded from their pages, the rest exact
// from the window.  Everything runs in the rotated domain: with H = H256
// (symmetric, H H = 256 I), q . k = (q H) . (c[code] n / 256) for an encoded
// key and (q H) . (k H) / 256 for a window key, and o = (1/256) (sum_j p_j y_j) H
// with y_j = n_j c[code_j] / 1 or v_j H: no cached vector is ever un-rotated.

#include "kvpage.cuh"

namespace hlwq {

namespace {

// What a kernel needs to know about the cache and the step.
struct KvAttn {
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq, ldo, T;
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

constexpr int kAtHeads = 8;  // query heads of one kv head that a CTA takes

// One CTA per (token, kv head, 8 query heads): 32 keys at a time, eight lanes
// per key.
__global__ void __launch_bounds__(256)
kv_attn_simple_kernel(const KvAttn a) {
  __shared__ __align__(16) float qs[kAtHeads * kKvQRow];
  __shared__ float vt[32][kKvDim];
  __shared__ float ss[kAtHeads][32];
  __shared__ float m_run[kAtHeads], l_run[kAtHeads], corr[kAtHeads];
  __shared__ float cb[kKvLevels];
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, g0 = blockIdx.z * kAtHeads, ng = min(kAtHeads, a.G - g0);
  const int lane = threadIdx.x & 31, l8 = lane & 7, warp = threadIdx.x >> 5, grp = threadIdx.x >> 3;
  kv_check_codebook(a.codebook);
  const int b = kv_request_of(a.cu, a.B, t);
  if (b < 0) return;
  const int64_t c0 = __ldg(a.cu + b), n = __ldg(a.cu + b + 1) - c0, p = __ldg(a.n_past + b);
  if (c0 < 0 || c0 > t || t >= c0 + n || c0 + n > a.T || p < 0) {
    if (threadIdx.x == 0) raise_device_error(HLWQ_DEVERR_KV_RANGE);
    return;
  }
  const int64_t n_enc = kv_enc(p + n, a.R), keys = p + (t - c0) + 1;
  if (threadIdx.x < kKvLevels) cb[threadIdx.x] = __ldg(a.codebook + threadIdx.x);
  if (threadIdx.x < kAtHeads) m_run[threadIdx.x] = -3.0e38f, l_run[threadIdx.x] = 0.0f;
  for (int m = warp * 4; m < ng; m += 32) {
    const int g = m + (lane >> 3);
    const bool on = g < ng;
    float v[32];
    const uint16_t* src = a.q + t * a.ldq + (h * a.G + g0 + (on ? g : 0)) * kKvDim + 32 * l8;
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = bf16_bits_to_float(__ldg(src + e));
    kv_fwht(v, lane);
    if (on) {
#pragma unroll
      for (int e = 0; e < 32; ++e) qs[kv_qpos(g, 32 * l8 + e)] = v[e] * (a.scale / 256.0f);
    }
  }
  __syncthreads();
  float acc[kAtHeads];
#pragma unroll
  for (int g = 0; g < kAtHeads; ++g) acc[g] = 0.0f;
  for (int64_t r0 = 0; r0 < keys; r0 += 32) {
    const int64_t r = r0 + grp;
    const bool on = r < keys, coded = on && r < n_enc;
    int64_t row = -1;
    if (coded) {
      const int64_t k = r / a.P;
      const int page = k < a.max_pages ? __ldg(a.table + b * a.max_pages + k) : -1;
      if (page < 0 || page >= a.num_pages) raise_device_error(HLWQ_DEVERR_KV_RANGE);
      else row = (static_cast<int64_t>(page) * a.H + h) * a.P + r % a.P;
    }
    const bool live = on && (!coded || row >= 0);
    for (int kv = 0; kv < 2; ++kv) {
      float v[32];
      float sc = 0.0f;
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0.0f;
      if (on && !coded) {
        const uint16_t* src = (kv ? a.vwin : a.kwin) + ((static_cast<int64_t>(b) * a.H + h) * a.R + r % a.R) * kKvDim + 32 * l8;
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = bf16_bits_to_float(__ldg(src + e));
        sc = 1.0f;
      }
      kv_fwht(v, lane);
      if (row >= 0) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>((kv ? a.vp : a.kp) + row * kKvBytes + 12 * l8);
        const uint32_t w[3] = {__ldg(src), __ldg(src + 1), __ldg(src + 2)};
        sc = half_bits_to_float(__ldg((kv ? a.vn : a.kn) + row));
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = cb[kv_code(w, e)];
      }
      if (kv == 0) {
        for (int g = 0; g < ng; ++g) {
          float d = 0.0f;
#pragma unroll
          for (int e = 0; e < 32; ++e) d = fmaf(v[e], qs[kv_qpos(g, 32 * l8 + e)], d);
          d = oct_sum(d);
          if (l8 == 0) ss[g][grp] = live ? d * sc : -INFINITY;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) vt[grp][32 * l8 + e] = live ? v[e] * sc : 0.0f;
      }
    }
    __syncthreads();
    for (int g = warp; g < ng; g += 8) {
      const float s = ss[g][lane];
      float m = s;
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = fmaxf(m, m_run[g]);
      float e = expf(s - m);
      ss[g][lane] = e;
#pragma unroll
      for (int o = 16; o; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
      if (lane == 0) {
        corr[g] = expf(m_run[g] - m);
        l_run[g] = l_run[g] * corr[g] + e;
        m_run[g] = m;
      }
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < kAtHeads; ++g)
      if (g < ng) {
        float s = acc[g] * corr[g];
        for (int k = 0; k < 32; ++k) s = fmaf(ss[g][k], vt[k][threadIdx.x], s);
        acc[g] = s;
      }
    __syncthreads();
  }
#pragma unroll
  for (int g = 0; g < kAtHeads; ++g)
    if (g < ng) qs[kv_qpos(g, threadIdx.x)] = acc[g];
  __syncthreads();
  for (int m = warp * 4; m < ng; m += 32) {
    const int g = m + (lane >> 3);
    const bool on = g < ng;
    float v[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = qs[kv_qpos(on ? g : 0, 32 * l8 + e)];
    kv_fwht(v, lane);
    if (on) {
      const float inv = l_run[g] > 0.0f ? 1.0f / (256.0f * l_run[g]) : l_run[g];
      uint16_t* dst = a.out + t * a.ldo + (h * a.G + g0 + g) * kKvDim + 32 * l8;
#pragma unroll
      for (int e = 0; e < 32; ++e) dst[e] = static_cast<uint16_t>(float_to_bf16_bits(v[e] * inv));
    }
  }
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

int launch_kv_attention(const KvAttn& a, int64_t, void*, size_t, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(a.H), static_cast<unsigned>(ceil_div(a.G, kAtHeads)));
  kv_attn_simple_kernel<<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? HLWQ_OK : HLWQ_ECUDA;
}

}  // namespace hlwq
