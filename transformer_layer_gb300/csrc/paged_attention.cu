// Attention of a few new tokens per sequence over a paged cache
// (ds_paged_attention), pages in 16 bits or in 4.
//
// Mathematics, per (sequence b, new token t, head h): s_j = scale q . k_j for
// positions j <= past[b] + t, p = softmax(s), out = sum_j p_j v_j; a 4-bit row
// stands for code * scale + minimum.  A row without positions is zeros.
//
// First form: one CTA per (row, head), its warps take every 4th position with
// a running maximum and sum each, and meet in shared memory.
#include "paged.cuh"

namespace ds {

constexpr int kSimpleThreads = 128;

template <typename ACT, int D, bool U4>
__global__ void __launch_bounds__(kSimpleThreads) paged_attention_kernel(const PagedAttnArgs a) {
  constexpr int C = D / 32;  // channels per lane
  constexpr int W = kSimpleThreads / 32;
  __shared__ float so[W][D], sm[W], sl[W];
  const int row = blockIdx.x, h = blockIdx.y;
  const int b = row / a.T, t = row % a.T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kh = h / (a.heads / a.c.kv_heads);
  const int n = a.past[b] + t + 1;
  const ACT* q = static_cast<const ACT*>(a.q) + (size_t)row * a.q_stride + (size_t)h * D + lane * C;
  float qv[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    qv[i] = Act<ACT>::to_f(q[i]) * a.scale_log2;
    o[i] = 0.f;
  }
  unsigned bad = 0;
  const long long cap = (long long)a.c.table_stride << a.c.page_shift;
  if (n > cap) bad |= kFlagCacheOverflow;
  for (int j = warp; j < n && j < cap; j += W) {
    unsigned why = 0;
    long long r = page_row(a.c, b, j, &why);
    bad |= why;
    if (r < 0) continue;
    r += (long long)kh << a.c.page_shift;
    float kv[C], vv[C];
    if constexpr (U4) {
      const float2 ks = __half22float2(static_cast<const __half2*>(a.c.k_scale)[r]);
      const float2 vs = __half22float2(static_cast<const __half2*>(a.c.v_scale)[r]);
#pragma unroll
      for (int i = 0; i < C; i += 2) {
        const size_t at = ((size_t)r * D + lane * C + i) / 2;
        const unsigned kb = static_cast<const uint8_t*>(a.c.k)[at], vb = static_cast<const uint8_t*>(a.c.v)[at];
        kv[i] = (kb & 15) * ks.x + ks.y;
        kv[i + 1] = (kb >> 4) * ks.x + ks.y;
        vv[i] = (vb & 15) * vs.x + vs.y;
        vv[i + 1] = (vb >> 4) * vs.x + vs.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        kv[i] = Act<ACT>::to_f(static_cast<const ACT*>(a.c.k)[r * D + lane * C + i]);
        vv[i] = Act<ACT>::to_f(static_cast<const ACT*>(a.c.v)[r * D + lane * C + i]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) s += qv[i] * kv[i];
    s = warp_sum(s);
    const float mn = fmaxf(m, s), al = exp2f(m - mn), p = exp2f(s - mn);
    l = l * al + p;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = o[i] * al + p * vv[i];
    m = mn;
  }
  if (bad != 0 && lane == 0) atomicOr(a.status, bad);
#pragma unroll
  for (int i = 0; i < C; ++i) so[warp][lane * C + i] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float M = -INFINITY;
    for (int w = 0; w < W; ++w) M = fmaxf(M, sm[w]);
    float L = 0.f, O = 0.f;
    for (int w = 0; w < W; ++w) {
      const float f = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - M);
      L += f * sl[w];
      O += f * so[w][threadIdx.x];
    }
    static_cast<ACT*>(a.out)[(size_t)row * a.out_stride + (size_t)h * D + threadIdx.x] =
        Act<ACT>::from_f(L > 0.f ? O / L : 0.f);
  }
}

size_t paged_attention_ws_bytes(const PagedView&, int, int, int, int) { return 256; }

template <typename ACT, int D>
static cudaError_t attention_launch(const PagedAttnArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.batch * a.T), (unsigned)a.heads);
  cfg.blockDim = dim3(kSimpleThreads);
  cfg.stream = st;
  if (a.c.u4) return cudaLaunchKernelEx(&cfg, paged_attention_kernel<ACT, D, true>, a);
  return cudaLaunchKernelEx(&cfg, paged_attention_kernel<ACT, D, false>, a);
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, void*, int, cudaStream_t st) {
  if (a.c.act == ActKind::F16)
    return a.c.head_dim == 64 ? attention_launch<__half, 64>(a, st) : attention_launch<__half, 128>(a, st);
  return a.c.head_dim == 64 ? attention_launch<__nv_bfloat16, 64>(a, st) : attention_launch<__nv_bfloat16, 128>(a, st);
}

}  // namespace ds
