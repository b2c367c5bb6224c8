// Causal attention over packed prompts of different lengths, grouped heads
// (ds_prompt_attention).
//
// Mathematics, per (query i of sequence b, head h): s_j = scale q_i . k_j for
// keys j <= Lk - Lq + i of the same sequence, out = softmax(s) V.
//
// First form: one CTA per (query, head), its warps take every 4th key with a
// running maximum and sum each, and meet in shared memory.
#include "paged.cuh"

namespace ds {

constexpr int kSimplePromptThreads = 128;

template <typename ACT, int D>
__global__ void __launch_bounds__(kSimplePromptThreads) prompt_attention_kernel(const PromptAttnArgs a) {
  constexpr int C = D / 32, W = kSimplePromptThreads / 32;
  __shared__ float so[W][D], sm[W], sl[W];
  const int row = blockIdx.x, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = find_sequence(a.cu_q, a.batch, row);
  if (b >= a.batch) return;
  const int kh = h / (a.heads / a.kv_heads);
  const int k0 = max(0, a.cu_k[b]), k1 = min(a.cu_k[b + 1], a.k_tokens);
  const int n = min(k1 - k0, (k1 - k0) - (a.cu_q[b + 1] - a.cu_q[b]) + (row - a.cu_q[b]) + 1);
  const ACT* q = static_cast<const ACT*>(a.q) + (size_t)row * a.q_stride + (size_t)h * D + lane * C;
  float qv[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    qv[i] = Act<ACT>::to_f(q[i]) * a.scale_log2;
    o[i] = 0.f;
  }
  for (int j = warp; j < n; j += W) {
    const ACT* k = static_cast<const ACT*>(a.k) + (size_t)(k0 + j) * a.k_stride + (size_t)kh * D + lane * C;
    const ACT* v = static_cast<const ACT*>(a.v) + (size_t)(k0 + j) * a.v_stride + (size_t)kh * D + lane * C;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) s += qv[i] * Act<ACT>::to_f(k[i]);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), al = exp2f(m - mn), p = exp2f(s - mn);
    l = l * al + p;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = o[i] * al + p * Act<ACT>::to_f(v[i]);
    m = mn;
  }
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

size_t prompt_attention_ws_bytes(int, int, int) { return 256; }

template <typename ACT, int D>
static cudaError_t prompt_launch(const PromptAttnArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.q_tokens, (unsigned)a.heads);
  cfg.blockDim = dim3(kSimplePromptThreads);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, prompt_attention_kernel<ACT, D>, a);
}

cudaError_t launch_prompt_attention(const PromptAttnArgs& a, void*, int, cudaStream_t st) {
  if (a.act == ActKind::F16) return a.head_dim == 64 ? prompt_launch<__half, 64>(a, st) : prompt_launch<__half, 128>(a, st);
  return a.head_dim == 64 ? prompt_launch<__nv_bfloat16, 64>(a, st) : prompt_launch<__nv_bfloat16, 128>(a, st);
}

}  // namespace ds
