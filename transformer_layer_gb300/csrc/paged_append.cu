// Paged cache, writing and reading back rows: new keys and values into the
// pages with the position rotation on the way (ds_paged_append), and rows of
// the pages as packed values (ds_paged_gather).
//
// Page cited: "DeepSpeed Inference 内核优化深度解析：多 GPU 自适应并行、算子融合推理内核
// 与 MoQ 量化支持", §3.2 region 1 appends the new keys and values to one
// contiguous cache; pages, rotation and 4-bit rows are this library's own
// extension of that append.
//
// Mathematics, per (token, head) row x[0 .. d) at position p:
//   rotation of pair (i1, i2) by the table's angle i:  x1 c - x2 s, x2 c + x1 s
//   in fp32, products and sums rounded separately (the same value whichever
//   lane computes it), then one rounding to the activation type;
//   4-bit row: m = fp16(min x), s = fp16((max x - m) / 15),
//   code = clamp(rne((x - m) / s), 0, 15), from the rotated fp32 values.
//
// Bound: memory.  Every row is read once and written once.  A row is held by
// d / 8 lanes, 16 bytes each, so loads and stores are whole rows; the partner
// of a rotated pair is at most d / 2 channels away, one shuffle.  A warp works
// on one token: its sequence, page and angles are looked up once and serve
// `iters` row groups, as many as still leave every SM several warps.
#include "paged.cuh"

namespace ds {

constexpr int kRowThreads = 128;

// What a lane needs of its token: position, cache row, angles of its channels.
template <int D, bool INTER>
struct Angles {
  float c[8], s[8];  // halves: of the lane's 8 channels; neighbours: of its 4 pairs
  __device__ __forceinline__ void load(const float* row, int rot, int ch) {
    const int half = rot >> 1;
    if constexpr (INTER) {
      if (8 * ch < rot) {
        const float4 a = *reinterpret_cast<const float4*>(row + 4 * ch);
        const float4 b = *reinterpret_cast<const float4*>(row + half + 4 * ch);
        c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
        s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
      }
    } else {
      if (8 * ch < rot) {
        const int i = 8 * ch < half ? 8 * ch : 8 * ch - half;
        const float4 a0 = *reinterpret_cast<const float4*>(row + i), a1 = *reinterpret_cast<const float4*>(row + i + 4);
        const float4 b0 = *reinterpret_cast<const float4*>(row + half + i);
        const float4 b1 = *reinterpret_cast<const float4*>(row + half + i + 4);
        c[0] = a0.x; c[1] = a0.y; c[2] = a0.z; c[3] = a0.w; c[4] = a1.x; c[5] = a1.y; c[6] = a1.z; c[7] = a1.w;
        s[0] = b0.x; s[1] = b0.y; s[2] = b0.z; s[3] = b0.w; s[4] = b1.x; s[5] = b1.y; s[6] = b1.z; s[7] = b1.w;
      }
    }
  }
  // Rotates the lane's 8 channels x of its row (all lanes of the warp call it).
  __device__ __forceinline__ void rotate(float (&x)[8], int rot, int ch) const {
    if constexpr (INTER) {
      if (8 * ch < rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
          x[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        }
      }
    } else {
      const int hc = rot >> 4;  // chunks of 8 channels in a half
      const int lane = threadIdx.x & 31;
      const int from = lane + (ch < hc ? hc : (ch < 2 * hc ? -hc : 0));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(0xffffffffu, x[i], from);
        if (ch < hc) x[i] = __fsub_rn(__fmul_rn(x[i], c[i]), __fmul_rn(y, s[i]));
        else if (ch < 2 * hc) x[i] = __fadd_rn(__fmul_rn(x[i], c[i]), __fmul_rn(y, s[i]));
      }
    }
  }
};

template <typename ACT>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Act<ACT>::unpack2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <typename ACT>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Act<ACT>::pack2(x[0], x[1]), Act<ACT>::pack2(x[2], x[3]), Act<ACT>::pack2(x[4], x[5]),
                    Act<ACT>::pack2(x[6], x[7]));
}

// Quantises the row whose 8-channel chunks the D / 8 lanes of this lane's
// group hold: returns the chunk's codes, and the row's (scale, minimum).
template <int D>
__device__ __forceinline__ uint32_t quantize_row(const float (&x)[8], __half2* scale) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const __half m = __float2half_rn(lo);
  const float mf = __half2float(m);
  const __half s = __float2half_rn(__fdiv_rn(__fsub_rn(hi, mf), 15.f));
  const float sf = __half2float(s);
  uint32_t codes = 0;
  if (sf > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = rintf(__fdiv_rn(__fsub_rn(x[i], mf), sf));
      codes |= (uint32_t)fminf(fmaxf(r, 0.f), 15.f) << (4 * i);
    }
  }
  *scale = __halves2half2(s, m);
  return codes;
}

template <typename ACT, int D, bool U4, bool INTER>
__global__ void __launch_bounds__(kRowThreads) paged_append_kernel(const PagedAppendArgs a, int subs, int iters) {
  constexpr int LPR = D / 8;     // lanes per row
  constexpr int RPI = 32 / LPR;  // rows a warp holds at once
  constexpr int U = 4;           // row groups loaded together
  const int lane = threadIdx.x & 31, ch = lane % LPR;
  pdl_wait();
  pdl_launch_dependents();
  const long long w = ((long long)blockIdx.x * kRowThreads + threadIdx.x) >> 5;
  const int t = (int)(w / subs), sub = (int)(w % subs);
  if (t >= a.tokens) return;
  const int b = find_sequence(a.cu, a.batch, t);
  if (b >= a.batch) return;
  const int pos = a.past[b] + (t - a.cu[b]);
  if (pos < 0) return;
  unsigned why = 0;
  const long long row0 = page_row(a.c, b, pos, &why);
  if (row0 >= 0 && a.cos_sin != nullptr && pos >= a.max_pos) why = kFlagCacheOverflow;
  if (why != 0) {
    if (lane == 0 && sub == 0) atomicOr(a.status, why);
    return;
  }
  const int rot = a.cos_sin != nullptr ? a.rotary_dim : 0;
  Angles<D, INTER> ang;
  if (rot) ang.load(a.cos_sin + (size_t)pos * rot, rot, ch);
  const int nq = a.q != nullptr ? a.heads : 0, nk = a.c.kv_heads, rows = nq + 2 * nk;
  const ACT* q = static_cast<const ACT*>(a.q) + (size_t)t * a.q_stride;
  const ACT* k = static_cast<const ACT*>(a.k) + (size_t)t * a.k_stride;
  const ACT* v = static_cast<const ACT*>(a.v) + (size_t)t * a.v_stride;
  ACT* qo = static_cast<ACT*>(a.q_out) + (size_t)t * a.q_out_stride;
  const int r_end = min(rows, (sub + 1) * iters * RPI);
  for (int base = sub * iters * RPI; base < r_end; base += U * RPI) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * RPI + lane / LPR;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < r_end) {
        const ACT* src = r < nq ? q + (size_t)r * D : (r < nq + nk ? k + (size_t)(r - nq) * D : v + (size_t)(r - nq - nk) * D);
        raw[u] = *reinterpret_cast<const uint4*>(src + 8 * ch);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * RPI >= r_end) break;  // the same for the whole warp
      const int r = base + u * RPI + lane / LPR;
      const bool is_v = r >= nq + nk;
      float x[8];
      unpack8<ACT>(raw[u], x);
      if (rot) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
        ang.rotate(y, rot, ch);
        if (!is_v)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = y[i];
      }
      uint32_t codes = 0;
      __half2 sc;
      if constexpr (U4) codes = quantize_row<D>(x, &sc);
      if (r >= r_end) continue;
      if (r < nq) {
        *reinterpret_cast<uint4*>(qo + (size_t)r * D + 8 * ch) = pack8<ACT>(x);
        continue;
      }
      const int h = is_v ? r - nq - nk : r - nq;
      const long long row = row0 + ((long long)h << a.c.page_shift);
      void* dst = is_v ? a.c.v : a.c.k;
      if constexpr (U4) {
        static_cast<uint32_t*>(dst)[row * (D / 8) + ch] = codes;
        if (ch == 0) static_cast<__half2*>(is_v ? a.c.v_scale : a.c.k_scale)[row] = sc;
      } else {
        *reinterpret_cast<uint4*>(static_cast<ACT*>(dst) + row * D + 8 * ch) = is_v ? raw[u] : pack8<ACT>(x);
      }
    }
  }
}

template <typename ACT, int D, bool U4>
__global__ void __launch_bounds__(kRowThreads) paged_gather_kernel(const PagedGatherArgs a, int subs, int iters) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, U = 4;
  const int lane = threadIdx.x & 31, ch = lane % LPR;
  pdl_wait();
  pdl_launch_dependents();
  const long long w = ((long long)blockIdx.x * kRowThreads + threadIdx.x) >> 5;
  const int t = (int)(w / subs), sub = (int)(w % subs);
  if (t >= a.tokens) return;
  const int b = find_sequence(a.cu, a.batch, t);
  if (b >= a.batch) return;
  const int pos = a.first[b] + (t - a.cu[b]);
  if (pos < 0) return;
  unsigned why = 0;
  const long long row0 = page_row(a.c, b, pos, &why);
  if (why != 0 && lane == 0 && sub == 0) atomicOr(a.status, why);
  const int nk = a.c.kv_heads;
  ACT* ko = static_cast<ACT*>(a.k) + (size_t)t * a.k_stride;
  ACT* vo = static_cast<ACT*>(a.v) + (size_t)t * a.v_stride;
  const int r_end = min(2 * nk, (sub + 1) * iters * RPI);
  for (int base = sub * iters * RPI; base < r_end; base += U * RPI) {
    uint4 raw[U];
    __half2 sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * RPI + lane / LPR;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      sc[u] = __float2half2_rn(0.f);
      if (r < r_end && row0 >= 0) {
        const long long row = row0 + ((long long)(r < nk ? r : r - nk) << a.c.page_shift);
        const void* src = r < nk ? a.c.k : a.c.v;
        if constexpr (U4) {
          raw[u].x = static_cast<const uint32_t*>(src)[row * (D / 8) + ch];
          sc[u] = static_cast<const __half2*>(r < nk ? a.c.k_scale : a.c.v_scale)[row];
        } else {
          raw[u] = *reinterpret_cast<const uint4*>(static_cast<const ACT*>(src) + row * D + 8 * ch);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * RPI + lane / LPR;
      if (r >= r_end) break;
      uint4 out = raw[u];
      if constexpr (U4) {
        const float s = __low2float(sc[u]), m = __high2float(sc[u]);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn((float)((raw[u].x >> (4 * i)) & 15u), s), m);
        out = pack8<ACT>(x);
      }
      *reinterpret_cast<uint4*>((r < nk ? ko + (size_t)r * D : vo + (size_t)(r - nk) * D) + 8 * ch) = out;
    }
  }
}

// Splits a token's `groups` row groups over as many warps as keep the GPU
// busy: one warp does up to 8 groups, fewer while there are under 16 warps an
// SM in the launch.
static void split_rows(int tokens, int groups, int num_sms, int* subs, int* iters) {
  int it = 8;
  while (it > 1 && (long long)tokens * ((groups + it - 1) / it) < 16LL * num_sms) it >>= 1;
  *iters = it;
  *subs = (groups + it - 1) / it;
}

template <typename ACT, int D>
static cudaError_t append_launch(const PagedAppendArgs& a, int num_sms, cudaStream_t st) {
  constexpr int RPI = 32 / (D / 8);
  const int rows = (a.q != nullptr ? a.heads : 0) + 2 * a.c.kv_heads;
  int subs, iters;
  split_rows(a.tokens, (rows + RPI - 1) / RPI, num_sms, &subs, &iters);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)a.tokens * subs + kRowThreads / 32 - 1) / (kRowThreads / 32)));
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.c.u4) {
    if (a.interleaved) return cudaLaunchKernelEx(&cfg, paged_append_kernel<ACT, D, true, true>, a, subs, iters);
    return cudaLaunchKernelEx(&cfg, paged_append_kernel<ACT, D, true, false>, a, subs, iters);
  }
  if (a.interleaved) return cudaLaunchKernelEx(&cfg, paged_append_kernel<ACT, D, false, true>, a, subs, iters);
  return cudaLaunchKernelEx(&cfg, paged_append_kernel<ACT, D, false, false>, a, subs, iters);
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, int num_sms, cudaStream_t st) {
  if (a.c.act == ActKind::F16)
    return a.c.head_dim == 64 ? append_launch<__half, 64>(a, num_sms, st) : append_launch<__half, 128>(a, num_sms, st);
  return a.c.head_dim == 64 ? append_launch<__nv_bfloat16, 64>(a, num_sms, st)
                            : append_launch<__nv_bfloat16, 128>(a, num_sms, st);
}

template <typename ACT, int D>
static cudaError_t gather_launch(const PagedGatherArgs& a, int num_sms, cudaStream_t st) {
  constexpr int RPI = 32 / (D / 8);
  int subs, iters;
  split_rows(a.tokens, (2 * a.c.kv_heads + RPI - 1) / RPI, num_sms, &subs, &iters);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)a.tokens * subs + kRowThreads / 32 - 1) / (kRowThreads / 32)));
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.c.u4) return cudaLaunchKernelEx(&cfg, paged_gather_kernel<ACT, D, true>, a, subs, iters);
  return cudaLaunchKernelEx(&cfg, paged_gather_kernel<ACT, D, false>, a, subs, iters);
}

cudaError_t launch_paged_gather(const PagedGatherArgs& a, int num_sms, cudaStream_t st) {
  if (a.c.act == ActKind::F16)
    return a.c.head_dim == 64 ? gather_launch<__half, 64>(a, num_sms, st) : gather_launch<__half, 128>(a, num_sms, st);
  return a.c.head_dim == 64 ? gather_launch<__nv_bfloat16, 64>(a, num_sms, st)
                            : gather_launch<__nv_bfloat16, 128>(a, num_sms, st);
}

}  // namespace ds
