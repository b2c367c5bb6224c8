// Internal launch interface of the paged-cache operators (paged_api.cu holds
// their C entry points).  Nothing here is exported from the shared library.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ds_layer.h"
#include "internal.h"

namespace ds {

// The caller's paged cache as the kernels see it.
struct PagedView {
  void *k = nullptr, *v = nullptr;
  void *k_scale = nullptr, *v_scale = nullptr;  // 4-bit pages: [row][2] fp16
  const int32_t* table = nullptr;
  int num_pages = 0, page_shift = 0, table_stride = 0, kv_heads = 0, head_dim = 0;
  bool u4 = false;
  ActKind act = ActKind::F16;
};

// Workspace of the attention calls: status word, then counters (at a place of
// their own, so that one workspace serves any of these calls in turn: every
// call leaves them at zero), then partial sums.
constexpr size_t kWsCounters = 256, kWsData = 256 + 4096;
constexpr int kWsMaxCounters = 1024;

struct PagedAppendArgs {
  PagedView c;
  const float* cos_sin = nullptr;  // null: no rotation
  int max_pos = 0, rotary_dim = 0, interleaved = 0;
  const void* q = nullptr;         // null: k and v only
  void* q_out = nullptr;
  const void *k = nullptr, *v = nullptr;
  long long q_stride = 0, q_out_stride = 0, k_stride = 0, v_stride = 0;
  int heads = 0, tokens = 0, batch = 0;
  const int32_t *cu = nullptr, *past = nullptr;  // cu null: T rows a sequence
  int T = 1;
  unsigned* status = nullptr;
};

struct PagedGatherArgs {
  PagedView c;
  void *k = nullptr, *v = nullptr;
  long long k_stride = 0, v_stride = 0;
  int tokens = 0, batch = 0;
  const int32_t *cu = nullptr, *first = nullptr;
  unsigned* status = nullptr;
};

struct PagedAttnArgs {
  PagedView c;
  const void* q = nullptr;
  void* out = nullptr;
  long long q_stride = 0, out_stride = 0;
  int heads = 0, batch = 0, T = 1;
  const int32_t* past = nullptr;
  float scale_log2 = 0.f;  // scale * log2(e)
  unsigned* status = nullptr;
};

struct PromptAttnArgs {
  const void *q = nullptr, *k = nullptr, *v = nullptr;
  void* out = nullptr;
  int heads = 0, kv_heads = 0, head_dim = 0;
  ActKind act = ActKind::F16;
  long long q_stride = 0, k_stride = 0, v_stride = 0, out_stride = 0;
  int q_tokens = 0, k_tokens = 0, batch = 0;
  const int32_t *cu_q = nullptr, *cu_k = nullptr;
  float scale_log2 = 0.f;
  unsigned* status = nullptr;
};

// What of a paged cache is refused before any launch; `dev` -1: not its pointers.
ds_status paged_check_cache(const ds_paged_cache* c, int dev);
ds_status paged_check_rotary(const ds_rotary* r, int head_dim, int dev);
PagedView paged_view(const ds_paged_cache* c);
bool paged_on_device(const void* p, int dev);

cudaError_t launch_paged_append(const PagedAppendArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_paged_gather(const PagedGatherArgs& a, int num_sms, cudaStream_t st);
// n values (a multiple of 8) between fp32 and the activation type.
cudaError_t launch_narrow(ActKind ak, const float* in, void* out, long long n, cudaStream_t st);
cudaError_t launch_widen(ActKind ak, const void* in, float* out, long long n, cudaStream_t st);
size_t paged_attention_ws_bytes(const PagedView& c, int heads, int batch, int T, int num_sms);
cudaError_t launch_paged_attention(const PagedAttnArgs& a, void* ws, int num_sms, cudaStream_t st);
size_t prompt_attention_ws_bytes(int batch, int tokens, int num_sms);
// *kernels: how many were launched.
cudaError_t launch_prompt_attention(const PromptAttnArgs& a, void* ws, int num_sms, cudaStream_t st, int* kernels);

}  // namespace ds
