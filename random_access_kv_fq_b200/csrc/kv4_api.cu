// extern "C" entry points of the 4-bit paged cache: argument validation and dispatch, as
// fq_api.cu does for the codec (nothing is allocated, nothing synchronises, no state is kept).
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "kv4.h"

using namespace fq;
using namespace fq::kv4;

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
fq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FQ_OK : FQ_ERR_CUDA; }

bool shape_ok(int d, int group) {
  return (d == 64 || d == 128) && (group == 32 || group == 64 || group == 128) && d % group == 0;
}
bool page_ok(int page) {
  return page >= kMinPage && page <= kMaxPage && (page & (page - 1)) == 0;
}
size_t elem(fq_dtype t) { return t == FQ_F32 ? 4 : 2; }

}  // namespace

extern "C" {

size_t fq_kv4_unit_bytes(int d, int group) {
  return shape_ok(d, group) ? (size_t)unit_bytes(d, group) : 0;
}

fq_status fq_page_step(const int32_t* lens, const int32_t* new_lens, int B, int32_t* block_tables,
                       int max_blocks, int page, int32_t* free_list, int n_blocks,
                       const int32_t* free_count, int32_t* lens_out, int32_t* free_count_out,
                       int32_t* cu_new, int32_t* slots, int n_slots, int32_t* refused,
                       void* stream) {
  if (B < 0 || max_blocks < 1 || n_blocks < 0 || n_slots < 0) return FQ_ERR_INVALID_ARG;
  if (B > kMaxRequests || !page_ok(page) || (int64_t)max_blocks * page > (1 << 30) ||
      (int64_t)n_blocks * page > INT_MAX || n_slots > (1 << 30))
    return FQ_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out || !cu_new || !refused || (n_slots > 0 && !slots) ||
      (n_blocks > 0 && !free_list) || (B > 0 && (!lens || !new_lens || !block_tables || !lens_out)))
    return FQ_ERR_INVALID_ARG;
  const void* all[] = {lens, new_lens, block_tables, free_list, free_count, lens_out,
                       free_count_out, cu_new, slots, refused};
  for (const void* p : all)
    if (!aligned(p, 4)) return FQ_ERR_ALIGNMENT;
  const PageArgs a{lens, new_lens, B, block_tables, max_blocks, page, free_list, n_blocks,
                   free_count, lens_out, free_count_out, cu_new, slots, n_slots, refused};
  return from_cuda(launch_page_step(a, static_cast<cudaStream_t>(stream)));
}

fq_status fq_kv4_write(const void* k, const void* v, fq_dtype type, int64_t n, int Hkv, int d,
                       int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                       int64_t v_head_stride, const int32_t* slots, uint8_t* cache,
                       int64_t n_blocks, int page, int group, void* k_values, void* v_values,
                       void* stream) {
  if (!shape_ok(d, group) || !page_ok(page)) return FQ_ERR_UNSUPPORTED;
  if (n < 0 || Hkv < 1 || n_blocks < 0 || (type != FQ_F16 && type != FQ_F32 && type != FQ_BF16))
    return FQ_ERR_INVALID_ARG;
  if (n_blocks > INT_MAX / page || n > INT_MAX / Hkv) return FQ_ERR_UNSUPPORTED;
  if (n == 0) return FQ_OK;
  if (!k || !v || !slots || (n_blocks > 0 && !cache)) return FQ_ERR_INVALID_ARG;
  if (!aligned(k, elem(type)) || !aligned(v, elem(type)) || !aligned(slots, 4) ||
      !aligned(cache, 16) || !aligned(k_values, 16) || !aligned(v_values, 16))
    return FQ_ERR_ALIGNMENT;
  const WriteArgs a{k, v, type, n, Hkv, d, k_token_stride, k_head_stride, v_token_stride,
                    v_head_stride, slots, cache, n_blocks, page, group, k_values, v_values};
  return from_cuda(launch_write(a, static_cast<cudaStream_t>(stream)));
}

size_t fq_kv4_attn_workspace_bytes(int B, int Hq, int Hkv, int d, int max_q, int max_blocks,
                                   int page) {
  if ((d != 64 && d != 128) || B < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || max_q < 1 ||
      max_blocks < 0 || !page_ok(page) || B > kMaxRequests || Hq > kMaxHeads ||
      (int64_t)max_blocks * page > (1 << 30) || max_q > (1 << 30) / Hq)
    return 0;
  return attn_workspace_bytes(B, Hq, Hkv, d, max_q, (int64_t)max_blocks * page);
}

fq_status fq_kv4_attn(const void* q, fq_dtype type, int64_t n_q, int Hq, int d,
                      int64_t q_token_stride, int64_t q_head_stride, const int32_t* cu_q, int B,
                      int max_q, const uint8_t* cache, int64_t n_blocks, int Hkv, int page,
                      int group, const int32_t* block_tables, int max_blocks,
                      const int32_t* kv_lens, int window, float scale, void* out,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!shape_ok(d, group) || !page_ok(page)) return FQ_ERR_UNSUPPORTED;
  if (B < 0 || n_q < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || n_blocks < 0 || max_blocks < 0 ||
      max_q < 0 || window < 0 || (type != FQ_F16 && type != FQ_BF16) || !std::isfinite(scale))
    return FQ_ERR_INVALID_ARG;
  if (!cu_q && (n_q != B || max_q != 1)) return FQ_ERR_INVALID_ARG;
  if (B > kMaxRequests || Hq > kMaxHeads || n_blocks > INT_MAX / page ||
      (int64_t)max_blocks * page > (1 << 30) || n_q > (1 << 30) / Hq || max_q > (1 << 30) / Hq)
    return FQ_ERR_UNSUPPORTED;
  if (B == 0 || n_q == 0 || max_q == 0) return FQ_OK;
  if (!q || !out || !kv_lens || (n_blocks > 0 && !cache) || (max_blocks > 0 && !block_tables))
    return FQ_ERR_INVALID_ARG;
  if (!aligned(q, 2) || !aligned(out, 16) || !aligned(cu_q, 4) || !aligned(cache, 16) ||
      !aligned(block_tables, 4) || !aligned(kv_lens, 4))
    return FQ_ERR_ALIGNMENT;
  const size_t need = attn_workspace_bytes(B, Hq, Hkv, d, max_q, (int64_t)max_blocks * page);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FQ_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return FQ_ERR_ALIGNMENT;
  const AttnArgs a{q, type, n_q, Hq, d, q_token_stride, q_head_stride, cu_q, B, max_q, cache,
                   n_blocks, Hkv, page, group, block_tables, max_blocks, kv_lens,
                   std::min(window, kMaxWindow), scale, out, workspace};
  return from_cuda(launch_attn(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
