// The extern "C" entry points of the dense-layer operators (declared in
// include/v4a_dense.h).  Each one forwards to the operator's .cu file.

#include "v4a_dense_internal.h"

extern "C" {

size_t v4a_plan_workspace_size(const v4a_plan_args* args) { return v4a::plan_workspace_size(args); }

int v4a_step_plan(const v4a_plan_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  return v4a::step_plan(args, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int64_t v4a_dense_block_bytes(int32_t num_kv_heads, int32_t dim, int32_t format) {
  if (num_kv_heads < 1 || num_kv_heads > 1024 || dim < 64 || dim > 256 || dim % 64) return 0;
  const int64_t rows = int64_t(2) * num_kv_heads * 256;
  return format == V4A_KV_BF16 ? rows * dim * 2 : format == V4A_KV_FP8_TOKEN ? rows * (dim + 4)
         : format == V4A_KV_FP8_GROUP ? rows * dim + rows / v4a::kGroupPositions * 4 : 0;
}

int v4a_dense_insert(const v4a_dense_insert_args* args, void* stream) {
  return v4a::dense_insert(args, false, nullptr, 0, static_cast<cudaStream_t>(stream));
}

int v4a_dense_insert_rows(const v4a_dense_insert_args* args, uint16_t* k_out, int64_t k_out_stride, void* stream) {
  return v4a::dense_insert(args, true, k_out, k_out_stride, static_cast<cudaStream_t>(stream));
}

int v4a_dense_read(const v4a_dense_read_args* args, void* stream) { return v4a::dense_read(args, static_cast<cudaStream_t>(stream)); }

size_t v4a_dense_attn_workspace_size(const v4a_dense_attn_args* args) { return v4a::dense_attn_workspace_size(args); }

int v4a_dense_attn(const v4a_dense_attn_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  return v4a::dense_attn(args, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

size_t v4a_prompt_attn_workspace_size(const v4a_prompt_attn_args* args) { return v4a::prompt_attn_workspace_size(args); }

int v4a_prompt_attn(const v4a_prompt_attn_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  return v4a::prompt_attn(args, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
