// Internal entry points of the dense-layer operators, called by the C ABI in dense_api.cu.
#pragma once
#include <cuda_runtime.h>
#include "v4a_dense.h"

namespace v4a {
// A group: the positions of a block that share a scale (V4A_KV_FP8_GROUP).
constexpr int kGroupPositions = 64, kGroupsPerBlock = 256 / kGroupPositions;

size_t plan_workspace_size(const v4a_plan_args* a);
int step_plan(const v4a_plan_args* a, void* ws, size_t ws_bytes, cudaStream_t stream);
// k_out: the keys as packed rows, or nullptr (`rows`: the call of v4a_dense_insert_rows).
int dense_insert(const v4a_dense_insert_args* a, bool rows, uint16_t* k_out, int64_t k_out_stride, cudaStream_t stream);
// The codes and scales of the groups that the call's tokens lie in, from the rows k_out and args.v (checked by dense_insert).
int dense_quant(const v4a_dense_insert_args& a, const uint16_t* k_out, int64_t k_out_stride, int64_t block_bytes, cudaStream_t stream);
int dense_read(const v4a_dense_read_args* a, cudaStream_t stream);
size_t prompt_attn_workspace_size(const v4a_prompt_attn_args* a);
int prompt_attn(const v4a_prompt_attn_args* a, void* ws, size_t ws_bytes, cudaStream_t stream);
size_t dense_attn_workspace_size(const v4a_dense_attn_args* a);
int dense_attn(const v4a_dense_attn_args* a, void* ws, size_t ws_bytes, cudaStream_t stream);
// Checks a cache's shape and pool and gives its block stride (the block table is the caller's to check).
int dense_cache_check(const v4a_dense_cache& c, int64_t* block_bytes);
}  // namespace v4a
