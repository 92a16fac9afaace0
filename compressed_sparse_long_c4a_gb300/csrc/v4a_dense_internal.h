// Internal entry points of the dense-layer operators, called by the C ABI in dense_api.cu.
#pragma once
#include <cuda_runtime.h>
#include "v4a_dense.h"

namespace v4a {
size_t plan_workspace_size(const v4a_plan_args* a);
int step_plan(const v4a_plan_args* a, void* ws, size_t ws_bytes, cudaStream_t stream);
int dense_insert(const v4a_dense_insert_args* a, cudaStream_t stream);
size_t dense_attn_workspace_size(const v4a_dense_attn_args* a);
int dense_attn(const v4a_dense_attn_args* a, void* ws, size_t ws_bytes, cudaStream_t stream);
// Checks a cache's shape and pool and gives its block stride (the block table is the caller's to check).
int dense_cache_check(const v4a_dense_cache& c, int64_t* block_bytes);
}  // namespace v4a
