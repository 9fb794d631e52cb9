// target.h -- host-side launchers of the target-pass operators (internal to the library).
#pragma once

#include "kernels.h"

namespace dspark {

cudaError_t launch_page_map(const dspark_page_map_args &a, cudaStream_t s);
cudaError_t launch_cache_store(const dspark_cache_store_args &a, cudaStream_t s);
size_t tree_attention_ws_bytes(const dspark_tree_attention_args &a);
cudaError_t launch_tree_attention(const dspark_tree_attention_args &a, void *ws, cudaStream_t s);
cudaError_t launch_logit_rules(const dspark_logit_rules_args &a, cudaStream_t s);

}  // namespace dspark
