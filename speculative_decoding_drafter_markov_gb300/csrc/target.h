// target.h -- host-side launchers of the target-pass operators (internal to the library).
#pragma once

#include "kernels.h"

namespace dspark {

// Launches a kernel whose CTAs may come up while the kernel before it on the stream
// drains (programmatic dependent launch): its first statement is `after_predecessor`.
// The kernels here run back to back, some for a few microseconds, of which the gap
// between two launches would be one.
template <typename... K, typename... A>
cudaError_t launch_close(void (*kern)(K...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchAttribute close{};
    close.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    close.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &close;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// waits until the kernels before on the stream are done and their writes visible
__device__ __forceinline__ void after_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

cudaError_t launch_page_map(const dspark_page_map_args &a, cudaStream_t s);
cudaError_t launch_cache_store(const dspark_cache_store_args &a, cudaStream_t s);
cudaError_t launch_rope_store(const dspark_rope_store_args &a, cudaStream_t s);
cudaError_t launch_cache_store4(const dspark_cache_store4_args &a, cudaStream_t s);
size_t tree_attention_ws_bytes(const dspark_tree_attention_args &a);
cudaError_t launch_tree_attention(const dspark_tree_attention_args &a, void *ws, cudaStream_t s);
// over caches in 4 bits
size_t tree_attention4_ws_bytes(const dspark_tree_attention_args &a);
cudaError_t launch_tree_attention4(const dspark_tree_attention_args &a, void *ws, cudaStream_t s);
cudaError_t launch_logit_rules(const dspark_logit_rules_args &a, cudaStream_t s);

}  // namespace dspark
