// mmq_prompt.cu -- the operators around the paged cache that prompts and trees
// of drafts need: norms and rotary positions with the cache append, attention
// of any number of new tokens or of a tree, and keeping a tree's path.  One
// translation unit with a status word of its own.
#include <cstdint>
#include <cuda_runtime.h>

#include "mmq_cache.cuh"

namespace mmq {

int take_prompt_status(int (&h)[8])
{
    if (!g_launched.load(std::memory_order_relaxed)) return MMQ_OK;        // h as the caller left it: zeros
    if (cudaMemcpyFromSymbol(h, g_status, sizeof(h)) != cudaSuccess) {
        cudaGetLastError();
        return MMQ_ERR_CUDA;
    }
    if (h[0] != 0) {
        const int zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        cudaMemcpyToSymbol(g_status, zero, sizeof(zero));
    }
    return MMQ_OK;
}

}  // namespace mmq

#include "mmq_norm_rope.cuh"
#include "mmq_prefill.cuh"
#include "mmq_keep.cuh"
