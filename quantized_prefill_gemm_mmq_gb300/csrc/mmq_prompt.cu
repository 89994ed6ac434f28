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

namespace {

// mmq_debug_fault_inject's mode, of each device: part of the launch here, so that the kernels need not read it.
std::atomic<int> g_withhold[64];

int withheld()
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 ? g_withhold[dev].load(std::memory_order_relaxed) : 0;
}

}  // namespace

int set_prompt_faults(int mode, unsigned long long wait_limit_ns)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaMemcpyToSymbol(g_wait_limit_ns, &wait_limit_ns, sizeof(wait_limit_ns)) != cudaSuccess) {
        cudaGetLastError();
        return MMQ_ERR_CUDA;
    }
    if (dev < 64) g_withhold[dev].store(mode, std::memory_order_relaxed);
    return MMQ_OK;
}

}  // namespace mmq

#include "mmq_norm_rope.cuh"
#include "mmq_prefill.cuh"
#include "mmq_keep.cuh"
