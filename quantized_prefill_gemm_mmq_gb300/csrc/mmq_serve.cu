// mmq_serve.cu -- the decode-side operators around the products: rotary
// positions with the cache append, attention of new tokens over the paged
// cache, eviction from it, and the verification of drafted tokens.  One
// translation unit, so that its kernels share a status word, which
// mmq_check_status reads after the GEMM unit's own.
#include <cstdint>
#include <cuda_runtime.h>

#include "mmq_cache.cuh"

namespace mmq {

namespace {

// streaming multiprocessors of the current device, looked up once per device
int sm_count()
{
    static int sms[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    if (sms[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 152;
        sms[dev] = n;
    }
    return sms[dev];
}

}  // namespace

int take_serve_status(int (&h)[8])
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

#include "mmq_rope.cuh"
#include "mmq_attn.cuh"
#include "mmq_evict.cuh"
#include "mmq_verify.cuh"
