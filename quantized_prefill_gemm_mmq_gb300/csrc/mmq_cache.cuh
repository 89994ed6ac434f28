// mmq_cache.cuh -- the paged key-value cache as the kernels see it: argument
// checks on the host, slot lookup and type conversion on the device.
#pragma once

#include <atomic>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mmq_dev.cuh"
#include "mmq_host.h"
#include "mmq_pdl.cuh"

namespace mmq {
namespace {

// kernel ids and sites in the status word
enum { KID_ROPE = 32, KID_ATTN = 33, KID_EVICT = 34, KID_VERIFY = 35, KID_PREFILL = 36, KID_NORM = 37, KID_KEEP = 38 };
enum { SITE_LEN = 1, SITE_PAGE = 2, SITE_COUNT = 3, SITE_TOKEN = 4, SITE_AXIS = 5, SITE_NODE = 6 };

// Division of 0 <= n < 2^31 by a d >= 1 that is fixed for a launch: a high
// product, an add and a shift (round-up method of Granlund and Montgomery).
struct FastDiv {
    uint32_t mul = 0;
    int shift = 0;
    FastDiv() = default;
    explicit FastDiv(int d)
    {
        while ((1ll << shift) < d) ++shift;
        mul = (uint32_t)((((1ull << shift) - (uint32_t)d) << 32) / (uint32_t)d + 1);
    }
    __device__ __forceinline__ int of(int n) const { return (int)((__umulhi(mul, (uint32_t)n) + (uint32_t)n) >> shift); }
};

// Checks of a cache descriptor that every call shares.
inline int check_cache(const mmq_kv_cache *c)
{
    if (!c) return MMQ_ERR_NULL;
    if (c->dtype != MMQ_F16 && c->dtype != MMQ_BF16) return MMQ_ERR_SHAPE;
    if (c->heads < 1 || c->heads > 65535 || c->dim < 8 || c->dim > 256 || (c->dim & 7) || c->page_size < 1 ||
        c->seqs < 0 || c->seqs > 65535 || c->cols < 1 || c->pages < 1 || c->pages > 0x7fffffff ||
        (int64_t)c->cols * c->page_size > (1 << 30))
        return MMQ_ERR_SHAPE;
    if (c->k_page < 0 || c->k_head < 0 || c->k_slot < 0 || c->v_page < 0 || c->v_head < 0 || c->v_slot < 0)
        return MMQ_ERR_SHAPE;
    if (c->seqs == 0) return MMQ_OK;
    if (!c->k || !c->v || !c->table || !c->len) return MMQ_ERR_NULL;
    if (!aligned16(c->k) || !aligned16(c->v) ||
        ((c->k_page | c->k_head | c->k_slot | c->v_page | c->v_head | c->v_slot) & 7))
        return MMQ_ERR_ALIGN;
    return MMQ_OK;
}

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

// Whether this process has launched a kernel of this unit (or captured one): before that its status word need not be
// read, which costs a status check 8 us, and the first one 14 ms for loading the unit.
std::atomic<bool> g_launched{false};

// Launch under programmatic dependent launch: the kernel may start while the
// one before it in the stream finishes, and waits for that one's end (pdl_wait)
// before it touches memory, the attention's joining launch excepted.  What the
// one before may have written is read with plain loads, not through the
// read-only path: that one promises data which nobody writes during the kernel.
// cluster: CTAs per cluster, 0 for none.
template <typename... P, typename... A>
int launch_pdl(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    g_launched.store(true, std::memory_order_relaxed);
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return launch_status();
    return launch_status();
}

// A sequence's length; 0 (reported) if its table row cannot hold it: table entries past the real length may hold other
// sequences' pages, which the largest length would reach.  L2: not through L1 (reads before pdl_wait).
template <bool L2 = false>
__device__ __forceinline__ int cache_len(const mmq_kv_cache &c, int b, int kid)
{
    const int n = L2 ? __ldcg(c.len + b) : *(c.len + b), cap = c.cols * c.page_size;
    const int r = (unsigned)n <= (unsigned)cap ? n : 0;
    if (r != n) record_error(MMQ_ERR_INDEX, kid, SITE_LEN);
    return r;
}

// A page id from the table, or -1 (reported) if it is none.
__device__ __forceinline__ int checked_page(const mmq_kv_cache &c, int pg, int kid)
{
    if (pg >= 0 && pg < c.pages) return pg;
    record_error(MMQ_ERR_INDEX, kid, SITE_PAGE);
    return -1;
}

// Page of table column `col` of sequence b, or -1 (reported) if it is none.
template <bool L2 = false>
__device__ __forceinline__ int cache_page(const mmq_kv_cache &c, int b, int col, int kid)
{
    const int32_t *at = c.table + (int64_t)b * c.cols + col;
    return checked_page(c, L2 ? __ldcg(at) : *at, kid);
}

// new tokens of sequence b, limited to 0..most
__device__ __forceinline__ int new_count(const int32_t *new_len, int b, int most, int kid)
{
    if (!new_len) return most;
    const int n = *(new_len + b);
    if (n >= 0 && n <= most) return n;
    record_error(MMQ_ERR_INDEX, kid, SITE_COUNT);
    return n < 0 ? 0 : most;
}

// two f32 values rounded to the pair type's 32 bits, the first in the low half
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u)
{
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

template <typename T>
__device__ __forceinline__ T to_cache(float x);
template <>
__device__ __forceinline__ __half to_cache<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 to_cache<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace
}  // namespace mmq
