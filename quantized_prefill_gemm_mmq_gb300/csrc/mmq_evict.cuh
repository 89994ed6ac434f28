// mmq_evict.cuh -- eviction from the paged cache by accumulated attention
// weight (mmq_kv_evict).
//
// Per sequence and head with L > budget entries, the `budget` largest keys
// stay, where a key is the weight's bits mapped to an unsigned order, or the
// largest number for an entry that is recent (pos >= keep_from).  The kept
// entries that lie past the budget move into the slots below it that were
// given up: as many as there are holes, each entry at most once, and sources
// (slots >= budget) and destinations (< budget) do not overlap, so the moves
// need no order.
//
// Two launches.  evict_select_kernel: a cluster of CTAs per (sequence, head)
// holds the keys in shared memory, finds the budget-th largest by three
// passes of a radix search (11, 11 and 10 bits; the CTAs' histograms are
// added through distributed shared memory), counts ties in slot order, and
// writes the list of moves and the bookkeeping of the entries that stay in
// place.  evict_move_kernel: 16-byte pieces of K and V, one per thread, and
// the moved entries' bookkeeping.
// Bound by memory: 8 B per entry and head for weight and position, 8 B for
// each that stays, 8 dim B per move.
#pragma once

namespace mmq {
namespace {

namespace evict {
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_CHUNK = 32768;       // keys per CTA: 128 KB
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_BATCH = 4;          // pieces a thread has in flight
}  // namespace evict

struct EvictParams {
    mmq_kv_cache c;
    const int32_t *keep_from;
    float *weight_out;
    int32_t *pos_out;
    int32_t *count;         // [seqs*heads] moves
    int32_t *src, *dst;     // [seqs*heads][most] slots
    int budget, most, chunk_cap;
};

// the address of `p` (this CTA's shared memory) in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t cluster_map(uint32_t a, int rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t cluster_ld(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Exclusive prefix over the block of one value per thread; `total` is the
// block's sum.  s: WARPS ints of shared memory.
__device__ __forceinline__ int block_prefix(int v, int *s, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < evict::WARPS; ++w) {
        if (w < warp) before += s[w];
        total += s[w];
    }
    return before + x - v;
}

__global__ void __launch_bounds__(evict::THREADS) evict_select_kernel(const EvictParams p)
{
    using namespace evict;
    extern __shared__ __align__(16) uint32_t keys[];       // [chunk_cap]
    __shared__ __align__(16) uint32_t hist[2][BINS];
    __shared__ int s_scan[WARPS];
    __shared__ uint32_t s_digit, s_above;
    __shared__ uint32_t s_xchg[3];                        // ties, holes, moves of this CTA
    const int tid = threadIdx.x;
    const int rank = (int)cluster_ctarank(), n_cta = (int)cluster_nctarank();
    const int row = blockIdx.x / n_cta, b = row / p.c.heads, h = row - b * p.c.heads;
    const int len = cache_len(p.c, b, KID_EVICT), ps = p.c.page_size;
    const bool whole = len <= p.budget;                    // nothing to evict

    const int chunk = (len + n_cta - 1) / n_cta;
    const int lo = min(len, rank * chunk), n = min(len, lo + chunk) - lo;
    const int keep_from = __ldg(p.keep_from + b);

    // entry address of slot, or -1
    auto entry = [&](int slot) -> int64_t {
        const int col = slot / ps, pg = cache_page(p.c, b, col, KID_EVICT);
        return pg < 0 ? -1 : ((int64_t)pg * p.c.heads + h) * ps + (slot - col * ps);
    };

    if (whole) {
        for (int i = tid; i < n; i += THREADS) {
            const int64_t e = entry(lo + i);
            if (e < 0) continue;
            p.weight_out[e] = __ldg(p.c.weight + e);
            p.pos_out[e] = __ldg(p.c.pos + e);
        }
        if (rank == 0 && tid == 0) p.count[row] = 0;
        return;                                            // the whole cluster leaves
    }

    for (int i = tid; i < n; i += THREADS) {
        const int64_t e = entry(lo + i);
        uint32_t key = 0;
        if (e >= 0) {
            if (__ldg(p.c.pos + e) >= keep_from) {
                key = 0xffffffffu;
            } else {
                const uint32_t u = __float_as_uint(__ldg(p.c.weight + e) + 0.f);    // -0 becomes 0
                key = u ^ (u & 0x80000000u ? 0xffffffffu : 0x80000000u);
            }
        }
        keys[i] = key;
    }

    // ---- the budget-th largest key, from its highest bits down
    uint32_t prefix = 0, mask = 0;
    int want = p.budget;                                   // of the keys that match the prefix
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        uint32_t *hs = hist[pass & 1];
        for (int i = tid; i < BINS; i += THREADS) hs[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += THREADS) {
            const uint32_t k = keys[i];
            if ((k & mask) == prefix) atomicAdd(&hs[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
        cluster_sync_all();
        // four bins per thread, from the highest down
        const int top = BINS - 4 - 4 * tid;
        uint32_t c[4] = {0, 0, 0, 0};
        for (int r = 0; r < n_cta; ++r) {
            const uint32_t a = cluster_map(smem_u32(hs + top), r);
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] += cluster_ld(a + 4 * k);
        }
        int total;
        const int mine = (int)(c[0] + c[1] + c[2] + c[3]);
        int before = block_prefix(mine, s_scan, total);
        if (before < want && want <= before + mine) {
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                if (before < want && want <= before + (int)c[k]) {
                    s_digit = (uint32_t)(top + k);
                    s_above = (uint32_t)before;
                }
                before += (int)c[k];
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        want -= (int)s_above;
    }
    // `want` of the keys equal to `prefix` stay, those in the lowest slots
    const int per = (n + THREADS - 1) / THREADS | 1;       // odd: a thread's run of keys meets every bank
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    int ties = 0, all;
    for (int i = i0; i < i1; ++i) ties += keys[i] == prefix;
    int tie_at = block_prefix(ties, s_scan, all);
    if (tid == 0) s_xchg[0] = (uint32_t)all;
    cluster_sync_all();
    for (int r = 0; r < rank; ++r) tie_at += (int)cluster_ld(cluster_map(smem_u32(&s_xchg[0]), r));
    int holes = 0, moves = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = keys[i];
        const bool keep = k > prefix || (k == prefix && tie_at++ < want);
        keys[i] = keep;
        if (lo + i < p.budget)
            holes += !keep;
        else
            moves += keep;
    }
    int hole_at = block_prefix(holes, s_scan, all);
    if (tid == 0) s_xchg[1] = (uint32_t)all;
    int move_at = block_prefix(moves, s_scan, all);
    if (tid == 0) s_xchg[2] = (uint32_t)all;
    cluster_sync_all();
    int n_holes = 0;
    for (int r = 0; r < n_cta; ++r) {
        const int x = (int)cluster_ld(cluster_map(smem_u32(&s_xchg[1]), r));
        const int y = (int)cluster_ld(cluster_map(smem_u32(&s_xchg[2]), r));
        n_holes += x;
        if (r < rank) {
            hole_at += x;
            move_at += y;
        }
    }
    if (rank == 0 && tid == 0) p.count[row] = n_holes;
    int32_t *src = p.src + (int64_t)row * p.most, *dst = p.dst + (int64_t)row * p.most;
    for (int i = i0; i < i1; ++i) {
        const bool keep = keys[i] != 0;
        if (lo + i < p.budget) {
            if (!keep) dst[hole_at++] = lo + i;
        } else if (keep) {
            src[move_at++] = lo + i;
        }
    }
    __syncthreads();
    // bookkeeping of what stays in place
    const int end = min(n, p.budget - lo);
    for (int i = tid; i < end; i += THREADS) {
        if (!keys[i]) continue;
        const int64_t e = entry(lo + i);
        if (e < 0) continue;
        p.weight_out[e] = __ldg(p.c.weight + e);
        p.pos_out[e] = __ldg(p.c.pos + e);
    }
    cluster_sync_all();                                    // no CTA leaves while another may read its shared memory
}

__global__ void __launch_bounds__(evict::MOVE_THREADS) evict_move_kernel(const EvictParams p)
{
    using namespace evict;
    const int row = blockIdx.y, b = row / p.c.heads, h = row - b * p.c.heads, ps = p.c.page_size;
    const int cpr = p.c.dim / 8, per_move = 2 * cpr;        // 16-byte pieces of an entry's k and v
    const int64_t pieces = (int64_t)p.count[row] * per_move;
    const int32_t *src = p.src + (int64_t)row * p.most, *dst = p.dst + (int64_t)row * p.most;
    for (int64_t at = (int64_t)blockIdx.x * MOVE_THREADS * MOVE_BATCH; at < pieces;
         at += (int64_t)gridDim.x * MOVE_THREADS * MOVE_BATCH) {
        uint4 w[MOVE_BATCH];
        uint4 *to[MOVE_BATCH];
#pragma unroll
        for (int i = 0; i < MOVE_BATCH; ++i) {
            const int64_t x = at + i * MOVE_THREADS + threadIdx.x;
            to[i] = nullptr;
            if (x >= pieces) continue;
            const int mv = (int)(x / per_move), pc = (int)(x - (int64_t)mv * per_move);
            const int s = src[mv], d = dst[mv];
            const int sc = s / ps, dc = d / ps;
            const int64_t sp = cache_page(p.c, b, sc, KID_EVICT), dp = cache_page(p.c, b, dc, KID_EVICT);
            if (sp < 0 || dp < 0) continue;
            const int so = s - sc * ps, dof = d - dc * ps;
            const bool is_v = pc >= cpr;
            uint8_t *base = static_cast<uint8_t *>(is_v ? p.c.v : p.c.k);
            const int64_t P = is_v ? p.c.v_page : p.c.k_page, H = is_v ? p.c.v_head : p.c.k_head,
                          S = is_v ? p.c.v_slot : p.c.k_slot;
            const int64_t off = (int64_t)h * H + (is_v ? pc - cpr : pc) * 8;
            w[i] = *reinterpret_cast<const uint4 *>(base + 2 * (sp * P + so * S + off));
            to[i] = reinterpret_cast<uint4 *>(base + 2 * (dp * P + dof * S + off));
            if (pc == 0) {
                const int64_t e0 = (sp * p.c.heads + h) * ps + so, e1 = (dp * p.c.heads + h) * ps + dof;
                p.weight_out[e1] = __ldg(p.c.weight + e0);
                p.pos_out[e1] = __ldg(p.c.pos + e0);
            }
        }
#pragma unroll
        for (int i = 0; i < MOVE_BATCH; ++i)
            if (to[i]) *to[i] = w[i];
    }
}

inline int evict_check(const mmq_kv_cache *c, int budget)
{
    const int rc = check_cache(c);
    if (rc != MMQ_OK) return rc;
    if (budget < 1 || (int64_t)c->cols * c->page_size > evict::MAX_CLUSTER * evict::MAX_CHUNK) return MMQ_ERR_SHAPE;
    return MMQ_OK;
}

// most moves of a row: entries past the budget, and slots below it
inline int evict_most(const mmq_kv_cache &c, int budget)
{
    const int past = c.cols * c.page_size - budget;
    return past < 1 ? 1 : past < budget ? past : budget;
}

}  // namespace
}  // namespace mmq

extern "C" int mmq_evict_sizes(const mmq_kv_cache *cache, int budget, int64_t *work_ints)
{
    const int rc = mmq::evict_check(cache, budget);
    if (rc != MMQ_OK) return rc;
    if (!work_ints) return MMQ_ERR_NULL;
    *work_ints = (int64_t)cache->seqs * cache->heads * (1 + 2 * (int64_t)mmq::evict_most(*cache, budget));
    return MMQ_OK;
}

extern "C" int mmq_kv_evict(const mmq_kv_cache *cache, int budget, const int32_t *keep_from, float *weight_out,
                            int32_t *pos_out, int32_t *work, mmq_stream_t stream)
{
    using namespace mmq;
    int rc = evict_check(cache, budget);
    if (rc != MMQ_OK) return rc;
    if (cache->seqs == 0) return MMQ_OK;
    if (!cache->weight || !cache->pos || !keep_from || !weight_out || !pos_out || !work) return MMQ_ERR_NULL;
    if (weight_out == cache->weight || pos_out == cache->pos) return MMQ_ERR_SHAPE;
    const int64_t rows = (int64_t)cache->seqs * cache->heads;
    if (rows > 65535) return MMQ_ERR_SHAPE;                // one grid row each
    if ((rc = check_arch()) != MMQ_OK) return rc;
    EvictParams p;
    p.c = *cache;
    p.keep_from = keep_from;
    p.weight_out = weight_out;
    p.pos_out = pos_out;
    p.budget = budget;
    p.most = evict_most(*cache, budget);
    p.count = work;
    p.src = work + rows;
    p.dst = p.src + rows * p.most;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    const int cap = cache->cols * cache->page_size;
    // CTAs per row: one up to 4096 keys (eight per thread), then twice as many
    // for twice the keys, up to a cluster of eight
    int cl = 1;
    while (cl < evict::MAX_CLUSTER && cap > 4096 * cl) cl *= 2;
    p.chunk_cap = (cap + cl - 1) / cl;
    static bool attr_done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return MMQ_ERR_ARCH;
    }
    if (!attr_done[dev]) {
        if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 evict::MAX_CHUNK * 4) != cudaSuccess)
            return launch_status();
        attr_done[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * cl));
    cfg.blockDim = dim3(evict::THREADS);
    cfg.dynamicSmemBytes = (size_t)p.chunk_cap * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, evict_select_kernel, p) != cudaSuccess) return launch_status();
    // rows in y; enough blocks along a row's moves to fill the device about four times
    const int64_t pieces = (int64_t)p.most * (cache->dim / 4);
    const int64_t per_block = evict::MOVE_THREADS * evict::MOVE_BATCH;
    int64_t x = (pieces + per_block - 1) / per_block;
    const int64_t enough = ((int64_t)sm_count() * 32 + rows - 1) / rows;
    if (x > enough) x = enough;
    evict_move_kernel<<<dim3((unsigned)x, (unsigned)rows), evict::MOVE_THREADS, 0, s>>>(p);
    return launch_status();
}
