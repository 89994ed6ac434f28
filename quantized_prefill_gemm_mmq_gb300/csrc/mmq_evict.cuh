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
// One launch: one CTA (a cluster of them where there are few rows) per
// sequence and head holds the keys in shared memory, finds the budget-th
// largest by three passes of a radix search (11, 11 and 10 bits; a cluster adds
// its histograms through distributed shared memory), counts ties in slot
// order, lists the moves, and makes them.  Slots are dealt to threads in
// stripes, so that every pass reads memory side by side; the order of slots is
// kept by counting per (stripe, warp) with ballots and one scan over those
// counts.  For the moves a warp looks up 32 at once, one per lane, then copies
// them one after the other, a 16-byte piece of K or V per lane.
// Bound by memory: 8 B per entry and head for weight and position, 8 B for
// each that stays, 8 dim B per move; with few moves by the latency of the
// selection's passes.
// Measured: 16 sequences up to 32768 entries of 8 heads of 128 down to 4096,
// 105 us, of which 72 us move 485 MB (6.7 TB/s); 1100 entries of 32 heads down
// to 1024, 8.6 us.
#pragma once

namespace mmq {
namespace {

namespace evict {
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int PER_SM = 2;
constexpr int BINS = 2048;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_CHUNK = 32768;               // keys per CTA: 128 KB
constexpr int STRIPES = MAX_CHUNK / THREADS;   // at most
constexpr int MAX_COLS = 4096;                 // page ids kept in shared memory
constexpr int BATCH = 8;                       // stripes whose loads a thread has in flight
constexpr int MOVE_BATCH = 3;                  // moves a warp has in flight
}  // namespace evict

struct EvictParams {
    mmq_kv_cache c;
    const int32_t *keep_from;
    float *weight_out;
    int32_t *pos_out;
    int32_t *src, *dst;     // [seqs*heads][most] slots
    int budget, most, chunk_cap, cols_cap;
    FastDiv page_div;
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

__device__ __forceinline__ uint4 cluster_ld4(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
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
    for (int w = 0; w < evict::WARPS; w += 4) {
        const int4 q = *reinterpret_cast<const int4 *>(s + w);
        before += (w < warp ? q.x : 0) + (w + 1 < warp ? q.y : 0) + (w + 2 < warp ? q.z : 0) + (w + 3 < warp ? q.w : 0);
        total += (q.x + q.y) + (q.z + q.w);
    }
    return before + x - v;
}

// Exclusive prefixes, in the order (stripe, warp), of counts that lane 0 of
// every warp has put into cnt[stripe*WARPS + warp], in place; returns the sum.
__device__ __forceinline__ int stripe_prefix(int *cnt, int stripes, int *s)
{
    constexpr int PER = evict::STRIPES * evict::WARPS / evict::THREADS;
    __syncthreads();
    const int n = stripes * evict::WARPS, i = threadIdx.x * PER;
    int v[PER], mine = 0, total;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        v[k] = i + k < n ? cnt[i + k] : 0;
        mine += v[k];
    }
    int before = block_prefix(mine, s, total);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (i + k < n) cnt[i + k] = before;
        before += v[k];
    }
    __syncthreads();
    return total;
}

__global__ void __launch_bounds__(evict::THREADS, evict::PER_SM) evict_kernel(const EvictParams p)
{
    using namespace evict;
    extern __shared__ __align__(16) uint32_t keys[];       // [chunk_cap], then the page ids [cols_cap]
    __shared__ __align__(16) uint32_t hist[2][BINS];
    __shared__ int s_cnt[2][STRIPES * WARPS];
    __shared__ __align__(16) int s_scan[WARPS];
    __shared__ uint32_t s_digit, s_above, s_match;
    __shared__ uint32_t s_xchg[2];                        // ties; holes and moves of this CTA
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t below = (1u << lane) - 1;
    pdl_wait();
    pdl_launch_dependents();
    const int rank = (int)cluster_ctarank(), n_cta = (int)cluster_nctarank();
    const int row = blockIdx.x / n_cta, b = row / p.c.heads, h = row - b * p.c.heads, ps = p.c.page_size;
    const int len = cache_len(p.c, b, KID_EVICT);

    const int chunk = (len + n_cta - 1) / n_cta;
    const int lo = min(len, rank * chunk), n = min(len, lo + chunk) - lo;
    const int stripes = (n + THREADS - 1) / THREADS;
    const int keep_from = *(p.keep_from + b);

    // page ids of this CTA's slots
    int32_t *pages = reinterpret_cast<int32_t *>(keys + p.chunk_cap);
    const int col0 = p.page_div.of(lo), cols = n > 0 ? p.page_div.of(lo + n - 1) - col0 + 1 : 0;
    for (int i = tid; i < min(cols, p.cols_cap); i += THREADS) pages[i] = cache_page(p.c, b, col0 + i, KID_EVICT);
    __syncthreads();
    // entry index of slot lo + i in the bookkeeping, or -1
    auto entry = [&](int i) -> int64_t {
        const int slot = lo + i, col = p.page_div.of(slot);
        const int pg = col - col0 < p.cols_cap ? pages[col - col0] : cache_page(p.c, b, col, KID_EVICT);
        return pg < 0 ? -1 : ((int64_t)pg * p.c.heads + h) * ps + (slot - col * ps);
    };
    const int edge = p.budget - lo;                        // slots i < edge lie below the budget
    const bool whole = len <= p.budget;                    // nothing to evict
    // Keys; and the bookkeeping of the slots below the budget as if they all
    // stayed: a moved entry overwrites it later.
    for (int i0 = tid; i0 < n; i0 += THREADS * BATCH) {
        float w[BATCH];
        int32_t x[BATCH];
        uint32_t there = 0;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k * THREADS;
            const int64_t e = i < n ? entry(i) : -1;
            if (e >= 0) {
                w[k] = *(p.c.weight + e);
                x[k] = *(p.c.pos + e);
                there |= 1u << k;
            }
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k * THREADS;
            if (i >= n) continue;
            uint32_t key = 0;
            if (there >> k & 1) {
                const uint32_t u = __float_as_uint(w[k] + 0.f);                     // -0 becomes 0
                key = x[k] >= keep_from ? 0xffffffffu : u ^ (u & 0x80000000u ? 0xffffffffu : 0x80000000u);
                if (whole || i < edge) {
                    const int64_t e = entry(i);
                    p.weight_out[e] = w[k];
                    p.pos_out[e] = x[k];
                }
            }
            if (!whole) keys[i] = key;
        }
    }
    if (whole) return;                                     // the whole cluster leaves

    // ---- the budget-th largest key, from its highest bits down
    uint32_t prefix = 0, mask = 0;
    int want = p.budget;                                   // of the keys that match the prefix
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        uint32_t *hs = hist[pass & 1];
        for (int i = tid; i < BINS; i += THREADS) hs[i] = 0;
        __syncthreads();
#pragma unroll 8
        for (int i = tid; i < n; i += THREADS) {
            const uint32_t k = keys[i];
            if ((k & mask) == prefix) atomicAdd(&hs[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
        // four bins per thread, from the highest down; a cluster's are added 16 bytes at a time
        constexpr int PER = 4;
        static_assert(BINS == PER * THREADS, "");
        const int top = BINS - PER - PER * tid;
        uint32_t c[PER];
        if (n_cta == 1) {
            __syncthreads();
            *reinterpret_cast<uint4 *>(c) = *reinterpret_cast<const uint4 *>(hs + top);
        } else {
            cluster_sync_all();
#pragma unroll
            for (int k = 0; k < PER; ++k) c[k] = 0;
            const uint32_t a = smem_u32(hs + top);
#pragma unroll 4
            for (int r = 0; r < n_cta; ++r) {
                const uint4 v = cluster_ld4(cluster_map(a, r));
                c[0] += v.x, c[1] += v.y, c[2] += v.z, c[3] += v.w;
            }
        }
        int total, mine = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) mine += (int)c[k];
        int before = block_prefix(mine, s_scan, total);
        if (before < want && want <= before + mine) {
#pragma unroll
            for (int k = PER - 1; k >= 0; --k) {
                if (before < want && want <= before + (int)c[k]) {
                    s_digit = (uint32_t)(top + k);
                    s_above = (uint32_t)before;
                    s_match = c[k];
                }
                before += (int)c[k];
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        want -= (int)s_above;
    }
    // What each CTA puts into s_xchg[k], two 16-bit counts: sums over the CTAs before this one, and of the lower
    // one over all.
    auto exchange = [&](int k, uint32_t mine, int &before_lo, int &before_hi) {
        before_lo = before_hi = 0;
        if (n_cta == 1) return (int)(mine & 0xffffu);
        if (tid == 0) s_xchg[k] = mine;
        cluster_sync_all();
        int all = 0;
        for (int r = 0; r < n_cta; ++r) {
            const uint32_t x = cluster_ld(cluster_map(smem_u32(&s_xchg[k]), r));
            all += (int)(x & 0xffffu);
            if (r < rank) {
                before_lo += (int)(x & 0xffffu);
                before_hi += (int)(x >> 16);
            }
        }
        return all;
    };

    // ---- `want` of the s_match keys equal to `prefix` stay, those in the lowest slots: where that is not all of
    // them, they are counted in order
    const bool choose = (int)s_match > want;
    int ties_before = 0, unused;
    if (choose) {
#pragma unroll 4
        for (int s = 0; s < stripes; ++s) {
            const int i = s * THREADS + tid;
            const unsigned tie = __ballot_sync(0xffffffffu, i < n && keys[i] == prefix);
            if (lane == 0) s_cnt[0][s * WARPS + warp] = __popc(tie);
        }
        const int ties = stripe_prefix(s_cnt[0], stripes, s_scan);
        exchange(0, (uint32_t)ties, ties_before, unused);
    }
    // holes (given up below the budget) and moves (kept past it), 16 bits each: at most 32768 per CTA
#pragma unroll 4
    for (int s = 0; s < stripes; ++s) {
        const int i = s * THREADS + tid;
        const uint32_t k = i < n ? keys[i] : 0u;
        bool keep = i < n && k >= prefix;
        if (choose) {
            const bool tie = i < n && k == prefix;
            const unsigned m = __ballot_sync(0xffffffffu, tie);
            if (tie) keep = ties_before + s_cnt[0][s * WARPS + warp] + __popc(m & below) < want;
        }
        const unsigned out = __ballot_sync(0xffffffffu, i < n && i < edge && !keep);
        const unsigned in = __ballot_sync(0xffffffffu, i >= edge && keep);
        if (i < n) keys[i] = keep;
        if (lane == 0) s_cnt[1][s * WARPS + warp] = __popc(out) | __popc(in) << 16;
    }
    const uint32_t both = (uint32_t)stripe_prefix(s_cnt[1], stripes, s_scan);
    int hole_at, move_at;
    const int holes = exchange(1, both, hole_at, move_at);
    int32_t *src = p.src + (int64_t)row * p.most, *dst = p.dst + (int64_t)row * p.most;
#pragma unroll 4
    for (int s = 0; s < stripes; ++s) {
        const int i = s * THREADS + tid;
        const bool keep = i < n && keys[i] != 0;
        const unsigned out = __ballot_sync(0xffffffffu, i < n && i < edge && !keep);
        const unsigned in = __ballot_sync(0xffffffffu, i >= edge && keep);
        const uint32_t at = (uint32_t)s_cnt[1][s * WARPS + warp];
        if (out >> lane & 1) dst[hole_at + (int)(at & 0xffffu) + __popc(out & below)] = lo + i;
        if (in >> lane & 1) src[move_at + (int)(at >> 16) + __popc(in & below)] = lo + i;
    }
    // ---- the moves, dealt to the cluster's warps evenly, at most 32 at a time (the lists are in global memory: L2)
    __syncthreads();
    if (n_cta > 1) {
        __threadfence();
        cluster_sync_all();                                // also: no CTA leaves while another may read its shared memory
    }
    const int cpr = p.c.dim / 8;                           // 16-byte pieces of a row
    const int share = min(32, (holes + WARPS * n_cta - 1) / (WARPS * n_cta));
    for (int m0 = share * (warp * n_cta + rank); m0 < holes; m0 += share * WARPS * n_cta) {
        // this lane's move: page and offset of where it comes from and goes to
        int sp = -1, so = 0, dp = -1, dof = 0;
        const int here = min(share, holes - m0);
        if (lane < here) {
            const int s = __ldcg(src + m0 + lane), d = __ldcg(dst + m0 + lane);
            const int sc = p.page_div.of(s), dc = p.page_div.of(d);
            so = s - sc * ps;
            dof = d - dc * ps;
            sp = cache_page(p.c, b, sc, KID_EVICT);
            dp = cache_page(p.c, b, dc, KID_EVICT);
            if (sp < 0 || dp < 0) {
                sp = -1;
            } else {
                const int64_t e0 = ((int64_t)sp * p.c.heads + h) * ps + so, e1 = ((int64_t)dp * p.c.heads + h) * ps + dof;
                p.weight_out[e1] = *(p.c.weight + e0);
                p.pos_out[e1] = *(p.c.pos + e0);
            }
        }
        for (int pc = lane; pc - lane < 2 * cpr; pc += 32) { // pieces of k, then of v (one round up to dim 128)
            const bool is_v = pc >= cpr, mine = pc < 2 * cpr;
            uint8_t *base = static_cast<uint8_t *>(is_v ? p.c.v : p.c.k) +
                            2 * ((int64_t)h * (is_v ? p.c.v_head : p.c.k_head) + (is_v ? pc - cpr : pc) * 8);
            const int64_t P = 2 * (is_v ? p.c.v_page : p.c.k_page), S = 2 * (is_v ? p.c.v_slot : p.c.k_slot);
            for (int i0 = 0; i0 < here; i0 += MOVE_BATCH) {
                uint4 w[MOVE_BATCH];
#pragma unroll
                for (int k = 0; k < MOVE_BATCH; ++k) {
                    const int64_t pg = __shfl_sync(0xffffffffu, sp, (i0 + k) & 31), of = __shfl_sync(0xffffffffu, so, (i0 + k) & 31);
                    if (mine && i0 + k < here && pg >= 0) w[k] = *reinterpret_cast<const uint4 *>(base + pg * P + of * S);
                }
#pragma unroll
                for (int k = 0; k < MOVE_BATCH; ++k) {
                    const int ok = __shfl_sync(0xffffffffu, sp, (i0 + k) & 31);
                    const int64_t pg = __shfl_sync(0xffffffffu, dp, (i0 + k) & 31), of = __shfl_sync(0xffffffffu, dof, (i0 + k) & 31);
                    if (mine && i0 + k < here && ok >= 0) *reinterpret_cast<uint4 *>(base + pg * P + of * S) = w[k];
                }
            }
        }
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

inline int launch_evict(const EvictParams &p, int64_t rows, int cl, cudaStream_t s)
{
    static bool attr_done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return MMQ_ERR_ARCH;
    }
    if (!attr_done[dev]) {
        if (cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (evict::MAX_CHUNK + evict::MAX_COLS) * 4) != cudaSuccess)
            return launch_status();
        attr_done[dev] = true;
    }
    return launch_pdl(evict_kernel, dim3((unsigned)(rows * cl)), evict::THREADS, (size_t)(p.chunk_cap + p.cols_cap) * 4, s, cl, p);
}

}  // namespace
}  // namespace mmq

extern "C" int mmq_evict_sizes(const mmq_kv_cache *cache, int budget, int64_t *work_ints)
{
    const int rc = mmq::evict_check(cache, budget);
    if (rc != MMQ_OK) return rc;
    if (!work_ints) return MMQ_ERR_NULL;
    *work_ints = (int64_t)cache->seqs * cache->heads * 2 * (int64_t)mmq::evict_most(*cache, budget);
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
    p.src = work;
    p.dst = p.src + rows * p.most;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    p.page_div = FastDiv(cache->page_size);

    const int cap = cache->cols * cache->page_size;
    // CTAs per row: as many as the keys need (32768 each), and more while all
    // are resident and each still has 2048 keys
    int cl = (cap + evict::MAX_CHUNK - 1) / evict::MAX_CHUNK;
    while (cl < evict::MAX_CLUSTER && rows * (cl + 1) <= evict::PER_SM * sm_count() && cap > 2048 * cl) ++cl;
    p.chunk_cap = (cap + cl - 1) / cl;
    p.cols_cap = cache->cols < evict::MAX_COLS ? cache->cols : evict::MAX_COLS;
    return launch_evict(p, rows, cl, s);
}
