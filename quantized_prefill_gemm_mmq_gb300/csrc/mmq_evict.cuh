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
// largest by up to three passes of a radix search (11, 11 and 10 bits), counts
// ties in slot order, lists the moves, and makes them.  The CTAs of a cluster
// read of each other's histograms, through distributed shared memory, the sums
// of 32 bins each and then the 32 bins they need (all 2048 bins of eight CTAs
// took 2 us a pass: 30 rows of 43382 entries 37 us, now 17).  Slots are dealt
// to threads in stripes, so that every pass reads memory side by side, four
// slots at a time where the pages allow; what happens to the 32 slots of a
// warp is a word of bits, and one scan over the words' counts keeps the order
// of slots.  For the moves a warp looks up 32 at once, one per lane, then
// copies them one after the other, a 16-byte piece of K or V per lane.
// Bound by memory: 8 B per entry and head for weight and position, 8 B for
// each that stays, 8 dim B per move; with few moves by the latency of the
// selection's passes.
// Measured: 16 sequences up to 32768 entries of 8 heads of 128 down to 4096,
// 98 us, of which 72 us move 485 MB (6.7 TB/s); 1100 entries of 32 heads down
// to 1024, 7.4 us.  Planned by what the table has room for, since lengths are on
// the device: shared memory and the cluster follow cols*page_size.
#pragma once

namespace mmq {
namespace {

namespace evict {
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int PER_SM = 2;
constexpr int BINS = 2048;
constexpr int GROUPS = BINS / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_CHUNK = 32768;               // keys per CTA: 128 KB
constexpr int STRIPES = MAX_CHUNK / THREADS;   // at most
constexpr int MAX_COLS = 4096;                 // page ids kept in shared memory
constexpr int BATCH = 8;                       // slots whose loads a thread has in flight,
constexpr int BATCH4 = 3;                      // and groups of four
constexpr int MOVE_BATCH = 3;                  // moves a warp has in flight
}  // namespace evict

struct EvictParams {
    mmq_kv_cache c;
    const int32_t *keep_from;
    float *weight_out;
    int32_t *pos_out;
    int32_t *src, *dst;     // [seqs*heads][most] slots
    int budget, most, chunk_cap, cols_cap;
    int wide;               // four slots at a time: pages of a multiple of four, bookkeeping on 16 bytes
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

__device__ __forceinline__ unsigned long long cluster_ld64(uint32_t a)
{
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
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

// Exclusive prefixes of count(w) over the words w = stripe*WARPS + warp, the
// order of slots, into cnt; returns the sum.
template <typename F>
__device__ __forceinline__ int stripe_prefix(int *cnt, int stripes, int *s, F count)
{
    constexpr int PER = evict::STRIPES * evict::WARPS / evict::THREADS;
    __syncthreads();
    const int n = stripes * evict::WARPS, i = threadIdx.x * PER;
    int v[PER], mine = 0, total;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        v[k] = i + k < n ? count(i + k) : 0;
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
    __shared__ __align__(8) uint32_t s_group[2][GROUPS];
    __shared__ uint32_t s_bits[STRIPES * WARPS];
    __shared__ int s_cnt[STRIPES * WARPS];
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

    const int chunk = ((len + n_cta - 1) / n_cta + 3) & ~3;
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
    // stayed: a moved entry overwrites it later.  Where four slots lie side by
    // side (`wide`) a thread takes them at once.  Keys past n are 0, the last in order.
    auto key_of = [&](float w, int32_t x) {
        const uint32_t u = __float_as_uint(w + 0.f);       // -0 becomes 0
        return x >= keep_from ? 0xffffffffu : u ^ (u & 0x80000000u ? 0xffffffffu : 0x80000000u);
    };
    if (p.wide) {
        for (int i0 = 4 * tid; i0 < n; i0 += 4 * THREADS * BATCH4) {
            float4 w[BATCH4];
            int4 x[BATCH4];
            int64_t e[BATCH4];
#pragma unroll
            for (int k = 0; k < BATCH4; ++k) {
                const int i = i0 + k * 4 * THREADS;
                e[k] = i < n ? entry(i) : -1;
                if (e[k] >= 0) {
                    w[k] = *reinterpret_cast<const float4 *>(p.c.weight + e[k]);
                    x[k] = *reinterpret_cast<const int4 *>(p.c.pos + e[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < BATCH4; ++k) {
                const int i = i0 + k * 4 * THREADS;
                if (i >= n) continue;
                const bool there = e[k] >= 0;
                const int stay = there ? min(n, edge) - i : 0;        // entries to write, of four
                if (stay >= 4) {
                    *reinterpret_cast<float4 *>(p.weight_out + e[k]) = w[k];
                    *reinterpret_cast<int4 *>(p.pos_out + e[k]) = x[k];
                } else if (stay > 0) {
                    const float ws[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                    const int xs[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (j < stay) {
                            p.weight_out[e[k] + j] = ws[j];
                            p.pos_out[e[k] + j] = xs[j];
                        }
                }
                if (whole) continue;
                uint4 key = make_uint4(0u, 0u, 0u, 0u);
                if (there) {
                    key.x = key_of(w[k].x, x[k].x);
                    if (i + 1 < n) key.y = key_of(w[k].y, x[k].y);
                    if (i + 2 < n) key.z = key_of(w[k].z, x[k].z);
                    if (i + 3 < n) key.w = key_of(w[k].w, x[k].w);
                }
                *reinterpret_cast<uint4 *>(keys + i) = key;
            }
        }
    } else {
        for (int i0 = tid; i0 < ((n + 3) & ~3); i0 += THREADS * BATCH) {
            float w[BATCH];
            int32_t x[BATCH];
            int64_t e[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int i = i0 + k * THREADS;
                e[k] = i < n ? entry(i) : -1;
                if (e[k] >= 0) {
                    w[k] = *(p.c.weight + e[k]);
                    x[k] = *(p.c.pos + e[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int i = i0 + k * THREADS;
                if (e[k] >= 0 && (whole || i < edge)) {
                    p.weight_out[e[k]] = w[k];
                    p.pos_out[e[k]] = x[k];
                }
                if (!whole && i < ((n + 3) & ~3)) keys[i] = e[k] >= 0 ? key_of(w[k], x[k]) : 0u;
            }
        }
    }
    if (whole) return;                                     // the whole cluster leaves

    // ---- the budget-th largest key, from its highest bits down
    uint32_t prefix = 0, mask = 0;
    int want = p.budget;                                   // of the keys that match the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        uint32_t *hs = hist[pass & 1];
        for (int i = tid; i < BINS; i += THREADS) hs[i] = 0;
        __syncthreads();
#pragma unroll 2
        for (int i = 4 * tid; i < n; i += 4 * THREADS) {
            const uint4 k = *reinterpret_cast<const uint4 *>(keys + i);
            auto add = [&](uint32_t x) {
                if ((x & mask) == prefix) atomicAdd(&hs[(x >> shift) & ((1u << bits) - 1)], 1u);
            };
            add(k.x);
            add(k.y);
            add(k.z);
            add(k.w);
        }
        // sums of 32 bins each: eight threads of four
        static_assert(BINS == 4 * THREADS && GROUPS * 32 == BINS && GROUPS == 64, "");
        __syncthreads();
        {
            const uint4 v = *reinterpret_cast<const uint4 *>(hs + 4 * tid);
            uint32_t x = (v.x + v.y) + (v.z + v.w);
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            if ((tid & 7) == 0) s_group[pass & 1][tid / 8] = x;
        }
        if (n_cta == 1) __syncthreads();
        else cluster_sync_all();
        // One warp finds the group of bins, two per lane from the highest down, then the bin, one per lane: of the
        // other CTAs' histograms it reads 64 sums and 32 bins, all CTAs' at once (past the last: that one's again).
        if (warp == 0) {
            const uint32_t *pair = &s_group[pass & 1][GROUPS - 2 - 2 * lane];
            uint32_t first = 0, second = 0;                // the higher group's and the lower one's
            if (n_cta == 1) {
                first = pair[1];
                second = pair[0];
            } else {
                unsigned long long v[MAX_CLUSTER];
#pragma unroll
                for (int r = 0; r < MAX_CLUSTER; ++r) v[r] = cluster_ld64(cluster_map(smem_u32(pair), min(r, n_cta - 1)));
#pragma unroll
                for (int r = 0; r < MAX_CLUSTER; ++r) {
                    first += r < n_cta ? (uint32_t)(v[r] >> 32) : 0u;
                    second += r < n_cta ? (uint32_t)v[r] : 0u;
                }
            }
            auto before = [&](int x) {                     // exclusive prefix over the lanes
                int y = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int z = __shfl_up_sync(0xffffffffu, y, o);
                    if (lane >= o) y += z;
                }
                return y - x;
            };
            int above = before((int)(first + second));
            const unsigned m = __ballot_sync(0xffffffffu, above < want && want <= above + (int)(first + second));
            const bool lower = want > above + (int)first;
            if (lower) above += (int)first;
            const int f = __ffs(m) - 1, group = __shfl_sync(0xffffffffu, GROUPS - 1 - 2 * lane - (lower ? 1 : 0), f);
            above = __shfl_sync(0xffffffffu, above, f);
            const int bin = group * 32 + 31 - lane;
            int c = 0;
            if (n_cta == 1) {
                c = (int)hs[bin];
            } else {
                uint32_t v[MAX_CLUSTER];
#pragma unroll
                for (int r = 0; r < MAX_CLUSTER; ++r) v[r] = cluster_ld(cluster_map(smem_u32(hs + bin), min(r, n_cta - 1)));
#pragma unroll
                for (int r = 0; r < MAX_CLUSTER; ++r) c += r < n_cta ? (int)v[r] : 0;
            }
            above += before(c);
            if (above < want && want <= above + c) {
                s_digit = (uint32_t)bin;
                s_above = (uint32_t)above;
                s_match = (uint32_t)c;
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        want -= (int)s_above;
        if (want == (int)s_match) break;                   // all that match stay: lower bits do not matter
    }
    // What each CTA puts into s_xchg[k], two 16-bit counts: sums over the CTAs before this one, and of the lower
    // one over all.
    auto exchange = [&](int k, uint32_t mine, int &before_lo, int &before_hi) {
        before_lo = before_hi = 0;
        if (n_cta == 1) return (int)(mine & 0xffffu);
        if (tid == 0) s_xchg[k] = mine;
        cluster_sync_all();
        const uint32_t x = lane < n_cta ? cluster_ld(cluster_map(smem_u32(&s_xchg[k]), lane)) : 0u;
        before_lo = (int)__reduce_add_sync(0xffffffffu, lane < rank ? x & 0xffffu : 0u);
        before_hi = (int)__reduce_add_sync(0xffffffffu, lane < rank ? x >> 16 : 0u);
        return (int)__reduce_add_sync(0xffffffffu, x & 0xffffu);
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
            if (lane == 0) s_bits[s * WARPS + warp] = tie;
        }
        const int ties = stripe_prefix(s_cnt, stripes, s_scan, [&](int w) { return __popc(s_bits[w]); });
        exchange(0, (uint32_t)ties, ties_before, unused);
    }
    // holes (given up below the budget) and moves (kept past it): a bit each for the 32 slots of a (stripe, warp), and
    // their counts, 16 bits each: at most 32768 per CTA
    auto under = [&](int w) {                              // the bits of slots below the budget
        const int k = edge - w * 32;
        return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1;
    };
#pragma unroll 4
    for (int s = 0; s < stripes; ++s) {
        const int i = s * THREADS + tid;
        const uint32_t k = i < n ? keys[i] : 0u;
        bool keep = k >= prefix;
        if (choose) {
            const bool tie = i < n && k == prefix;
            const unsigned m = __ballot_sync(0xffffffffu, tie);
            if (tie) keep = ties_before + s_cnt[s * WARPS + warp] + __popc(m & below) < want;
        }
        const unsigned m = __ballot_sync(0xffffffffu, i < n && keep != (i < edge));
        if (lane == 0) s_bits[s * WARPS + warp] = m;
    }
    const uint32_t both = (uint32_t)stripe_prefix(s_cnt, stripes, s_scan, [&](int w) {
        const uint32_t m = s_bits[w], u = under(w);
        return __popc(m & u) | __popc(m & ~u) << 16;
    });
    int hole_at, move_at;
    const int holes = exchange(1, both, hole_at, move_at);
    int32_t *src = p.src + (int64_t)row * p.most, *dst = p.dst + (int64_t)row * p.most;
#pragma unroll 4
    for (int s = 0; s < stripes; ++s) {
        const int w = s * WARPS + warp;
        const uint32_t m = s_bits[w];
        if ((m >> lane & 1) == 0) continue;
        const uint32_t u = under(w), at = (uint32_t)s_cnt[w];
        const int i = s * THREADS + tid;
        if (u >> lane & 1) dst[hole_at + (int)(at & 0xffffu) + __popc(m & u & below)] = lo + i;
        else src[move_at + (int)(at >> 16) + __popc(m & ~u & below)] = lo + i;
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
    if (budget < 1 || (int64_t)c->cols * c->page_size > evict::MAX_CLUSTER * evict::MAX_CHUNK ||
        (int64_t)c->seqs * c->heads > 0x7fffffff / evict::MAX_CLUSTER)        // a cluster per row in the grid's x
        return MMQ_ERR_SHAPE;
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
    p.chunk_cap = ((cap + cl - 1) / cl + 3) & ~3;
    p.wide = cache->page_size % 4 == 0 && aligned16(cache->weight) && aligned16(cache->pos) && aligned16(weight_out) && aligned16(pos_out);
    p.cols_cap = cache->cols < evict::MAX_COLS ? cache->cols : evict::MAX_COLS;
    return launch_evict(p, rows, cl, s);
}
