// mmq_keep.cuh -- the accepted path of a tree of drafts moves to the front of
// the tree's entries (mmq_kv_keep).
//
// Of a sequence's last n entries (nodes), node keep[i] goes to node i's place,
// for keep ascending.  A source keep[i] >= i is never the destination of an
// earlier i, so one thread can move its 16 bytes of every entry in order, a
// batch of loads before the batch's stores.
//
// Bound by latency: a few entries per sequence.  A block takes one sequence and
// some of its heads' 16-byte pieces, so that even one sequence's moves are a
// single round of loads spread over the device.  Measured: eight entries of 32
// heads of 128, one sequence, 5.5 us; 64 sequences of 8 heads 6.5 us.
#pragma once

namespace mmq {
namespace {

constexpr int KEEP_THREADS = 128, KEEP_MAX = 64, KEEP_BATCH = 8;

struct KeepParams {
    mmq_kv_cache c;
    const int32_t *keep, *count, *new_len;
    int width, nodes;
    FastDiv page_div;
};

__global__ void __launch_bounds__(KEEP_THREADS) keep_kernel(const KeepParams p)
{
    __shared__ int2 s_from[KEEP_MAX], s_to[KEEP_MAX];          // page (negative: stays), offset
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x;
    const int len = cache_len(p.c, b, KID_KEEP), n = new_count(p.new_len, b, p.nodes, KID_KEEP);
    const int kept = new_count(p.count, b, p.width, KID_KEEP);
    const int start = len - n;
    if (start < 0) {
        if (threadIdx.x == 0) record_error(MMQ_ERR_INDEX, KID_KEEP, SITE_LEN);
        return;
    }
    for (int i = threadIdx.x; i < kept; i += KEEP_THREADS) {
        const int32_t *at = p.keep + (int64_t)b * p.width + i;
        const int from = *at, before = i > 0 ? *(at - 1) : -1;
        int2 src = make_int2(-1, 0), dst = make_int2(-1, 0);
        if (from <= before || from >= n || from < i) record_error(MMQ_ERR_INDEX, KID_KEEP, SITE_NODE);
        else if (from != i) {
            int col = p.page_div.of(start + from);
            src = make_int2(cache_page(p.c, b, col, KID_KEEP), start + from - col * p.c.page_size);
            col = p.page_div.of(start + i);
            dst = make_int2(cache_page(p.c, b, col, KID_KEEP), start + i - col * p.c.page_size);
            if (dst.x < 0) src.x = -1;
        }
        s_from[i] = src;
        s_to[i] = dst;
    }
    __syncthreads();
    const int pieces = p.c.dim / 8;                            // of a head; then one for weight and pos
    const int per_head = 2 * pieces + 1, unit = blockIdx.y * KEEP_THREADS + threadIdx.x;
    const int h = unit / per_head, piece = unit - h * per_head;
    if (h >= p.c.heads) return;
    if (piece == 2 * pieces) {
        if (!p.c.weight && !p.c.pos) return;
        for (int i = 0; i < kept; ++i) {
            if (s_from[i].x < 0) continue;
            const int64_t s = ((int64_t)s_from[i].x * p.c.heads + h) * p.c.page_size + s_from[i].y;
            const int64_t d = ((int64_t)s_to[i].x * p.c.heads + h) * p.c.page_size + s_to[i].y;
            if (p.c.weight) p.c.weight[d] = p.c.weight[s];
            if (p.c.pos) p.c.pos[d] = p.c.pos[s];
        }
        return;
    }
    const bool is_v = piece >= pieces;
    uint16_t *pool = static_cast<uint16_t *>(is_v ? p.c.v : p.c.k) + (is_v ? piece - pieces : piece) * 8;
    const int64_t page = is_v ? p.c.v_page : p.c.k_page, slot = is_v ? p.c.v_slot : p.c.k_slot;
    pool += h * (is_v ? p.c.v_head : p.c.k_head);
    for (int i0 = 0; i0 < kept; i0 += KEEP_BATCH) {
        uint4 x[KEEP_BATCH];
#pragma unroll
        for (int i = 0; i < KEEP_BATCH; ++i)
            if (i0 + i < kept && s_from[i0 + i].x >= 0)
                x[i] = *reinterpret_cast<const uint4 *>(pool + s_from[i0 + i].x * page + s_from[i0 + i].y * slot);
#pragma unroll
        for (int i = 0; i < KEEP_BATCH; ++i)
            if (i0 + i < kept && s_from[i0 + i].x >= 0)
                *reinterpret_cast<uint4 *>(pool + s_to[i0 + i].x * page + s_to[i0 + i].y * slot) = x[i];
    }
}

}  // namespace
}  // namespace mmq

extern "C" int mmq_kv_keep(const mmq_kv_cache *cache, const int32_t *keep, const int32_t *count, const int32_t *new_len, int width,
                           int nodes, mmq_stream_t stream)
{
    using namespace mmq;
    int rc = check_cache(cache);
    if (rc != MMQ_OK) return rc;
    if (nodes < 0 || nodes > KEEP_MAX || width < 0 || width > nodes) return MMQ_ERR_SHAPE;
    if (cache->seqs == 0 || width == 0) return MMQ_OK;
    if (!keep) return MMQ_ERR_NULL;
    const int64_t units = (int64_t)cache->heads * (2 * (cache->dim / 8) + 1), blocks = (units + KEEP_THREADS - 1) / KEEP_THREADS;
    if (blocks > 65535) return MMQ_ERR_SHAPE;
    if ((rc = check_arch()) != MMQ_OK) return rc;
    const KeepParams p = {*cache, keep, count, new_len, width, nodes, FastDiv(cache->page_size)};
    return launch_pdl(keep_kernel, dim3((unsigned)cache->seqs, (unsigned)blocks), KEEP_THREADS, 0,
                      reinterpret_cast<cudaStream_t>(stream), 0, p);
}
