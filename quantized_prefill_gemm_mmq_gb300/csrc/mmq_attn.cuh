// mmq_attn.cuh -- attention of the newest tokens over the paged cache
// (mmq_attn_decode).
//
// Per query row r (a token t and a query head of the key-value head's group):
//     s = scale q.k,  p = exp(s - m),  out = sum p v / sum p
// in one pass over the cache with a running maximum m: when a tile raises m,
// what was summed so far is multiplied by exp(m_old - m_new).  m is taken off
// before the multiplication by scale, so that scores may be of any size.
//
// Work.  The cache is read once; everything else is small, so the kernel is
// bound by memory (4 dim bytes per entry and head) as long as the rows that
// share a key-value head are few.  All tiles of TILE entries of all sequences
// and heads are numbered in a row, and the persistent grid's CTA c takes tiles
// [c W/G, (c+1) W/G): every CTA reads the same amount whatever the lengths.
// A run of tiles that belongs to one (sequence, head) is a segment; a CTA that
// has all of a segment writes its output, the others leave their part (max,
// sum, sum p v) in the workspace, and a second launch joins the parts in CTA
// order.  No result depends on timing.  (Joining by the last CTA to arrive,
// with a counter per segment, took 7 to 14 us at the end of a launch with 33
// parts of 20 rows: one CTA reads all parts of its segment.)
//
// Tiles.  K and V rows are gathered through the page table with 16-byte
// cp.async into a ring of stages (any page size and stride; entries past
// the length arrive as zeros), chunk-XOR swizzled so that ldmatrix reads
// without bank conflicts.  The addresses of a tile's rows are computed once,
// an iteration before its copies are issued (per copy they were more than half
// of all instructions: 131071 entries took 120 us).
//
// Products run on the warp-level tensor core (16-row operand), with q and p
// split into parts of the cache's type that add up to 22 bits (f16, two parts)
// or 24 (bf16, three); K and V are used as they are.  The parts of few rows
// share one operand, and the result's parts are added: up to four rows of bf16
// (MODE 0), rows 0-3 hold the first parts, 4-7 the second, 8-11 the third; up
// to eight rows (MODE 1), the upper eight hold the first part, the lower eight
// the second, and bf16's third takes a second product into the lower ones (the
// tensor core cuts its sums off, so the large part's takes as few as it can).
// More rows (MODE 2): sixteen rows per operand, one product per part.  q is
// scaled by a power of two per row to lie below 4, and for f16 p carries 2^15,
// so that f16's range does not clip either.  The sums over a tile's entries stay in f32 and are
// added to the running sums with f32 FMAs.
//
// UG warps of the four take these rows each over the same entries and 4/UG
// warps split a tile's entries (with their own running maximum, joined at the
// segment's end), so that up to 64 rows share one read of the cache.
//
// Measured (device time, both launches): one token over 131071 entries of 8
// heads of 128, f16, 85 us = 6.3 TB/s; a ragged batch of 16 up to 32768, bf16,
// 186 us = 6.8 TB/s (the copy rate is 6.8); over 513 entries of 32 heads 7.4 us;
// five tokens of 8 sequences up to 4099, heads of 64 (20 rows), 27 us, where the
// tensor pipe is 27 % active and two warps per scheduler set the pace.  More
// rows cost more: 8 sequences of 4096 entries of 8 heads of 128 in bf16 take 34
// us with 8 rows, 50 with 16, 62 with 32 and 106 with 64.  Some kernels of many
// rows spill: <256, bf16, 1, 4> 504 bytes, <128, bf16, 2, 4> 360,
// <64, bf16, 2, 4> 332, <80, bf16, 2, 4> 244, <128, bf16, 2, 1> 184,
// <128, half, 2, 4> 136, the others at most 52.
#pragma once

#include <type_traits>

namespace mmq {
namespace {

namespace attn {
constexpr int THREADS = 128;

template <typename T>
constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
template <typename T>
constexpr float kExp = kBf16<T> ? 0.f : 15.f;      // p carries 2^kExp

// DP: dim padded to 64, 80 (as 96 it took 5 to 14 % longer), 96, 128, 192 or 256; MODE, UG: see above
template <int DP, int MODE, int UG>
struct Shape {
    static constexpr int kPerWarp = MODE == 0 ? 4 : MODE == 1 ? 8 : 16;   // rows
    static constexpr int kTile = DP == 64 ? 128 : DP > 128 && UG > 1 ? 32 : 64;       // entries per tile
    static constexpr int kStages = DP == 192 && UG == 1 ? 2 : 3;      // tiles in the ring
    static constexpr int kPerSm = 2;                                  // CTAs resident per SM
    static constexpr int kStride = DP == 80 || DP == 96 ? 256 : DP * 2;           // bytes from row to row: the swizzle takes eight pieces
    static constexpr int kHalf = kTile * kStride;                     // bytes of K (or V) per stage
    static constexpr int kSmem = kStages * 2 * kHalf;
    static constexpr bool kFull = DP == 128 && MODE == 2;             // registers are
    static constexpr int kNg = kFull ? 1 : UG == 1 ? 2 : 8;           // eight-entry groups of scores at a time
    static constexpr int kDg = kFull ? 2 : DP == 80 ? 10 : 4;                         // eight-value groups of sums at a time
    static constexpr int kRows = kPerWarp * UG;                       // rows per CTA
    // the four warps' sums are joined in one stage's memory, in as many rounds of columns as fit
    static constexpr int fit(int rounds) { return 4 * kPerWarp * (DP / rounds + 8) * 4 <= 2 * kHalf ? rounds : fit(rounds * 2); }
    static constexpr int kRounds = fit(1);
    static constexpr int kCols = DP / kRounds;
    static constexpr int kPad = kCols + 8;                            // floats per row there: no bank conflicts
};

// 16 bytes to shared memory: `size` (16 or 0) of them from src, zeros after
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t size)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (x, y) split into parts of the cache's type: hi + mid (+ lo) = (x, y) to 22
// (f16) or 24 (bf16) bits
template <typename T>
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    hi = pack2<T>(x, y);
    const float2 h = unpack2<T>(hi);
    x -= h.x;
    y -= h.y;
    mid = pack2<T>(x, y);
    if constexpr (kBf16<T>) {
        const float2 m = unpack2<T>(mid);
        lo = pack2<T>(x - m.x, y - m.y);
    } else {
        lo = 0;
    }
}

// 2^x to two ulp; 0 for -inf and where the result is below the normal range
__device__ __forceinline__ float pow2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// quad = the four lanes that hold one row
__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// 1 / sum, 0 for a row that saw nothing; a NaN stays one
__device__ __forceinline__ float inverse(float sum) { return sum > 0.f ? 1.f / sum : sum; }
// A row's maximum and a factor: pow2(score - x) * y is an entry's weight, at most 1 however large the scores.  (Their
// log-sum in one number is off by whole powers of two where m is past 2^24.)  A row that saw nothing adds nothing.
template <typename T>
__device__ __forceinline__ float2 row_norm(float m, float sum)
{
    return sum > 0.f ? make_float2(m, (kBf16<T> ? 1.f : 32768.f) / sum) : make_float2(INFINITY, 0.f);
}

// whether one of two values has all exponent bits set
template <typename T>
__device__ __forceinline__ bool not_finite2(uint32_t u)
{
    constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    return (u & e) == e || (u & (e << 16)) == (e << 16);
}
}  // namespace attn

struct AttnParams {
    mmq_kv_cache c;
    const float *q;
    const int32_t *new_len;
    float *out;
    int64_t ldq;
    float scale_log2;        // scale * log2(e): exponentials are powers of two
    int new_tokens, group;   // rows per key-value head: r = t*group + g
    int rows, row_tiles;     // rows, and parts of kRows rows
    float *part;             // [2*grid][kRows][DP] sums, then [2*grid][kRows][2] (max, sum)
    int3 *parts;             // [seqs*heads][row_tiles]: first part, its CTA, last CTA (-1: output written)
    float *scores;           // [seqs*heads][rows][cap] in powers of two (weights only)
    float2 *norm;            // [seqs*heads][rows] of whole rows, see row_norm (weights only, else NULL)
    int64_t cap;
    FastDiv page_div, group_div;
};

// A place in the row of tiles: sequence, head, part of the rows, tile.
struct AttnCursor {
    int b, h, rt, tile, tiles, len;
};

template <int TILE>
__device__ __forceinline__ int attn_tiles(int len)
{
    return len > 0 ? (len + TILE - 1) / TILE : 1;     // an empty sequence still has outputs to write
}

template <int TILE>
__device__ __forceinline__ void attn_advance(const AttnParams &p, AttnCursor &u)
{
    if (++u.tile < u.tiles) return;
    u.tile = 0;
    if (++u.rt < p.row_tiles) return;
    u.rt = 0;
    if (++u.h < p.c.heads) return;
    u.h = 0;
    if (++u.b >= p.c.seqs) return;
    u.len = cache_len(p.c, u.b, KID_ATTN);
    u.tiles = attn_tiles<TILE>(u.len);
}

template <int DP, typename T, int MODE, int UG>
__global__ void __launch_bounds__(attn::THREADS, attn::Shape<DP, MODE, UG>::kPerSm) attn_kernel(const AttnParams p)
{
    using namespace attn;
    using S = Shape<DP, MODE, UG>;
    constexpr bool BF = kBf16<T>;
    constexpr int RP = MODE == 2 ? 2 : 1;                            // rows per quad of lanes
    constexpr int PARTS = MODE == 0 ? 1 : MODE == 1 ? (BF ? 2 : 1) : (BF ? 3 : 2);     // products per tensor-core step
    constexpr int TILE = S::kTile, STAGES = S::kStages, TG = 4 / UG, TW = TILE / TG;    // TW: entries per warp and tile
    constexpr int NT = TW / 8, KS = DP / 16, DT = DP / 8, ROWS = S::kRows;
    constexpr int CPR = DP / 8, PASSES = TILE * CPR / THREADS;              // 16-byte copies per row, and per thread and tile
    static_assert(TILE * CPR % THREADS == 0, "copies come out even");
    // A page id is loaded an iteration before the address it gives is computed: under load a miss in L1 takes longer
    // than a tile (11 sequences of 4637 in pages of 16, f16, heads of 64: 90 us and 75).  Not where the registers are
    // full, and the place that waits is spilled (bf16, 16 rows of 128: 51 us and 54; 60 rows of 64: 63 and 70).
    constexpr bool AHEAD = !(BF && (S::kFull || (DP == 64 && UG == 4)));

    pdl_wait();
    pdl_launch_dependents();       // the joining launch may start; what this one writes it reads after this one's end
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ ulonglong2 s_row[STAGES][TILE];
    __shared__ float2 s_ml[4][S::kPerWarp];         // (max, sum) of every warp's rows
    const uint32_t ring = smem_u32(smem);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // which rows and entries the warp takes: turned by two in every other CTA of an SM, so that warps without rows
    // (33 to 48 rows of 64) are not all on the same scheduler
    const int turned = UG == 4 && blockIdx.x >= gridDim.x / 2 ? (warp + 2) % 4 : warp;
    const int ug = turned % UG, tg = turned / UG;
    const int g = lane >> 2, j = lane & 3;
    const int gr = MODE == 0 ? g & 3 : g;                     // the quad's (first) row in the warp
    const bool holds = MODE != 0 || g < 4;                    // MODE 0: quads 4-7 compute the rows of 0-3 again
    const int hrs = p.c.heads * p.row_tiles;

    // ---- this CTA's tiles [u0, u1) of all W: every warp for itself, 32 sequences at a time
    int W = 0;
    for (int b = lane; b < p.c.seqs; b += 32) W += attn_tiles<TILE>(cache_len(p.c, b, KID_ATTN));
    W = __reduce_add_sync(0xffffffffu, W) * hrs;
    const int G = min(W, (int)gridDim.x);                     // CTAs with work: none between two of them is idle
    if ((int)blockIdx.x >= G) return;
    const int u0 = (int)((long long)W * blockIdx.x / G), n_units = (int)((long long)W * (blockIdx.x + 1) / G) - u0;
    AttnCursor cur;
    {
        int at = 0;                                           // first tile of sequence b
        for (int b0 = 0;; b0 += 32) {
            const int len = b0 + lane < p.c.seqs ? cache_len(p.c, b0 + lane, KID_ATTN) : 0;
            const int tiles = b0 + lane < p.c.seqs ? attn_tiles<TILE>(len) : 0;
            int upto = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, at + upto * hrs > u0);
            if (past) {
                const int f = __ffs(past) - 1;
                cur.b = b0 + f;
                cur.len = __shfl_sync(0xffffffffu, len, f);
                cur.tiles = __shfl_sync(0xffffffffu, tiles, f);
                at += (__shfl_sync(0xffffffffu, upto, f) - cur.tiles) * hrs;
                break;
            }
            at += __shfl_sync(0xffffffffu, upto, 31) * hrs;
        }
        const int rem = u0 - at, hr = rem / cur.tiles;
        cur.tile = rem - hr * cur.tiles;
        cur.h = hr / p.row_tiles;
        cur.rt = hr - cur.h * p.row_tiles;
    }
    int seg_base = u0 - cur.tile;                             // first tile of the segment at `cur`
    AttnCursor inf = cur;                                     // next tile to look up

    // Where entry `tid` of the tile at `inf` lies, and its row's addresses: 0 past the length; an entry with a bad page,
    // which is reported, gets the pool's first row.
    struct Place {
        int page, off, h;                                     // off: slot within the page, -1 for none
    };
    auto look_up = [&](bool there) {
        Place r = {0, -1, 0};
        if (there) {
            const int slot = inf.tile * TILE + tid;
            if (tid < TILE && slot < inf.len) {
                const int col = p.page_div.of(slot);
                r.off = slot - col * p.c.page_size;
                r.page = *(p.c.table + (int64_t)inf.b * p.c.cols + col);
                r.h = inf.h;
            }
            attn_advance<TILE>(p, inf);
        }
        return r;
    };
    auto addresses = [&](const Place &x) {
        ulonglong2 r = make_ulonglong2(0, 0);
        if (x.off >= 0) {
            int64_t pg = checked_page(p.c, x.page, KID_ATTN);
            int off = x.off;
            if (pg < 0) pg = off = 0;
            r = make_ulonglong2(
                (unsigned long long)(static_cast<const T *>(p.c.k) + pg * p.c.k_page + x.h * p.c.k_head + off * p.c.k_slot),
                (unsigned long long)(static_cast<const T *>(p.c.v) + pg * p.c.v_page + x.h * p.c.v_head + off * p.c.v_slot));
        }
        return r;
    };
    // This thread's 16-byte pieces of a tile: number tid + k*THREADS, row by row.  Past dim: zeros.
    constexpr bool EVEN = THREADS % CPR == 0;                 // the same piece of every (THREADS/CPR)th row
    auto copy = [&](int stage) {
        const uint32_t base = ring + stage * 2 * S::kHalf;
        const bool full = s_row[stage][TILE - 1].x != 0;      // a whole tile: its last entry is there
        auto place = [&](int k, int &row, int &cc, uint32_t &dst, uint32_t &piece) {
            row = EVEN ? tid / CPR + k * (THREADS / CPR) : (tid + k * THREADS) / CPR;
            cc = EVEN ? tid % CPR : (tid + k * THREADS) % CPR;
            dst = base + row * S::kStride + ((cc ^ (row & 7)) << 4);
            piece = cc * 8 < p.c.dim ? 16 : 0;
        };
        int row, cc;
        uint32_t dst, piece;
        if (full) {
#pragma unroll
            for (int k = 0; k < PASSES; ++k) {
                place(k, row, cc, dst, piece);
                const ulonglong2 w = s_row[stage][row];
                cp16(dst, reinterpret_cast<const uint8_t *>(w.x) + cc * piece, piece);
                cp16(dst + S::kHalf, reinterpret_cast<const uint8_t *>(w.y) + cc * piece, piece);
            }
            return;
        }
#pragma unroll 1
        for (int k = 0; k < PASSES; ++k) {
            place(k, row, cc, dst, piece);
            const ulonglong2 w = s_row[stage][row];
            const uint32_t size = w.x != 0 ? piece : 0;
            cp16(dst, size ? reinterpret_cast<const uint8_t *>(w.x) + cc * 16 : p.c.k, size);
            cp16(dst + S::kHalf, size ? reinterpret_cast<const uint8_t *>(w.y) + cc * 16 : p.c.v, size);
        }
    };

    Place next;                                               // in the tile STAGES ahead
    {
        Place r[STAGES];
#pragma unroll
        for (int k = 0; k < STAGES; ++k) r[k] = look_up(k < n_units);
        if (AHEAD) next = look_up(STAGES < n_units);
#pragma unroll
        for (int k = 0; k < STAGES; ++k)
            if (tid < TILE) s_row[k][tid] = addresses(r[k]);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < STAGES - 1; ++k) {
            if (k < n_units) copy(k);
            cp_commit();
        }
    }

    // the rows of this thread's quad: one, or two eight apart
    uint32_t qf[PARTS][KS][4];                   // query fragments
    float o[DT][RP][2], m[RP], l[RP], sfac[RP];
    int limit[RP], n_new = 0;
    bool fresh = true;

    for (int i = 0; i < n_units; ++i) {
        const int h = cur.h, rt = cur.rt;
        const int row0 = rt * ROWS + ug * S::kPerWarp + gr;
        if (fresh) {                              // a new segment: its query rows, while its first tile is on the way
            fresh = false;
            n_new = new_count(p.new_len, cur.b, p.new_tokens, KID_ATTN);
#pragma unroll
            for (int rp = 0; rp < RP; ++rp) {
                const int r = row0 + 8 * rp, t = p.group_div.of(r);
                const bool valid = r < p.rows && t < n_new;
                limit[rp] = valid ? cur.len - n_new + t + 1 : 0;
                const float *qr = p.q + ((int64_t)cur.b * p.new_tokens + (valid ? t : 0)) * p.ldq +
                                  (int64_t)(h * p.group + (valid ? r - t * p.group : 0)) * p.c.dim;
                float2 x[KS][2];
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = ks * 16 + e * 8 + 2 * j;
                        x[ks][e] = valid && d < p.c.dim ? *reinterpret_cast<const float2 *>(qr + d) : make_float2(0.f, 0.f);
                        top = fmaxf(top, fmaxf(fabsf(x[ks][e].x), fabsf(x[ks][e].y)));
                    }
                top = quad_max(top);
                // the row's power of two, where it and its inverse are normal numbers (q then lies below 4 at most); the
                // sign of the scale goes to q, so that sfac > 0
                int ex = (int)(__float_as_uint(top) >> 23) - 127;
                ex = min(max(ex, -126), 126);
                const float down = copysignf(__uint_as_float((uint32_t)(127 - ex) << 23), p.scale_log2);
                sfac[rp] = fmaxf(fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + ex) << 23), 1e-37f);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t hi, mid, lo;
                        split<T>(x[ks][e].x * down, x[ks][e].y * down, hi, mid, lo);
                        if constexpr (MODE == 0) {
                            qf[0][ks][2 * e] = g < 4 ? hi : mid;
                            qf[0][ks][2 * e + 1] = g < 4 ? lo : 0u;
                        } else if constexpr (RP == 1) {
                            qf[0][ks][2 * e] = hi;
                            qf[0][ks][2 * e + 1] = mid;
                            if constexpr (BF) {
                                qf[PARTS - 1][ks][2 * e] = 0;
                                qf[PARTS - 1][ks][2 * e + 1] = lo;
                            }
                        } else {
                            qf[0][ks][2 * e + rp] = hi;
                            qf[1 % PARTS][ks][2 * e + rp] = mid;
                            if constexpr (BF) qf[PARTS - 1][ks][2 * e + rp] = lo;
                        }
                    }
                m[rp] = -INFINITY;
                l[rp] = 0.f;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) o[dt][rp][0] = o[dt][rp][1] = 0.f;
            }
        }
        cp_wait<STAGES - 2>();
        __syncthreads();
        const int stage = i % STAGES;
        if (i + STAGES - 1 < n_units) copy((i + STAGES - 1) % STAGES);
        cp_commit();
        // the rows of tile i + STAGES take the place of tile i's, which has been copied
        if (AHEAD && tid < TILE) s_row[stage][tid] = addresses(next);
        next = look_up(i + STAGES + AHEAD < n_units);
        const ulonglong2 late = AHEAD ? make_ulonglong2(0, 0) : addresses(next);

        const int base = cur.tile * TILE + tg * TW;           // the warp's first entry
        if (base < cur.len && rt * ROWS + ug * S::kPerWarp < p.rows) {
            const uint32_t kb = ring + stage * 2 * S::kHalf + tg * TW * S::kStride, vb = kb + S::kHalf;
            // ---- scores, before their row's factor
            float s[NT][RP][2];
            const int seen = cur.len - n_new + 1;             // entries that every row sees
            const bool edge = base + TW > seen;               // some row may not see all of the warp's
            // Independent chains of products side by side, since one takes some 20 cycles after the one before it:
            // NG times eight entries at a time, each in one chain, or two (even and odd steps) where NG is small: a
            // shorter chain is also cut off less.  (Sixteen rows of 128 values fill the registers: there more chains
            // spill, and 163 us became 172; so do eight rows of 256 in bf16, 78 us became 82.)
            constexpr int NG = S::kNg < NT ? S::kNg : NT, CH = NG <= 2 && !(BF && MODE == 1 && DP == 256) ? 2 : 1;
#pragma unroll
            for (int n0 = 0; n0 < NT; n0 += NG) {
                float acc[NG][CH][4];
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int x = 0; x < CH; ++x) acc[n][x][0] = acc[n][x][1] = acc[n][x][2] = acc[n][x][3] = 0.f;
#pragma unroll
                for (int k2 = 0; k2 < (KS + 1) / 2; ++k2)       // an odd last step: half of what is loaded is not used
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        uint32_t b[4];                        // lane's row: entry nt*8 + lane%8, piece k2*4 + lane/8
                        ldsm4(b, kb + ((n0 + n) * 8 + (lane & 7)) * S::kStride + (((k2 * 4 + (lane >> 3)) ^ (lane & 7)) << 4));
#pragma unroll
                        for (int x = 0; x < PARTS; ++x)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                if (2 * k2 + e >= KS) continue;
                                const uint32_t(&a)[4] = qf[x][2 * k2 + e];
                                mma16816<T>(acc[n][e % CH], RP == 1 && x == 1 ? 0u : a[0], a[1], RP == 1 && x == 1 ? 0u : a[2], a[3],
                                            b[2 * e], b[2 * e + 1]);
                            }
                    }
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int rp = 0; rp < RP; ++rp)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = acc[n][0][2 * rp + e];
                            if (CH == 2) x += acc[n][CH - 1][2 * rp + e];
                            if (RP == 1) x += CH == 2 ? acc[n][0][2 + e] + acc[n][CH - 1][2 + e] : acc[n][0][2 + e];
                            if (MODE == 0) x += __shfl_xor_sync(0xffffffffu, x, 16);
                            s[n0 + n][rp][e] = x;
                        }
            }
            if (base + TW > min(limit[0], limit[RP - 1])) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int rp = 0; rp < RP; ++rp)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (base + nt * 8 + 2 * j + e >= limit[rp]) s[nt][rp][e] = -INFINITY;
            }
            if (p.norm) {
#pragma unroll
                for (int rp = 0; rp < RP; ++rp)
                    if (holds && row0 + 8 * rp < p.rows) {
                        float *dst = p.scores + (((int64_t)cur.b * p.c.heads + h) * p.rows + row0 + 8 * rp) * p.cap + base + 2 * j;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            *reinterpret_cast<float2 *>(dst + nt * 8) = make_float2(s[nt][rp][0] * sfac[rp], s[nt][rp][1] * sfac[rp]);
                    }
            }
            // ---- running maximum, powers, sums
            float alpha[RP];
            uint32_t pf[PARTS][NT / 2][4];
#pragma unroll
            for (int rp = 0; rp < RP; ++rp) {
                float mx = s[0][rp][0];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(s[nt][rp][0], s[nt][rp][1]));
                // The maximum is kept before the row's factor, and scores are multiplied after it is taken off: the
                // largest gives kExp exactly.  (As fma(s, sfac, -max of s*sfac) past 2^24, where the rounded maximum
                // is off by whole numbers, p left f16's range and finite inputs gave NaN.)
                mx = fmaxf(m[rp], quad_max(mx));
                const float ref = mx == -INFINITY ? 0.f : mx; // nothing seen yet: every power is 0
                alpha[rp] = pow2((m[rp] - ref) * sfac[rp]);
                m[rp] = mx;
                l[rp] *= alpha[rp];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float p0 = pow2(fmaf(s[nt][rp][0] - ref, sfac[rp], kExp<T>)), p1 = pow2(fmaf(s[nt][rp][1] - ref, sfac[rp], kExp<T>));
                    l[rp] += p0 + p1;
                    uint32_t hi, mid, lo;
                    split<T>(p0, p1, hi, mid, lo);
                    const int k = nt / 2, e = nt & 1;
                    if constexpr (MODE == 0) {
                        pf[0][k][2 * e] = g < 4 ? hi : mid;
                        pf[0][k][2 * e + 1] = g < 4 ? lo : 0u;
                    } else if constexpr (RP == 1) {
                        pf[0][k][2 * e] = hi;
                        pf[0][k][2 * e + 1] = mid;
                        if constexpr (BF) {
                            pf[PARTS - 1][k][2 * e] = 0;
                            pf[PARTS - 1][k][2 * e + 1] = lo;
                        }
                    } else {
                        pf[0][k][2 * e + rp] = hi;
                        pf[1 % PARTS][k][2 * e + rp] = mid;
                        if constexpr (BF) pf[PARTS - 1][k][2 * e + rp] = lo;
                    }
                }
            }
            // ---- p v.  Entries that only some of the rows see must not reach the others even as 0 * Inf:
            // if one of them is not finite, the products run once per new token with the entries beyond its
            // view cleared, each row taking the pass of its own token.
            int passes = 1;
            if (n_new > 1 && edge) {
                bool bad = false;
                const int e1 = min(cur.len, base + TW) - base;
                for (int e = max(seen - base, 0); e < e1; ++e)
                    for (int w = lane; w < DP / 2; w += 32) {
                        uint32_t v;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(vb + e * S::kStride + (((w >> 2) ^ (e & 7)) << 4) + (w & 3) * 4));
                        bad |= not_finite2<T>(v);
                    }
                if (__any_sync(0xffffffffu, bad)) passes = n_new;
            }
#pragma unroll 1
            for (int pass = 0; pass < passes; ++pass) {
                const int view = passes > 1 ? seen + pass : 0x7fffffff;
                bool take[RP];
                float keep[RP];
#pragma unroll
                for (int rp = 0; rp < RP; ++rp) {
                    take[rp] = passes == 1 || limit[rp] == view;
                    keep[rp] = take[rp] ? alpha[rp] : 1.f;
                }
#pragma unroll
                for (int dg = 0; dg < DT / S::kDg; ++dg) {    // kDg chains side by side
                    float y[S::kDg][4];
#pragma unroll
                    for (int c = 0; c < S::kDg; ++c) y[c][0] = y[c][1] = y[c][2] = y[c][3] = 0.f;
#pragma unroll
                    for (int k = 0; k < NT / 2; ++k)
#pragma unroll
                        for (int d2 = 0; d2 < S::kDg / 2; ++d2) {
                            uint32_t b[4];
                            const int e = k * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, ch = dg * S::kDg + d2 * 2 + (lane >> 4);
                            ldsm4t(b, vb + e * S::kStride + ((ch ^ (e & 7)) << 4));
                            if (passes > 1) {
                                const int tok = base + k * 16 + 2 * j;
                                const uint32_t m0 = (tok < view ? 0xffffu : 0u) | (tok + 1 < view ? 0xffff0000u : 0u);
                                const uint32_t m1 = (tok + 8 < view ? 0xffffu : 0u) | (tok + 9 < view ? 0xffff0000u : 0u);
                                b[0] &= m0, b[1] &= m1, b[2] &= m0, b[3] &= m1;
                            }
#pragma unroll
                            for (int x = 0; x < PARTS; ++x) {
                                const uint32_t(&a)[4] = pf[x][k];
                                const uint32_t a0 = RP == 1 && x == 1 ? 0u : a[0], a2 = RP == 1 && x == 1 ? 0u : a[2];
                                mma16816<T>(y[2 * d2], a0, a[1], a2, a[3], b[0], b[1]);
                                mma16816<T>(y[2 * d2 + 1], a0, a[1], a2, a[3], b[2], b[3]);
                            }
                        }
#pragma unroll
                    for (int c = 0; c < S::kDg; ++c)
#pragma unroll
                        for (int rp = 0; rp < RP; ++rp)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float add = RP == 1 ? y[c][e] + y[c][2 + e] : y[c][2 * rp + e];
                                float &sum = o[S::kDg * dg + c][rp][e];
                                sum = fmaf(sum, keep[rp], take[rp] ? add : 0.f);
                            }
                }
            }
        }
        if (!AHEAD && tid < TILE) s_row[stage][tid] = late;

        const AttnCursor was = cur;
        attn_advance<TILE>(p, cur);
        if (i + 1 < n_units && cur.tile != 0) continue;

        // ---- the segment's end (or this CTA's): join the warps that split its entries.  Their sums go
        // through the stage that was just used up: its next copies are issued after the next barrier.
        fresh = true;
        float *sums = reinterpret_cast<float *>(smem + stage * 2 * S::kHalf);
        const int rows_here = min(ROWS, p.rows - rt * ROWS);
        const int64_t seg = (int64_t)was.b * p.c.heads + h;
        const bool whole = seg_base >= u0 && was.tile + 1 == was.tiles;
        // slot in the workspace of a part of a segment: 0 if it is the CTA's first, else 1
        const int64_t part = 2 * (int64_t)blockIdx.x + (seg_base > u0 ? 1 : 0);
        float *const ml_all = p.part + 2 * (int64_t)gridDim.x * ROWS * DP;
        auto out_row = [&](int r) {
            const int rg = rt * ROWS + r, t = p.group_div.of(rg);
            return p.out + (((int64_t)was.b * p.new_tokens + t) * p.c.heads * p.group + h * p.group + (rg - t * p.group)) * (int64_t)p.c.dim;
        };
#pragma unroll
        for (int rp = 0; rp < RP; ++rp) {
            l[rp] = quad_sum(l[rp]);
            if (j == 0 && holds) s_ml[turned][gr + 8 * rp] = make_float2(m[rp] * sfac[rp], l[rp]);
        }
        if constexpr (MODE == 0) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int e = 0; e < 2; ++e) o[dt][0][e] += __shfl_xor_sync(0xffffffffu, o[dt][0][e], 16);
        }
#pragma unroll
        for (int round = 0; round < S::kRounds; ++round) {
            __syncthreads();
#pragma unroll
            for (int rp = 0; rp < RP; ++rp)
                if (holds && row0 + 8 * rp < p.rows) {
                    float *mine = sums + (turned * S::kPerWarp + gr + 8 * rp) * S::kPad + 2 * j;
#pragma unroll
                    for (int x = 0; x < DT / S::kRounds; ++x) {
                        const int dt = round * (DT / S::kRounds) + x;
                        *reinterpret_cast<float2 *>(mine + x * 8) = make_float2(o[dt][rp][0], o[dt][rp][1]);
                    }
                }
            __syncthreads();
            constexpr int C4 = S::kCols / 4;                  // 16-byte pieces of a row
            for (int x = tid; x < rows_here * C4; x += THREADS) {
                const int r = x / C4, c4 = x % C4, w0 = r / S::kPerWarp, rw = r % S::kPerWarp;      // row r: warps w0, w0 + UG, ...
                const int col = round * S::kCols + c4 * 4;
                float2 ml[TG];
                float top = -INFINITY, tot = 0.f;
#pragma unroll
                for (int k = 0; k < TG; ++k) {
                    ml[k] = s_ml[w0 + k * UG][rw];
                    top = fmaxf(top, ml[k].x);
                }
                const float ref = top == -INFINITY ? 0.f : top;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < TG; ++k) {
                    const float w = pow2(ml[k].x - ref);
                    const float4 v = *reinterpret_cast<const float4 *>(sums + ((w0 + k * UG) * S::kPerWarp + rw) * S::kPad + c4 * 4);
                    tot = fmaf(ml[k].y, w, tot);
                    y.x = fmaf(v.x, w, y.x), y.y = fmaf(v.y, w, y.y), y.z = fmaf(v.z, w, y.z), y.w = fmaf(v.w, w, y.w);
                }
                if (whole) {
                    const float inv = inverse(tot);
                    if (inv == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);      // saw nothing: its 0 * Inf must not show
                    if (col < p.c.dim)
                        *reinterpret_cast<float4 *>(out_row(r) + col) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
                    if (p.norm && col == 0) p.norm[seg * p.rows + rt * ROWS + r] = row_norm<T>(top, tot);
                } else {
                    *reinterpret_cast<float4 *>(p.part + (part * ROWS + r) * DP + col) = y;
                    if (col == 0) *reinterpret_cast<float2 *>(ml_all + (part * ROWS + r) * 2) = make_float2(top, tot);
                }
            }
        }
        // The CTA with the segment's first tile says which CTAs hold parts of it: itself up to the one of the last
        // tile (itself alone, and no part, if it holds all)
        if (seg_base >= u0 && tid == 0)
            p.parts[seg * p.row_tiles + rt] =
                make_int3((int)part, (int)blockIdx.x, whole ? -1 : (int)((((long long)seg_base + was.tiles) * G - 1) / W));
        seg_base = u0 + i + 1;
    }
}

// The second launch.  Its first blocks join the parts of rows, `row_blocks` of
// them for the rows that a CTA of the first launch takes together, each every
// row_blocks-th row, if the row has parts: groups of dim/4 threads take every
// ways-th part, four in flight, with a running maximum, and meet in shared
// memory.  The blocks after them (weights wanted) take JOIN_WEIGHTS entries of
// a (sequence, head) each: weight[entry] += sum over the rows of
// 2^(score - maximum) / sum, the scores read side by side along the entries,
// maxima and sums of split rows from their parts, eight lanes to a row.
// Seven blocks per SM (72 registers, 8 bytes spilled): with six, 30 sequences of
// 1500 with five tokens of bf16 and weights took 99 us, and take 94.
constexpr int JOIN_THREADS = 128;
constexpr int JOIN_WEIGHTS = 1024;
constexpr int JOIN_ROWS = 2048;      // most rows of a key-value head

template <typename T>
__global__ void __launch_bounds__(JOIN_THREADS, 7) attn_join_kernel(const AttnParams p, int dp, int kept_rows, int grid, int row_blocks, int64_t join_blocks,
                                                                 int chunks)
{
    using namespace attn;
    __shared__ __align__(16) float4 s_y[JOIN_THREADS];
    __shared__ float2 s_ml[JOIN_THREADS];
    __shared__ float2 s_norm[JOIN_ROWS];
    const int tid = threadIdx.x;
    const float2 *ml_all = reinterpret_cast<const float2 *>(p.part + 2 * (int64_t)grid * kept_rows * dp);
    if (blockIdx.x < join_blocks) {
        pdl_wait();
        pdl_launch_dependents();
        const int64_t x = blockIdx.x / row_blocks, seg = x / p.row_tiles;
        const int rt = (int)(x - seg * p.row_tiles);
        const int3 at = p.parts[x];
        if (at.z < 0) return;
        const int per = dp / 4, ways = JOIN_THREADS / per, way = tid / per, col = (tid - way * per) * 4;
        const int rows_here = min(kept_rows, p.rows - rt * kept_rows);
        const int64_t b = seg / p.c.heads, h = seg - b * p.c.heads;
        for (int rr = (int)(blockIdx.x - x * row_blocks); rr < rows_here; rr += row_blocks) {
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = -INFINITY, tot = 0.f;
            for (int c = at.y + way; c <= at.z; c += ways * 4) {
                float2 ml[4];
                float4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {                 // past the end: the last part again, without weight
                    const int cc = min(c + k * ways, at.z);
                    const int64_t sl = (int64_t)(cc == at.y ? at.x : 2 * cc) * kept_rows + rr;
                    ml[k] = __ldcg(ml_all + sl);
                    v[k] = __ldcg(reinterpret_cast<const float4 *>(p.part + sl * dp + col));
                }
                const float mx = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), top);
                const float ref = mx == -INFINITY ? 0.f : mx, old = pow2(top - ref);
                top = mx;
                tot *= old;
                y.x *= old, y.y *= old, y.z *= old, y.w *= old;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // A part that saw nothing (its sum is 0) adds nothing, whatever its entries hold.  One that saw
                    // something is added even if its weight is 0: a NaN, or 0 * Inf, has to come through.
                    if (c + k * ways > at.z || ml[k].y == 0.f) continue;
                    const float w = pow2(ml[k].x - ref);
                    tot = fmaf(ml[k].y, w, tot);
                    y.x = fmaf(v[k].x, w, y.x), y.y = fmaf(v[k].y, w, y.y), y.z = fmaf(v[k].z, w, y.z), y.w = fmaf(v[k].w, w, y.w);
                }
            }
            __syncthreads();                                  // the row before has been read
            s_y[tid] = y;
            s_ml[tid] = make_float2(top, tot);
            __syncthreads();
            if (way > 0 || col >= p.c.dim) continue;
            for (int k = 1; k < ways; ++k) top = fmaxf(top, s_ml[tid + k * per].x);
            const float ref = top == -INFINITY ? 0.f : top;
            tot = 0.f;
            y = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < ways; ++k) {
                const float2 ml = s_ml[tid + k * per];
                const float4 v = s_y[tid + k * per];
                const float w = pow2(ml.x - ref);
                tot = fmaf(ml.y, w, tot);
                y.x = fmaf(v.x, w, y.x), y.y = fmaf(v.y, w, y.y), y.z = fmaf(v.z, w, y.z), y.w = fmaf(v.w, w, y.w);
            }
            const float inv = inverse(tot);
            const int r = rt * kept_rows + rr, t = p.group_div.of(r);
            *reinterpret_cast<float4 *>(p.out + ((b * p.new_tokens + t) * p.c.heads * p.group + h * p.group + (r - t * p.group)) * p.c.dim + col) =
                make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        }
        return;
    }
    const int64_t x = blockIdx.x - join_blocks, seg = x / chunks;
    const int b = (int)(seg / p.c.heads), h = (int)(seg - (int64_t)b * p.c.heads);
    const int len = cache_len<true>(p.c, b, KID_ATTN), first = (int)(x - seg * chunks) * JOIN_WEIGHTS;
    // Eight neighbouring entries per thread.  What the first launch does not write is read before its end: lengths,
    // page ids and the weights so far.  (The first launch lets this one start only after the launches before it have
    // ended.)  From L2, since nothing before pdl_wait says that lines left in L1 are of today.
    constexpr int EACH = JOIN_WEIGHTS / JOIN_THREADS;
    static_assert(EACH == 8, "two 16-byte accesses");
    const int mine = first + tid * EACH, n = min(EACH, len - mine);
    const bool together = p.c.page_size % EACH == 0 && n == EACH;        // one page, 32-byte aligned
    float w[EACH];
    float *at[EACH];
    if (together) {
        const int c = p.page_div.of(mine), pg = cache_page<true>(p.c, b, c, KID_ATTN);
        at[0] = pg < 0 ? nullptr : p.c.weight + ((int64_t)pg * p.c.heads + h) * p.c.page_size + (mine - c * p.c.page_size);
        if (at[0]) {
            *reinterpret_cast<float4 *>(w) = __ldcg(reinterpret_cast<const float4 *>(at[0]));
            *reinterpret_cast<float4 *>(w + 4) = __ldcg(reinterpret_cast<const float4 *>(at[0] + 4));
        }
    } else {
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            at[k] = nullptr;
            if (k >= n) continue;
            const int c = p.page_div.of(mine + k), pg = cache_page<true>(p.c, b, c, KID_ATTN);
            if (pg < 0) continue;
            at[k] = p.c.weight + ((int64_t)pg * p.c.heads + h) * p.c.page_size + (mine + k - c * p.c.page_size);
            w[k] = __ldcg(at[k]);
        }
    }
    pdl_wait();
    pdl_launch_dependents();
    if (first >= len) return;
    for (int r0 = 0; r0 < p.rows; r0 += JOIN_THREADS / 8) {               // eight lanes per row's sum
        const int r = r0 + tid / 8, rt = r / kept_rows, rr = r - rt * kept_rows;
        const int3 at = r < p.rows ? p.parts[seg * p.row_tiles + rt] : make_int3(0, 0, -1);
        float top = -INFINITY, tot = 0.f;
#pragma unroll 4
        for (int c = at.y + tid % 8; c <= at.z; c += 8) {
            const float2 ml = __ldcg(ml_all + (int64_t)(c == at.y ? at.x : 2 * c) * kept_rows + rr);
            const float mx = fmaxf(top, ml.x), ref = mx == -INFINITY ? 0.f : mx;
            tot = tot * pow2(top - ref) + ml.y * pow2(ml.x - ref);
            top = mx;
        }
        float mx = top;
#pragma unroll
        for (int o = 4; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        tot *= pow2(top - (mx == -INFINITY ? 0.f : mx));
#pragma unroll
        for (int o = 4; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
        if (r < p.rows && tid % 8 == 0) s_norm[r] = at.z < 0 ? __ldcg(p.norm + seg * p.rows + r) : row_norm<T>(mx, tot);
    }
    __syncthreads();
    if (n <= 0) return;
    const float *s = p.scores + seg * p.rows * p.cap + mine;             // 32-byte aligned, readable past len
    float add[EACH];
#pragma unroll
    for (int k = 0; k < EACH; ++k) add[k] = 0.f;
#pragma unroll 4
    for (int r = 0; r < p.rows; ++r) {
        const float4 a = __ldcg(reinterpret_cast<const float4 *>(s + r * p.cap));
        const float4 c = __ldcg(reinterpret_cast<const float4 *>(s + r * p.cap) + 1);
        const float2 f = s_norm[r];
        const float v[EACH] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < EACH; ++k) add[k] = fmaf(pow2(v[k] - f.x), f.y, add[k]);
    }
    if (together) {
        if (!at[0]) return;
        *reinterpret_cast<float4 *>(at[0]) = make_float4(w[0] + add[0], w[1] + add[1], w[2] + add[2], w[3] + add[3]);
        *reinterpret_cast<float4 *>(at[0] + 4) = make_float4(w[4] + add[4], w[5] + add[5], w[6] + add[6], w[7] + add[7]);
    } else {
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            if (at[k]) *at[k] = w[k] + add[k];
    }
}

// Which kernel: dim padded, rows per operand (MODE) and warps along the rows.
// Up to 16, 32 and 64 rows, one, two and four warps take sixteen each, the
// remaining warps split the entries; for heads above 128 sixteen rows do not
// fit the registers, and warps take eight.  Heads above 192 leave two warps of
// four without rows rather than splitting 64 entries four ways: tiles of 32
// let two CTAs share an SM (8 sequences of 20000 entries of 256 values, f16: 137
// us against 158).  More rows than a CTA takes are dealt to further CTAs, which read the
// cache again (from L2).
struct AttnPlan {
    int dp, mode, ug, rows, kept_rows, row_tiles, grid;
    int64_t tiles, cap, part_floats, score_floats, norm_floats, parts;
};

// f(type, DP, MODE, UG) with the plan's kernel as compile-time values
template <typename F>
int attn_dispatch(const AttnPlan &a, int dtype, F f)
{
    using std::integral_constant;
    const auto with_ug = [&](auto t, auto DPc, auto Mc) {
        return a.ug == 1   ? f(t, DPc, Mc, integral_constant<int, 1>())
               : a.ug == 2 ? f(t, DPc, Mc, integral_constant<int, 2>())
                           : f(t, DPc, Mc, integral_constant<int, 4>());
    };
    const auto with_dp = [&](auto t, auto DPc) {
        constexpr integral_constant<int, 1> one;
        if constexpr (attn::kBf16<decltype(t)>) {
            if (a.mode == 0) return f(t, DPc, integral_constant<int, 0>(), integral_constant<int, DPc.value == 256 ? 2 : 1>());
        }
        if constexpr (DPc.value == 256)
            return a.ug == 2 ? f(t, DPc, one, integral_constant<int, 2>()) : f(t, DPc, one, integral_constant<int, 4>());
        else if constexpr (DPc.value == 192) return with_ug(t, DPc, one);
        else return a.mode == 1 ? f(t, DPc, one, one) : with_ug(t, DPc, integral_constant<int, 2>());
    };
    const auto with_type = [&](auto t) {
        return a.dp == 64    ? with_dp(t, integral_constant<int, 64>())
               : a.dp == 80  ? with_dp(t, integral_constant<int, 80>())
               : a.dp == 96  ? with_dp(t, integral_constant<int, 96>())
               : a.dp == 128 ? with_dp(t, integral_constant<int, 128>())
               : a.dp == 192 ? with_dp(t, integral_constant<int, 192>())
                             : with_dp(t, integral_constant<int, 256>());
    };
    return dtype == MMQ_F16 ? with_type(__half()) : with_type(__nv_bfloat16());
}

inline AttnPlan attn_plan(const mmq_kv_cache &c, int q_heads, int new_tokens, bool save)
{
    AttnPlan a;
    a.dp = c.dim <= 64 ? 64 : c.dim <= 80 ? 80 : c.dim <= 96 ? 96 : c.dim <= 128 ? 128 : c.dim <= 192 ? 192 : 256;
    a.rows = q_heads / c.heads * new_tokens;
    a.mode = c.dtype == MMQ_BF16 && a.rows <= 4 ? 0 : a.rows <= 8 || a.dp > 128 ? 1 : 2;
    const int per_warp = a.mode == 2 ? 16 : 8;
    a.ug = a.rows <= per_warp && a.dp < 256 ? 1 : a.rows <= 2 * per_warp ? 2 : 4;
    int tile = 0, per_sm = 0;
    attn_dispatch(a, c.dtype, [&](auto, auto DPc, auto Mc, auto UGc) {
        using S = attn::Shape<DPc.value, Mc.value, UGc.value>;
        tile = S::kTile;
        per_sm = S::kPerSm;
        a.kept_rows = S::kRows;
        return 0;
    });
    const int rows = a.kept_rows;                                        // per CTA
    a.row_tiles = (a.rows + rows - 1) / rows;
    a.tiles = ((int64_t)c.cols * c.page_size + tile - 1) / tile * c.seqs * c.heads * a.row_tiles;
    const int64_t full = (int64_t)sm_count() * per_sm;                   // every CTA resident
    a.grid = (int)(a.tiles < full ? a.tiles : full);
    a.cap = ((int64_t)c.cols * c.page_size + 127) / 128 * 128;
    a.part_floats = 2 * (int64_t)a.grid * rows * (a.dp + 2);
    a.score_floats = save ? (int64_t)c.seqs * c.heads * a.rows * a.cap : 0;
    a.norm_floats = save ? 2 * (int64_t)c.seqs * c.heads * a.rows : 0;
    a.parts = (int64_t)c.seqs * c.heads * a.row_tiles;
    return a;
}

inline int attn_check(const mmq_kv_cache *c, int q_heads, int new_tokens)
{
    const int rc = check_cache(c);
    if (rc != MMQ_OK) return rc;
    if (q_heads < 1 || q_heads > 65535 || q_heads % c->heads || q_heads / c->heads > 128 || new_tokens < 1 ||
        new_tokens > 16)
        return MMQ_ERR_SHAPE;
    return MMQ_OK;
}

// Whether a plan fits: tiles are counted in an int, and so are the second launch's blocks.
inline bool attn_fits(const mmq_kv_cache &c, const AttnPlan &a, bool save)
{
    const int64_t chunks = save ? (a.cap + JOIN_WEIGHTS - 1) / JOIN_WEIGHTS : 0;
    return a.tiles <= 0x7fffffff && (int64_t)c.seqs * c.heads * (a.rows + chunks) <= 0x7fffffff;
}

template <int DP, typename T, int MODE, int UG>
int launch_attn(const AttnParams &p, int grid, cudaStream_t stream)
{
    const auto kernel = attn_kernel<DP, T, MODE, UG>;
    constexpr int smem = attn::Shape<DP, MODE, UG>::kSmem;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return MMQ_ERR_ARCH;
    }
    static bool attr_done[64];
    if (!attr_done[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return launch_status();
        attr_done[dev] = true;
    }
    return launch_pdl(kernel, dim3((unsigned)grid), attn::THREADS, smem, stream, 0, p);
}

}  // namespace
}  // namespace mmq

extern "C" int mmq_attn_sizes(const mmq_kv_cache *cache, int q_heads, int new_tokens, int accumulate,
                              int64_t *work_floats)
{
    using namespace mmq;
    const int rc = attn_check(cache, q_heads, new_tokens);
    if (rc != MMQ_OK) return rc;
    if (!work_floats) return MMQ_ERR_NULL;
    const AttnPlan a = attn_plan(*cache, q_heads, new_tokens, accumulate != 0);
    if (!attn_fits(*cache, a, accumulate != 0)) return MMQ_ERR_SHAPE;
    *work_floats = a.part_floats + a.score_floats + a.norm_floats + 3 * a.parts;
    return MMQ_OK;
}

extern "C" int mmq_attn_decode(const mmq_kv_cache *cache, const float *q, int64_t ldq, const int32_t *new_len,
                               float *out, int q_heads, int new_tokens, float scale, int accumulate, float *work,
                               mmq_stream_t stream)
{
    using namespace mmq;
    int rc = attn_check(cache, q_heads, new_tokens);
    if (rc != MMQ_OK) return rc;
    if (ldq < (int64_t)q_heads * cache->dim || !(scale - scale == 0.f)) return MMQ_ERR_SHAPE;
    if (cache->seqs == 0) return MMQ_OK;
    if (out == q) return MMQ_ERR_SHAPE;                   // rows are read by several CTAs, at any time
    if (!q || !out || !work || (accumulate && !cache->weight)) return MMQ_ERR_NULL;
    if (!aligned16(q) || (ldq & 3) || !aligned16(out) || !aligned16(work) || (accumulate && !aligned16(cache->weight)))
        return MMQ_ERR_ALIGN;
    if ((rc = check_arch()) != MMQ_OK) return rc;
    const bool save = accumulate != 0;
    const AttnPlan a = attn_plan(*cache, q_heads, new_tokens, save);
    if (!attn_fits(*cache, a, save)) return MMQ_ERR_SHAPE;
    AttnParams p;
    p.c = *cache;
    p.q = q;
    p.new_len = new_len;
    p.out = out;
    p.ldq = ldq;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.new_tokens = new_tokens;
    p.group = q_heads / cache->heads;
    p.rows = a.rows;
    p.row_tiles = a.row_tiles;
    p.scores = work;                                   // rows of a multiple of 128 floats: 16-byte aligned
    p.part = work + a.score_floats;
    p.norm = save ? reinterpret_cast<float2 *>(p.part + a.part_floats) : nullptr;        // 8-byte aligned: part_floats is even
    p.parts = reinterpret_cast<int3 *>(p.part + a.part_floats + a.norm_floats);
    p.cap = a.cap;
    p.page_div = FastDiv(cache->page_size);
    p.group_div = FastDiv(p.group);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    rc = attn_dispatch(a, cache->dtype, [&](auto t, auto DPc, auto Mc, auto UGc) {
        return launch_attn<DPc.value, decltype(t), Mc.value, UGc.value>(p, a.grid, s);
    });
    if (rc != MMQ_OK) return rc;
    const int64_t segs = (int64_t)cache->seqs * cache->heads;
    // Blocks for the rows of a segment's part: one each while that is at most sixteen blocks per SM; four where weights
    // are wanted, whose blocks wait for a place behind them (30 sequences of 1500 with five tokens of bf16: with
    // weights 98 us at sixteen and 93 at four, without 80 and 84).
    int64_t row_blocks = (int64_t)sm_count() * (save ? 4 : 16) / a.parts;
    const int most = a.rows < a.kept_rows ? a.rows : a.kept_rows;
    row_blocks = row_blocks < 1 ? 1 : row_blocks > most ? most : row_blocks;
    const int64_t join_blocks = a.parts * row_blocks;
    const int chunks = save ? (int)((a.cap + JOIN_WEIGHTS - 1) / JOIN_WEIGHTS) : 0;
    const auto join = cache->dtype == MMQ_F16 ? attn_join_kernel<__half> : attn_join_kernel<__nv_bfloat16>;
    return launch_pdl(join, dim3((unsigned)(join_blocks + segs * chunks)), JOIN_THREADS, 0, s, 0, p, a.dp, a.kept_rows, a.grid,
                      (int)row_blocks, join_blocks, chunks);
}
