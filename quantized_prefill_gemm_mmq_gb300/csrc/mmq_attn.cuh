// mmq_attn.cuh -- attention of the newest tokens over the paged cache
// (mmq_attn_decode).
//
// Per query row r (a token t and a query head of the key-value head's group):
//     s = scale q.k,  p = exp(s - m),  out = sum p v / sum p
// in one pass over the cache with a running maximum m: when a tile raises m,
// what was summed so far is multiplied by exp(m_old - m_new).
//
// Work.  The cache is read once; everything else is small, so the kernel is
// bound by memory (4 dim bytes per entry and head) as long as the rows that
// share a key-value head are few.  All tiles of TILE entries of all sequences
// and heads are numbered in a row, and the persistent grid's CTA c takes tiles
// [c W/G, (c+1) W/G): every CTA reads the same amount whatever the lengths.
// A run of tiles that belongs to one (sequence, head) is a segment; a CTA that
// has all of a segment writes its output, the others leave their part (m, sum,
// sum p v) in the workspace, and the last of them to arrive joins the parts in
// CTA order.  The counters only say who is last: no result depends on timing.
//
// Tiles.  K and V rows are gathered through the page table with 16-byte
// cp.async into a three-stage ring (any page size and stride; entries past
// the length arrive as zeros), chunk-XOR swizzled so that ldmatrix reads
// without bank conflicts.  The table entries of a tile are fetched one
// iteration before its copies are issued.
//
// Products run on the warp-level tensor core, whose 16-row operand is filled
// with eight query rows twice: the upper eight rows hold the rounded values
// (f16 or bf16, the cache's type), the lower eight what rounding left, and the
// two halves of the result are added.  For f16 that makes 22 bits of q and of
// p; for bf16 a second product with a third part makes 24.  q is scaled by a
// power of two per row to lie below 2 and p by 2^15, so that f16's range does
// not clip either.  K and V are used as they are.  The sums over a tile's
// entries stay in f32 and are added to the running sums with f32 FMAs.
//
// UG warps of the four take eight rows each over the same entries and 4/UG
// warps split a tile's entries (with their own running maximum, joined at the
// segment's end), so that up to 8*UG rows share one read of the cache.
#pragma once

#include <type_traits>

namespace mmq {
namespace {

namespace attn {
constexpr int THREADS = 128;
constexpr int STAGES = 3;
constexpr float P_EXP = 15.f;         // p carries 2^15

template <int DP>
struct Shape {
    static constexpr int kTile = DP == 64 ? 128 : 64;                 // entries per tile
    static constexpr int kHalf = kTile * DP * 2;                      // bytes of K (or V) per stage
    static constexpr int kSmem = STAGES * 2 * kHalf;
    static constexpr int kPerSm = DP <= 128 ? 2 : 1;
    static constexpr int kPad = DP + 8;                               // floats per row of a warp's sums in shared memory
    static_assert(4 * 8 * kPad * 4 <= 2 * kHalf, "four warps' sums fit in one stage");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
    if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value) {
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
// log2 of a row's sum of powers, so that pow2(score - it) is its weight
__device__ __forceinline__ float log_sum(float m, float sum) { return sum > 0.f ? m + log2f(sum) - P_EXP : INFINITY; }

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
    int rows, row_tiles;     // rows, and parts of 8*UG rows
    float *part;             // [2*grid][8*UG][DP] sums, then [2*grid][8*UG][2] (max, sum)
    int32_t *cnt;            // [seqs*heads*row_tiles]
    float *scores;           // [seqs*heads][rows][cap] in powers of two (weights only)
    float *lse;              // [seqs*heads][rows] (weights only, else NULL)
    int64_t cap;
    FastDiv page_div;
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

template <int DP, typename T, int UG>
__global__ void __launch_bounds__(attn::THREADS, attn::Shape<DP>::kPerSm) attn_kernel(const AttnParams p)
{
    using namespace attn;
    using S = Shape<DP>;
    constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    constexpr int TILE = S::kTile, TG = 4 / UG, TW = TILE / TG;    // entries per warp and tile
    constexpr int NT = TW / 8, KS = DP / 16, DT = DP / 8, ROWS = 8 * UG;
    constexpr int CPR = DP / 8, RPP = THREADS / CPR, PASSES = TILE / RPP;   // 16-byte copies per row, rows per pass

    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ ulonglong2 s_row[2][TILE];
    __shared__ int s_last;
    __shared__ float2 s_ml[4][8];              // (max, sum) of every warp's rows
    __shared__ float2 s_row_ml[ROWS];          // of the joined rows; the joining CTA: (max, 1 / sum)
    const uint32_t ring = smem_u32(smem);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ug = warp % UG, tg = warp / UG;
    const int g = lane >> 2, j = lane & 3;
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

    // addresses of K and V of entry `tid` of the tile at `inf`; 0 if there is none
    auto look_up = [&](bool there) {
        ulonglong2 r = make_ulonglong2(0, 0);
        if (there) {
            const int slot = inf.tile * TILE + tid;
            if (tid < TILE && slot < inf.len) {
                const int col = p.page_div.of(slot), off = slot - col * p.c.page_size;
                const int64_t pg = cache_page(p.c, inf.b, col, KID_ATTN);
                if (pg >= 0)
                    r = make_ulonglong2(
                        (unsigned long long)(static_cast<const T *>(p.c.k) + pg * p.c.k_page + inf.h * p.c.k_head + off * p.c.k_slot),
                        (unsigned long long)(static_cast<const T *>(p.c.v) + pg * p.c.v_page + inf.h * p.c.v_head + off * p.c.v_slot));
            }
            attn_advance<TILE>(p, inf);
        }
        return r;
    };
    // this thread's 16-byte piece of rows cr, cr + RPP, ...
    const int cc = tid % CPR, cr = tid / CPR;
    const bool piece = cc * 8 < p.c.dim;
    auto copy = [&](int stage, int buf) {
        const uint32_t base = ring + stage * 2 * S::kHalf + cr * (DP * 2);
        const ulonglong2 *rows = s_row[buf] + cr;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const ulonglong2 w = rows[i * RPP];
            const bool there = w.x != 0 && piece;
            const uint32_t dst = base + i * RPP * (DP * 2) + ((cc ^ ((cr + i * RPP) & 7)) << 4);
            cp16(dst, there ? reinterpret_cast<const uint8_t *>(w.x) + cc * 16 : p.c.k, there);
            cp16(dst + S::kHalf, there ? reinterpret_cast<const uint8_t *>(w.y) + cc * 16 : p.c.v, there);
        }
    };

    {
        const ulonglong2 r0 = look_up(true), r1 = look_up(n_units > 1);
        if (tid < TILE) {
            s_row[0][tid] = r0;
            s_row[1][tid] = r1;
        }
        __syncthreads();
        copy(0, 0);
        cp_commit();
        if (n_units > 1) copy(1, 1);
        cp_commit();
        const ulonglong2 r2 = look_up(n_units > 2);
        __syncthreads();
        if (tid < TILE) s_row[0][tid] = r2;
    }

    uint32_t qa[KS][4], ql[BF ? KS : 1][2];      // query fragments: rounded | rest, and the third part
    float o[DT][2], m = -INFINITY, l = 0.f, sfac = 0.f;
    int limit = 0, r_global = 0, n_new = 0;
    bool fresh = true;

    for (int i = 0; i < n_units; ++i) {
        const int h = cur.h, rt = cur.rt;
        if (fresh) {                              // a new segment: its query rows, while its first tile is on the way
            fresh = false;
            n_new = new_count(p.new_len, cur.b, p.new_tokens, KID_ATTN);
            r_global = rt * ROWS + ug * 8 + g;
            const int t = r_global / p.group;
            const bool valid = r_global < p.rows && t < n_new;
            limit = valid ? cur.len - n_new + t + 1 : 0;
            const float *qr = p.q + ((int64_t)cur.b * p.new_tokens + (valid ? t : 0)) * p.ldq +
                              (int64_t)(h * p.group + (valid ? r_global - t * p.group : 0)) * p.c.dim;
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
            // the row's power of two, away from f32's ends
            int ex = (int)(__float_as_uint(top) >> 23) - 127;
            ex = min(max(ex, -100), 100);
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
            sfac = p.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t l0, l1;
                split<T>(x[ks][0].x * down, x[ks][0].y * down, qa[ks][0], qa[ks][1], l0);
                split<T>(x[ks][1].x * down, x[ks][1].y * down, qa[ks][2], qa[ks][3], l1);
                if constexpr (BF) {
                    ql[ks][0] = l0;
                    ql[ks][1] = l1;
                }
            }
            m = -INFINITY;
            l = 0.f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) o[dt][0] = o[dt][1] = 0.f;
        }

        cp_wait<1>();
        __syncthreads();
        const int stage = i % STAGES;
        if (i + 2 < n_units) copy((i + 2) % STAGES, i & 1);
        cp_commit();
        const ulonglong2 nrow = look_up(i + 3 < n_units);

        const int base = cur.tile * TILE + tg * TW;           // the warp's first entry
        if (base < cur.len) {
            const uint32_t kb = ring + stage * 2 * S::kHalf + tg * TW * (DP * 2), vb = kb + S::kHalf;
            // ---- scores
            float s[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                // lane's row address: entry nt*8 + lane%8, chunk group lane/8
                const uint32_t ra = kb + (nt * 8 + (lane & 7)) * (DP * 2);
#pragma unroll
                for (int k2 = 0; k2 < KS / 2; ++k2) {
                    uint32_t b[4];
                    ldsm4(b, ra + (((k2 * 4 + (lane >> 3)) ^ (lane & 7)) << 4));
                    mma16816<T>(acc, qa[2 * k2][0], qa[2 * k2][1], qa[2 * k2][2], qa[2 * k2][3], b[0], b[1]);
                    mma16816<T>(acc, qa[2 * k2 + 1][0], qa[2 * k2 + 1][1], qa[2 * k2 + 1][2], qa[2 * k2 + 1][3], b[2], b[3]);
                    if constexpr (BF) {
                        mma16816<T>(acc, ql[2 * k2][0], 0u, ql[2 * k2][1], 0u, b[0], b[1]);
                        mma16816<T>(acc, ql[2 * k2 + 1][0], 0u, ql[2 * k2 + 1][1], 0u, b[2], b[3]);
                    }
                }
                const int tok = base + nt * 8 + 2 * j;
                s[nt][0] = tok < limit ? (acc[0] + acc[2]) * sfac : -INFINITY;
                s[nt][1] = tok + 1 < limit ? (acc[1] + acc[3]) * sfac : -INFINITY;
            }
            if (p.lse) {
                if (r_global < p.rows) {
                    float *dst = p.scores + (((int64_t)cur.b * p.c.heads + h) * p.rows + r_global) * p.cap + base + 2 * j;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        *reinterpret_cast<float2 *>(dst + nt * 8) = make_float2(s[nt][0], s[nt][1]);
                }
            }
            // ---- running maximum, powers, sums
            float mx = m;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(s[nt][0], s[nt][1]));
            mx = quad_max(mx);
            const float ref = mx == -INFINITY ? 0.f : mx;     // nothing seen yet: every power is 0
            const float alpha = pow2(m - ref);
            m = mx;
            l *= alpha;
            uint32_t ph[NT / 2][4], pl[BF ? NT / 2 : 1][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float p0 = pow2(s[nt][0] - ref) * 0x1p15f, p1 = pow2(s[nt][1] - ref) * 0x1p15f;
                l += p0 + p1;
                uint32_t lo;
                split<T>(p0, p1, ph[nt / 2][(nt & 1) * 2], ph[nt / 2][(nt & 1) * 2 + 1], lo);
                if constexpr (BF) pl[nt / 2][nt & 1] = lo;
            }
            // ---- p v.  Entries that only some of the rows see must not reach the others even as 0 * Inf:
            // if one of them is not finite, the products run once per new token with the entries beyond its
            // view cleared, each row taking the pass of its own token.
            int pass = 0, passes = 1;
            const int seen = cur.len - n_new + 1;             // entries that every row sees
            if (n_new > 1 && base + TW > seen) {
                bool bad = false;
                const int e0 = max(seen, base) - base, e1 = min(cur.len, base + TW) - base;
                for (int e = max(e0, 0); e < e1; ++e)
                    for (int w = lane; w < DP / 2; w += 32) {
                        uint32_t v;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(vb + e * (DP * 2) + w * 4));
                        bad |= not_finite2<T>(v);
                    }
                if (__any_sync(0xffffffffu, bad)) passes = n_new;
            }
#pragma unroll 1
            for (; pass < passes; ++pass) {
                const int view = passes > 1 ? seen + pass : 0x7fffffff;
                const bool take = passes == 1 || limit == view;
                const float keep = take ? alpha : 1.f;
#pragma unroll
                for (int d2 = 0; d2 < DT / 2; ++d2) {
                    float a0[4] = {0.f, 0.f, 0.f, 0.f}, a1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < NT / 2; ++k) {
                        uint32_t b[4];
                        const int e = k * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, ch = d2 * 2 + (lane >> 4);
                        ldsm4t(b, vb + e * (DP * 2) + ((ch ^ (e & 7)) << 4));
                        if (passes > 1) {
                            const int tok = base + k * 16 + 2 * j;
                            const uint32_t m0 = (tok < view ? 0xffffu : 0u) | (tok + 1 < view ? 0xffff0000u : 0u);
                            const uint32_t m1 = (tok + 8 < view ? 0xffffu : 0u) | (tok + 9 < view ? 0xffff0000u : 0u);
                            b[0] &= m0, b[1] &= m1, b[2] &= m0, b[3] &= m1;
                        }
                        mma16816<T>(a0, ph[k][0], ph[k][1], ph[k][2], ph[k][3], b[0], b[1]);
                        mma16816<T>(a1, ph[k][0], ph[k][1], ph[k][2], ph[k][3], b[2], b[3]);
                        if constexpr (BF) {
                            mma16816<T>(a0, pl[k][0], 0u, pl[k][1], 0u, b[0], b[1]);
                            mma16816<T>(a1, pl[k][0], 0u, pl[k][1], 0u, b[2], b[3]);
                        }
                    }
                    o[2 * d2][0] = fmaf(o[2 * d2][0], keep, take ? a0[0] + a0[2] : 0.f);
                    o[2 * d2][1] = fmaf(o[2 * d2][1], keep, take ? a0[1] + a0[3] : 0.f);
                    o[2 * d2 + 1][0] = fmaf(o[2 * d2 + 1][0], keep, take ? a1[0] + a1[2] : 0.f);
                    o[2 * d2 + 1][1] = fmaf(o[2 * d2 + 1][1], keep, take ? a1[1] + a1[3] : 0.f);
                }
            }
        }
        if (tid < TILE) s_row[(i + 1) & 1][tid] = nrow;

        const AttnCursor was = cur;
        attn_advance<TILE>(p, cur);
        if (i + 1 < n_units && cur.tile != 0) continue;

        // ---- the segment's end (or this CTA's): join the warps that split its entries.  Their sums go
        // through the stage that was just used up: its next copies are issued after the next barrier.
        fresh = true;
        l = quad_sum(l);
        float *sums = reinterpret_cast<float *>(smem + stage * 2 * S::kHalf);
        __syncthreads();
        if (r_global < p.rows) {
            float *mine = sums + (warp * 8 + g) * S::kPad + 2 * j;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) *reinterpret_cast<float2 *>(mine + dt * 8) = make_float2(o[dt][0], o[dt][1]);
            if (j == 0) s_ml[warp][g] = make_float2(m, l);
        }
        __syncthreads();
        const int rows_here = min(ROWS, p.rows - rt * ROWS);
        const int64_t seg = (int64_t)was.b * p.c.heads + h;
        const bool whole = seg_base >= u0 && was.tile + 1 == was.tiles;
        // slot in the workspace of a part of a segment: 0 if it is the CTA's first, else 1
        const int64_t part = 2 * (int64_t)blockIdx.x + (seg_base > u0 ? 1 : 0);
        float *const ml_all = p.part + 2 * (int64_t)gridDim.x * ROWS * DP;
        auto out_row = [&](int r) {
            const int rg = rt * ROWS + r, t = rg / p.group;
            return p.out + (((int64_t)was.b * p.new_tokens + t) * p.c.heads * p.group + h * p.group + (rg - t * p.group)) * (int64_t)p.c.dim;
        };
        constexpr int C4 = DP / 4;                            // 16-byte pieces of a row
        for (int x = tid; x < rows_here * C4; x += THREADS) {
            const int r = x / C4, c4 = x % C4, w0 = r / 8;    // row r: warps w0, w0 + UG, ...
            float2 ml[TG];
            float top = -INFINITY, tot = 0.f;
#pragma unroll
            for (int k = 0; k < TG; ++k) {
                ml[k] = s_ml[w0 + k * UG][r & 7];
                top = fmaxf(top, ml[k].x);
            }
            const float ref = top == -INFINITY ? 0.f : top;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < TG; ++k) {
                const float w = pow2(ml[k].x - ref);
                const float4 v = *reinterpret_cast<const float4 *>(sums + ((w0 + k * UG) * 8 + (r & 7)) * S::kPad + c4 * 4);
                tot = fmaf(ml[k].y, w, tot);
                y.x = fmaf(v.x, w, y.x), y.y = fmaf(v.y, w, y.y), y.z = fmaf(v.z, w, y.z), y.w = fmaf(v.w, w, y.w);
            }
            if (whole) {
                const float inv = inverse(tot);
                if (c4 * 4 < p.c.dim)
                    *reinterpret_cast<float4 *>(out_row(r) + c4 * 4) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
                if (p.lse && c4 == 0) p.lse[seg * p.rows + rt * ROWS + r] = log_sum(top, tot);
            } else {
                *reinterpret_cast<float4 *>(p.part + (part * ROWS + r) * DP + c4 * 4) = y;
                if (c4 == 0) *reinterpret_cast<float2 *>(ml_all + (part * ROWS + r) * 2) = make_float2(top, tot);
            }
        }
        if (!whole) {
            // CTAs that hold tiles of the segment: those of its first and last tile, and all between
            const int c0 = (int)(((seg_base + 1ll) * G - 1) / W), c1 = (int)((((long long)seg_base + was.tiles) * G - 1) / W);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                int32_t *cnt = p.cnt + seg * p.row_tiles + rt;
                s_last = atomicAdd(cnt, 1) == c1 - c0;
                if (s_last) *cnt = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                // slot of CTA c: 1 only for the first, if the segment starts inside it
                const int first = 2 * c0 + (seg_base > (int)((long long)W * c0 / G) ? 1 : 0);
                auto slot_of = [&](int c) { return (int64_t)(c == c0 ? first : 2 * c); };
                for (int r = warp; r < rows_here; r += 4) {   // the rows' statistics, CTAs side by side
                    float top = -INFINITY, tot = 0.f;
                    for (int c = c0 + lane; c <= c1; c += 32) {
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(ml_all) + slot_of(c) * ROWS + r);
                        const float mx = fmaxf(top, ml.x), ref = mx == -INFINITY ? 0.f : mx;
                        tot = tot * pow2(top - ref) + ml.y * pow2(ml.x - ref);
                        top = mx;
                    }
                    float mx = top;
#pragma unroll
                    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    tot *= pow2(top - (mx == -INFINITY ? 0.f : mx));
#pragma unroll
                    for (int o = 16; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
                    if (lane == 0) {
                        s_row_ml[r] = make_float2(mx == -INFINITY ? 0.f : mx, inverse(tot));
                        if (p.lse) p.lse[seg * p.rows + rt * ROWS + r] = log_sum(mx, tot);
                    }
                }
                __syncthreads();
                // the sums: with few rows, groups of threads take every ways-th CTA each and join in shared memory
                const int items = rows_here * C4, ways = items <= THREADS / 4 ? 4 : items <= THREADS / 2 ? 2 : 1;
                const int per = THREADS / ways;
                for (int x0 = 0; x0 < items; x0 += per) {
                    const int x = x0 + tid % per, way = tid / per, r = x / C4, c4 = x % C4;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    float2 st = make_float2(0.f, 0.f);
                    if (x < items) {
                        st = s_row_ml[r];
#pragma unroll 8
                        for (int c = c0 + way; c <= c1; c += ways) {
                            const int64_t sl = slot_of(c) * ROWS + r;
                            const float w = pow2(__ldcg(ml_all + sl * 2) - st.x);
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part + sl * DP) + c4);
                            y.x = fmaf(v.x, w, y.x), y.y = fmaf(v.y, w, y.y), y.z = fmaf(v.z, w, y.z), y.w = fmaf(v.w, w, y.w);
                        }
                    }
                    if (ways > 1) {
                        float4 *way_sums = reinterpret_cast<float4 *>(sums);
                        way_sums[tid] = y;
                        __syncthreads();
                        if (way == 0)
                            for (int k = 1; k < ways; ++k) {
                                const float4 v = way_sums[tid + k * per];
                                y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
                            }
                    }
                    if (way == 0 && x < items && c4 * 4 < p.c.dim)
                        *reinterpret_cast<float4 *>(out_row(r) + c4 * 4) = make_float4(y.x * st.y, y.y * st.y, y.z * st.y, y.w * st.y);
                }
            }
        }
        seg_base = u0 + i + 1;
    }
}

// weight[entry] += sum over the rows of 2^(score - log-sum): one thread per
// entry reads its rows' saved scores (coalesced along the entries).
__global__ void __launch_bounds__(256) attn_weight_kernel(const AttnParams p)
{
    const int h = blockIdx.y, b = blockIdx.z;
    const int len = cache_len(p.c, b, KID_ATTN), slot = blockIdx.x * 256 + threadIdx.x;
    if (slot >= len) return;
    const int64_t seg = (int64_t)b * p.c.heads + h;
    const float *s = p.scores + seg * p.rows * p.cap + slot, *lse = p.lse + seg * p.rows;
    float w = 0.f;
#pragma unroll 4
    for (int r = 0; r < p.rows; ++r) w += attn::pow2(__ldg(s + r * p.cap) - __ldg(lse + r));
    const int col = p.page_div.of(slot), pg = cache_page(p.c, b, col, KID_ATTN);
    if (pg < 0) return;
    p.c.weight[((int64_t)pg * p.c.heads + h) * p.c.page_size + (slot - col * p.c.page_size)] += w;
}

struct AttnPlan {
    int dp, ug, rows, row_tiles, grid;
    int64_t tiles, cap, part_floats, score_floats, lse_floats, counters;
};

inline AttnPlan attn_plan(const mmq_kv_cache &c, int q_heads, int new_tokens, bool save)
{
    AttnPlan a;
    a.dp = c.dim <= 64 ? 64 : c.dim <= 128 ? 128 : 256;
    a.rows = q_heads / c.heads * new_tokens;
    // warps along the rows: as few as cover them, so that the others split the entries
    a.ug = a.rows <= 8 ? 1 : a.rows <= 16 ? 2 : 4;
    a.row_tiles = (a.rows + 8 * a.ug - 1) / (8 * a.ug);
    const int tile = a.dp == 64 ? 128 : 64;
    a.tiles = ((int64_t)c.cols * c.page_size + tile - 1) / tile * c.seqs * c.heads * a.row_tiles;
    const int64_t full = (int64_t)sm_count() * (a.dp <= 128 ? 2 : 1);     // every CTA resident
    a.grid = (int)(a.tiles < full ? a.tiles : full);
    a.cap = ((int64_t)c.cols * c.page_size + 127) / 128 * 128;
    a.part_floats = 2 * (int64_t)a.grid * 8 * a.ug * (a.dp + 2);
    a.score_floats = save ? (int64_t)c.seqs * c.heads * a.rows * a.cap : 0;
    a.lse_floats = save ? (int64_t)c.seqs * c.heads * a.rows : 0;
    a.counters = (int64_t)c.seqs * c.heads * a.row_tiles;
    return a;
}

inline int attn_check(const mmq_kv_cache *c, int q_heads, int new_tokens)
{
    const int rc = check_cache(c);
    if (rc != MMQ_OK) return rc;
    if (q_heads < 1 || q_heads > 65535 || q_heads % c->heads || new_tokens < 1 || new_tokens > 16) return MMQ_ERR_SHAPE;
    return MMQ_OK;
}

template <int DP, typename T, int UG>
int launch_attn(const AttnParams &p, int grid, cudaStream_t stream)
{
    const auto kernel = attn_kernel<DP, T, UG>;
    constexpr int smem = attn::Shape<DP>::kSmem;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return MMQ_ERR_ARCH;
    }
    static bool attr_done[64];
    if (!attr_done[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return launch_status();
        attr_done[dev] = true;
    }
    kernel<<<grid, attn::THREADS, smem, stream>>>(p);
    return launch_status();
}

template <int DP, typename T>
int launch_attn_ug(const AttnParams &p, const AttnPlan &a, cudaStream_t s)
{
    return a.ug == 1   ? launch_attn<DP, T, 1>(p, a.grid, s)
           : a.ug == 2 ? launch_attn<DP, T, 2>(p, a.grid, s)
                       : launch_attn<DP, T, 4>(p, a.grid, s);
}
template <typename T>
int launch_attn_dp(const AttnParams &p, const AttnPlan &a, cudaStream_t s)
{
    return a.dp == 64    ? launch_attn_ug<64, T>(p, a, s)
           : a.dp == 128 ? launch_attn_ug<128, T>(p, a, s)
                         : launch_attn_ug<256, T>(p, a, s);
}

}  // namespace
}  // namespace mmq

extern "C" int mmq_attn_sizes(const mmq_kv_cache *cache, int q_heads, int new_tokens, int accumulate,
                              int64_t *work_floats, int64_t *n_counters)
{
    using namespace mmq;
    const int rc = attn_check(cache, q_heads, new_tokens);
    if (rc != MMQ_OK) return rc;
    if (!work_floats || !n_counters) return MMQ_ERR_NULL;
    const AttnPlan a = attn_plan(*cache, q_heads, new_tokens, accumulate != 0);
    if (a.tiles > 0x7fffffff) return MMQ_ERR_SHAPE;
    *work_floats = a.part_floats + a.score_floats + a.lse_floats;
    *n_counters = a.counters;
    return MMQ_OK;
}

extern "C" int mmq_attn_decode(const mmq_kv_cache *cache, const float *q, int64_t ldq, const int32_t *new_len,
                               float *out, int q_heads, int new_tokens, float scale, int accumulate, float *work,
                               int32_t *counters, mmq_stream_t stream)
{
    using namespace mmq;
    int rc = attn_check(cache, q_heads, new_tokens);
    if (rc != MMQ_OK) return rc;
    if (ldq < (int64_t)q_heads * cache->dim || !(scale - scale == 0.f)) return MMQ_ERR_SHAPE;
    if (cache->seqs == 0) return MMQ_OK;
    if (!q || !out || !work || !counters || (accumulate && !cache->weight)) return MMQ_ERR_NULL;
    if (!aligned16(q) || (ldq & 3) || !aligned16(out) || !aligned16(work)) return MMQ_ERR_ALIGN;
    if ((rc = check_arch()) != MMQ_OK) return rc;
    const bool save = accumulate != 0;
    const AttnPlan a = attn_plan(*cache, q_heads, new_tokens, save);
    if (a.tiles > 0x7fffffff) return MMQ_ERR_SHAPE;       // tiles are counted in an int
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
    p.lse = save ? p.part + a.part_floats : nullptr;
    p.cnt = counters;
    p.cap = a.cap;
    p.page_div = FastDiv(cache->page_size);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    rc = cache->dtype == MMQ_F16 ? launch_attn_dp<__half>(p, a, s) : launch_attn_dp<__nv_bfloat16>(p, a, s);
    if (rc != MMQ_OK || !save) return rc;
    const dim3 grid((unsigned)(a.cap / 128 + 1) / 2, (unsigned)cache->heads, (unsigned)cache->seqs);
    attn_weight_kernel<<<grid, 256, 0, s>>>(p);
    return launch_status();
}
