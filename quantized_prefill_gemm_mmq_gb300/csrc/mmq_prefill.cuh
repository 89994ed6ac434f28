// mmq_prefill.cuh -- attention of any number of new tokens over the paged cache
// (mmq_attn_prefill), and of a tree of drafted tokens (mmq_attn_tree).
//
// Row i of a sequence (its slot) sees the slots lo <= j < hi, or for a tree all
// slots before the nodes and the nodes of its 64-bit word:
//     s = scale q.k;  s = cap tanh(s / cap);  s += slope (j - i)
//     p = exp(s - m),  out = sum p v / sum p
// in one pass over the entries with a running maximum m.  m is only raised where
// a tile's largest score lies more than 8 powers of two above it, so that the
// sums so far are multiplied again in few tiles.
//
// Work.  The `group` query heads that share a key-value head are rows beside the
// tokens: row r is token r / group and head r % group.  A unit is 128 or 256
// rows of one sequence and head.  What bounds it is the tensor core (4 dim flops
// per row and entry) for prompts, memory (4 dim bytes per entry and head) for
// few rows.
//
// Roles.  Q, K and V come through tensor copies (boxes of one page's entries; row
// by row with cp.async where pages or strides allow none) into a ring in shared
// memory, 128-byte swizzled.  S = Q K^T and O += P V run on the tensor core
// (tcgen05, sums in tensor memory), one thread per 128 rows issuing; V is used
// as it lies, its operand is the transposed form of the same swizzle.  One warp
// of every four reads S of 32 rows, one row per thread, writes P over it in the
// cache's type, and keeps maximum and sum in f32.  With 256 rows one K and V tile
// serves both halves, and the halves take turns on the tensor core; with up to
// 128 rows S has two buffers instead.  One loader warp finds the CTA's units and
// tells the others.
//
// Units.  Where they are many every CTA takes one, the longest first, and then
// those whose CTAs have not started (cluster launch control).  Otherwise all tiles
// of all units are numbered in a row and every CTA takes an equal part; units that
// are cut leave (max, sum, sum p v) in the workspace, and a second launch joins
// them in order.  No result depends on timing.
//
// What the time went to, and what it took (a prompt of 4096 rows of 32 heads of
// 128, f16, whose beginning sees itself whole; 149 GFLOP):
//   330 us  everything copied row by row, one issuing thread for both halves
//   232     tensor copies; registers moved from the other warps to the softmax
//   204     products issued under elect.sync: an issue took 156 cycles, 64 now; the
//           halves take turns (together they wait for scores, then for products)
//   181     Q, and tiles that rows see in part, by tensor copies as well
//   156     capped, biased and masked scores are worked over in tensor memory in a
//           rolled loop: unrolled, the code did not stay in the instruction cache
//   146     exponentials begin with the maximum so far; the softmax spills nothing
//           (local memory shares its path with the tensor core's operands: 604
//           bytes of it cost 30 to 70 %)
//   144     packed arithmetic under a cap, one chain for the maximum
//   138     the softmax's warp index uniform, and with it the barriers' addresses
//           (8192 rows under a cap 430 us before, 401 after)
// It is 1.08 PFLOP/s, 0.56 of cuBLAS' burst rate; 2048 rows of four heads over a
// window of 8192 entries, bf16, 235 us = 1.2 PFLOP/s (0.61), the tensor pipe 60 %
// active.  A tile of 256 rows took 3300 cycles (at 146 us), its products 2048: the chain scores
// -> exponentials -> P -> products of one half is longer than the other half's
// products.  Not kept: two threads per row (212 us: they swap maxima through shared
// memory, where a word takes some 200 cycles while operands are read), reading the
// scores twice instead of holding 128 of them (172), caps applied in registers
// (671 us and 442 for 8192 rows under a cap: code size again).  Trees of 48 nodes over 16 sequences of up to
// 16384 entries (8 heads of 128, groups of four) take 146 us = 4.4 TB/s, one token
// over 513 entries of 32 heads 20 us.
#pragma once

#include <type_traits>

namespace mmq {
namespace {

namespace pre {
constexpr int LOADERS = 2;            // warps
constexpr int PARTS = 2;              // of a tile's P, each announced by itself
constexpr int LAG = 2;                // copies a loader has under way before it waits for the oldest
constexpr int MAX_SLOTS = 12;
constexpr uint32_t SMEM = 232448;     // all of it dynamic

enum { W_Q = 1, W_K, W_V, W_P, W_S, W_EMPTY, W_QEMPTY, W_PV, W_TURN, W_SCAN, W_NEXT, W_RUN, W_DRAIN };     // sites of waits

// By whole warps; the lanes may wait for different barriers: a wait for one that is over already takes some 200 cycles while
// the tensor core reads shared memory, so several are better waited for in one go.
__device__ __forceinline__ bool wait(uint32_t bar, int parity, volatile uint32_t *abort, int site)
{
    if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, (uint32_t)parity, 1000))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)parity, abort, KID_PREFILL, site));
}

template <typename T>
constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
// p carries 2^kLift: f16 keeps 11 bits down to 2^-21 of the row's largest, and 2^(kLift + 8) still fits
template <typename T>
constexpr float kLift = kBf<T> ? 0.f : 7.f;
constexpr float kLazy = 8.f;

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t size)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 2^x to two ulp; 0 for -inf and where the result is below the normal range
__device__ __forceinline__ float pow2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A row's weights are 2^(s c + lifted(m)), or 2^((s - m) c + kLift) where m c is kLarge or more.
constexpr float kLarge = 4096.f;
template <typename T>
__device__ __forceinline__ float lifted(float m, float c) { return __fsub_rn(kLift<T>, __fmul_rn(m, c)); }
// By how much kLift - m c lies above that exponent, which is rounded twice (the product, the difference): below kLarge by up to
// 1.5 * 2^-12.
template <typename T>
__device__ __forceinline__ float lost(float m, float c)
{
    const float a = __fmul_rn(m, c);
    return fabsf(a) < kLarge ? (kLift<T> - (lifted<T>(m, c) + a)) - fmaf(m, c, -a) : 0.f;
}
// What sums of weights with the maximum m are multiplied by to go with the maximum `to`.  The exponents' roundings count:
// without them tiles before and after a raise, and parts that are joined, lie off by 2^-12 of a power of two against one
// another, a third of f16's rounding.
template <typename T>
__device__ __forceinline__ float rescale(float m, float to, float c)
{
    return pow2(fmaf(m - to, c, lost<T>(m, c) - lost<T>(to, c)));
}
// Asks for a CTA of this launch that has not started: its index comes to `at` (16 bytes) and counts on the barrier.
__device__ __forceinline__ void ask_next(uint32_t at, uint32_t bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(at), "r"(bar) : "memory");
}
// The answer: the index of the CTA whose work this one has taken over, or -1 when all have started.
__device__ __forceinline__ int answer(uint32_t at)
{
    uint32_t got, x = 0;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(got), "+r"(x)
        : "r"(at)
        : "memory");
    return got ? (int)x : -1;
}

// True in one thread of a converged warp, always the same.  Products issued under it take their descriptors from uniform
// registers; under lane == 0 each of them took 156 cycles to issue (64 to execute).
__device__ __forceinline__ bool elect()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// two at a time
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// the largest of three; a NaN does not count
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// NaN if one of them is
__device__ __forceinline__ float max3_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Columns of the warp's 32 lanes, to be used after tmem_ld_wait on each 32 of them.
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[32]) { tmem_ld32(at, r); }
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[64])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
                 "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
                 "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
                   "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
                   "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
                   "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
                   "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
                 : "r"(at)
                 : "memory");
}

// 32 scores (of the columns at `at`) under a cap, in powers of two: cap tanh(s / cap) = cap - 2 cap / (1 + e^(2 s / cap)).  Four share a reciprocal (8
// cycles a warp, an exponential 4); e^ is held below 2^30, where the fraction no longer counts, so that their product is
// finite, and a NaN, which that would hide, is looked for first.
__device__ __forceinline__ void cap32(uint32_t at, uint32_t (&y)[32], float cap_in, float cap_out)
{
    float nan = 0.f;
#pragma unroll
    for (int j = 0; j < 32; j += 2) nan = max3_nan(nan, __uint_as_float(y[j]), __uint_as_float(y[j + 1]));
    const bool any_nan = __any_sync(0xffffffffu, nan != nan);
    const uint64_t in2 = pair(cap_in, cap_in), one2 = pair(1.f, 1.f), out2 = pair(cap_out, cap_out);
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        // d = 1 + e^ of the elements 0 and 2, 1 and 3: the pairs' products are (lo, hi)
        float d[4];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            float a, b;
            unpair(mul2(pair(__uint_as_float(y[k + j]), __uint_as_float(y[k + j + 1])), in2), a, b);
            d[j] = fminf(pow2(a), 0x1p30f);
            d[j + 1] = fminf(pow2(b), 0x1p30f);
        }
        const uint64_t even = add2(pair(d[0], d[2]), one2), odd = add2(pair(d[1], d[3]), one2), both = mul2(even, odd);
        float lo, hi;
        unpair(both, lo, hi);
        const float r = rcp(lo * hi) * (-2.f * cap_out);
        const uint64_t inv = mul2(pair(hi, lo), pair(r, r));
        float z0, z1, z2, z3;
        unpair(fma2(inv, odd, out2), z0, z2);
        unpair(fma2(inv, even, out2), z1, z3);
        y[k] = __float_as_uint(z0);
        y[k + 1] = __float_as_uint(z1);
        y[k + 2] = __float_as_uint(z2);
        y[k + 3] = __float_as_uint(z3);
    }
    if (any_nan) {
        uint32_t was[32];
        tmem_ld32(at, was);
        tmem_ld_wait(was);
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = was[j] << 1 > 0xff000000u ? was[j] : y[j];
    }
}

__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// eight columns of the warp's lanes times f
__device__ __forceinline__ void scale8(uint32_t at, float f)
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at)
                 : "memory");
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * f);
    tmem_st8(at, r);
}

// 32 bytes to where 16 or (wide) 32 bytes are aligned: a whole sector by one thread
__device__ __forceinline__ void store32(void *dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f, uint32_t g, uint32_t h,
                                        int wide)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g),
                     "r"(h)
                     : "memory");
    } else {
        static_cast<uint4 *>(dst)[0] = make_uint4(a, b, c, d);
        static_cast<uint4 *>(dst)[1] = make_uint4(e, f, g, h);
    }
}

// kind::f16 descriptor: f16 or bf16 operands, f32 sums, A K-major; B K-major or (mn) with its N values contiguous
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool mn)
{
    return (1u << 4) | ((kBf<T> ? 1u : 0u) << 7) | ((kBf<T> ? 1u : 0u) << 10) | ((mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Operand whose N values lie contiguous, 64 to a 128-byte swizzled row of one k: eight rows are an atom of 1024 bytes,
// the next eight k follow it, the next 64 values of N are `chunk` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr, uint32_t chunk)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)((chunk >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
}  // namespace pre

struct PrefillParams {
    mmq_kv_cache c;
    const void *q;
    const int32_t *new_len, *prefix, *first;
    const uint64_t *tree;
    const float *slopes;
    void *out;
    int64_t ldq;
    float scale_log2;          // scale * log2(e)
    float cap_in, cap_out;     // 2 log2(e) scale / cap, cap log2(e); cap_out 0: no cap
    int out_f32, window;
    int out_wide, part_wide;   // rows of out, and of the parts, begin on 32 bytes
    int new_tokens, group, q_heads;
    int rows, row_tiles;       // rows per sequence and key-value head, units of them
    int whole;                 // one unit per CTA
    int part_rows;             // rows of a part
    int chunks, ksteps;        // 64-value pieces and 16-value steps of a head
    int slots;                 // of the ring
    int box;                   // rows of a tensor copy, 0: none are used
    float *part;               // [2*grid][part_rows][dim], then [2*grid][part_rows] (max, sum), then [grid] int2 (unit, last CTA)
    float2 *part_ml;
    int2 *joins;
    FastDiv page_div, group_div;
    int q_box;                 // q rows come by tensor copies
    int withhold;              // test-only: the last K tile of a run never comes
    CUtensorMap k_map, v_map;  // [pages][heads][page_size][dim], boxes of 64 values of `box` entries
    CUtensorMap q_map;         // [rows][q_heads][dim], boxes of 64 values of a group's heads of 128/group tokens
};

// What a unit's rows see.
struct PrefillRow {
    int lo, hi;
};

struct PrefillUnit {
    int b, h, rt;
    int len, n, ctx, prefix;   // ctx: entries before the new ones; prefix 0 for none
    int t0, t1;                // tiles
    int max_lo, min_hi;        // every live row sees max_lo <= j < min_hi
};

__device__ __forceinline__ PrefillRow prefill_row(const PrefillParams &p, const PrefillUnit &u, int t, bool with_first)
{
    PrefillRow r;
    const int i = u.ctx + t;
    r.hi = p.tree ? u.len : max(i + 1, u.prefix);
    r.lo = p.window > 0 ? max(0, i - p.window + 1) : 0;
    if (with_first && p.first) r.lo = max(r.lo, *(p.first + (int64_t)u.b * p.new_tokens + t));
    return r;
}

// Lengths and counts of sequence b: the loads first, then their checks.
__device__ __forceinline__ void prefill_sequence(const PrefillParams &p, PrefillUnit &u)
{
    const int len = *(p.c.len + u.b), n = p.new_len ? *(p.new_len + u.b) : p.new_tokens, prefix = p.prefix ? *(p.prefix + u.b) : 0;
    const int cap = p.c.cols * p.c.page_size;
    u.len = (unsigned)len <= (unsigned)cap ? len : 0;
    u.n = min(max(n, 0), p.new_tokens);
    if (u.len != len || u.n != n || u.n > u.len) {
        record_error(MMQ_ERR_INDEX, KID_PREFILL, u.n != n ? SITE_COUNT : SITE_LEN);
        if (u.n > u.len) u.n = 0;                 // more new tokens than entries: none of them is there
    }
    u.ctx = u.len - u.n;
    u.prefix = min(max(prefix, 0), u.len);
}

// Tiles of unit (b, rt) as far as lengths, window and prefix say: the same for every head, and without reading `first`.
template <int RT, int TN>
__device__ __forceinline__ int2 prefill_span(const PrefillParams &p, const PrefillUnit &u)
{
    const int ta = p.group_div.of(u.rt * RT), tb = min(p.group_div.of(min(p.rows, (u.rt + 1) * RT) - 1), u.n - 1);
    if (ta > tb) return make_int2(0, 0);
    const int lo = prefill_row(p, u, ta, false).lo, hi = prefill_row(p, u, tb, false).hi;
    return lo < hi ? make_int2(lo / TN, (hi + TN - 1) / TN) : make_int2(0, 0);
}

// The unit's tiles within [t0, t1), and what all of its rows see; by a whole warp.
template <int RT, int TN>
__device__ __forceinline__ void prefill_bounds(const PrefillParams &p, PrefillUnit &u)
{
    const int ta = p.group_div.of(u.rt * RT), tb = min(p.group_div.of(min(p.rows, (u.rt + 1) * RT) - 1), u.n - 1);
    int lo = 0x7fffffff;
    u.max_lo = 0;
    u.min_hi = 0x7fffffff;
    if (ta > tb) {
        u.t0 = u.t1 = 0;
        return;
    }
    if (p.first) {
        for (int t = ta + (int)(threadIdx.x & 31); t <= tb; t += 32) {
            const PrefillRow r = prefill_row(p, u, t, true);
            lo = min(lo, r.lo);
            u.max_lo = max(u.max_lo, r.lo);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        u.max_lo = __reduce_max_sync(0xffffffffu, u.max_lo);
    } else {
        lo = prefill_row(p, u, ta, false).lo;
        u.max_lo = prefill_row(p, u, tb, false).lo;
    }
    const int hi = prefill_row(p, u, tb, false).hi;
    u.min_hi = p.tree ? u.ctx : prefill_row(p, u, ta, false).hi;
    u.t0 = max(u.t0, lo / TN);
    u.t1 = min(u.t1, (hi + TN - 1) / TN);
    if (lo >= hi || u.t0 >= u.t1) u.t0 = u.t1 = 0;
}

// Runs of tiles that a CTA takes, one unit (or part of one) after the other; one loader warp finds them and tells the other
// warps.  Units are numbered (sequence, rows, head): the heads of one (sequence, rows) pair have the same span of tiles.
template <int RT, int TN>
struct PrefillWalk {
    PrefillUnit u;
    int left;                  // tiles still to come
    int at;                    // tile within the unit's span where the next run starts
    int2 span;
    bool begins, ends;         // the run has the unit's first, last tile
    int each, extra;           // split: CTA c has each + (c < extra) tiles of all units
    int place;                 // split: tiles of all units up to the run's end
    int rest;                  // tiles of the unit after the run
    int asked;                 // whole: units taken over

    __device__ __forceinline__ static int count(int2 s) { return max(1, s.y - s.x); }        // an empty unit still has outputs

    __device__ __forceinline__ void split(const PrefillParams &p)
    {
        const int lane = threadIdx.x & 31, pairs = p.c.seqs * p.row_tiles;
        auto tiles_of = [&](int i) {
            if (i >= pairs) return 0;
            PrefillUnit w;
            w.b = i / p.row_tiles;
            w.rt = i - w.b * p.row_tiles;
            prefill_sequence(p, w);
            return count(prefill_span<RT, TN>(p, w));
        };
        at = place = 0;
        const int first32 = tiles_of(lane);
        int W = first32;
        for (int i = lane + 32; i < pairs; i += 32) W += tiles_of(i);
        W = __reduce_add_sync(0xffffffffu, W) * p.c.heads;
        each = W / (int)gridDim.x;
        extra = W - each * (int)gridDim.x;
        place = each * (int)blockIdx.x + min((int)blockIdx.x, extra);
        left = each + ((int)blockIdx.x < extra ? 1 : 0);
        if (left == 0) return;
        int before = 0;                                       // tiles before pair i0
        for (int i0 = 0;; i0 += 32) {
            const int mine = i0 == 0 ? first32 : tiles_of(i0 + lane);
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + upto * p.c.heads > place);
            if (past) {
                const int f = __ffs(past) - 1, each = __shfl_sync(0xffffffffu, mine, f);
                const int rem = place - before - (__shfl_sync(0xffffffffu, upto, f) - each) * p.c.heads;
                u.b = (i0 + f) / p.row_tiles;
                u.rt = i0 + f - u.b * p.row_tiles;
                u.h = rem / each;
                at = rem - u.h * each;
                break;
            }
            before += __shfl_sync(0xffffffffu, upto, 31) * p.c.heads;
        }
        prefill_sequence(p, u);
        span = prefill_span<RT, TN>(p, u);
    }

    // The CTA that has tile x.
    __device__ __forceinline__ int owner(int x) const
    {
        const int first = (each + 1) * extra;
        return x < first ? x / (each + 1) : extra + (x - first) / each;
    }

    // The next run of a CTA with an equal share of all tiles, false when there is none.
    __device__ __forceinline__ bool next_split(const PrefillParams &p, bool first)
    {
        if (left <= 0) return false;
        if (!first) {
            at = 0;
            if (++u.h == p.c.heads) {
                u.h = 0;
                if (++u.rt == p.row_tiles) {
                    u.rt = 0;
                    ++u.b;
                    prefill_sequence(p, u);
                }
                span = prefill_span<RT, TN>(p, u);
            }
        }
        const int all = count(span), take = min(left, all - at);
        begins = at == 0;
        ends = at + take == all;
        left -= take;
        place += take;
        rest = all - at - take;
        u.t0 = span.x + at;
        u.t1 = min(span.y, span.x + at + take);
        prefill_bounds<RT, TN>(p, u);
        return true;
    }

    // The next whole unit: the CTA's own, then those whose CTAs have not started.  It asks when its copies for the unit
    // before are on their way: asked a unit ahead, long units wait for busy CTAs.  -1: none left, -2: a wait ran out.
    __device__ __forceinline__ int next_whole(const PrefillParams &p, bool first, uint32_t answer_at, uint32_t bar, volatile uint32_t *abort)
    {
        int id = (int)blockIdx.x;
        if (!first) {
            if ((threadIdx.x & 31) == 0) {
                mbar_arrive_expect_tx(bar, 16);
                pre::ask_next(answer_at, bar);
            }
            __syncwarp();
            if (!pre::wait(bar, asked & 1, abort, pre::W_NEXT)) return -2;
            id = pre::answer(answer_at);
            fence_proxy_async_smem();
            __syncwarp();
            ++asked;
            if (id < 0) return -1;
        }
        const int per = p.c.seqs * p.c.heads, back = id / per, bh = id - back * per;
        u.rt = p.row_tiles - 1 - back;                        // the longest first
        u.b = bh / p.c.heads;
        u.h = bh - u.b * p.c.heads;
        prefill_sequence(p, u);
        span = prefill_span<RT, TN>(p, u);
        begins = ends = true;
        u.t0 = span.x;
        u.t1 = span.y;
        prefill_bounds<RT, TN>(p, u);
        return 0;
    }
};

// What the warps of a CTA are told of a run.
struct PrefillRun {
    PrefillUnit u;
    int flags;                 // 1: has the unit's first tile, 2: its last, 4: there is none any more
};

template <typename T, int NQ, int TN>
struct PrefillShape {
    static constexpr int RT = 128 * NQ;
    static constexpr int SOFT = 4 * NQ;                        // softmax warps; then two issuing and two loading ones
    static constexpr int kThreads = (SOFT + 4) * 32;
    static constexpr int kBuf = 2;                             // S buffers: one per half, or two for the only half
    static constexpr int kO = kBuf * TN;                       // tensor-memory column of the sums
    static constexpr int kOPitch = (512 - kO) / NQ;
    static constexpr int kMaxDim = kOPitch < 256 ? kOPitch / 64 * 64 : 256;
};

// Shared memory behind the tiles.
template <int NQ, int TN>
struct PrefillShared {
    static constexpr int RUNS = 3;
    uint64_t q_full, q_empty, drain[2];
    uint64_t full[pre::MAX_SLOTS], empty[pre::MAX_SLOTS];
    uint64_t s[2], pv[2], turn[2], scan[2], p[2 * pre::PARTS];          // p [S buffer][part of P]
    uint64_t run_full[RUNS], run_empty[RUNS], next;
    uint64_t pad;
    uint4 answer;
    PrefillRun run[RUNS];
    uint32_t bad[pre::MAX_SLOTS][TN / 32];                     // entries of a V tile that were not finite and are taken as 0
    uint32_t tmem, abort;
};

template <typename T, int NQ, int TN>
__global__ void __launch_bounds__(PrefillShape<T, NQ, TN>::kThreads, 1) prefill_kernel(const __grid_constant__ PrefillParams p)
{
    using namespace pre;
    using S = PrefillShape<T, NQ, TN>;
    using Shared = PrefillShared<NQ, TN>;
    constexpr int RT = S::RT, SOFT = S::SOFT;
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t base = smem_u32(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t q_bytes = (uint32_t)p.chunks * (128 * 128), slot_bytes = (uint32_t)p.chunks * (TN * 128);
    const uint32_t ring = base + NQ * q_bytes;
    Shared &sh = *reinterpret_cast<Shared *>(raw + NQ * q_bytes + p.slots * slot_bytes);
    volatile uint32_t *abort = &sh.abort;
    auto bar = [&](uint64_t &b) { return smem_u32(&b); };

    if (threadIdx.x == 0) {
        sh.abort = 0;
        mbar_init(bar(sh.q_full), LOADERS);
        mbar_init(bar(sh.q_empty), NQ);
        for (int i = 0; i < MAX_SLOTS; ++i) {
            mbar_init(bar(sh.full[i]), LOADERS);
            mbar_init(bar(sh.empty[i]), NQ);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(sh.drain[i]), 1);
            mbar_init(bar(sh.s[i]), 1);
            mbar_init(bar(sh.pv[i]), 1);
            mbar_init(bar(sh.turn[i]), 1);
            mbar_init(bar(sh.scan[i]), 4);
            for (int k = 0; k < PARTS; ++k) mbar_init(bar(sh.p[i * PARTS + k]), 4);
        }
        for (int i = 0; i < Shared::RUNS; ++i) {
            mbar_init(bar(sh.run_full[i]), 1);
            mbar_init(bar(sh.run_empty[i]), SOFT + NQ + 1);
        }
        mbar_init(bar(sh.next), 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {                                   // the maps are part of the launch
        if (p.q_box) tma_prefetch(&p.q_map);
        if (p.box) {
            tma_prefetch(&p.k_map);
            tma_prefetch(&p.v_map);
        }
    }
    // Tensor memory is taken after the launch before has ended: its blocks may still have to take theirs.
    pdl_wait();
    if (warp == SOFT) {
        tmem_alloc(smem_u32(&sh.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = *(volatile uint32_t *)&sh.tmem;

    // The next run, as told; false at the end, or when a wait ran out.
    int run_at = 0, run_phase = 0;
    auto hear = [&](PrefillRun &r) {
        if (!wait(bar(sh.run_full[run_at]), run_phase, abort, W_RUN)) return false;
        r = sh.run[run_at];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.run_empty[run_at]));
        if (++run_at == Shared::RUNS) run_at = 0, run_phase ^= 1;
        return (r.flags & 4) == 0;
    };

    if (warp < SOFT) {
        // ------------------------------------------------------------------ softmax: one row per thread
        // With 256 rows these warps need more registers than an equal share (168): 2 * 216 + 72 = 3 * 168.
        if (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int soft = __shfl_sync(0xffffffffu, warp, 0);    // uniform: the barriers' addresses are, then
        const int half = soft >> 2, quarter = soft & 3, in_half = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t o_col = tmem + lanes + S::kO + half * S::kOPitch;
        const bool general = p.cap_out != 0.f || p.slopes || !(p.scale_log2 > 0.f);
        const float c = general ? 1.f : p.scale_log2;
        int g = 0, runs = 0, scans = 0, vslot = 1, vphase = 0;
        PrefillRun run;
        while (hear(run)) {
            const PrefillUnit &u = run.u;
            const int r = u.rt * RT + half * 128 + in_half;
            const int t = p.group_div.of(min(r, p.rows - 1));
            const bool live = r < p.rows && t < u.n;
            const int head = u.h * p.group + (min(r, p.rows - 1) - t * p.group);
            PrefillRow see = {0, 0};
            if (live) see = prefill_row(p, u, t, true);
            uint64_t word = 0;
            if (p.tree && live) {
                word = p.tree[(int64_t)u.b * p.new_tokens + t];
                if (u.n < 64) word &= (1ull << u.n) - 1;
                see.hi = u.ctx;
            }
            const bool any = __any_sync(0xffffffffu, live);
            // what every live row of this warp sees
            const int max_lo = __reduce_max_sync(0xffffffffu, live ? see.lo : 0);
            const int min_hi = __reduce_min_sync(0xffffffffu, live ? see.hi : 0x7fffffff);
            const float slope = p.slopes && live ? p.slopes[head] * 1.44269504088896341f : 0.f;
            float m = -INFINITY, l = 0.f, off = kLift<T>;      // off: lifted(m)
            bool poison = false, any_large = false;            // any_large: of the warp, see below

            for (int tile = u.t0; tile < u.t1; ++tile, ++g) {
                const int sb = NQ == 2 ? half : g & 1, sph = NQ == 2 ? g & 1 : (g >> 1) & 1;
                const uint32_t s_col = tmem + lanes + sb * TN;
                const int e0 = tile * TN;
                auto sees = [&](int k) {                       // which of the tile's 32 entries from the k-th on this row sees
                    const int a = min(max(see.lo - e0 - k, 0), 32), z = min(max(see.hi - e0 - k, 0), 32);
                    const uint32_t from = a == 32 ? 0u : 0xffffffffu << a, to = z == 32 ? 0xffffffffu : (1u << z) - 1u;
                    uint32_t nodes = 0;
                    if (p.tree) {
                        const int d = e0 + k - u.ctx;          // node of the first of them
                        if (d >= 0 && d < 64) nodes = (uint32_t)(word >> d);
                        else if (d < 0 && d > -32) nodes = (uint32_t)(word << -d);
                    }
                    return from & (to | nodes);
                };
                // In a tile that some row of the unit sees in part only, entries of V that are not finite are taken as 0
                // (0 times them would be NaN in rows that do not see them) and noted: a row that sees one is not finite.
                // The halves both look, and both take away what either has noted (a half that comes second may find zeros
                // already): a half's product reads V after that half's own stores, fenced before its P is announced.
                const bool scan = e0 < u.max_lo || e0 + TN > u.min_hi;
                if (scan) {
                    if (!wait(bar(sh.full[vslot]), vphase, abort, W_V)) goto done;
                    constexpr int PER = 128 / TN;              // threads per entry
                    const int at = in_half, e = at / PER;
                    const uint32_t row = ring + vslot * slot_bytes + e * 128;
                    auto piece = [&](int k) { return row + (k >> 3) * (TN * 128) + (((k & 7) ^ (e & 7)) << 4); };
                    uint32_t acc = 0;
#pragma unroll 1
                    for (int k = at % PER; k < p.c.dim / 8; k += PER) {
                        uint32_t v[4];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(piece(k)) : "memory");
                        constexpr uint32_t one = kBf<T> ? 0x00800080u : 0x04000400u;       // on top of a full exponent: bit 15
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc |= (v[i] & 0x7fff7fffu) + one;
                    }
                    if ((acc & 0x80008000u) != 0) atomicOr(&sh.bad[vslot][e >> 5], 1u << (e & 31));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(sh.scan[half]));
                    if (!wait(bar(sh.scan[half]), scans & 1, abort, W_SCAN)) goto done;
                    ++scans;
                    bool mine = false;                         // this thread's entry is noted
#pragma unroll 1
                    for (int k = 0; k < TN; k += 32) {
                        const uint32_t bad = *(volatile uint32_t *)&sh.bad[vslot][k / 32];
                        poison |= (bad & sees(k)) != 0;
                        if ((e & ~31) == k) mine = (bad >> (e & 31) & 1u) != 0;
                    }
                    if (mine) {
                        for (int k = at % PER; k < p.c.dim / 8; k += PER)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(piece(k)), "r"(0u) : "memory");
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                }
                vslot += 2;
                if (vslot >= p.slots) {
                    vslot -= p.slots;
                    vphase ^= 1;
                }
                if (!wait(bar(sh.s[sb]), sph, abort, W_S)) goto done;
                tc_fence_after();
                // With two S buffers the scores come before the last tile's product has been added.  Its barrier is waited for in
                // every tile before P is announced: one that is left out would be taken for the next but one.
                auto added = [&]() {
                    const bool ok = g == 0 || wait(bar(sh.pv[0]), (g - 1) & 1, abort, W_PV);
                    tc_fence_after();
                    return ok;
                };
                if (!any) {
                    if (NQ == 1 && !added()) goto done;
                    tc_fence_before();
                    __syncwarp();
                    if (lane < PARTS) mbar_arrive(bar(sh.p[sb * PARTS + lane]));
                    continue;
                }
                // Scores that need more than the plain softmax are worked over where they lie, 32 at a time: few tiles (or all,
                // with a cap or a bias), and unrolled beside the rest the code would not stay in its cache.
                const bool cut = e0 < max_lo || e0 + TN > min_hi;
                if (general || cut) {
#pragma unroll 1
                    for (int k = 0; k < TN; k += 32) {
                        const bool cut32 = e0 + k < max_lo || e0 + k + 32 > min_hi;
                        if (!general && !cut32) continue;
                        uint32_t y[32];
                        tmem_ld32(s_col + k, y);
                        tmem_ld_wait(y);
                        if (p.cap_out != 0.f) cap32(s_col + k, y, p.cap_in, p.cap_out);
                        else if (general)
#pragma unroll
                            for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * p.scale_log2);
                        if (p.slopes) {
                            const float bias = slope * (float)(e0 + k - u.ctx - t);
#pragma unroll
                            for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) + fmaf(slope, (float)j, bias));
                        }
                        if (cut32) {
                            const uint32_t bits = sees(k);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!(bits >> j & 1u)) y[j] = 0xff800000u;
                        }
                        tmem_st32(s_col + k, y);
                    }
                    tmem_st_wait();
                }
                // Scores are read once: the tensor core's own traffic in tensor memory goes first.  The first part's exponentials
                // are begun with the maximum so far, while the tile's is found; where that has to be raised, which is rare, they
                // are done again.
                constexpr int W = TN / PARTS;
                uint32_t x[TN];
                auto load = [&](int part) { tmem_ld(s_col + part * W, reinterpret_cast<uint32_t(&)[W]>(x[part * W])); };
                auto loaded = [&](int part) {
#pragma unroll
                    for (int k = part * W; k < (part + 1) * W; k += 32) tmem_ld_wait(reinterpret_cast<uint32_t(&)[32]>(x[k]));
                };
                float top;
                auto largest = [&](int k0, int k1) {
#pragma unroll
                    for (int k = k0; k < k1; k += 2) top = max3(top, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                };
                uint64_t sum;
                float by = c, add = off;
                auto power = [&](int k0, int k1) {             // scores to P, in place of the first half of them
#pragma unroll
                    for (int j = k0; j < k1; j += 2) {
                        const float a = pow2(fmaf(__uint_as_float(x[j]), by, add)), b = pow2(fmaf(__uint_as_float(x[j + 1]), by, add));
                        sum = add2(sum, pair(a, b));
                        x[j / 2] = pack2<T>(a, b);
                    }
                };
#pragma unroll 1
                for (bool again = false;; again = true) {
                    load(0);
                    loaded(0);
                    load(1);                                   // under way during the first part's exponentials
                    top = -INFINITY;
                    largest(0, W);
                    sum = 0;
                    power(0, W);
                    loaded(1);
                    largest(W, TN);
                    const float mx = top;
                    const bool raise = mx > m && !((mx - m) * c <= kLazy);
                    if (again || !__any_sync(0xffffffffu, raise || any_large)) break;
                    float f = 1.f;
                    if (raise) {
                        f = rescale<T>(m, mx, c);
                        m = mx;
                        l *= f;
                        off = lifted<T>(m, c);
                    }
                    const bool large = m != -INFINITY && !(fabsf(m * c) < kLarge);
                    any_large = __any_sync(0xffffffffu, large);
                    if (tile != u.t0 && __any_sync(0xffffffffu, raise)) {
                        if (NQ == 1 && !added()) goto done;    // the last product may still be adding
#pragma unroll 1
                        for (int d = 0; d < p.ksteps * 16; d += 8) scale8(o_col + d, f);
                    }
                    add = off;
                    if (any_large) {                           // m is taken off first in rows of such scores, and in these alone
#pragma unroll 1
                        for (int k = 0; k < TN; k += 32) {
                            uint32_t y[32];
                            tmem_ld32(s_col + k, y);
                            tmem_ld_wait(y);
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float s = __uint_as_float(y[j]);
                                y[j] = __float_as_uint(large ? fmaf(s - m, c, kLift<T>) : fmaf(s, c, off));
                            }
                            tmem_st32(s_col + k, y);
                        }
                        tmem_st_wait();
                        by = 1.f;
                        add = 0.f;
                    }
                }
                // P goes over scores that are read; a part is announced once it is stored, which the next exponentials cover.
                auto store = [&](int part) {
#pragma unroll
                    for (int k = part * W / 2; k < (part + 1) * W / 2; k += 16) tmem_st16(s_col + k, reinterpret_cast<uint32_t(&)[16]>(x[k]));
                };
                auto stored = [&](int part) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(sh.p[sb * PARTS + part]));
                };
                static_assert(PARTS == 2, "two parts");
                if (NQ == 1 && !added()) goto done;
                store(0);
                power(W, W + W / 2);
                stored(0);
                power(W + W / 2, TN);
                store(1);
                stored(1);
                float la, lb;
                unpair(sum, la, lb);
                l += la + lb;
            }

            // the run's sums
            const bool some = u.t0 < u.t1;
            if (some) {
                if (!wait(bar(sh.pv[half]), NQ == 2 ? runs & 1 : (g - 1) & 1, abort, W_PV)) goto done;
                tc_fence_after();
                ++runs;
            }
            if (poison) l = NAN;
            if (!live) l = 0.f;
            const bool whole = (run.flags & 3) == 3;
            const int64_t row = ((int64_t)u.b * p.new_tokens + t) * p.q_heads + head;
            const int64_t part = (2ll * blockIdx.x + (run.flags & 1)) * p.part_rows + half * 128 + in_half;
            const float f = !whole ? 1.f : l > 0.f ? 1.f / l : l;   // a NaN stays one
            const bool sums = some && !(l == 0.f);
            if (__any_sync(0xffffffffu, r < p.rows)) {
                const bool wide = whole ? p.out_wide : p.part_wide;
#pragma unroll 1
                for (int d = 0; d < p.c.dim; d += 32) {
                    uint32_t o[32];                            // the columns past the last are there, whatever they hold
                    if (some) {
                        tmem_ld32(o_col + d, o);
                        tmem_ld_wait(o);
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = sums ? __float_as_uint(__uint_as_float(o[k]) * f) : 0u;
                    if (r < p.rows) {
                        if (!whole || p.out_f32) {
                            float *dst = whole ? static_cast<float *>(p.out) + row * p.c.dim : p.part + part * p.c.dim;
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                if (d + e < p.c.dim) store32(dst + d + e, o[e], o[e + 1], o[e + 2], o[e + 3], o[e + 4], o[e + 5], o[e + 6], o[e + 7], wide);
                        } else {
                            T *dst = static_cast<T *>(p.out) + row * p.c.dim;
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = pack2<T>(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
#pragma unroll
                            for (int e = 0; e < 32; e += 16) {
                                const int k = e / 2;
                                if (d + e + 8 < p.c.dim)
                                    store32(dst + d + e, o[k], o[k + 1], o[k + 2], o[k + 3], o[k + 4], o[k + 5], o[k + 6], o[k + 7], wide);
                                else if (d + e < p.c.dim)
                                    *reinterpret_cast<uint4 *>(dst + d + e) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (!whole && r < p.rows) p.part_ml[part] = make_float2(m, l);
            }
            tc_fence_before();
        }
    } else {
        // The other four warps give up theirs in one instruction, as a warpgroup has to.
        if (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp < SOFT + 2) {
            // ------------------------------------------------------------------ one thread per half issues its products
            constexpr uint32_t kIdS = idesc<T>(TN, false);
            const uint32_t id_o = idesc<T>(p.ksteps * 16, true);
            const int i = __shfl_sync(0xffffffffu, warp, 0) - SOFT;    // the half, uniform; with one half the second warp has nothing to do
            int g = 0, runs = 0, slot = 0, phase = 0;              // slot: of the next tile's K
            constexpr int KSTEPS = S::kMaxDim / 16;
            auto product_s = [&](int sb, int at, bool last) {      // S buffer sb, K in slot `at`
                const uint64_t a = sdesc_k_sw128(base + i * q_bytes), b = sdesc_k_sw128(ring + at * slot_bytes);
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < KSTEPS; ++k)
                        if (k < p.ksteps)
                            umma_f16(tmem + sb * TN, a + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                                     b + (((k >> 2) * (TN * 128) + (k & 3) * 32) >> 4), kIdS, k > 0);
                    umma_commit(bar(sh.s[sb]));
                    umma_commit(bar(sh.empty[at]));
                    if (last) umma_commit(bar(sh.q_empty));
                }
                __syncwarp();
            };
            auto product_o = [&](int sb, int at, int part, bool add, bool last) {
                constexpr int STEPS = TN / 16 / PARTS;
                const uint64_t b = sdesc_mn_sw128(ring + at * slot_bytes + part * STEPS * 2048, TN * 128);
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < STEPS; ++k)
                        umma_f16_ts(tmem + S::kO + i * S::kOPitch, tmem + sb * TN + 8 * (part * STEPS + k), b + ((k * 2048) >> 4), id_o,
                                    add || k > 0);
                    if (part == PARTS - 1) {
                        umma_commit(bar(sh.empty[at]));
                        if (last) umma_commit(bar(sh.pv[i]));
                    }
                }
                __syncwarp();
            };
            auto waits = [&](uint64_t &b, int parity, int site) {
                const bool ok = wait(bar(b), parity, abort, site);
                tc_fence_after();
                return ok;
            };
            auto work = [&](int nt) {
                if (!waits(sh.q_full, runs & 1, W_Q) || !waits(sh.full[slot], phase, W_K)) return false;
                product_s(NQ == 2 ? i : g & 1, slot, nt == 1);
                for (int j = 0; j < nt; ++j, ++g) {
                    int vs = slot + 1, vp = phase;
                    if (vs >= p.slots) vs = 0, vp ^= 1;
                    int ks = vs + 1, kp = vp;
                    if (ks >= p.slots) ks = 0, kp ^= 1;
                    const bool more = j + 1 < nt;
                    const int sb = NQ == 2 ? i : g & 1;
                    // V and the next K are waited for before P, so that nothing but P holds the products up.  The halves take
                    // turns, a tile's products at a time: otherwise both wait for scores, then both for the tensor core.
                    if (!waits(sh.full[vs], vp, W_V)) return false;
                    if (more && !waits(sh.full[ks], kp, W_K)) return false;
                    if (NQ == 1 && more) product_s((g + 1) & 1, ks, j + 2 == nt);      // while this tile's scores are worked on
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        if (!waits(sh.p[sb * PARTS + part], NQ == 2 ? g & 1 : (g >> 1) & 1, W_P)) return false;
                        if (NQ == 2 && part == 0 && !waits(sh.turn[i], i == 0 ? (g & 1) ^ 1 : g & 1, W_TURN)) return false;
                        product_o(sb, vs, part, j > 0 || part > 0, NQ == 1 || !more);
                    }
                    if (NQ == 2) {
                        if (more) product_s(sb, ks, j + 2 == nt);
                        if (lane == 0) mbar_arrive(bar(sh.turn[i ^ 1]));
                        __syncwarp();
                    }
                    slot = ks;
                    phase = kp;
                }
                ++runs;
                return true;
            };
            if (i < NQ) {
                PrefillRun run;
                while (hear(run)) {
                    const int nt = run.u.t1 - run.u.t0;
                    if (nt > 0 && !work(nt)) break;
                }
                if (elect()) umma_commit(bar(sh.drain[i]));        // nothing is under way when tensor memory is given back
                __syncwarp();
                uint32_t never = 0;
                mbar_wait_warp(bar(sh.drain[i]), 0, &never, KID_PREFILL, W_DRAIN);
            }
        } else {
            // ------------------------------------------------------------------ loaders; the first finds the runs
            const int lw = warp - SOFT - 2;
            const int pieces = p.ksteps * 2;                       // 16-byte pieces of a row, past `dim` zeros
            const int step_row = 32 / pieces, step_piece = 32 - step_row * pieces;
            const int row0 = lane / pieces, piece0 = lane - row0 * pieces;
            constexpr int BATCH = TN / 32 / LOADERS;               // batches of 32 rows per warp and tile
            uint32_t queue[LAG];                                   // barriers of the copies under way, 0 for none
#pragma unroll
            for (int i = 0; i < LAG; ++i) queue[i] = 0;
            // 32 rows whose addresses the lanes hold (null: zeros), `pitch` bytes between their 64-value chunks
            auto copy_rows = [&](const T *at, uint32_t dst, int first_row, uint32_t pitch) {
                int row = row0, piece = piece0;
#pragma unroll 1
                for (int i = 0; i < pieces; ++i) {
                    const T *src = reinterpret_cast<const T *>(__shfl_sync(0xffffffffu, (unsigned long long)at, row));
                    const bool there = src != nullptr && piece * 8 < p.c.dim;
                    const int rr = first_row + row;
                    cp16(dst + (piece >> 3) * pitch + rr * 128 + (((piece & 7) ^ (rr & 7)) << 4),
                         there ? static_cast<const void *>(src + piece * 8) : p.c.k, there ? 16u : 0u);
                    row += step_row;
                    piece += step_piece;
                    if (piece >= pieces) piece -= pieces, ++row;
                }
            };
            auto announce = [&](uint32_t b) {                      // the oldest copies have arrived
                if (b == 0) return;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b);
            };
            auto push = [&](uint32_t b) {
                cp_commit();
                cp_wait<LAG>();
                announce(queue[0]);
#pragma unroll
                for (int i = 0; i + 1 < LAG; ++i) queue[i] = queue[i + 1];
                queue[LAG - 1] = b;
            };
            auto flush = [&]() {
                cp_wait<0>();
#pragma unroll
                for (int i = 0; i < LAG; ++i) {
                    announce(queue[i]);
                    queue[i] = 0;
                }
            };
            // Before a wait that others may have to end with what is still under way here.
            auto waits = [&](uint64_t &b, int parity, int site) {
                if (__all_sync(0xffffffffu, mbar_try_wait(bar(b), (uint32_t)parity))) return true;
                flush();
                return wait(bar(b), parity, abort, site);
            };
            int runs = 0, slot = 0, phase = 0;                     // runs: whose q is copied
            auto load = [&](const PrefillUnit &u) {
                if (!waits(sh.q_empty, (runs & 1) ^ 1, W_QEMPTY)) return false;
                if (p.q_box) {                                     // rows of other sequences, or zeros, in place of rows that are not there
                    if (lane == 0) {
                        if (lw == 0) mbar_arrive_expect_tx(bar(sh.q_full), (uint32_t)(NQ * p.chunks * (128 * 128)));
                        else mbar_arrive(bar(sh.q_full));
                    }
                    __syncwarp();
                    if (lw == 0 && lane < NQ * p.chunks) {
                        const int i = lane / p.chunks, ch = lane - i * p.chunks;
                        tma_load_4d(base + i * q_bytes + ch * (128 * 128), &p.q_map, bar(sh.q_full), ch * 64, u.h * p.group,
                                    u.b * p.new_tokens + p.group_div.of(u.rt * RT + i * 128), 0);
                    }
                } else {
#pragma unroll 1
                    for (int bt = lw; bt < RT / 32; bt += LOADERS) {
                        const int r = u.rt * RT + bt * 32 + lane, t = p.group_div.of(min(r, p.rows - 1));
                        const bool live = r < p.rows && t < u.n;
                        const T *at = live ? static_cast<const T *>(p.q) + ((int64_t)u.b * p.new_tokens + t) * p.ldq +
                                                 (int64_t)(u.h * p.group + (r - t * p.group)) * p.c.dim
                                           : nullptr;
                        copy_rows(at, base + (bt >> 2) * q_bytes, (bt & 3) * 32, 128 * 128);
                    }
                    push(bar(sh.q_full));
                }
                ++runs;
                for (int tile = u.t0; tile < u.t1; ++tile) {
                    if (p.box) {                                   // boxes of entries of one page
                        const int boxes = TN / p.box;
                        const bool mine = lane < boxes && lane % LOADERS == lw;
                        int pg = 0, off = 0;
                        if (mine) {
                            const int e = tile * TN + lane * p.box, col = p.page_div.of(e);
                            off = e - col * p.c.page_size;
                            // past the length lies a page that does not exist: zeros
                            pg = e < u.len ? cache_page(p.c, u.b, col, KID_PREFILL) : (int)p.c.pages;
                            if (pg < 0) pg = off = 0;
                        }
                        const int many = __popc(__ballot_sync(0xffffffffu, mine));
#pragma unroll
                        for (int kv = 0; kv < 2; ++kv) {
                            if (!waits(sh.empty[slot], phase ^ 1, W_EMPTY)) return false;
                            const uint32_t b = bar(sh.full[slot]), dst = ring + slot * slot_bytes + lane * p.box * 128;
                            if (lw == 0 && lane < TN / 32) sh.bad[slot][lane] = 0;
                            __syncwarp();
                            const bool skip = p.withhold && lw == 0 && kv == 0 && tile == u.t1 - 1;
                            if (lane == 0 && !skip) {
                                if (many) mbar_arrive_expect_tx(b, (uint32_t)(many * p.chunks * p.box * 128));
                                else mbar_arrive(b);
                            }
                            __syncwarp();
                            if (mine && !skip)
                                for (int ch = 0; ch < p.chunks; ++ch)
                                    tma_load_4d(dst + ch * (TN * 128), kv ? &p.v_map : &p.k_map, b, ch * 64, off, u.h, pg);
                            if (++slot == p.slots) slot = 0, phase ^= 1;
                        }
                        flush();                                   // what was copied otherwise
                        continue;
                    }
                    const T *ka[BATCH], *va[BATCH];
#pragma unroll
                    for (int bt = 0; bt < BATCH; ++bt) {
                        const int e = tile * TN + (bt * LOADERS + lw) * 32 + lane;
                        ka[bt] = va[bt] = nullptr;
                        if (e < u.len) {
                            const int col = p.page_div.of(e);
                            int off = e - col * p.c.page_size;
                            int64_t pg = cache_page(p.c, u.b, col, KID_PREFILL);
                            if (pg < 0) pg = off = 0;
                            ka[bt] = static_cast<const T *>(p.c.k) + pg * p.c.k_page + u.h * p.c.k_head + off * p.c.k_slot;
                            va[bt] = static_cast<const T *>(p.c.v) + pg * p.c.v_page + u.h * p.c.v_head + off * p.c.v_slot;
                        }
                    }
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (!waits(sh.empty[slot], phase ^ 1, W_EMPTY)) return false;
                        if (lw == 0 && lane < TN / 32) sh.bad[slot][lane] = 0;
                        if (!(p.withhold && lw == 0 && kv == 0 && tile == u.t1 - 1)) {
#pragma unroll
                            for (int bt = 0; bt < BATCH; ++bt)
                                copy_rows(kv ? va[bt] : ka[bt], ring + slot * slot_bytes, (bt * LOADERS + lw) * 32, TN * 128);
                            push(bar(sh.full[slot]));
                        }
                        if (++slot == p.slots) slot = 0, phase ^= 1;
                    }
                }
                return true;
            };
            bool ok = true;
            int asking = -1;                                       // whole: phase of an answer that has not come
            if (lw == 0) {
                PrefillWalk<RT, TN> w;
                w.asked = 0;
                if (!p.whole) w.split(p);
                int2 join = make_int2(-1, 0);
                for (bool first = true; ok; first = false) {
                    int none = 0;
                    if (p.whole) {
                        const int st = w.next_whole(p, first, smem_u32(&sh.answer), bar(sh.next), abort);
                        if (st == -2) asking = w.asked & 1;
                        if (st == -2) break;
                        none = st;
                    } else if (!w.next_split(p, first)) {
                        none = -1;
                    }
                    if (!none && w.begins && !w.ends) {            // the CTA's last run: who has the rest of the unit
                        join = make_int2((w.u.b * p.row_tiles + w.u.rt) * p.c.heads + w.u.h, w.owner(w.place + w.rest - 1));
                    }
                    if (!waits(sh.run_empty[run_at], run_phase ^ 1, W_RUN)) break;
                    if (lane == 0) {
                        sh.run[run_at].u = w.u;
                        sh.run[run_at].flags = none ? 4 : (w.begins ? 1 : 0) | (w.ends ? 2 : 0);
                        mbar_arrive(bar(sh.run_full[run_at]));
                    }
                    __syncwarp();
                    if (++run_at == Shared::RUNS) run_at = 0, run_phase ^= 1;
                    if (none) break;
                    if (w.u.t0 < w.u.t1) ok = load(w.u);
                    flush();                                       // before a wait for warps that may wait for these copies
                }
                if (!p.whole && lane == 0) p.joins[blockIdx.x] = ok && !*abort ? join : make_int2(-1, 0);
            } else {
                PrefillRun run;
                while (ok && hear(run)) {
                    if (run.u.t0 < run.u.t1) ok = load(run.u);
                    flush();
                }
            }
            flush();
            // A wait ran out: the copies under way still come to their end.  Each barrier is waited for in the phase of this warp's
            // last copy; where one runs out here too (the other warp had no copy to add), all copies have had that time.
            if (!ok || *abort) {
                uint32_t never = 0;
                for (int i = 0; i < p.slots; ++i) {
                    const int before = i < slot ? phase : phase ^ 1;       // of the slot's last copy; none: over already
                    if (lane == 0 && p.box) mbar_wait(bar(sh.full[i]), (uint32_t)before, &never, KID_PREFILL, W_DRAIN);
                }
                if (lane == 0 && asking >= 0) mbar_wait(bar(sh.next), (uint32_t)asking, &never, KID_PREFILL, W_DRAIN);
                if (lane == 0 && p.q_box && runs > 0) mbar_wait(bar(sh.q_full), (uint32_t)((runs - 1) & 1), &never, KID_PREFILL, W_DRAIN);
                __syncwarp();
            }
        }
    }
done:
    tc_fence_before();
    __syncthreads();
    if (warp == SOFT) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of the unit that CTA blockIdx.x starts and does not end: one row per warp.
template <typename T>
__global__ void __launch_bounds__(128) prefill_join_kernel(const __grid_constant__ PrefillParams p, int rt_rows)
{
    using namespace pre;
    pdl_wait();
    pdl_launch_dependents();
    const int2 join = p.joins[blockIdx.x];
    if (join.x < 0) return;
    const int lane = threadIdx.x & 31, n = join.y - (int)blockIdx.x + 1;
    const int pair = join.x / p.c.heads, h = join.x - pair * p.c.heads, b = pair / p.row_tiles, rt = pair - b * p.row_tiles;
    const float c = p.cap_out != 0.f || p.slopes || !(p.scale_log2 > 0.f) ? 1.f : p.scale_log2;
    const int rows = min(rt_rows, p.rows - rt * rt_rows);
    for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < rows; r += gridDim.y * 4) {
        // the part that begins the unit is its CTA's second, the others are their CTAs' first
        auto at = [&](int i) { return (2ll * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * p.part_rows + r; };
        auto weighed = [&](int i) { return i < n ? p.part_ml[at(i)] : make_float2(-INFINITY, 0.f); };
        constexpr int BATCH = 4;                               // parts whose sums are loaded together, the first before their weights
        float4 v[BATCH][2];
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (i0 + i < n && (lane + 32 * e) * 4 < p.c.dim)
                        v[i][e] = reinterpret_cast<const float4 *>(p.part + at(i0 + i) * p.c.dim)[lane + 32 * e];
        };
        float2 ml = weighed(lane);
        load(0);
        float top = ml.y > 0.f ? ml.x : -INFINITY;
        for (int i = lane + 32; i < n; i += 32) {
            const float2 w = weighed(i);
            if (w.y > 0.f) top = fmaxf(top, w.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.f;
        float4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        for (int i0 = 0; i0 < n; i0 += 32) {
            if (i0 > 0) ml = weighed(i0 + lane);
            float wt = 0.f;
            if (ml.y > 0.f) wt = rescale<T>(ml.x, top, c);
            sum += ml.y > 0.f ? wt * ml.y : ml.y;              // 0, or a NaN
            for (int j = 0; j < 32 && i0 + j < n; j += BATCH) {
                if (i0 + j > 0) load(i0 + j);
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const float wi = __shfl_sync(0xffffffffu, wt, j + i);
                    if (wi == 0.f) continue;                   // not there, or nothing in it
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if ((lane + 32 * e) * 4 >= p.c.dim) continue;
                        acc[e].x = fmaf(wi, v[i][e].x, acc[e].x);
                        acc[e].y = fmaf(wi, v[i][e].y, acc[e].y);
                        acc[e].z = fmaf(wi, v[i][e].z, acc[e].z);
                        acc[e].w = fmaf(wi, v[i][e].w, acc[e].w);
                    }
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float f = sum > 0.f ? 1.f / sum : sum;           // a row that saw nothing is 0, a NaN stays one
        const int rr = rt * rt_rows + r, t = p.group_div.of(rr);
        const int64_t row = ((int64_t)b * p.new_tokens + t) * p.q_heads + h * p.group + (rr - t * p.group);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int d = lane + 32 * e;
            if (d * 4 >= p.c.dim) continue;
            const float4 v = make_float4(acc[e].x * f, acc[e].y * f, acc[e].z * f, acc[e].w * f);
            if (p.out_f32) *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row * p.c.dim + 4 * d) = v;
            else
                *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + row * p.c.dim + 4 * d) =
                    make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
        }
    }
}

namespace pre {
// How a call is cut up: the same for the sizes and the launch.
struct Plan {
    int rows, row_tiles, rt, tn, whole, grid, part_rows, slots, chunks, ksteps;
    int64_t floats;
    uint32_t smem;
};

inline int make_plan(const mmq_kv_cache *c, int q_heads, int new_tokens, Plan &q)
{
    if (q_heads < 1 || q_heads > 65535 || q_heads % c->heads || q_heads / c->heads > 128 || new_tokens < 1 ||
        (int64_t)new_tokens * (q_heads / c->heads) > 0x7fffff00 || (int64_t)c->seqs * new_tokens > 0x7fffffff)
        return MMQ_ERR_SHAPE;
    q.rows = new_tokens * (q_heads / c->heads);
    // 256 rows share a tile of K and V where there are that many and tensor memory holds their sums
    q.rt = q.rows > 128 && c->dim <= 192 ? 256 : 128;
    q.tn = c->dim <= 128 ? 128 : 64;
    q.row_tiles = (q.rows + q.rt - 1) / q.rt;
    q.chunks = (c->dim + 63) / 64;
    q.ksteps = (c->dim + 15) / 16;
    const int64_t units = (int64_t)c->seqs * c->heads * q.row_tiles, cap = (int64_t)c->cols * c->page_size;
    if (units > 0x7fffff00 || units * ((cap + q.tn - 1) / q.tn) > 0x7fffff00) return MMQ_ERR_SHAPE;
    const int sms = sm_count();
    // A unit per CTA where that keeps the device busy (2048 rows of four heads over 8192 entries, 256 units: 255 us, cut into
    // equal parts 274), or where no sequence can be so long that cutting it would pay for the joining launch (5 us; one token
    // over 513 entries of 32 heads 20 and 21).  The lengths are on the device: the table's columns go for them.
    const int64_t waves = (units + sms - 1) / sms;
    q.whole = (q.row_tiles > 1 && (units >= 3 * sms || units * 5 >= waves * sms * 4)) || cap <= 6 * q.tn;
    q.grid = q.whole ? (int)units : sms;
    q.part_rows = q.rows < q.rt ? q.rows : q.rt;
    q.floats = q.whole ? 4 : 2ll * sms * q.part_rows * (c->dim + 2) + 2ll * sms;
    const uint32_t slot = (uint32_t)q.chunks * q.tn * 128, queries = (uint32_t)q.chunks * q.rt * 128;
    const uint32_t rest = q.rt == 256 ? (q.tn == 128 ? sizeof(PrefillShared<2, 128>) : sizeof(PrefillShared<2, 64>))
                                      : (q.tn == 128 ? sizeof(PrefillShared<1, 128>) : sizeof(PrefillShared<1, 64>));
    q.slots = (int)((SMEM - rest - queries) / slot);
    if (q.slots > MAX_SLOTS) q.slots = MAX_SLOTS;
    q.smem = queries + q.slots * slot + rest;
    return MMQ_OK;
}

template <typename T, int NQ, int TN>
int launch(const PrefillParams &p, const Plan &q, cudaStream_t stream)
{
    static std::atomic<unsigned long long> set{0};             // devices whose limit is raised
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return launch_status();
    if (!(set.load(std::memory_order_relaxed) >> dev & 1)) {
        if (cudaFuncSetAttribute(prefill_kernel<T, NQ, TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM) != cudaSuccess)
            return launch_status();
        set.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    int rc = launch_pdl(prefill_kernel<T, NQ, TN>, dim3((unsigned)q.grid), PrefillShape<T, NQ, TN>::kThreads, q.smem, stream, 0, p);
    if (rc != MMQ_OK || q.whole) return rc;
    const int by = (q.part_rows + 3) / 4;
    return launch_pdl(prefill_join_kernel<T>, dim3((unsigned)q.grid, (unsigned)(by < 64 ? by : 64)), 128, 0, stream, 0, p, q.rt);
}

template <typename T>
int launch_any(const PrefillParams &p, const Plan &q, cudaStream_t stream)
{
    if (q.rt == 256) return q.tn == 128 ? launch<T, 2, 128>(p, q, stream) : launch<T, 2, 64>(p, q, stream);
    return q.tn == 128 ? launch<T, 1, 128>(p, q, stream) : launch<T, 1, 64>(p, q, stream);
}

struct Call {
    const void *q;
    int64_t ldq;
    const int32_t *new_len, *prefix, *first;
    const uint64_t *tree;
    const float *slopes;
    void *out;
    int out_dtype, q_heads, new_tokens;
    float scale, cap;
    int window;
    float *work;
};

// Tensor maps of K and V, where boxes of at least eight entries fit the pages (and the swizzle's groups of eight rows), and of
// q, where a box holds whole tokens.  A layout that has no map is copied row by row.
void make_maps(PrefillParams &p, const Plan &q)
{
    const mmq_kv_cache &c = p.c;
    const CUtensorMapDataType type = c.dtype == MMQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (c.dim < 64) return;                                    // a box is 64 values wide
    constexpr uint64_t kMostStride = 1ull << 40;
    if (128 % p.group == 0 && (uint64_t)p.ldq * 2 < kMostStride) {
        const uint64_t dims[4] = {(uint64_t)c.dim, (uint64_t)p.q_heads, (uint64_t)c.seqs * p.new_tokens, 1};
        const uint64_t strides[3] = {(uint64_t)c.dim * 2, (uint64_t)p.ldq * 2, 16};
        const uint32_t extent[4] = {64, (uint32_t)p.group, (uint32_t)(128 / p.group), 1};
        p.q_box = make_tmap_4d(&p.q_map, p.q, type, dims, strides, extent, CU_TENSOR_MAP_SWIZZLE_128B) == MMQ_OK;
    }
    int box = 1;
    while (2 * box <= q.tn && c.page_size % (2 * box) == 0) box *= 2;
    if (box < 8) return;
    const uint64_t dims[4] = {(uint64_t)c.dim, (uint64_t)c.page_size, (uint64_t)c.heads, (uint64_t)c.pages};
    const uint32_t extent[4] = {64, (uint32_t)box, 1, 1};
    for (int kv = 0; kv < 2; ++kv) {
        uint64_t strides[3] = {(uint64_t)(kv ? c.v_slot : c.k_slot) * 2, (uint64_t)(kv ? c.v_head : c.k_head) * 2,
                               (uint64_t)(kv ? c.v_page : c.k_page) * 2};
        for (int i = 0; i < 3; ++i) {
            if (dims[i + 1] == 1) strides[i] = 16;             // never used
            if (strides[i] == 0 || strides[i] >= kMostStride) return;
        }
        if (make_tmap_4d(kv ? &p.v_map : &p.k_map, kv ? c.v : c.k, type, dims, strides, extent, CU_TENSOR_MAP_SWIZZLE_128B) != MMQ_OK) return;
    }
    p.box = box;
}

int attend(const mmq_kv_cache *cache, const Call &a, mmq_stream_t stream)
{
    int rc = check_cache(cache);
    if (rc != MMQ_OK) return rc;
    Plan q;
    if ((rc = make_plan(cache, a.q_heads, a.new_tokens, q)) != MMQ_OK) return rc;
    if ((a.out_dtype != MMQ_F32 && a.out_dtype != cache->dtype) || a.ldq < (int64_t)a.q_heads * cache->dim ||
        !isfinite(a.scale * 1.44269504088896341f) || !(a.cap >= 0.f && a.cap <= 1024.f) || a.window < 0 || (a.q && a.q == a.out))
        return MMQ_ERR_SHAPE;
    if (cache->seqs == 0) return MMQ_OK;
    if (!a.q || !a.out || !a.work) return MMQ_ERR_NULL;
    if (!aligned16(a.q) || !aligned16(a.out) || !aligned16(a.work) || (a.ldq & 7)) return MMQ_ERR_ALIGN;
    if ((rc = check_arch()) != MMQ_OK) return rc;
    PrefillParams p = {};
    p.c = *cache;
    p.q = a.q;
    p.new_len = a.new_len;
    p.prefix = a.prefix;
    p.first = a.first;
    p.tree = a.tree;
    p.slopes = a.slopes;
    p.out = a.out;
    p.ldq = a.ldq;
    p.scale_log2 = a.scale * 1.44269504088896341f;
    if (a.cap > 0.f) {
        p.cap_in = 2.f * 1.44269504088896341f * (a.scale / a.cap);
        p.cap_out = a.cap * 1.44269504088896341f;
    }
    p.out_f32 = a.out_dtype == MMQ_F32;
    p.out_wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && (p.out_f32 || cache->dim % 16 == 0);
    p.window = a.window;
    p.new_tokens = a.new_tokens;
    p.group = a.q_heads / cache->heads;
    p.q_heads = a.q_heads;
    p.rows = q.rows;
    p.row_tiles = q.row_tiles;
    p.whole = q.whole;
    p.part_rows = q.part_rows;
    p.chunks = q.chunks;
    p.ksteps = q.ksteps;
    p.slots = q.slots;
    p.part = a.work;
    p.part_wide = (reinterpret_cast<uintptr_t>(a.work) & 31) == 0;
    p.part_ml = reinterpret_cast<float2 *>(a.work + 2ll * q.grid * q.part_rows * cache->dim);
    p.joins = reinterpret_cast<int2 *>(p.part_ml + 2ll * q.grid * q.part_rows);
    p.page_div = FastDiv(cache->page_size);
    p.group_div = FastDiv(p.group);
    p.withhold = withheld();
    make_maps(p, q);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return cache->dtype == MMQ_F16 ? launch_any<__half>(p, q, st) : launch_any<__nv_bfloat16>(p, q, st);
}
}  // namespace pre

}  // namespace
}  // namespace mmq

extern "C" int mmq_prefill_sizes(const mmq_kv_cache *cache, int q_heads, int new_tokens, int64_t *work_floats)
{
    using namespace mmq;
    const int rc = check_cache(cache);
    if (rc != MMQ_OK) return rc;
    if (!work_floats) return MMQ_ERR_NULL;
    pre::Plan q;
    const int st = pre::make_plan(cache, q_heads, new_tokens, q);
    if (st != MMQ_OK) return st;
    *work_floats = q.floats;
    return MMQ_OK;
}

extern "C" int mmq_attn_prefill(const mmq_kv_cache *cache, const void *q, int64_t ldq, const int32_t *new_len, const int32_t *prefix,
                                const int32_t *first, const float *slopes, void *out, int out_dtype, int q_heads, int new_tokens,
                                float scale, float cap, int window, float *work, mmq_stream_t stream)
{
    return mmq::pre::attend(cache, {q, ldq, new_len, prefix, first, nullptr, slopes, out, out_dtype, q_heads, new_tokens, scale, cap, window, work},
                            stream);
}

extern "C" int mmq_attn_tree(const mmq_kv_cache *cache, const void *q, int64_t ldq, const uint64_t *tree, const int32_t *new_len,
                             const int32_t *first, void *out, int out_dtype, int q_heads, int new_tokens, float scale, float cap,
                             float *work, mmq_stream_t stream)
{
    using namespace mmq;
    const int rc = check_cache(cache);
    if (rc != MMQ_OK) return rc;
    if (new_tokens > 64) return MMQ_ERR_SHAPE;
    if (cache->seqs > 0 && !tree) return MMQ_ERR_NULL;
    return pre::attend(cache, {q, ldq, new_len, nullptr, first, tree, nullptr, out, out_dtype, q_heads, new_tokens, scale, cap, 0, work}, stream);
}
