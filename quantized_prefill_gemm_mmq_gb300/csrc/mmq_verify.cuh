// mmq_verify.cuh -- verification of drafted tokens (mmq_spec_verify).
//
// Draft i is accepted while u_i q_i(x) < p_i(x).  At the first that is not,
// the token is drawn from max(p - q, 0), else from the target's last row, by
// inverting the cumulative sum.  The sum is of whole numbers
// w_j = round(2^40 max(p_j - q_j, 0)), so any order of adding gives the same,
// and the row can be split over a cluster's CTAs, warps and lanes and still
// draw what a serial sum would.
//
// A cluster per sequence.  Every CTA finds the first rejection by itself (a
// few loads) and adds up its part of the row in spans of 2 x 32 x 16 bytes, one
// per warp at a time, keeping the spans' sums; the CTAs exchange their totals
// through distributed shared memory; the one whose part the threshold falls
// into reads the one span again and finds the value.  So the row is read once.
// A row of an odd vocabulary does not start on 16 bytes: the parts are laid out
// from the last 16-byte boundary before the target's row, and of the draft's
// row, where it lies otherwise, a lane takes its 16 bytes out of two aligned
// ones.
// Bound by memory (one or two rows of the vocabulary per sequence) and, near
// it, by some eleven instructions per value, so a span that lies inside the rows
// is loaded without the checks that the rows' ends need (64 sequences: 13.3 us
// with the checks everywhere and a 64-bit sum by shuffles, 11.7 without).
// Measured: 64 sequences of 7 drafts over 128001 values in bf16 11.3 us (2.5
// TB/s; the first 2.5 us find the rejections), 3 drafts over 32000 4.6 us.
#pragma once

namespace mmq {
namespace {

namespace ver {
constexpr int THREADS = 256;
constexpr int PER_SM = 4;               // CTAs resident per SM: 64 registers a thread
constexpr int WARPS = THREADS / 32;
constexpr int BATCH = 2;                // 16-byte pieces per lane and span
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_VOCAB = 1 << 20;
constexpr int MAX_DRAFTS = 64;
template <typename T>
constexpr int kPer = 16 / sizeof(T);    // values per lane and span
template <typename T>
constexpr int kSpan = BATCH * 32 * kPer<T>;
}  // namespace ver

struct VerifyParams {
    const void *target, *draft;
    const int32_t *tokens;
    const float *uniform;
    const int32_t *count;
    int32_t *out, *accepted;
    int drafts, vocab, spans;           // spans per CTA
};

__device__ __forceinline__ float ver_f(float x) { return x; }
__device__ __forceinline__ float ver_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float ver_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// w = round(2^40 d), d = max(p - q, 0) limited to 1, in two parts: added to hi
// the upper 17 bits, to lo the 23 below them (up to 2^23).  With 2^23 added, a
// float's bits count in ones: the upper part by rounding down, the lower, of
// the exact rest, to nearest even.  The bits of 2^23 itself, 0x4b000000, stay
// in the sums: ver_join takes them off.
__device__ __forceinline__ void ver_add(float p, float q, uint32_t &hi, uint32_t &lo)
{
    const float d = __saturatef(__fsub_rn(p, q));
    const float t = __fmaf_rd(d, 0x1p17f, 0x1p23f);
    const float rest = __fmaf_rn(d, 0x1p17f, -__fsub_rn(t, 0x1p23f));
    hi += __float_as_uint(t);
    lo += __float_as_uint(__fmaf_rn(rest, 0x1p23f, 0x1p23f));
}
// the sum of n values' w
__device__ __forceinline__ unsigned long long ver_join(uint32_t hi, uint32_t lo, uint32_t n)
{
    return ((unsigned long long)(hi - n * 0x4b000000u) << 23) + (lo - n * 0x4b000000u);
}

// bytes odd .. odd+15 of the 32 in x and y; odd is the same for the whole warp
__device__ __forceinline__ uint4 ver_shift(const uint4 &x, const uint4 &y, uint32_t odd)
{
    const uint32_t s = (odd & 3) * 8;
    const auto by = [&](uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e) {
        return make_uint4(__funnelshift_r(a, b, s), __funnelshift_r(b, c, s), __funnelshift_r(c, d, s), __funnelshift_r(d, e, s));
    };
    switch (odd >> 2) {
    case 0: return by(x.x, x.y, x.z, x.w, y.x);
    case 1: return by(x.y, x.z, x.w, y.x, y.y);
    case 2: return by(x.z, x.w, y.x, y.y, y.z);
    default: return by(x.w, y.x, y.y, y.z, y.w);
    }
}

// A row of n values.  load(j): the 16 bytes from value j on, zeros outside the
// row.  `odd`: how far value j (a multiple of 16 bytes from `first`) lies past
// a 16-byte boundary, the same for every j.
template <typename T>
struct VerRow {
    const T *row;
    uint32_t odd;
    __device__ VerRow(const T *r, int first) : row(r), odd((uint32_t)(reinterpret_cast<uintptr_t>(r + first) & 15u)) {}
    __device__ __forceinline__ uint4 load(int j, int n) const
    {
        constexpr int N = ver::kPer<T>;
        // the aligned words around the 16 bytes must lie in the row themselves: its ends are read value by value
        if (j < (odd ? N : 0) || j + (odd ? 2 * N : N) > n) {
            T v[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                v[k] = T(0.f);
                if (j + k >= 0 && j + k < n) v[k] = row[j + k];
            }
            return *reinterpret_cast<const uint4 *>(v);
        }
        const uint4 *a = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(row + j) - odd);
        const uint4 x = *a;
        if (odd == 0) return x;
        const uint4 y = *(a + 1);
        return ver_shift(x, y, odd);
    }
};

// ver_add of two values, with packed products and sums: one instruction for two
__device__ __forceinline__ void ver_add2(float p0, float p1, float q0, float q1, uint32_t &hi, uint32_t &lo)
{
    const float d0 = __saturatef(__fsub_rn(p0, q0)), d1 = __saturatef(__fsub_rn(p1, q1));
    uint32_t t0, t1, l0, l1;
    asm("{\n\t"
        ".reg .b64 d, t, m, r, c17, c23;\n\t"
        "mov.b64 d, {%4, %5};\n\t"
        "mov.b64 c17, {%6, %6};\n\t"
        "mov.b64 c23, {%7, %7};\n\t"
        "fma.rm.f32x2 t, d, c17, c23;\n\t"
        "sub.rn.f32x2 m, c23, t;\n\t"
        "fma.rn.f32x2 r, d, c17, m;\n\t"
        "fma.rn.f32x2 r, r, c23, c23;\n\t"
        "mov.b64 {%0, %1}, t;\n\t"
        "mov.b64 {%2, %3}, r;\n\t"
        "}"
        : "=r"(t0), "=r"(t1), "=r"(l0), "=r"(l1)
        : "f"(d0), "f"(d1), "f"(0x1p17f), "f"(0x1p23f));
    hi += t0 + t1;
    lo += l0 + l1;
}

// adds the w_j of 16 bytes' worth of values to hi and lo
template <typename T>
__device__ __forceinline__ void ver_sum(const uint4 &pv, const uint4 &qv, uint32_t &hi, uint32_t &lo)
{
    const T *p = reinterpret_cast<const T *>(&pv), *q = reinterpret_cast<const T *>(&qv);
#pragma unroll
    for (int k = 0; k < ver::kPer<T>; k += 2) ver_add2(ver_f(p[k]), ver_f(p[k + 1]), ver_f(q[k]), ver_f(q[k + 1]), hi, lo);
}

template <typename T>
__global__ void __launch_bounds__(ver::THREADS, ver::PER_SM) spec_verify_kernel(const VerifyParams p)
{
    using namespace ver;
    constexpr int PER = kPer<T>, SPAN = kSpan<T>;
    extern __shared__ __align__(16) unsigned long long s_span[];    // [spans]
    __shared__ unsigned long long s_total[2], s_warp[WARPS];
    __shared__ int s_first, s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_ctarank(), n_cta = (int)cluster_nctarank(), b = blockIdx.x / n_cta;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t V = p.vocab;
    const T *target = static_cast<const T *>(p.target) + (int64_t)b * (p.drafts + 1) * V;
    const T *draft = p.draft ? static_cast<const T *>(p.draft) + (int64_t)b * p.drafts * V : nullptr;
    const int n = new_count(p.count, b, p.drafts, KID_VERIFY);

    if (warp == 0) {                                        // the first rejection
        int first = n;
        bool bad = false;
        for (int i0 = 0; i0 < n && first == n; i0 += 32) {
            const int i = i0 + lane;
            bool no = false, off = false;
            if (i < n) {
                const int x = *(p.tokens + (int64_t)b * p.drafts + i);
                off = x < 0 || x >= p.vocab;
                if (off) {
                    no = true;
                } else {
                    const float pt = ver_f(target[i * V + x]), q = draft ? ver_f(draft[i * V + x]) : 1.f;
                    no = !(__fmul_rn(*(p.uniform + (int64_t)b * (p.drafts + 1) + i), q) < pt);
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, no);
            if (m) {
                first = i0 + __ffs(m) - 1;
                bad = __shfl_sync(0xffffffffu, off ? 1 : 0, __ffs(m) - 1) != 0;
            }
        }
        if (lane == 0) {
            s_first = first;
            s_bad = bad;
            if (bad && rank == 0) record_error(MMQ_ERR_INDEX, KID_VERIFY, SITE_TOKEN);
        }
    }
    __syncthreads();
    const int a = s_first;
    const T *pr = target + a * V;
    // what is taken off the target: the draft's row, or (draft == nullptr) the drafted token itself
    const bool rejected = a < n && !s_bad;
    const T *qr = rejected && draft ? draft + a * V : nullptr;
    const int whole_tok = rejected && !draft ? *(p.tokens + (int64_t)b * p.drafts + a) : -1;
    // the CTA's first value: `origin` is up to 16 bytes before the row's start, on a boundary
    const int origin = -(int)((reinterpret_cast<uintptr_t>(pr) & 15u) / sizeof(T)), lo = origin + rank * p.spans * SPAN;
    const VerRow<T> prow(pr, origin), qrow(qr ? qr : pr, origin);
    // the values of a lane: the row less what is taken off it
    auto load_q = [&](int j, bool plain) {
        if (plain || (!qr && (whole_tok < j || whole_tok >= j + PER))) return make_uint4(0u, 0u, 0u, 0u);
        if (qr) return qrow.load(j, p.vocab);
        T v[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) v[k] = T(j + k == whole_tok ? 1.f : 0.f);
        return *reinterpret_cast<const uint4 *>(v);
    };

    unsigned long long r = 0, before = 0, mine = 0;
    for (int tries = 0; tries < 2; ++tries) {
        const bool plain = tries == 1;                      // the target alone, if nothing of the difference is left
        unsigned long long sum = 0;
#pragma unroll (sizeof(T) == 4 ? 1 : 2)                  // two f32 spans do not fit the registers
        for (int sp = warp; sp < p.spans; sp += WARPS) {
            uint4 pv[BATCH], qv[BATCH];
            const int j0 = lo + sp * SPAN;
            // a span whose 16-byte words all lie in the rows, and where nothing but a draft's row is taken off
            if (j0 >= PER && j0 + SPAN + PER <= p.vocab && (qr || plain || whole_tok < j0 || whole_tok >= j0 + SPAN)) {
                const bool with = qr && !plain;
                const uint4 *a = reinterpret_cast<const uint4 *>(pr + j0) + lane;
                const uint4 *c = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(qrow.row + j0) - qrow.odd) + lane;
                uint4 next[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    pv[k] = a[k * 32];
                    qv[k] = next[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (with) {
                        qv[k] = c[k * 32];
                        if (qrow.odd) next[k] = c[k * 32 + 1];
                    }
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) qv[k] = ver_shift(qv[k], next[k], qrow.odd);
            } else {
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int j = j0 + (k * 32 + lane) * PER;
                    pv[k] = qv[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (j < p.vocab) {
                        pv[k] = prow.load(j, p.vocab);
                        qv[k] = load_q(j, plain);
                    }
                }
            }
            uint32_t hi = 0, low = 0;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) ver_sum<T>(pv[k], qv[k], hi, low);
            // the warp's: per lane hi is up to 2^21 and low up to 2^27, the latter added in two parts
            hi -= BATCH * PER * 0x4b000000u;
            low -= BATCH * PER * 0x4b000000u;
            const unsigned long long w = ((unsigned long long)__reduce_add_sync(0xffffffffu, hi) << 23) +
                                         ((unsigned long long)__reduce_add_sync(0xffffffffu, low >> 16) << 16) +
                                         __reduce_add_sync(0xffffffffu, low & 0xffffu);
            if (lane == 0) s_span[sp] = w;
            sum += w;
        }
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        if (tid == 0) {
            unsigned long long t = 0;
            for (int w = 0; w < WARPS; ++w) t += s_warp[w];
            s_total[tries] = t;
        }
        cluster_sync_all();
        unsigned long long total = 0;
        before = 0;
        for (int c = 0; c < n_cta; ++c) {
            const unsigned long long t = cluster_ld64(cluster_map(smem_u32(&s_total[tries]), c));
            if (c < rank) before += t;
            total += t;
        }
        mine = s_total[tries];
        const unsigned long long u = (unsigned long long)(fminf(fmaxf(*(p.uniform + (int64_t)b * (p.drafts + 1) + p.drafts), 0.f), 1.f - 0x1p-24f) * 0x1p24f);
        r = (total >> 24) * u + (((total & 0xffffffull) * u) >> 24);     // floor(total u / 2^24), below total
        if (total > 0 || tries == 1) {
            if (total == 0) mine = 0;
            // ---- the span, then the value, where the sum passes r
            if (before <= r && r < before + mine && warp == 0) {
                unsigned long long at = before;
                int sp = 0;
                for (int s0 = 0; s0 < p.spans; s0 += 32) {
                    unsigned long long x = s0 + lane < p.spans ? s_span[s0 + lane] : 0, c = x;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const unsigned long long y = __shfl_up_sync(0xffffffffu, c, o);
                        if (lane >= o) c += y;
                    }
                    const unsigned m = __ballot_sync(0xffffffffu, at + c > r);
                    if (m) {
                        const int f = __ffs(m) - 1;
                        sp = s0 + f;
                        at += __shfl_sync(0xffffffffu, c - x, f);
                        break;
                    }
                    at += __shfl_sync(0xffffffffu, c, 31);
                }
                for (int half = 0; half < BATCH; ++half) {  // the span's pieces, in order
                    const int j = lo + sp * SPAN + (half * 32 + lane) * PER;
                    uint4 pv = make_uint4(0u, 0u, 0u, 0u), qv = pv;
                    if (j < p.vocab) {
                        pv = prow.load(j, p.vocab);
                        qv = load_q(j, plain);
                    }
                    uint32_t hi = 0, low = 0;
                    ver_sum<T>(pv, qv, hi, low);
                    const unsigned long long x = ver_join(hi, low, PER);
                    unsigned long long c = x;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const unsigned long long y = __shfl_up_sync(0xffffffffu, c, o);
                        if (lane >= o) c += y;
                    }
                    const unsigned m = __ballot_sync(0xffffffffu, at + c > r);
                    if (m == 0) {
                        at += __shfl_sync(0xffffffffu, c, 31);
                        continue;
                    }
                    if (lane == __ffs(m) - 1) {
                        at += c - x;
                        const T *pk = reinterpret_cast<const T *>(&pv), *qk = reinterpret_cast<const T *>(&qv);
                        int tok = -1;
#pragma unroll
                        for (int k = 0; k < PER; ++k) {
                            uint32_t h1 = 0, l1 = 0;
                            ver_add(ver_f(pk[k]), ver_f(qk[k]), h1, l1);
                            at += ver_join(h1, l1, 1);
                            if (tok < 0 && at > r) tok = j + k;
                        }
                        p.out[(int64_t)b * (p.drafts + 1) + a] = tok;
                    }
                    break;
                }
            }
            if (total == 0 && rank == 0 && tid == 0) p.out[(int64_t)b * (p.drafts + 1) + a] = 0;
            break;
        }
        __syncthreads();
    }
    if (rank == 0) {
        for (int i = tid; i <= p.drafts; i += THREADS)
            if (i != a)
                p.out[(int64_t)b * (p.drafts + 1) + i] = i < a ? *(p.tokens + (int64_t)b * p.drafts + i) : -1;
        if (tid == 0) p.accepted[b] = a;
    }
    cluster_sync_all();                                    // no CTA leaves while another may read its shared memory
}

template <typename T>
int launch_verify(VerifyParams &p, int seqs, cudaStream_t stream)
{
    // CTAs per sequence: one per 16 KB of a row, up to a cluster of eight
    constexpr int each = 16384 / (int)sizeof(T);
    int cl = 1;
    while (cl < ver::MAX_CLUSTER && p.vocab > each * cl) cl *= 2;
    const int per = (p.vocab + ver::kPer<T> + cl - 1) / cl;       // up to 16 bytes before the row's start besides
    p.spans = (per + ver::kSpan<T> - 1) / ver::kSpan<T>;
    return launch_pdl(spec_verify_kernel<T>, dim3((unsigned)(seqs * cl)), ver::THREADS, (size_t)p.spans * 8 /* <= 8 KB */, stream, cl, p);
}

}  // namespace
}  // namespace mmq

extern "C" int mmq_spec_verify(const void *target, const void *draft, int dtype, const int32_t *tokens,
                               const float *uniform, const int32_t *count, int32_t *out, int32_t *accepted, int seqs,
                               int drafts, int vocab, mmq_stream_t stream)
{
    using namespace mmq;
    if (seqs < 0 || seqs > 65535 || drafts < 1 || drafts > ver::MAX_DRAFTS || vocab < 1 || vocab > ver::MAX_VOCAB ||
        (dtype != MMQ_F16 && dtype != MMQ_BF16 && dtype != MMQ_F32))
        return MMQ_ERR_SHAPE;
    if (seqs == 0) return MMQ_OK;
    if (!target || !tokens || !uniform || !out || !accepted) return MMQ_ERR_NULL;
    if (!aligned16(target) || (draft && !aligned16(draft))) return MMQ_ERR_ALIGN;
    const int rc = check_arch();
    if (rc != MMQ_OK) return rc;
    VerifyParams p = {target, draft, tokens, uniform, count, out, accepted, drafts, vocab, 0};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == MMQ_F32   ? launch_verify<float>(p, seqs, s)
           : dtype == MMQ_F16 ? launch_verify<__half>(p, seqs, s)
                              : launch_verify<__nv_bfloat16>(p, seqs, s);
}
