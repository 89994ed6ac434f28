// mmq_norm_rope.cuh -- norms of every q and k head, rotary positions with one
// or several axes, and the append of the new keys and values to the paged cache
// (mmq_norm_rope_append).
//
// A head's values x become y = x rsqrt(mean x^2 + eps) w; pair i of the first
// `rot` of them turns by 2 pi frac(x_a f_i / 2^64), x_a being the row's position
// on the pair's axis a and f_i turns per position as a 64-bit fraction, whose
// product keeps the fraction of the turns exactly.
//
// Bound by memory: per row 4 + (4 or 2) bytes per q value and 6 per k and v
// value.  Eight values of a head (four pairs) lie with one thread, a head with a
// group of 1 to 32 neighbouring threads that add their squares by shuffles.  A
// block takes a row (or part of its heads): its groups take heads side by side,
// two ahead, and the row's sines are computed once while the first ones come.
// q, k and v heads have a loop each, and the norm's weights are folded into the
// sines and cosines: with one loop that asked for every head what it is, the
// instructions took longer than the memory (4096 rows of 32 + 2*32 heads of 128,
// f16: 89 us, and 61 now = 4.9 TB/s; three heads ahead 70 us, more blocks per row
// 76).  What bounds 4096 rows are still the instructions beside the memory (0.73
// of the copy rate), 1000 rows with three axes (11.7 us, 0.47) two rounds of
// blocks and the latency of a row, a single row (3.5 us) latency alone.
#pragma once

#include <type_traits>

namespace mmq {
namespace {

constexpr int NR_THREADS = 256;
constexpr int NR_BATCH = 2;          // heads whose loads a thread has in flight
constexpr int NR_BLOCKS = 4;         // resident blocks per multiprocessor

struct NormRopeParams {
    mmq_kv_cache c;
    const int64_t *freq;
    const int32_t *axis;             // [rot/2] or NULL
    const float *q_norm, *k_norm;    // [dim] or NULL
    const float *q, *k, *v;
    const int32_t *pos, *new_len;    // pos [axes][rows]
    void *q_out;
    int64_t ldq, ldk, ldv, ldo, rows;
    float magnitude, eps, inv_dim;
    int rot, interleaved, axes, q_heads, new_tokens, q_f32;
    int heads_per_block;             // of the row's q_heads + 2*heads
    int group;                       // threads per head
    FastDiv page_div;
};

// WIDE: rot is a multiple of 8, so that a thread's values are two aligned groups of four.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(NR_THREADS, NR_BLOCKS) norm_rope_kernel(const NormRopeParams p)
{
    enum { Q, K, V };
    __shared__ float s_cos[128], s_sin[128];
    pdl_wait();
    pdl_launch_dependents();
    const int D = p.c.dim, half = p.rot / 2;
    const int u = threadIdx.x & (p.group - 1), hl = threadIdx.x / p.group, lanes = blockDim.x / p.group;
    const int64_t row = blockIdx.x;
    const int b = (int)(row / p.new_tokens), t = (int)(row - (int64_t)b * p.new_tokens);
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(p.q_heads + 2 * p.c.heads, h0 + p.heads_per_block);
    const bool owner = u * 8 < D;                                // groups are rounded up to a power of two
    // The thread's pairs are (a[j], b[j]).  Where they lie: WIDE in two runs of four (halves apart, or side by side),
    // else pair k = 4u + j at (k, k + half), (2k, 2k + 1) interleaved or past the rotated ones.
    const bool apart = !p.interleaved && u * 8 < p.rot;
    const int d0 = apart ? u * 4 : u * 8, d1 = apart ? half + u * 4 : u * 8 + 4;
    auto place = [&](int j, int &x, int &y, bool rotated) {      // !WIDE
        const int k = u * 4 + j;
        x = rotated && k < half && !p.interleaved ? k : 2 * k;
        y = rotated && k < half && !p.interleaved ? k + half : 2 * k + 1;
    };
    auto read = [&](const float *src, bool rotated, float (&a)[4], float (&c)[4]) {
        if constexpr (WIDE) {
            const float4 x = *reinterpret_cast<const float4 *>(src + (rotated ? d0 : u * 8));
            const float4 y = *reinterpret_cast<const float4 *>(src + (rotated ? d1 : u * 8 + 4));
            const bool ap = rotated && apart;
            a[0] = x.x, a[1] = ap ? x.y : x.z, a[2] = ap ? x.z : y.x, a[3] = ap ? x.w : y.z;
            c[0] = ap ? y.x : x.y, c[1] = ap ? y.y : x.w, c[2] = ap ? y.z : y.y, c[3] = y.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                int x, y;
                place(j, x, y, rotated);
                a[j] = src[x];
                c[j] = src[y];
            }
        }
    };
    // eight values to f32, or rounded to the cache's type
    auto write = [&](auto *dst, bool rotated, const float (&a)[4], const float (&c)[4]) {
        using O = typename std::remove_pointer<decltype(dst)>::type;
        if constexpr (WIDE) {
            const bool ap = rotated && apart;
            const float4 x = make_float4(a[0], ap ? a[1] : c[0], ap ? a[2] : a[1], ap ? a[3] : c[1]);
            const float4 y = make_float4(ap ? c[0] : a[2], ap ? c[1] : c[2], ap ? c[2] : a[3], c[3]);
            if constexpr (std::is_same<O, float>::value) {
                *reinterpret_cast<float4 *>(dst + (rotated ? d0 : u * 8)) = x;
                *reinterpret_cast<float4 *>(dst + (rotated ? d1 : u * 8 + 4)) = y;
            } else {
                const uint2 w0 = make_uint2(pack2<O>(x.x, x.y), pack2<O>(x.z, x.w)), w1 = make_uint2(pack2<O>(y.x, y.y), pack2<O>(y.z, y.w));
                if (!ap) {
                    *reinterpret_cast<uint4 *>(dst + u * 8) = make_uint4(w0.x, w0.y, w1.x, w1.y);
                } else {
                    *reinterpret_cast<uint2 *>(dst + d0) = w0;
                    *reinterpret_cast<uint2 *>(dst + d1) = w1;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                int x, y;
                place(j, x, y, rotated);
                if constexpr (std::is_same<O, float>::value) dst[x] = a[j], dst[y] = c[j];
                else dst[x] = to_cache<O>(a[j]), dst[y] = to_cache<O>(c[j]);
            }
        }
    };
    const int n = new_count(p.new_len, b, p.new_tokens, KID_NORM);
    if (t >= n) {                                                // a row that is not there: q is 0
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        for (int h = h0 + hl; h < min(h1, p.q_heads); h += lanes) {
            if (!owner) continue;
            if (p.q_f32) write(static_cast<float *>(p.q_out) + row * p.ldo + (int64_t)h * D, true, zero, zero);
            else write(static_cast<T *>(p.q_out) + row * p.ldo + (int64_t)h * D, true, zero, zero);
        }
        return;
    }
    float a[NR_BATCH][4], c[NR_BATCH][4];
    // heads h + i lanes < end of rows at src
    auto load = [&](const float *src, int h, int end, bool rotated) {
#pragma unroll
        for (int i = 0; i < NR_BATCH; ++i) {
            if (h + i * lanes < end && owner) {
                read(src + (int64_t)(h + i * lanes) * D, rotated, a[i], c[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) a[i][j] = c[i][j] = 0.f;
            }
        }
    };
    // the block's heads of each kind
    const int kv = p.c.heads, q0 = min(h0, p.q_heads), q1 = min(h1, p.q_heads);
    const int k0 = min(max(h0 - p.q_heads, 0), kv), k1 = min(max(h1 - p.q_heads, 0), kv);
    const int v0 = min(max(h0 - p.q_heads - kv, 0), kv), v1 = min(max(h1 - p.q_heads - kv, 0), kv);
    const float *q_src = p.q + row * p.ldq, *k_src = p.k + row * p.ldk, *v_src = p.v + row * p.ldv;
    const int first = q0 < q1 ? Q : k0 < k1 ? K : V;             // its first heads come while the sines are computed
    load(first == Q ? q_src : first == K ? k_src : v_src, (first == Q ? q0 : first == K ? k0 : v0) + hl, first == Q ? q1 : first == K ? k1 : v1,
         first != V);

    const int slot = cache_len(p.c, b, KID_NORM) - n + t;
    bool store = slot >= 0;
    int64_t page = 0;
    int off = 0;
    if (store) {
        const int col = p.page_div.of(slot);
        off = slot - col * p.c.page_size;
        const int pg = cache_page(p.c, b, col, KID_NORM);
        store = pg >= 0;
        page = pg;
    } else {
        record_error(MMQ_ERR_INDEX, KID_NORM, SITE_LEN);
    }
    const int first_pos = *(p.pos + row);
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
        int ax = p.axis ? *(p.axis + i) : 0;
        if (ax < 0 || ax >= p.axes) {
            record_error(MMQ_ERR_INDEX, KID_NORM, SITE_AXIS);
            ax = 0;
        }
        const int x = ax == 0 ? first_pos : *(p.pos + ax * p.rows + row);
        const uint64_t turned = (uint64_t)(int64_t)x * (uint64_t)*(p.freq + i);
        float sine, cosine;
        sincospif((float)(int32_t)(turned >> 32) * 0x1p-31f, &sine, &cosine);
        s_cos[i] = cosine * p.magnitude;
        s_sin[i] = sine * p.magnitude;
    }
    __syncthreads();

    // All threads take the same number of steps: the shuffles need whole warps.
    auto heads = [&](auto kind_, const float *src, int from, int to) {
        constexpr int kind = decltype(kind_)::value;
        if (from >= to) return;
        // y0 = r (x0 w0 cos - x1 w1 sin), y1 = r (x0 w0 sin + x1 w1 cos); pairs that do not turn have cos 1 and no sine (0 times
        // a value that is not finite would be NaN in the other one)
        const float *weight = kind == Q ? p.q_norm : p.k_norm;
        const bool normed = kind != V && weight != nullptr;
        float c0[4], s0[4], c1[4], s1[4];
        if (kind != V) {
            float w0[4] = {1.f, 1.f, 1.f, 1.f}, w1[4] = {1.f, 1.f, 1.f, 1.f};
            if (normed && owner) read(weight, true, w0, w1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool turns = WIDE ? u * 4 < half : u * 4 + j < half;
                const float cs = turns ? s_cos[u * 4 + j] : 1.f, sn = turns ? s_sin[u * 4 + j] : 0.f;
                c0[j] = w0[j] * cs, s0[j] = w0[j] * sn, c1[j] = w1[j] * cs, s1[j] = w1[j] * sn;
            }
        }
        for (int hb = from; hb < to; hb += lanes * NR_BATCH) {
            if (kind != first || hb != from) load(src, hb + hl, to, kind != V);
#pragma unroll
            for (int i = 0; i < NR_BATCH; ++i) {
                const int h = hb + hl + i * lanes;
                if (normed) {
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) ss = fmaf(a[i][j], a[i][j], fmaf(c[i][j], c[i][j], ss));
                    for (int o = p.group >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float r = rsqrtf(ss * p.inv_dim + p.eps);
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[i][j] *= r, c[i][j] *= r;
                }
                if (h >= to || !owner) continue;
                if (kind != V) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool turns = WIDE ? u * 4 < half : u * 4 + j < half;
                        const float x0 = a[i][j], x1 = c[i][j];
                        a[i][j] = turns ? x0 * c0[j] - x1 * s1[j] : x0 * c0[j];
                        c[i][j] = turns ? x0 * s0[j] + x1 * c1[j] : x1 * c1[j];
                    }
                }
                if (kind == Q) {
                    if (p.q_f32) write(static_cast<float *>(p.q_out) + row * p.ldo + (int64_t)h * D, true, a[i], c[i]);
                    else write(static_cast<T *>(p.q_out) + row * p.ldo + (int64_t)h * D, true, a[i], c[i]);
                } else if (store) {
                    write(kind == V ? static_cast<T *>(p.c.v) + page * p.c.v_page + h * p.c.v_head + off * p.c.v_slot
                                    : static_cast<T *>(p.c.k) + page * p.c.k_page + h * p.c.k_head + off * p.c.k_slot,
                          kind != V, a[i], c[i]);
                    if (kind == K && u == 0) {
                        const int64_t e = (page * kv + h) * p.c.page_size + off;
                        if (p.c.weight) p.c.weight[e] = 0.f;
                        if (p.c.pos) p.c.pos[e] = first_pos;
                    }
                }
            }
        }
    };
    heads(std::integral_constant<int, Q>{}, q_src, q0, q1);
    heads(std::integral_constant<int, K>{}, k_src, k0, k1);
    heads(std::integral_constant<int, V>{}, v_src, v0, v1);
}

template <typename T>
int launch_norm_rope(NormRopeParams &p, cudaStream_t stream)
{
    const int total = p.q_heads + 2 * p.c.heads;
    p.group = 1;
    while (p.group * 8 < p.c.dim) p.group *= 2;
    const int lanes = NR_THREADS / p.group;
    // One block walks all heads of a row when there are rows enough to fill the device; with few rows, a row's heads are
    // spread over blocks down to one pass of the block's groups each.
    int64_t parts = ((int64_t)sm_count() * 4 + p.rows - 1) / p.rows;
    const int most = (total + lanes - 1) / lanes;
    if (parts > most) parts = most;
    p.heads_per_block = (int)((total + parts - 1) / parts);
    p.heads_per_block = (p.heads_per_block + lanes - 1) / lanes * lanes;
    const dim3 grid((unsigned)p.rows, (unsigned)((total + p.heads_per_block - 1) / p.heads_per_block));
    return launch_pdl(p.rot % 8 == 0 ? norm_rope_kernel<T, true> : norm_rope_kernel<T, false>, grid, NR_THREADS, 0, stream, 0, p);
}

}  // namespace
}  // namespace mmq

extern "C" int mmq_norm_rope_append(const mmq_kv_cache *cache, const int64_t *freq, const int32_t *axis, int rot, float magnitude,
                                    int interleaved, const float *q_norm, const float *k_norm, float eps, const float *q, int64_t ldq,
                                    const float *k, int64_t ldk, const float *v, int64_t ldv, const int32_t *pos, int axes,
                                    const int32_t *new_len, void *q_out, int64_t ldo, int q_dtype, int q_heads, int new_tokens,
                                    mmq_stream_t stream)
{
    using namespace mmq;
    int rc = check_cache(cache);
    if (rc != MMQ_OK) return rc;
    const int64_t D = cache->dim;
    if (rot < 2 || rot > D || (rot & 1) || q_heads < 1 || q_heads > 65535 || new_tokens < 0 || axes < 1 || axes > 8 ||
        (int64_t)cache->seqs * new_tokens > 0x7fffffff || ldq < q_heads * D || ldo < q_heads * D || ldk < cache->heads * D ||
        ldv < cache->heads * D || !(eps >= 0.f) || (q_dtype != MMQ_F32 && q_dtype != cache->dtype) ||
        (q && q == q_out && (ldq != ldo || q_dtype != MMQ_F32)))
        return MMQ_ERR_SHAPE;
    if (cache->seqs == 0 || new_tokens == 0) return MMQ_OK;
    if (!freq || !q || !k || !v || !pos || !q_out || (axes > 1 && !axis)) return MMQ_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(q_norm) || !aligned16(k_norm) ||
        ((ldq | ldk | ldv) & 3) || (ldo & (q_dtype == MMQ_F32 ? 3 : 7)))
        return MMQ_ERR_ALIGN;
    if ((rc = check_arch()) != MMQ_OK) return rc;
    NormRopeParams p = {*cache, freq, axis, q_norm, k_norm, q, k, v, pos, new_len, q_out, ldq, ldk, ldv, ldo,
                        (int64_t)cache->seqs * new_tokens, magnitude, eps, 1.f / (float)D, rot, interleaved ? 1 : 0, axes, q_heads, new_tokens,
                        q_dtype == MMQ_F32 ? 1 : 0, 0, 0, FastDiv(cache->page_size)};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return cache->dtype == MMQ_F16 ? launch_norm_rope<__half>(p, st) : launch_norm_rope<__nv_bfloat16>(p, st);
}
