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
// group of 1 to 32 neighbouring threads that add their squares by shuffles; a
// block's groups take heads side by side, with several heads' loads under way,
// and the row's sines are computed once per block meanwhile.
#pragma once

namespace mmq {
namespace {

constexpr int NR_THREADS = 256;
constexpr int NR_BATCH = 3;          // heads whose loads a thread has in flight

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
__global__ void __launch_bounds__(NR_THREADS, 4) norm_rope_kernel(const NormRopeParams p)
{
    __shared__ float s_cos[128], s_sin[128];
    pdl_wait();
    pdl_launch_dependents();
    const int D = p.c.dim, half = p.rot / 2;
    const int u = threadIdx.x & (p.group - 1), hl = threadIdx.x / p.group, lanes = blockDim.x / p.group;
    const int64_t row = blockIdx.x;
    const int b = (int)(row / p.new_tokens), t = (int)(row - (int64_t)b * p.new_tokens);
    const int total = p.q_heads + 2 * p.c.heads;
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(total, h0 + p.heads_per_block);
    const bool owner = u * 8 < D;                                // groups are rounded up to a power of two
    const bool turns = WIDE ? u * 8 < p.rot : true;
    // The thread's pairs are (a[j], b[j]).  Where they lie: WIDE in two runs of four (halves apart, or side by side),
    // else pair k = 4u + j at (k, k + half), (2k, 2k + 1) interleaved or past the rotated ones.
    const bool apart = !p.interleaved && turns;
    const int e0 = apart ? u * 4 : u * 8, e1 = apart ? half + u * 4 : u * 8 + 4;
    auto place = [&](int j, int &x, int &y, bool rotated) {      // !WIDE
        const int k = u * 4 + j;
        x = rotated && k < half && !p.interleaved ? k : 2 * k;
        y = rotated && k < half && !p.interleaved ? k + half : 2 * k + 1;
    };
    auto read = [&](const float *src, bool rotated, float (&a)[4], float (&c)[4]) {
        if constexpr (WIDE) {
            const bool ap = rotated && apart;
            const float4 x = *reinterpret_cast<const float4 *>(src + (ap ? e0 : u * 8));
            const float4 y = *reinterpret_cast<const float4 *>(src + (ap ? e1 : u * 8 + 4));
            if (ap) {
                a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
                c[0] = y.x, c[1] = y.y, c[2] = y.z, c[3] = y.w;
            } else {
                a[0] = x.x, c[0] = x.y, a[1] = x.z, c[1] = x.w;
                a[2] = y.x, c[2] = y.y, a[3] = y.z, c[3] = y.w;
            }
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
    const int n = new_count(p.new_len, b, p.new_tokens, KID_NORM);
    const int len = cache_len(p.c, b, KID_NORM);
    const int slot = len - n + t;
    const bool live = t < n;
    bool store = live;
    int64_t page = 0;
    int off = 0;
    if (live) {
        if (slot < 0) {
            record_error(MMQ_ERR_INDEX, KID_NORM, SITE_LEN);
            store = false;
        } else {
            const int col = p.page_div.of(slot);
            off = slot - col * p.c.page_size;
            const int pg = cache_page(p.c, b, col, KID_NORM);
            store = pg >= 0;
            page = pg;
        }
    }
    float a[NR_BATCH][4], c[NR_BATCH][4];
    auto load = [&](int hb) {
#pragma unroll
        for (int i = 0; i < NR_BATCH; ++i) {
            const int h = hb + i * lanes;
#pragma unroll
            for (int j = 0; j < 4; ++j) a[i][j] = c[i][j] = 0.f;
            if (h >= h1 || !live || !owner) continue;
            const bool is_v = h >= p.q_heads + p.c.heads;
            const float *src = h < p.q_heads ? p.q + row * p.ldq + (int64_t)h * D
                               : !is_v       ? p.k + row * p.ldk + (int64_t)(h - p.q_heads) * D
                                             : p.v + row * p.ldv + (int64_t)(h - p.q_heads - p.c.heads) * D;
            read(src, !is_v, a[i], c[i]);
        }
    };
    load(h0 + hl);
    float qa[4], qc[4], ka[4], kc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) qa[j] = qc[j] = ka[j] = kc[j] = 1.f;
    if (owner && p.q_norm) read(p.q_norm, true, qa, qc);
    if (owner && p.k_norm) read(p.k_norm, true, ka, kc);
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
    float cs[4], sn[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool r = u * 4 + j < half;
        cs[j] = r ? s_cos[u * 4 + j] : 1.f;
        sn[j] = r ? s_sin[u * 4 + j] : 0.f;
    }

    // every thread takes the same number of steps: the shuffles need whole warps
    for (int hb = h0; hb < h1; hb += lanes * NR_BATCH) {
        if (hb != h0) load(hb + hl);
#pragma unroll
        for (int i = 0; i < NR_BATCH; ++i) {
            const int h = hb + hl + i * lanes;
            const bool is_v = h >= p.q_heads + p.c.heads, is_q = h < p.q_heads;
            const bool normed = is_q ? p.q_norm != nullptr : !is_v && p.k_norm != nullptr;
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fmaf(a[i][j], a[i][j], fmaf(c[i][j], c[i][j], ss));
            for (int o = p.group >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (h >= h1 || !owner) continue;
            float y0[4], y1[4];
            const float r = normed ? rsqrtf(ss * p.inv_dim + p.eps) : 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v0 = a[i][j], v1 = c[i][j];
                if (normed) {
                    v0 = v0 * r * (is_q ? qa[j] : ka[j]);
                    v1 = v1 * r * (is_q ? qc[j] : kc[j]);
                }
                y0[j] = is_v ? v0 : v0 * cs[j] - v1 * sn[j];
                y1[j] = is_v ? v1 : v0 * sn[j] + v1 * cs[j];
                // pairs that do not turn pass as they are
                if (!is_v && u * 4 + j >= half) {
                    y0[j] = v0;
                    y1[j] = v1;
                }
                if (!live) y0[j] = y1[j] = 0.f;
            }
            if (!is_q && !store) continue;
            const int kh = is_v ? h - p.q_heads - p.c.heads : h - p.q_heads;
            const bool as_f32 = is_q && p.q_f32;
            T *dst = is_q   ? static_cast<T *>(p.q_out) + (as_f32 ? 0 : row * p.ldo + (int64_t)h * D)
                     : is_v ? static_cast<T *>(p.c.v) + page * p.c.v_page + kh * p.c.v_head + off * p.c.v_slot
                            : static_cast<T *>(p.c.k) + page * p.c.k_page + kh * p.c.k_head + off * p.c.k_slot;
            float *dst32 = static_cast<float *>(p.q_out) + row * p.ldo + (int64_t)h * D;
            if constexpr (WIDE) {
                const bool ap = !is_v && apart;
                float4 x = ap ? make_float4(y0[0], y0[1], y0[2], y0[3]) : make_float4(y0[0], y1[0], y0[1], y1[1]);
                float4 y = ap ? make_float4(y1[0], y1[1], y1[2], y1[3]) : make_float4(y0[2], y1[2], y0[3], y1[3]);
                const int d0 = ap ? e0 : u * 8, d1 = ap ? e1 : u * 8 + 4;
                if (as_f32) {
                    *reinterpret_cast<float4 *>(dst32 + d0) = x;
                    *reinterpret_cast<float4 *>(dst32 + d1) = y;
                } else {
                    const uint2 w0 = make_uint2(pack2<T>(x.x, x.y), pack2<T>(x.z, x.w));
                    const uint2 w1 = make_uint2(pack2<T>(y.x, y.y), pack2<T>(y.z, y.w));
                    if (!ap) {
                        *reinterpret_cast<uint4 *>(dst + d0) = make_uint4(w0.x, w0.y, w1.x, w1.y);
                    } else {
                        *reinterpret_cast<uint2 *>(dst + d0) = w0;
                        *reinterpret_cast<uint2 *>(dst + d1) = w1;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    int x, y;
                    place(j, x, y, !is_v);
                    if (as_f32) {
                        dst32[x] = y0[j];
                        dst32[y] = y1[j];
                    } else {
                        dst[x] = to_cache<T>(y0[j]);
                        dst[y] = to_cache<T>(y1[j]);
                    }
                }
            }
            if (!is_q && !is_v && u == 0) {
                const int64_t e = (page * p.c.heads + kh) * p.c.page_size + off;
                if (p.c.weight) p.c.weight[e] = 0.f;
                if (p.c.pos) p.c.pos[e] = first_pos;
            }
        }
    }
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
