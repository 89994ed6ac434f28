// mmq_rope.cuh -- rotary positions on f32 q and k rows, and the append of the
// new keys and values to the paged cache (mmq_rope_append).
//
// Pair (a, b) at position x turns by 2 pi frac(x f / 2^64), f being turns per
// position as a 64-bit fraction.  The 64-bit product keeps the low 64 bits,
// which is the fraction of the turns exactly; its high 32 bits as a signed
// number, times 2^-31, are the half turns in [-1, 1) that sincospi takes, so
// no range reduction is needed and no position is too large.
//
// Bound by memory: per row 8 B per q value (read, write) and 6 B per k and v
// value.  One thread owns the same eight values (four pairs) of several heads;
// a block's threads cover whole heads side by side, one block per row and part
// of its heads.  The row's sines and cosines are computed once per block, while
// the first heads' loads are in flight.
// Measured: 4096 rows of 32 + 2*32 heads of 128, 58 us = 5.8 TB/s (the copy
// rate is 6.8); 512 rows of 32 + 2*8, 6.8 us; one row 2.4 us.
#pragma once

namespace mmq {
namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_BATCH = 3;        // heads whose loads a thread has in flight

struct RopeParams {
    mmq_kv_cache c;
    const int64_t *freq;
    const float *q, *k, *v;
    const int32_t *pos, *new_len;
    float *q_out;
    int64_t ldq, ldk, ldv, ldo;
    float magnitude;
    int rot, interleaved, q_heads, new_tokens;
    int heads_per_block;             // of the row's q_heads + 2*heads
    FastDiv page_div;
};

// P pairs per thread: 4 where rot and dim are multiples of 8 (16-byte
// accesses), else 1.
template <typename T, int P>
__global__ void __launch_bounds__(ROPE_THREADS, 4) rope_append_kernel(const RopeParams p)
{
    __shared__ __align__(16) float s_cos[128], s_sin[128];
    pdl_wait();
    pdl_launch_dependents();
    const int D = p.c.dim, units = D / (2 * P);
    const int u = threadIdx.x % units, hl = threadIdx.x / units, lanes = blockDim.x / units;
    const int row = blockIdx.x, b = row / p.new_tokens, t = row - b * p.new_tokens;
    const int total = p.q_heads + 2 * p.c.heads;
    const int h0 = blockIdx.y * p.heads_per_block;
    const int h1 = min(total, h0 + p.heads_per_block);
    const bool rotated = u * 2 * P < p.rot;
    // element offsets of the thread's first and second P values within a head
    int e0 = u * 2 * P, e1 = e0 + P;
    if (rotated && !p.interleaved) {
        e0 = u * P;
        e1 = p.rot / 2 + u * P;
    }
    const int n = new_count(p.new_len, b, p.new_tokens, KID_ROPE);
    const int len = cache_len(p.c, b, KID_ROPE);
    const int slot = len - n + t;
    bool live = t < n, store = live;
    int64_t page = 0;
    int off = 0;
    if (live) {
        if (slot < 0) {
            record_error(MMQ_ERR_INDEX, KID_ROPE, SITE_LEN);
            store = false;
        } else {
            const int col = p.page_div.of(slot);
            off = slot - col * p.c.page_size;
            const int pg = cache_page(p.c, b, col, KID_ROPE);
            store = pg >= 0;
            page = pg;
        }
    }
    // The row's heads: q, k, v.  A batch of heads is in flight at a time, the first while the sines are computed.
    const int x = *(p.pos + row);
    float a[ROPE_BATCH][P], c[ROPE_BATCH][P];
    auto load = [&](int hb) {
#pragma unroll
        for (int i = 0; i < ROPE_BATCH; ++i) {
            const int h = hb + i * lanes;
            if (h >= h1 || !live) continue;
            const bool is_v = h >= p.q_heads + p.c.heads;
            const float *src = h < p.q_heads ? p.q + row * p.ldq + (int64_t)h * D
                               : !is_v       ? p.k + row * p.ldk + (int64_t)(h - p.q_heads) * D
                                             : p.v + row * p.ldv + (int64_t)(h - p.q_heads - p.c.heads) * D;
            const int s0 = is_v ? u * 2 * P : e0, s1 = is_v ? u * 2 * P + P : e1;
            if constexpr (P == 4) {
                *reinterpret_cast<float4 *>(a[i]) = *reinterpret_cast<const float4 *>(src + s0);
                *reinterpret_cast<float4 *>(c[i]) = *reinterpret_cast<const float4 *>(src + s1);
            } else {
                a[i][0] = src[s0];
                c[i][0] = src[s1];
            }
        }
    };
    load(h0 + hl);
    for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) {
        const uint64_t turns = (uint64_t)(int64_t)x * (uint64_t)*(p.freq + i);
        float sine, cosine;
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sine, &cosine);
        s_cos[i] = cosine * p.magnitude;
        s_sin[i] = sine * p.magnitude;
    }
    __syncthreads();
    if (hl >= lanes) return;
    float cs[P], sn[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        cs[i] = rotated ? s_cos[u * P + i] : 1.f;
        sn[i] = rotated ? s_sin[u * P + i] : 0.f;
    }

    for (int hb = h0 + hl; hb < h1; hb += lanes * ROPE_BATCH) {
        if (hb != h0 + hl) load(hb);
#pragma unroll
        for (int i = 0; i < ROPE_BATCH; ++i) {
            const int h = hb + i * lanes;
            if (h >= h1) continue;
            const bool is_v = h >= p.q_heads + p.c.heads, turn = rotated && !is_v;
            const int d0 = is_v ? u * 2 * P : e0, d1 = is_v ? u * 2 * P + P : e1;
            float y0[P], y1[P];
            if (P == 4 && turn && p.interleaved) {              // pairs side by side: (a0 a1) (a2 a3) (c0 c1) (c2 c3)
#pragma unroll
                for (int j = 0; j < P; j += 2) {
                    const int n = (j + 1) % P, s = j / 2, w = (P / 2 + j / 2) % P;
                    y0[j] = a[i][j] * cs[s] - a[i][n] * sn[s];
                    y0[n] = a[i][j] * sn[s] + a[i][n] * cs[s];
                    y1[j] = c[i][j] * cs[w] - c[i][n] * sn[w];
                    y1[n] = c[i][j] * sn[w] + c[i][n] * cs[w];
                }
            } else {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    y0[j] = turn ? a[i][j] * cs[j] - c[i][j] * sn[j] : a[i][j];
                    y1[j] = turn ? a[i][j] * sn[j] + c[i][j] * cs[j] : c[i][j];
                }
            }
            if (h < p.q_heads) {
                float *dst = p.q_out + row * p.ldo + (int64_t)h * D;
                if (!live) {
#pragma unroll
                    for (int j = 0; j < P; ++j) y0[j] = y1[j] = 0.f;
                }
                if constexpr (P == 4) {
                    *reinterpret_cast<float4 *>(dst + d0) = *reinterpret_cast<float4 *>(y0);
                    *reinterpret_cast<float4 *>(dst + d1) = *reinterpret_cast<float4 *>(y1);
                } else {
                    dst[d0] = y0[0];
                    dst[d1] = y1[0];
                }
                continue;
            }
            if (!store) continue;
            const int kh = is_v ? h - p.q_heads - p.c.heads : h - p.q_heads;
            T *dst = is_v ? static_cast<T *>(p.c.v) + page * p.c.v_page + kh * p.c.v_head + off * p.c.v_slot
                          : static_cast<T *>(p.c.k) + page * p.c.k_page + kh * p.c.k_head + off * p.c.k_slot;
            if constexpr (P == 4) {
                const uint2 w0 = make_uint2(pack2<T>(y0[0], y0[1]), pack2<T>(y0[2], y0[3]));
                const uint2 w1 = make_uint2(pack2<T>(y1[0], y1[1]), pack2<T>(y1[2], y1[3]));
                if (d1 == d0 + 4) {
                    *reinterpret_cast<uint4 *>(dst + d0) = make_uint4(w0.x, w0.y, w1.x, w1.y);
                } else {
                    *reinterpret_cast<uint2 *>(dst + d0) = w0;
                    *reinterpret_cast<uint2 *>(dst + d1) = w1;
                }
            } else {
                dst[d0] = to_cache<T>(y0[0]);
                dst[d1] = to_cache<T>(y1[0]);
            }
            if (!is_v && u == 0) {
                const int64_t e = (page * p.c.heads + kh) * p.c.page_size + off;
                if (p.c.weight) p.c.weight[e] = 0.f;
                if (p.c.pos) p.c.pos[e] = x;
            }
        }
    }
}

template <typename T>
int launch_rope(RopeParams &p, int sms, cudaStream_t stream)
{
    const int D = p.c.dim, total = p.q_heads + 2 * p.c.heads;
    const bool wide = p.rot % 8 == 0;
    const int units = wide ? D / 8 : D / 2;
    const int lanes = ROPE_THREADS / units > 0 ? ROPE_THREADS / units : 1;
    const int64_t rows = (int64_t)p.c.seqs * p.new_tokens;
    // One block walks all heads of a row when there are rows enough to fill the
    // device; with few rows, a row's heads are spread over blocks down to one
    // pass of the block's lanes each.
    const int64_t want = (int64_t)sms * 4;                // resident blocks
    int64_t parts = (want + rows - 1) / rows;
    const int most = (total + lanes - 1) / lanes;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    p.heads_per_block = (int)((total + parts - 1) / parts);
    p.heads_per_block = (p.heads_per_block + lanes - 1) / lanes * lanes;
    const dim3 grid((unsigned)rows, (unsigned)((total + p.heads_per_block - 1) / p.heads_per_block));
    return launch_pdl(wide ? rope_append_kernel<T, 4> : rope_append_kernel<T, 1>, grid, units * lanes, 0, stream, 0, p);
}

}  // namespace
}  // namespace mmq

extern "C" int mmq_rope_append(const mmq_kv_cache *cache, const int64_t *freq, int rot, float magnitude,
                               int interleaved, const float *q, int64_t ldq, const float *k, int64_t ldk,
                               const float *v, int64_t ldv, const int32_t *pos, const int32_t *new_len, float *q_out,
                               int64_t ldo, int q_heads, int new_tokens, mmq_stream_t stream)
{
    using namespace mmq;
    int rc = check_cache(cache);
    if (rc != MMQ_OK) return rc;
    const int64_t D = cache->dim;
    if (rot < 2 || rot > D || (rot & 1) || q_heads < 1 || q_heads > 65535 || new_tokens < 0 ||
        (int64_t)cache->seqs * new_tokens > 0x7fffffff || ldq < q_heads * D || ldo < q_heads * D ||
        ldk < cache->heads * D || ldv < cache->heads * D || (q == q_out && ldq != ldo))
        return MMQ_ERR_SHAPE;
    if (cache->seqs == 0 || new_tokens == 0) return MMQ_OK;
    if (!freq || !q || !k || !v || !pos || !q_out) return MMQ_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || ((ldq | ldk | ldv | ldo) & 3))
        return MMQ_ERR_ALIGN;
    if ((rc = check_arch()) != MMQ_OK) return rc;
    RopeParams p = {*cache, freq, q, k, v, pos, new_len, q_out, ldq, ldk, ldv, ldo, magnitude, rot, interleaved ? 1 : 0,
                    q_heads, new_tokens, 0, FastDiv(cache->page_size)};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return cache->dtype == MMQ_F16 ? launch_rope<__half>(p, sm_count(), st)
                                   : launch_rope<__nv_bfloat16>(p, sm_count(), st);
}
