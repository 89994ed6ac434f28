"""GPU tests of the decode-side operators (rotary append, paged attention,
eviction, verification) against plain 64-bit implementations.

Tolerances, derived before any run:
* rotation, f32: the half-turn argument is rounded once (an angle error of at
  most pi 2^-25), sine and cosine to 2 ulp, magnitude, two products and a sum
  to half an ulp each: together below 8 ulp of 2^-24 of (|a| + |b|) magnitude;
  a stored key or value adds half an ulp of its type.
* attention: q enters as 22 bits of the row's largest value or better and the
  dot products and their scaling round in f32, so a score is off by at most
  2^-20 of scale sum|q||k|, and a probability by twice that, relatively; p
  keeps 22 bits, and the sums over entries add at most 2^-19 relatively.  The
  output is off by at most (2 ds + 2^-19) max|v|.  Accumulated weights: the
  same without max|v|, per row that adds to them.
* eviction and verification: equal.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import serve_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_prefill_gemm_mmq_gb300 import ops as _ops
    from quantized_prefill_gemm_mmq_gb300 import _lib
    _lib.load()
    return _ops


def make_cache(ops, lens, heads, dim, page, dtype=torch.float16, layout="hnd", seed=0, extra=0, track=True, fill=None):
    """A cache with shuffled pages, one spare page, and random entries; what lies past the lengths is `fill`."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    cols = max(1, -(-(max(lens + [1]) + extra) // page))
    pages = B * cols + 1
    perm = torch.randperm(pages, generator=g)[:B * cols].to(torch.int32).view(B, cols)
    pools = []
    for _ in range(2):
        p = torch.randn((pages, heads, page, dim), generator=g).to(dtype)
        if fill is not None:
            keep = torch.zeros((pages, page), dtype=torch.bool)
            for b in range(B):
                for s in range(lens[b]):
                    keep[perm[b, s // page], s % page] = True
            p = torch.where(keep[:, None, :, None], p, torch.full((), fill, dtype=dtype))
        p = p.cuda()
        pools.append(p if layout == "hnd" else p.transpose(1, 2).contiguous().transpose(1, 2))
    w = torch.rand((pages, heads, page), generator=g).cuda() if track else None
    pos = torch.zeros((pages, heads, page), dtype=torch.int32).cuda() if track else None
    return ops.KVCache(pools[0], pools[1], perm.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), w, pos)


# --------------------------------------------------------------- rotation ---

@pytest.mark.parametrize("B,N,Hq,H,dim,rot,inter,dtype,page,layout,scaling", [
    (1, 1, 4, 4, 128, 128, False, torch.float16, 16, "hnd", "none"),
    (1, 1, 1, 1, 8, 8, True, torch.bfloat16, 1, "hnd", "linear"),
    (3, 5, 8, 2, 128, 64, True, torch.bfloat16, 7, "nhd", "by_parts"),
    (2, 70, 6, 3, 80, 40, False, torch.float16, 24, "nhd", "base"),
    (1, 33, 2, 1, 256, 256, False, torch.float16, 64, "hnd", "by_parts"),
    (2, 3, 4, 2, 64, 6, False, torch.float16, 5, "hnd", "none"),      # pairs that no 16-byte access fits
    (2, 3, 4, 2, 72, 70, True, torch.bfloat16, 5, "hnd", "none"),
    (1, 700, 32, 8, 128, 128, False, torch.float16, 64, "hnd", "none"),
])
def test_rope_append(ops, B, N, Hq, H, dim, rot, inter, dtype, page, layout, scaling):
    g = torch.Generator().manual_seed(B * N + dim)
    new = [N] + [max(0, N - 2 * b) for b in range(1, B)]
    lens = [N + 3 + 11 * b for b in range(B)]
    cache = make_cache(ops, lens, H, dim, page, dtype, layout)
    before = [t.cpu().clone() for t in (cache.k, cache.v, cache.weight, cache.pos)]
    row = torch.randn((B * N, (Hq + 2 * H) * dim), generator=g)
    pos = torch.randint(0, 40000, (B * N,), generator=g, dtype=torch.int32)
    pos[0] = 1 << 30
    factor = 1.0 if scaling == "none" else 4.0
    table = ops.rope_table(rot, base=10000.0, scaling=scaling, factor=factor, context=512)
    inv, mag = ops.rope_frequencies(rot, 10000.0, scaling, factor, 512)
    d = row.cuda()
    q, k, v = (d[:, a * dim:b * dim].view(B * N, b - a, dim) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    out = ops.rope_append(cache, table, q, k, v, pos.cuda(), interleaved=inter,
                          new=torch.tensor(new, dtype=torch.int32).cuda() if B > 1 else None)
    ops.check_status()
    # the angle of the 64-bit table itself: 2 pi frac(x f / 2^64)
    fixed = ops.rope_fixed(inv)
    def rotate(x):
        y = x.double().clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            ang = torch.tensor([2 * math.pi * (((int(p) * fixed[i]) % (1 << 64)) / 2.0 ** 64) for p in pos], dtype=torch.float64)
            c, s = (torch.cos(ang) * mag)[:, None], (torch.sin(ang) * mag)[:, None]
            u, w = x[:, :, a].double(), x[:, :, b].double()
            y[:, :, a], y[:, :, b] = u * c - w * s, u * s + w * c
        return y
    def bound(x):
        e = x.double().abs()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            e[:, :, a] = e[:, :, b] = (x[:, :, a].double().abs() + x[:, :, b].double().abs()) * mag
        return e * 8 * 2.0 ** -24
    qc, kc, vc = (t.cpu() for t in (q, k, v))
    live = torch.tensor([t < new[b] for b in range(B) for t in range(N)])
    want, tol = rotate(qc), bound(qc)
    want[~live] = 0
    assert bool(((out.cpu().double() - want).abs() <= tol).all())
    # the f64 definition by frequency agrees where positions are small
    small = pos < 2000
    assert torch.allclose(rotate(qc)[small], ref.rope(qc, pos, inv, mag, rot, inter)[small], rtol=0, atol=1e-9)
    kw, kt = rotate(kc), bound(kc)
    half = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    got_k, got_v, got_w, got_p = (t.cpu() for t in (cache.k, cache.v, cache.weight, cache.pos))
    tab = cache.table.cpu()
    touched = torch.zeros(got_w.shape[0], got_w.shape[2], dtype=torch.bool)
    for b in range(B):
        for t in range(new[b]):
            pg, off = ref.slot_place(tab, page, b, lens[b] - new[b] + t)
            r = b * N + t
            assert bool(((got_k[pg, :, off].double() - kw[r]).abs() <= kt[r] + kw[r].abs() * half * 1.01 + 2.0 ** -25).all())
            assert torch.equal(got_v[pg, :, off], vc[r].to(dtype))
            assert bool((got_w[pg, :, off] == 0).all()) and bool((got_p[pg, :, off] == pos[r]).all())
            touched[pg, off] = True
    for got, was in zip((got_k, got_v, got_w, got_p), before):           # nothing else is written
        same = (got == was) if got.dim() == 3 else (got == was).all(-1)
        assert bool((same | touched[:, None]).all())


def test_rope_in_place_and_no_bookkeeping(ops):
    cache = make_cache(ops, [9, 40], 2, 64, 16, track=False)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((2, h, 64), generator=g).cuda() for h in (4, 2, 2))
    pos = torch.tensor([8, 39], dtype=torch.int32).cuda()
    table = ops.rope_table(64)
    want = ops.rope_append(cache, table, q, k, v, pos)
    got = ops.rope_append(cache, table, q, k, v, pos, out=q)
    assert got is q and torch.equal(q, want)
    ops.check_status()


def test_rope_position_zero_is_identity(ops):
    cache = make_cache(ops, [1], 1, 128, 16)
    q = torch.randn((1, 3, 128)).cuda()
    k, v = torch.randn((1, 1, 128)).cuda(), torch.randn((1, 1, 128)).cuda()
    out = ops.rope_append(cache, ops.rope_table(128), q, k, v, torch.zeros(1, dtype=torch.int32).cuda())
    assert torch.equal(out, q)


# -------------------------------------------------------------- attention ---

def check_attention(ops, lens, N, Hq, H, dim, page, dtype, layout="hnd", new=None, accumulate=False, seed=1, qscale=1.0,
                    scale=None, fill=None, cache=None, q=None):
    B = len(lens)
    cache = cache or make_cache(ops, lens, H, dim, page, dtype, layout, seed=seed, fill=fill)
    g = torch.Generator().manual_seed(seed + 100)
    q = torch.randn((B * N, Hq, dim), generator=g) * qscale if q is None else q
    nw = new if new is not None else [N] * B
    w0 = cache.weight.cpu().double()
    ws = ops.attn_workspace(cache, Hq, N, accumulate)
    newt = torch.tensor(new, dtype=torch.int32).cuda() if new is not None else None
    out = ops.attn_decode(cache, q.cuda(), scale=scale, new=newt, accumulate=accumulate, workspace=ws)
    again = None if accumulate else ops.attn_decode(cache, q.cuda(), scale=scale, new=newt, workspace=ws)
    ops.check_status()
    tab = cache.table.cpu()
    kp, vp = cache.k.cpu(), cache.v.cpu()
    sc = dim ** -0.5 if scale is None else scale
    want, weights, reach = ref.attention(q, kp, vp, tab, lens, nw, page, sc)
    seen = [vp[ref.slot_place(tab, page, b, s)[0], :, s % page].double().abs().max() for b in range(B) for s in range(lens[b])]
    vmax = float(max([x for x in seen if math.isfinite(x)] + [0.0]))
    ds = reach * 2.0 ** -20
    tol = (2 * ds + 2.0 ** -19) * vmax
    got = out.cpu().double()
    assert bool(torch.isfinite(got).all())
    err = float((got - want).abs().max()) if got.numel() else 0.0
    assert err <= tol, (err, tol)
    if again is not None:
        assert torch.equal(out, again)
    w1 = cache.weight.cpu().double()
    if not accumulate:
        assert torch.equal(w0, w1)
        return cache
    rows = N * Hq // H
    covered = torch.zeros_like(w0, dtype=torch.bool)
    for b in range(B):
        for h in range(H):
            for s in range(lens[b]):
                pg, off = ref.slot_place(tab, page, b, s)
                add = float(weights[b, h][s])
                assert abs(float(w1[pg, h, off] - w0[pg, h, off]) - add) <= add * (2 * ds + 2.0 ** -19) + (1 + rows) * 2.0 ** -23
                covered[pg, h, off] = True
    assert torch.equal(w1[~covered], w0[~covered])
    return cache


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens", [[0], [1], [15], [16], [17], [63], [64], [65], [127], [128], [129], [0, 1, 200, 0, 64], [513]])
def test_attn_lengths(ops, lens, dtype):
    check_attention(ops, lens, 1, 4, 2, 128, 16, dtype, seed=len(lens) + lens[0])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [8, 16, 56, 64, 72, 80, 96, 128, 136, 192, 256])
@pytest.mark.parametrize("group", [1, 3, 12])
def test_attn_dims(ops, dim, group, dtype):
    check_attention(ops, [150, 37], 1, 2 * group, 2, dim, 24, dtype, seed=dim + group)


@pytest.mark.parametrize("page", [1, 7, 16, 64, 100, 1024])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_attn_pages_and_layouts(ops, page, layout):
    check_attention(ops, [130, 61, 300], 1, 4, 4, 64, page, torch.float16, layout, accumulate=page == 7, fill=float("nan"))


@pytest.mark.parametrize("N,group,dim,dtype", [(2, 1, 128, torch.float16), (5, 4, 64, torch.bfloat16), (16, 1, 128, torch.bfloat16),
                                               (16, 8, 64, torch.float16), (7, 5, 256, torch.float16), (4, 8, 128, torch.bfloat16),
                                               (3, 8, 256, torch.bfloat16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_attn_new_tokens(ops, N, group, dim, dtype, accumulate):
    lens = [N, N + 63, 64 + N - 1, 190, 2]
    new = [N, N, max(1, N - 1), 0, min(N, 2)]
    check_attention(ops, lens, N, 2 * group, 2, dim, 16, dtype, new=new, accumulate=accumulate, seed=N, fill=float("inf"))


def test_attn_more_new_than_entries(ops):
    # rows whose mask leaves nothing: the first new tokens of a sequence with fewer entries than that
    cache = make_cache(ops, [2, 70], 2, 64, 16)
    q = torch.randn((10, 4, 64))
    out = ops.attn_decode(cache, q.cuda()).cpu()
    assert bool((out[:3] == 0).all()) and bool((out[3:] != 0).any(-1).all())
    check_attention(ops, [2, 70], 5, 4, 2, 64, 16, torch.float16, new=[2, 5])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,dim,group", [(torch.float16, 128, 1), (torch.bfloat16, 64, 4), (torch.float16, 256, 4)])
def test_attn_masked_entries_do_not_reach_earlier_rows(ops, bad, dtype, dim, group):
    N, lens = 4, [67, 131]
    cache = make_cache(ops, lens, 2, dim, 16, dtype)
    q = torch.randn((8, 2 * group, dim), generator=torch.Generator().manual_seed(5)).cuda()
    want = ops.attn_decode(cache, q)
    tab = cache.table.cpu()
    for b, n in enumerate(lens):                       # the last two new entries are not finite
        for s in (n - 2, n - 1):
            pg, off = ref.slot_place(tab, 16, b, s)
            cache.v[pg, :, off] = bad
            cache.k[pg, :, off] = bad
    got = ops.attn_decode(cache, q)
    ops.check_status()
    for b in range(2):
        a, w = got[b * N:b * N + 2], want[b * N:b * N + 2]
        assert bool(torch.isfinite(a).all())
        assert float((a - w).abs().max()) <= 2.0 ** -18 * float(w.abs().max())
        assert not bool(torch.isfinite(got[b * N + 2:b * N + 4]).any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,dim,group", [(torch.float16, 128, 1), (torch.bfloat16, 64, 1), (torch.bfloat16, 128, 4), (torch.bfloat16, 256, 4)])
def test_attn_rows_that_are_not_there_stay_zero(ops, bad, dtype, dim, group):
    # an entry that the other rows see is not finite; in one CTA's segments and in split ones
    N, lens, new = 3, [20, 90, 4000, 5], [1, 2, 1, 0]
    cache = make_cache(ops, lens, 2, dim, 16, dtype)
    tab = cache.table.cpu()
    for b in range(4):
        cache.v[ref.slot_place(tab, 16, b, 0)[0], :, 0] = bad
    q = torch.randn((12, 2 * group, dim), generator=torch.Generator().manual_seed(6)).cuda()
    for accumulate in (False, True):
        got = ops.attn_decode(cache, q, new=torch.tensor(new, dtype=torch.int32).cuda(), accumulate=accumulate)
        ops.check_status()
        for b in range(4):
            assert not bool(torch.isfinite(got[b * N:b * N + new[b]]).any())
            assert bool((got[b * N + new[b]:(b + 1) * N] == 0).all())
        assert bool(torch.isfinite(cache.weight).all())


@pytest.mark.parametrize("H,group,N,dim,dtype", [(1, 128, 16, 64, torch.bfloat16), (2, 20, 5, 128, torch.float16), (1, 71, 1, 192, torch.bfloat16),
                                                 (1, 33, 3, 256, torch.float16), (1, 12, 3, 96, torch.bfloat16)])
def test_attn_many_rows(ops, H, group, N, dim, dtype):
    # more rows than a CTA takes at once, up to the most there may be; and warps without rows
    for accumulate in (False, True):
        check_attention(ops, [150, 40], N, H * group, H, dim, 16, dtype, accumulate=accumulate, seed=group)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attn_long_split(ops, dtype):
    # one sequence over many CTAs, and a ragged batch whose CTAs hold several segments
    check_attention(ops, [30000], 1, 4, 1, 64, 64, dtype, seed=9)
    check_attention(ops, [5000] + [3] * 40 + [900], 1, 8, 8, 64, 16, dtype, seed=10)


def test_attn_shared_pages(ops):
    # two sequences with a common beginning in the same pages
    cache = make_cache(ops, [100, 130], 2, 64, 16)
    cache.table[1, :5] = cache.table[0, :5]
    check_attention(ops, [100, 130], 1, 4, 2, 64, 16, torch.float16, cache=cache)


def test_attn_many_sequences(ops):
    check_attention(ops, [1 + (37 * i) % 90 for i in range(300)], 1, 2, 1, 64, 16, torch.float16, seed=4)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("qscale,scale", [(1e6, 1e-7), (1e-6, 1e5), (1.0, 4.0), (0.0, None), (3.0, -0.1)])
def test_attn_magnitudes(ops, qscale, scale, dtype):
    check_attention(ops, [300, 20], 2, 4, 2, 128, 16, dtype, qscale=qscale, scale=scale)


def test_attn_lowest_scores(ops):
    # keys of the type's lowest value: every score is far below the others' range, the softmax is still exact
    cache = make_cache(ops, [70], 1, 64, 16)
    cache.k.fill_(-65504.0)
    q = torch.ones((1, 1, 64)).cuda()
    out = ops.attn_decode(cache, q)
    tab = cache.table.cpu()
    v = ref.gather(cache.v.cpu(), tab, 16, 0, 0, 70)
    assert float((out.cpu().double()[0, 0] - v.mean(0)).abs().max()) <= 2.0 ** -18 * float(v.abs().max())


def test_attn_stream_graph_and_strided_rows(ops):
    cache = make_cache(ops, [200, 77], 4, 128, 16)
    wide = torch.randn((2, 3 * 8 * 128)).cuda()
    q = wide[:, 8 * 128:16 * 128].view(2, 8, 128)
    want = ops.attn_decode(cache, q.contiguous())
    ws, out = ops.attn_workspace(cache, 8), torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.attn_decode(cache, q, out=out, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.attn_decode(cache, q, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    cache.lens.copy_(torch.tensor([33, 150], dtype=torch.int32))     # a replay follows the lengths on the device
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ops.attn_decode(cache, q))


def test_attn_offsets_past_32_bits(ops):
    """A pool of more than 2^31 elements: the last page is read and written."""
    pages, page, H, dim = 33000, 64, 8, 128                          # 2.16e9 elements, 4.3 GB each
    k = torch.empty((pages, H, page, dim), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    k[[0, pages - 1]] = torch.randn((2, H, page, dim), device="cuda", dtype=torch.float16)
    v[[0, pages - 1]] = torch.randn((2, H, page, dim), device="cuda", dtype=torch.float16)
    big = ops.KVCache(k, v, table, lens)
    small = ops.KVCache(k[[pages - 1, 0]].contiguous(), v[[pages - 1, 0]].contiguous(),
                        torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), lens)
    q = torch.randn((1, 8, dim), device="cuda")
    assert torch.equal(ops.attn_decode(big, q), ops.attn_decode(small, q))
    lens.fill_(3)
    row = torch.randn((1, 8, dim), device="cuda")
    ops.rope_append(big, ops.rope_table(dim), row, row, row, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert torch.equal(k[pages - 1, :, 2], row[0].half())
    ops.check_status()


def test_bad_page_and_length_are_reported(ops):
    """Device-side values out of range are skipped and reported, and the next call is clean."""
    from quantized_prefill_gemm_mmq_gb300._lib import MMQError
    cache = make_cache(ops, [100, 50], 2, 64, 16)
    q = torch.randn((2, 4, 64)).cuda()
    keep = cache.table.clone()
    for bad in (-1, 1 << 20):
        want = ops.attn_decode(cache, q)
        cache.table[0, 2] = bad
        got = ops.attn_decode(cache, q)
        with pytest.raises(MMQError) as e:
            ops.check_status()
        assert e.value.status == -11
        assert torch.equal(got[1], want[1])
        ops.rope_append(cache, ops.rope_table(64), q, q[:, :2], q[:, :2].contiguous(), torch.zeros(2, dtype=torch.int32).cuda())
        ops.check_status()                                           # the new entry's page is a good one
        cache.table.copy_(keep)
    cache.lens[1] = 1 << 29
    ops.attn_decode(cache, q)
    with pytest.raises(MMQError):
        ops.check_status()
    cache.lens[1] = 50
    a, b = ops.attn_decode(cache, q), ops.attn_decode(cache, q)
    ops.check_status()
    assert torch.equal(a, b)


def test_bad_pages_are_not_written(ops):
    """Append and eviction skip entries whose page is none, report it, and write the others."""
    from quantized_prefill_gemm_mmq_gb300._lib import MMQError
    cache = make_cache(ops, [40, 40], 2, 64, 16)
    pages = cache.table.clone()
    for bad in (-1, cache.k.shape[0]):
        rows = [torch.randn((2, h, 64)).cuda() for h in (4, 2, 2)]
        cache.table[0, 2] = bad
        k, v = cache.k.clone(), cache.v.clone()
        out = ops.rope_append(cache, ops.rope_table(64), *rows, torch.tensor([39, 39], dtype=torch.int32).cuda())
        with pytest.raises(MMQError) as e:
            ops.check_status()
        assert e.value.status == -11 and bool(torch.isfinite(out).all())
        changed = ((cache.k != k) | (cache.v != v)).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(pages[1, 2])]
    cache.lens.fill_(41)
    cache.pos.zero_()
    k, v = cache.k.clone(), cache.v.clone()
    wo, po = torch.full_like(cache.weight, -7.0), torch.full_like(cache.pos, -7)
    ops.kv_evict(cache, 20, torch.tensor([1, 1], dtype=torch.int32).cuda(), wo, po)
    with pytest.raises(MMQError) as e:
        ops.check_status()
    assert e.value.status == -11
    allowed = set(pages[:, :2].flatten().tolist())                   # the pages of slots below the budget
    for got, was in ((cache.k, k), (cache.v, v), (wo, torch.full_like(wo, -7.0)), (po, torch.full_like(po, -7))):
        assert set((got != was).flatten(1).any(1).nonzero().flatten().tolist()) <= allowed
    cache.table.copy_(pages)
    ops.attn_decode(cache, rows[0])
    ops.check_status()


# --------------------------------------------------------------- eviction ---

def check_evict(ops, lens, H, dim, page, budget, recent, dtype=torch.float16, layout="hnd", weights="random", seed=2, extra=0):
    cache = make_cache(ops, lens, H, dim, page, dtype, layout, seed=seed, extra=extra)
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    tab = cache.table.cpu()
    w, pos = cache.weight.cpu(), cache.pos.cpu()
    for b in range(B):
        perm = torch.randperm(max(1, lens[b]), generator=g)
        for s in range(lens[b]):
            pg, off = ref.slot_place(tab, page, b, s)
            pos[pg, :, off] = int(perm[s])
    if weights == "ties":
        w = torch.randint(0, 3, w.shape, generator=g).float()
    elif weights == "equal":
        w.fill_(0.5)
    elif weights == "signed":
        w = torch.randn(w.shape, generator=g)
        w[w.abs() < 0.3] = -0.0
        w[w > 2] = float("inf")
    cache.set_bookkeeping(w.cuda(), pos.cuda())
    keep_from = [n - recent for n in lens]
    k0, v0 = cache.k.cpu().clone(), cache.v.cpu().clone()
    wo, po = torch.full_like(cache.weight, -7.0), torch.full_like(cache.pos, -7)
    for _ in range(2):                                               # a repeated call gives the same
        ops.kv_evict(cache, budget, torch.tensor(keep_from, dtype=torch.int32).cuda(), wo, po)
        ops.check_status()
        want_k, want_v = k0.clone(), v0.clone()
        want_w, want_p = torch.full_like(w, -7.0), torch.full_like(pos, -7)
        for b in range(B):
            places = [ref.slot_place(tab, page, b, s) for s in range(lens[b])]
            for h in range(H):
                if lens[b] <= budget:
                    src = list(range(lens[b]))
                else:
                    src = ref.evict_row([float(w[p, h, o]) for p, o in places], [int(pos[p, h, o]) for p, o in places],
                                        keep_from[b], budget)
                for d, s in enumerate(src):
                    (dp, do), (sp, so) = places[d], places[s]
                    want_k[dp, h, do], want_v[dp, h, do] = k0[sp, h, so], v0[sp, h, so]
                    want_w[dp, h, do], want_p[dp, h, do] = w[sp, h, so], pos[sp, h, so]
        assert torch.equal(cache.k.cpu(), want_k) and torch.equal(cache.v.cpu(), want_v)
        assert torch.equal(wo.cpu(), want_w) and torch.equal(po.cpu(), want_p)
    assert torch.equal(cache.weight.cpu(), w) and torch.equal(cache.pos.cpu(), pos)


@pytest.mark.parametrize("weights", ["random", "ties", "equal", "signed"])
@pytest.mark.parametrize("lens,budget,recent", [([100], 64, 16), ([0, 1, 65, 64, 300], 64, 0), ([500, 499], 1, 1), ([257], 256, 256),
                                                ([200, 90], 100, 300), ([700], 699, 5)])
def test_evict(ops, lens, budget, recent, weights):
    check_evict(ops, lens, 2, 64, 16, budget, recent, weights=weights)


@pytest.mark.parametrize("dim,page,dtype,layout", [(8, 1, torch.float16, "hnd"), (80, 7, torch.bfloat16, "nhd"), (256, 100, torch.float16, "nhd"),
                                                   (128, 64, torch.bfloat16, "hnd")])
def test_evict_layouts(ops, dim, page, dtype, layout):
    check_evict(ops, [150, 333], 3, dim, page, 70, 20, dtype, layout)


@pytest.mark.parametrize("length,extra", [(4100, 0), (9000, 3000), (20001, 0), (33000, 0)])
@pytest.mark.parametrize("weights", ["random", "ties"])
def test_evict_long(ops, length, extra, weights):
    check_evict(ops, [length, 50], 1, 8, 64, length // 3, 40, weights=weights, extra=extra)


@pytest.mark.parametrize("page", [7, 10, 12])
@pytest.mark.parametrize("weights", ["random", "ties", "equal"])
def test_evict_pages_across_clusters(ops, page, weights):
    # pages that do and do not hold whole groups of four slots; lengths that end inside a group, in a part of a cluster
    check_evict(ops, [6001, 2050, 4099, 3], 1, 16, page, 1001, 300, weights=weights, extra=3000)


def test_evict_longest(ops):
    """The most slots a row may have, ties everywhere: the lowest slots stay and nothing moves."""
    n, budget = 262144, 100000
    k = torch.arange(n, device="cuda").remainder(1000).half().view(n // 64, 1, 64, 1).expand(-1, -1, -1, 8).contiguous()
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda").view(1, -1)
    w, pos = torch.ones((n // 64, 1, 64), device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda").view(-1, 1, 64).contiguous()
    cache = ops.KVCache(k, k.clone(), table, torch.tensor([n], dtype=torch.int32, device="cuda"), w, pos)
    wo, po = torch.zeros_like(w), torch.zeros_like(pos)
    ops.kv_evict(cache, budget, torch.tensor([n - 1000], dtype=torch.int32, device="cuda"), wo, po)
    ops.check_status()
    want = torch.arange(budget, dtype=torch.int32)
    want[budget - 1000:] = torch.arange(n - 1000, n, dtype=torch.int32)
    assert torch.equal(po.view(-1)[:budget].cpu(), want)
    assert torch.equal(cache.k.view(-1, 8)[:budget, 0].cpu().float(), want.remainder(1000).float())


def test_evict_offsets_past_32_bits(ops):
    """Pools of more than 2^31 elements: an entry of the last page moves into the page before it."""
    pages, page, H, dim = 33000, 64, 8, 128
    k = torch.empty((pages, H, page, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    last = [pages - 2, pages - 1]
    table = torch.tensor([last], dtype=torch.int32, device="cuda")
    k[last], v[last] = torch.randn((2, 2, H, page, dim), device="cuda").bfloat16().unbind(0)
    w, pos = torch.zeros((pages, H, page), device="cuda"), torch.zeros((pages, H, page), dtype=torch.int32, device="cuda")
    w[last] = 1.0
    w[pages - 2, :, 5] = 0.5
    pos[pages - 1, :, 36] = 100
    cache = ops.KVCache(k, v, table, torch.tensor([101], dtype=torch.int32, device="cuda"), w, pos)
    want_k, want_v = k[pages - 1, :, 36].clone(), v[pages - 1, :, 36].clone()
    wo, po = torch.zeros_like(w), torch.zeros_like(pos)
    ops.kv_evict(cache, 100, torch.tensor([100], dtype=torch.int32, device="cuda"), wo, po)
    ops.check_status()
    assert torch.equal(k[pages - 2, :, 5], want_k) and torch.equal(v[pages - 2, :, 5], want_v)
    assert bool((wo[pages - 2] == 1).all()) and bool((po[pages - 2, :, 5] == 100).all())


def test_chained_calls_see_each_other(ops):
    """Append, attention with weights and eviction back to back (each may start while the one before it ends) and with
    a synchronisation after every call: the same cache and outputs.  Pages of 16 put two heads' weights in one line."""
    g = torch.Generator().manual_seed(11)
    B, H, Hq, D, budget = 3, 4, 8, 64, 60
    rows = [(torch.randn((B, Hq, D), generator=g).cuda(), torch.randn((B, H, D), generator=g).cuda(), torch.randn((B, H, D), generator=g).cuda())
            for _ in range(24)]
    table = ops.rope_table(D)
    got = []
    for sync in (False, True):
        cache = make_cache(ops, [64, 70, 61], H, D, 16, seed=12, extra=60)
        spare = (torch.zeros_like(cache.weight), torch.zeros_like(cache.pos))
        cache.pos.copy_(torch.arange(cache.pos.numel(), dtype=torch.int32, device="cuda").view(cache.pos.shape) % 50)
        ws, ew, outs = ops.attn_workspace(cache, Hq, 1, True), ops.evict_workspace(cache, budget), []
        done = (lambda: torch.cuda.synchronize()) if sync else (lambda: None)
        for i, (q, k, v) in enumerate(rows):
            pos = torch.full((B,), 50 + i, dtype=torch.int32, device="cuda")
            cache.lens.add_(1)
            done()
            qr = ops.rope_append(cache, table, q, k, v, pos)
            done()
            outs.append(ops.attn_decode(cache, qr, accumulate=True, workspace=ws))
            done()
            old = (cache.weight, cache.pos)
            ops.kv_evict(cache, budget, pos - 5, *spare, workspace=ew)
            done()
            cache.set_bookkeeping(*spare)
            spare = old
            cache.lens.clamp_(max=budget)
        ops.check_status()
        got.append((torch.stack(outs), cache.k, cache.v, cache.weight, cache.pos, cache.table.long()))
    (o1, k1, v1, w1, p1, t1), (o2, k2, v2, w2, p2, _) = got
    pages = t1[:, :4].reshape(-1)                                    # the pages of the first 64 slots
    assert torch.equal(o1, o2) and torch.equal(k1, k2) and torch.equal(v1, v2)
    assert torch.equal(w1[pages], w2[pages]) and torch.equal(p1[pages], p2[pages])


# ----------------------------------------------------------- verification ---

def check_verify(ops, target, draft, tokens, uniform, count=None):
    got, acc = ops.spec_verify(target.cuda(), draft.cuda() if draft is not None else None, tokens.cuda(), uniform.cuda(),
                               count=count.cuda() if count is not None else None)
    n = count.tolist() if count is not None else [tokens.shape[1]] * tokens.shape[0]
    want, wacc = ref.verify(target.float().numpy(), draft.float().numpy() if draft is not None else None, tokens.numpy(),
                            uniform.numpy(), n)
    assert np.array_equal(acc.cpu().numpy(), wacc)
    assert np.array_equal(got.cpu().numpy(), want)
    return got, acc


def make_verify(B, N, V, dtype, seed, spread=0.7):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((B, N + 1, V), generator=g) * 2
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :N] + spread * torch.randn((B, N, V), generator=g), -1)
    tokens = torch.multinomial(draft.reshape(B * N, V), 1, generator=g).view(B, N).to(torch.int32)
    return target.to(dtype), draft.to(dtype), tokens, torch.rand((B, N + 1), generator=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,N,V", [(1, 1, 1), (5, 3, 2), (7, 4, 31), (4, 7, 256), (3, 5, 4097), (2, 64, 300), (40, 33, 33), (2, 3, 32001)])
def test_verify(ops, B, N, V, dtype):
    args = make_verify(B, N, V, dtype, B + N + V)
    check_verify(ops, *args)
    count = torch.randint(0, N + 1, (B,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    check_verify(ops, *args, count=count)
    check_verify(ops, args[0], None, args[2], args[3], count=count)
    ops.check_status()


def test_verify_edges(ops):
    target, draft, tokens, uniform = make_verify(6, 3, 1000, torch.float32, 3)
    check_verify(ops, target, target[:, :3].contiguous(), tokens, uniform)          # equal: everything is accepted
    check_verify(ops, target, draft, tokens, torch.full_like(uniform, 1 - 2.0 ** -24))
    check_verify(ops, target, draft, tokens, torch.zeros_like(uniform))
    zero = target.clone()
    zero[:, 0] = 0                                                                 # rejected, and nothing to draw from
    got, acc = check_verify(ops, zero, draft, tokens, uniform)
    assert bool((acc == 0).all()) and bool((got[:, 0] == 0).all())
    over = target.clone()
    over[0, 0] = draft[0, 0] * 0.5                                                 # the draft is above the target everywhere
    check_verify(ops, over, draft, tokens, torch.full_like(uniform, 0.75))
    tiny = torch.full((1, 2, 5000), 2.0 ** -41)                                    # half of the smallest step: to even, 0
    tiny[0, :, 4999] = 3 * 2.0 ** -41
    check_verify(ops, tiny, tiny[:, :1].contiguous(), torch.zeros((1, 1), dtype=torch.int32), torch.rand((1, 2)))
    ops.check_status()


def test_verify_distribution(ops):
    """Accepted or redrawn, the first token follows the target: 2^16 evenly spaced pairs of uniforms on 8 tokens."""
    n = 1 << 8
    target = torch.tensor([0.3, 0.25, 0.2, 0.1, 0.05, 0.05, 0.03, 0.02])
    draft = torch.tensor([0.1, 0.1, 0.1, 0.1, 0.15, 0.15, 0.15, 0.15])
    u = (torch.arange(n) + 0.5) / n
    u0, u1 = u.repeat_interleave(n), u.repeat(n)
    total = torch.zeros(8, dtype=torch.float64)
    B = n * n // 4
    for x in range(8):                                                             # each drafted token with its probability
        for i in range(4):
            s = slice(i * B, (i + 1) * B)
            got, _ = ops.spec_verify(target.expand(B, 2, 8).contiguous().cuda(), draft.expand(B, 1, 8).contiguous().cuda(),
                                     torch.full((B, 1), x, dtype=torch.int32).cuda(), torch.stack((u0[s], u1[s]), 1).contiguous().cuda())
            total += draft[x].double() * torch.bincount(got[:, 0].cpu().long(), minlength=8).double() / (n * n)
    # every threshold falls between two of the 2^8 points of a uniform: off by at most 2^-8 for each of the 8 + 8 steps
    assert float((total - target.double()).abs().max()) <= 16 / n


def test_verify_bad_tokens_and_counts_are_reported(ops):
    from quantized_prefill_gemm_mmq_gb300._lib import MMQError
    target, draft, tokens, uniform = make_verify(3, 2, 50, torch.float32, 8)
    tokens[1, 0] = 50
    tokens[2, 0] = -1
    check_verify(ops, target, draft, tokens, uniform)
    with pytest.raises(MMQError) as e:
        ops.check_status()
    assert e.value.status == -11
    tokens.clamp_(0, 49)
    ops.spec_verify(target.cuda(), draft.cuda(), tokens.cuda(), uniform.cuda(), count=torch.tensor([1, 9, -1], dtype=torch.int32).cuda())
    with pytest.raises(MMQError):
        ops.check_status()
    check_verify(ops, target, draft, tokens, uniform)
    ops.check_status()


# ---------------------------------------------------------------- outputs ---

def test_outputs_are_the_callers(ops):
    """Small outputs come out of shared blocks: none is handed out twice, on whatever stream, and a captured graph's
    output is not one of them."""
    cache = make_cache(ops, [30], 2, 64, 16)
    qs = [torch.randn((1, 4, 64)).cuda() for _ in range(70)]
    first = [ops.attn_decode(cache, q) for q in qs]
    kept = [o.clone() for o in first]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = [ops.attn_decode(cache, q) for q in qs]
    side.synchronize()
    every = first + second
    spans = sorted((o.data_ptr(), o.data_ptr() + o.numel() * 4) for o in every)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    assert all(torch.equal(a, b) for a, b in zip(first, kept)) and all(torch.equal(a, b) for a, b in zip(second, kept))
    ws = ops.attn_workspace(cache, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.attn_decode(cache, qs[3], workspace=ws)
    more = [ops.attn_decode(cache, q) for q in qs]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, kept[3]) and all(torch.equal(a, b) for a, b in zip(more, kept))
    assert not any(o.data_ptr() == out.data_ptr() for o in more)


# --------------------------------------------------------------- refusals ---

def test_refusals(ops):
    from quantized_prefill_gemm_mmq_gb300._lib import MMQError
    cache = make_cache(ops, [20, 30], 2, 64, 16)
    bare = make_cache(ops, [20, 30], 2, 64, 16, track=False)
    q, kv = torch.zeros((2, 4, 64)).cuda(), torch.zeros((2, 2, 64)).cuda()
    pos, table = torch.zeros(2, dtype=torch.int32).cuda(), ops.rope_table(64)
    for bad in (lambda: ops.attn_decode(cache, q.half()), lambda: ops.attn_decode(cache, q[:, :3].contiguous()),
                lambda: ops.attn_decode(cache, q[:1]), lambda: ops.attn_decode(cache, q.repeat(17, 1, 1)),
                lambda: ops.attn_decode(cache, q.cpu()), lambda: ops.attn_decode(bare, q, accumulate=True),
                lambda: ops.attn_decode(cache, q, out=torch.zeros((2, 4, 32)).cuda()),
                lambda: ops.attn_decode(cache, q, new=torch.zeros(3, dtype=torch.int32).cuda()),
                lambda: ops.rope_append(cache, ops.rope_table(128), q, kv, kv, pos),
                lambda: ops.rope_append(cache, table, q, kv[:1], kv, pos), lambda: ops.rope_append(cache, table, q, kv, kv, pos.long()),
                lambda: ops.rope_append(cache, table, q[..., ::2], kv, kv, pos),
                lambda: ops.kv_evict(bare, 8, pos, None, None), lambda: ops.kv_evict(cache, 8, pos, cache.weight, cache.pos),
                lambda: ops.spec_verify(torch.zeros((2, 3, 9)).cuda(), torch.zeros((2, 3, 9)).cuda(), torch.zeros((2, 2), dtype=torch.int32).cuda(), torch.zeros((2, 3)).cuda()),
                lambda: ops.spec_verify(torch.zeros((2, 1, 9)).cuda(), None, pos, pos),
                lambda: ops.KVCache(cache.k[..., ::2], cache.v[..., ::2], cache.table, cache.lens),
                lambda: ops.KVCache(cache.k, cache.v.bfloat16(), cache.table, cache.lens),
                lambda: ops.KVCache(cache.k, cache.v, cache.table.long(), cache.lens),
                lambda: ops.KVCache(cache.k, cache.v, cache.table, cache.lens[:1])):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: ops.attn_decode(cache, q, scale=float("nan")), -1), (lambda: ops.attn_decode(cache, q, out=q), -1), (lambda: ops.attn_decode(cache, q, scale=float("inf")), -1),
                        (lambda: ops.evict_workspace(cache, 0), -1)):
        with pytest.raises(MMQError) as e:
            bad()
        assert e.value.status == status
    ops.check_status()
