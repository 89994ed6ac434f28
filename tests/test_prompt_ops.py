"""GPU tests of the operators for prompts and trees of drafts (normed rotary append, attention of any number of new tokens
or of a tree, keeping a path) against plain 64-bit implementations; the tolerances are derived in prompt_ref.py."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from tests import prompt_ref as ref  # noqa: E402
from tests import serve_ref  # noqa: E402
from tests.test_serve_ops import make_cache, ops  # noqa: E402, F401

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def queries(cache, lens, N, group, scale=1.0, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((len(lens) * N, cache.heads * group, cache.dim), generator=g) * scale).to(cache.k.dtype)


def dev(x, dtype=torch.int32):
    return None if x is None else torch.tensor(x, dtype=dtype).cuda()


def signed(words):
    return [[w - (1 << 64) if w >> 63 else w for w in row] for row in words]


def check(ops, cache, q, lens, new=None, scale=None, cap=0.0, slopes=None, window=0, prefix=None, first=None, tree=None,
          out_dtype=None, **call):
    """One call against 64 bits; returns the call's output."""
    N = q.shape[0] // len(lens)
    first_t = None if first is None else dev(first).reshape(-1)
    if tree is None:
        got = ops.attn_prefill(cache, q.cuda(), scale=scale, cap=cap, slopes=dev(slopes, F32), window=window, prefix=dev(prefix),
                               first=first_t, new=dev(new), out_dtype=out_dtype, **call)
    else:
        got = ops.attn_tree(cache, q.cuda(), dev(signed(tree), torch.int64), scale=scale, cap=cap, first=first_t, new=dev(new),
                            out_dtype=out_dtype, **call)
    ops.check_status()
    counts = new if new is not None else [N] * len(lens)
    want, tol = ref.attention(q, cache.k.cpu(), cache.v.cpu(), cache.table.cpu(), lens, counts, cache.page_size,
                              cache.dim ** -0.5 if scale is None else scale, cap, slopes, window=window, prefix=prefix, first=first, tree=tree)
    assert got.dtype == (out_dtype or cache.k.dtype)
    half = 0.0 if got.dtype == F32 else ref.HALF[got.dtype]
    tol = tol + (want.abs() + tol) * half + (2.0 ** -25 if got.dtype == F16 else 0.0)
    off = (got.cpu().double() - want).abs()
    assert bool((off <= tol).all()), float((off / (tol + 1e-30)).max())
    return got


# ---------------------------------------------------------------- attention ---

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,N,H,group,dim,page,layout", [
    ([1], 1, 1, 1, 8, 1, "hnd"),                         # one token that sees itself alone
    ([1], 1, 2, 4, 128, 16, "nhd"),
    ([513], 1, 4, 1, 128, 16, "hnd"),
    ([700, 3, 129], 1, 2, 8, 64, 24, "hnd"),             # single tokens, lengths of all sizes
    ([130], 130, 2, 1, 128, 16, "hnd"),                  # two halves of 128 rows, the second nearly empty
    ([300], 300, 1, 1, 64, 100, "nhd"),
    ([257, 64], 64, 2, 3, 80, 24, "hnd"),                # 192 rows
    ([400], 33, 1, 7, 72, 7, "nhd"),                     # a head that is no multiple of 16
    ([200, 90], 90, 2, 2, 192, 64, "hnd"),
    ([200, 77], 77, 1, 4, 256, 32, "nhd"),
    ([150], 20, 1, 2, 256, 128, "hnd"),                  # 40 rows of the largest heads
    ([90], 9, 1, 3, 160, 16, "hnd"),
    ([1100], 1000, 1, 1, 128, 64, "hnd"),
])
def test_causal(ops, lens, N, H, group, dim, page, layout, dtype):
    cache = make_cache(ops, lens, H, dim, page, dtype, layout, fill=float("nan"))
    check(ops, cache, queries(cache, lens, N, group), lens)


@pytest.mark.parametrize("dtype,out", [(F16, F32), (BF16, F32), (F16, F16)])
def test_outputs_of_both_types_and_ragged_counts(ops, dtype, out):
    lens, new = [200, 150, 30, 5], [64, 1, 0, 5]
    cache = make_cache(ops, lens, 2, 64, 16, dtype)
    q = queries(cache, lens, 64, 4)
    got = check(ops, cache, q, lens, new=new, out_dtype=out)
    rows = got.view(4, 64, -1)
    assert all(bool((rows[b, n:] == 0).all()) for b, n in enumerate(new))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("N,dim,group", [(1, 128, 4), (40, 128, 2), (140, 64, 2), (70, 192, 2), (70, 256, 1)])
@pytest.mark.parametrize("what", ["cap", "slopes", "cap_slopes", "window", "prefix", "first", "all", "minus"])
def test_forms(ops, what, N, dim, group, dtype):
    lens = [400, 290]
    cache = make_cache(ops, lens, 2, dim, 24, dtype, fill=float("inf"))
    kw = {}
    if what in ("cap", "cap_slopes", "all"):
        kw["cap"] = 5.0
    if what in ("slopes", "cap_slopes", "all"):
        kw["slopes"] = [2.0 ** -(1 + h) for h in range(2 * group)]
    if what in ("window", "all"):
        kw["window"] = 33
    if what in ("prefix", "all"):
        kw["prefix"] = [400 - N // 2, 290]
    if what in ("first", "all"):                         # rows 1/3 and on begin at their own place, one sees nothing
        kw["first"] = [[0 if t < N // 3 else ln - N + N // 3 for t in range(N)] for ln in lens]
        kw["first"][0][-1] = 400
    if what == "minus":
        kw["scale"] = -0.2
    got = check(ops, cache, queries(cache, lens, N, group, 3.0), lens, **kw)
    if what == "first":
        assert bool((got[N - 1] == 0).all())


@pytest.mark.parametrize("window", [1, 2, 127, 128, 129, 5000])
def test_windows(ops, window):
    lens = [900]
    cache = make_cache(ops, lens, 1, 64, 16)
    check(ops, cache, queries(cache, lens, 600, 1), lens, window=window)


def test_units_one_per_cta(ops):
    """Enough rows that no unit is cut: 64 heads of 10 units."""
    lens, N = [1300, 700], 1300
    cache = make_cache(ops, lens, 48, 16, 64, BF16)
    check(ops, cache, queries(cache, lens, N, 1), lens, new=[1300, 650], window=400)


@pytest.mark.parametrize("dtype,dim,N,group", [(F16, 128, 1, 1), (BF16, 64, 5, 4), (BF16, 128, 150, 1), (F16, 256, 3, 2)])
def test_long_contexts_are_joined(ops, dtype, dim, N, group):
    lens = [9000, 17, 4000]
    cache = make_cache(ops, lens, 1, dim, 64, dtype)
    new = [N, min(N, 17), 0]
    a = check(ops, cache, queries(cache, lens, N, group, 2.0), lens, new=new)
    b = check(ops, cache, queries(cache, lens, N, group, 2.0), lens, new=new)
    assert torch.equal(a, b)


def trees(B, N, seed=0):
    g = torch.Generator().manual_seed(seed)
    parents = [[-1 if t == 0 or torch.rand((), generator=g) < 0.1 else int(torch.randint(max(0, t - 5), t, (), generator=g)) for t in range(N)]
               for _ in range(B)]
    words = []
    for row in parents:
        w = []
        for t, p in enumerate(row):
            w.append((w[p] if p >= 0 else 0) | 1 << t)
        words.append(w)
    return parents, words


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens,N,new,H,group,dim,page", [
    ([1], 1, None, 1, 1, 64, 16),
    ([500], 16, None, 2, 1, 128, 16),
    ([300, 64, 190], 64, None, 2, 4, 128, 24),           # one sequence is nothing but its tree
    ([5000, 130, 20, 9], 33, [33, 7, 0, 9], 1, 8, 64, 64),
    ([200, 128], 48, None, 1, 2, 192, 100),
    ([150], 63, None, 1, 4, 256, 7),
])
def test_trees(ops, lens, N, new, H, group, dim, page, dtype):
    cache = make_cache(ops, lens, H, dim, page, dtype, fill=float("nan"))
    parents, words = trees(len(lens), N)
    assert torch.equal(ops.tree_words(parents).cpu(), torch.tensor(signed(words), dtype=torch.int64))
    q = queries(cache, lens, N, group)
    check(ops, cache, q, lens, new=new, tree=words)
    check(ops, cache, q, lens, new=new, tree=words, cap=3.0, out_dtype=F32,
          first=[[max(0, ln - N - 20 + t % 3) for t in range(N)] for ln in lens])


def test_tree_words_of_any_kind(ops):
    """Bits that are no tree: rows that see no node, nodes behind them, or nothing at all."""
    cache = make_cache(ops, [64, 70], 1, 64, 16)
    words = [[(0x9E3779B97F4A7C15 * (t + 1) * (b + 3)) % (1 << 64) for t in range(64)] for b in range(2)]
    words[0][5] = 0
    got = check(ops, cache, queries(cache, [64, 70], 64, 1), [64, 70], tree=words)
    assert bool((got[5] == 0).all())


def test_a_chain_is_the_causal_mask(ops):
    lens, N = [333, 90], 20
    cache = make_cache(ops, lens, 2, 128, 16, BF16)
    q = queries(cache, lens, N, 2).cuda()
    chain = ops.tree_words([list(range(-1, N - 1))] * 2)
    assert torch.equal(ops.attn_tree(cache, q, chain), ops.attn_prefill(cache, q))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,dim,N,group,window", [(F16, 64, 100, 1, 0), (BF16, 128, 200, 2, 0), (F16, 256, 60, 2, 50), (BF16, 192, 40, 4, 0)])
def test_what_is_not_seen_does_not_matter(ops, bad, dtype, dim, N, group, window):
    """V and K entries that are not finite: rows that do not see them are the same bit for bit, the others not finite (V)."""
    ln = N + 150
    where = [3, 140, ln - N // 2, ln - 2]
    q = None
    for pool in ("v", "k"):
        cache = make_cache(ops, [ln], 1, dim, 16, dtype)
        q = queries(cache, [ln], N, group).cuda()
        want = ops.attn_prefill(cache, q, window=window)
        first = torch.zeros(N, dtype=torch.int32)
        first[N // 4:] = 145                                 # the later rows' document begins after the first two
        want_first = ops.attn_prefill(cache, q, window=window, first=first.cuda())
        for s in where:
            pg, off = serve_ref.slot_place(cache.table.cpu(), 16, 0, s)
            getattr(cache, pool)[pg, 0, off, dim // 2] = bad
        for f, clean in ((None, want), (first, want_first)):
            got = ops.attn_prefill(cache, q, window=window, first=None if f is None else f.cuda())
            ops.check_status()
            hit = torch.zeros(N, dtype=torch.bool)
            for t in range(N):
                i = ln - N + t
                lo = max(0, i - window + 1) if window else 0
                lo = lo if f is None else max(lo, int(f[t]))
                hit[t] = any(lo <= s <= i for s in where)
            assert torch.equal(got[~hit.cuda()], clean[~hit.cuda()])
            if pool == "v":
                assert not bool(torch.isfinite(got[hit.cuda()]).all(-1).any())
            elif bad != bad:
                assert bool(torch.isnan(got[hit.cuda()]).all())


def test_trees_do_not_see_what_is_beside_them(ops):
    lens, N = [100], 40
    cache = make_cache(ops, lens, 1, 64, 16, BF16)
    _, words = trees(1, N, 3)
    q, tree = queries(cache, lens, N, 1).cuda(), dev(signed(words), torch.int64)
    want = ops.attn_tree(cache, q, tree)
    pg, off = serve_ref.slot_place(cache.table.cpu(), 16, 0, 60 + 7)
    cache.v[pg, 0, off] = float("nan")
    got = ops.attn_tree(cache, q, tree)
    hit = torch.tensor([bool(w >> 7 & 1) for w in words[0]])
    assert 0 < int(hit.sum()) < N
    assert torch.equal(got[~hit.cuda()], want[~hit.cuda()]) and bool(torch.isnan(got[hit.cuda()]).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [1e2, 1e4])
def test_large_scores(ops, dtype, size):
    """Where the largest score leads by far, its value comes out; every output is a mean of values."""
    lens, N, dim = [500], 150, 64
    cache = make_cache(ops, lens, 1, dim, 16, dtype)
    q = queries(cache, lens, N, 1, size)
    got = ops.attn_prefill(cache, q.cuda(), scale=4.0).cpu().double()
    ops.check_status()
    k, v = (serve_ref.gather(x.cpu(), cache.table.cpu(), 16, 0, 0, 500) for x in (cache.k, cache.v))
    clear = 0
    for t in range(N):
        m = 350 + t + 1
        s = k[:m] @ q[t, 0].double() * 4.0
        off = 2.0 ** -20 * 4.0 * float((k[:m].abs() @ q[t, 0].double().abs()).max())
        best, at = s.topk(2)
        # a value is a sum of rounded weights over their sum, rounded
        slack = 3 * ref.HALF[dtype] * float(v[:m].abs().max())
        assert bool(((got[t, 0] >= v[:m].amin(0) - slack) & (got[t, 0] <= v[:m].amax(0) + slack)).all())
        if float(best[0] - best[1]) > 4 * off + 40:
            assert float((got[t, 0] - v[at[0]]).abs().max()) <= slack
            clear += 1
    assert clear > 10


def test_scores_that_rise_and_fall(ops):
    """Running maxima that rise in every tile, by little and by much, and masked tiles in front."""
    lens, N, dim = [1500], 200, 64
    cache = make_cache(ops, lens, 1, dim, 16)
    flat = cache.table[0].long()
    k = torch.randn((len(flat) * 16, dim), generator=torch.Generator().manual_seed(5)) * 0.1
    ramp = torch.linspace(-3, 3, len(flat) * 16)
    ramp[700:900] = -3
    k[:, 0] = ramp
    cache.k[flat, 0] = k.view(-1, 16, dim).to(F16).cuda()
    q = queries(cache, lens, N, 1, 0.3)
    q[:, :, 0] = torch.linspace(-12, 12, N)[:, None].to(F16)
    check(ops, cache, q, lens, scale=1.0)
    check(ops, cache, q, lens, scale=1.0, first=[[1000 + t for t in range(N)]])


@pytest.mark.parametrize("extra", [0, 1000], ids=["one launch", "joined"])
@pytest.mark.parametrize("units", range(8))
def test_weights_of_tiles_whose_maxima_are_large(ops, units, extra):
    """Scores of -4093 and -4084 in powers of two, exact to 2^-12: a tile's weights against another tile's.  f32 has steps of
    2^-11 from 4096 on and of 2^-12 below, so that a maximum of which 7 is taken off may be rounded; then the weights of one
    tile lie off by the rounding, together.  The entry that is looked at weighs 2^6 and some steps of 2^-12 more or less, which
    f16 rounds by up to half a step; nothing else is rounded by more than the f32 sums and the exponentials (2^-18)."""
    import math
    step, scale = 2.0 ** -12, 0.693147182464599609375        # log 2 in f32: times log2(e) it is 1 in f32
    cache = make_cache(ops, [256], 1, 64, 16, F16, extra=extra)
    k, v = torch.zeros((256, 64)), torch.zeros((256, 64))
    k[:128, 0], k[:128, 1], k[:128, 2] = -4092, -1, -3 * step            # the first tile's maximum: -(4093 + 3 steps)
    k[7, 0], k[7, 1], k[7, 2] = -4094, 0, (units - 1) * step             # 1 less, and units + 2 steps
    k[128:, 0] = -4084                                                   # the second tile's
    v[7, 0] = 1
    flat = cache.table[0, :16].long()
    for pool, x in ((cache.k, k), (cache.v, v)):
        pool[flat] = x.view(16, 1, 16, 64).to(F16).cuda()
    q = torch.zeros((1, 1, 64), dtype=F16)
    q[0, 0, :3] = 1
    got = float(ops.attn_prefill(cache, q.cuda(), scale=scale, out_dtype=F32)[0, 0, 0])
    ops.check_status()
    s = [float(k[j, 0]) + float(k[j, 1]) + float(k[j, 2]) + 4084 for j in range(256)]
    weights = [math.exp2(x * scale / math.log(2)) for x in s]
    want = weights[7] / math.fsum(weights)
    assert abs(got / want - 1) <= ref.HALF[F16] + 2.0 ** -18


# --------------------------------------------------------------- how it is called ---

def test_rows_out_and_workspace_of_the_caller(ops):
    lens, N = [300, 200], 30
    cache = make_cache(ops, lens, 2, 64, 16, BF16)
    wide = torch.randn((2 * N, 12 * 64), generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    q = wide[:, 128:128 + 4 * 64].view(2 * N, 4, 64)
    want = ops.attn_prefill(cache, q.contiguous())
    out = torch.full((2 * N, 4, 64), 9.0, dtype=F32).cuda()
    work = ops.prefill_workspace(cache, 4, N)
    work.work.fill_(float("nan"))
    got = ops.attn_prefill(cache, q, out=out, workspace=work)
    assert got is out and torch.equal(got.to(BF16), want)
    one = ops.attn_prefill(cache, q, workspace=ops.AttnWorkspace(cache.device, 4))     # too small: one for the call
    assert torch.equal(one, want)
    ops.check_status()


def test_another_stream_and_captured_calls(ops):
    lens, N = [1000, 333], 40
    cache = make_cache(ops, lens, 2, 128, 16)
    q = queries(cache, lens, N, 2).cuda()
    tree = ops.tree_words([list(range(-1, N - 1))] * 2)
    want, want_tree = ops.attn_prefill(cache, q, cap=20.0), ops.attn_tree(cache, q, tree)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ops.attn_prefill(cache, q, cap=20.0)
    s.synchronize()
    assert torch.equal(got, want)
    work = ops.prefill_workspace(cache, 4, N)
    a, b = torch.empty_like(want), torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):                            # both calls use the workspace, in order
        ops.attn_prefill(cache, q, cap=20.0, out=a, workspace=work)
        ops.attn_tree(cache, q, tree, out=b, workspace=work)
    for _ in range(3):
        a.fill_(7), b.fill_(7)
        g.replay()
        assert torch.equal(a, want) and torch.equal(b, want_tree)
    cache.lens[0] = 500                                  # a replay reads what the tensors hold then
    g.replay()
    assert torch.equal(a, ops.attn_prefill(cache, q, cap=20.0)) and not torch.equal(a, want)
    ops.check_status()


def test_calls_in_a_row_see_what_the_one_before_wrote(ops):
    """Append, attention and keeping without a wait between: the same as with one."""
    lens, N, H, dim = [200, 90], 24, 2, 64
    outs = []
    for wait in (False, True):
        cache = make_cache(ops, lens, H, dim, 16, BF16)
        g = torch.Generator().manual_seed(4)
        table = ops.rope_table(dim)
        res = []
        for _ in range(20):
            row = torch.randn((2 * N, 8 * dim), generator=g).cuda()
            q, k, v = (row[:, a * dim:b * dim].view(2 * N, b - a, dim) for a, b in ((0, 4), (4, 6), (6, 8)))
            pos = torch.randint(0, 300, (2 * N,), generator=g, dtype=torch.int32).cuda()
            keep = torch.stack([torch.randperm(N, generator=g)[:5].sort().values for _ in range(2)]).to(torch.int32).cuda()
            steps = [lambda: ops.norm_rope_append(cache, table, q, k, v, pos, out_dtype=BF16)]
            qr = steps[0]()
            if wait:
                torch.cuda.synchronize()
            res.append(ops.attn_prefill(cache, qr))
            if wait:
                torch.cuda.synchronize()
            ops.kv_keep(cache, keep, None, N)
            if wait:
                torch.cuda.synchronize()
            res.append(ops.attn_prefill(cache, qr, slopes=torch.ones(4).cuda()))
        outs.append(torch.stack(res))
        ops.check_status()
    assert torch.equal(*outs)


def test_caches_past_32_bit_offsets(ops):
    """Pages whose addresses lie past 2^32 values."""
    page, dim, H = 64, 128, 8
    pages = (1 << 32) // (page * dim * H) + 40
    k = torch.zeros((pages, H, page, dim), dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    last = torch.arange(pages - 4, pages, dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    for x in (k, v):
        x[last.long().cuda()] = torch.randn((4, H, page, dim), generator=g).to(BF16).cuda()
    cache = ops.KVCache(k, v, last.view(1, 4).cuda(), torch.tensor([250], dtype=torch.int32).cuda())
    small = ops.KVCache(k[-4:].clone(), v[-4:].clone(), torch.arange(4, dtype=torch.int32).view(1, 4).cuda(), cache.lens)
    q = queries(small, [250], 50, 2).cuda()
    assert torch.equal(ops.attn_prefill(cache, q), ops.attn_prefill(small, q))
    keep = torch.tensor([[3, 20, 49]], dtype=torch.int32).cuda()
    for c in (cache, small):
        ops.kv_keep(c, keep, None, 50)
    ops.check_status()
    assert torch.equal(cache.k[-4:], small.k) and torch.equal(cache.v[-4:], small.v)


def test_bad_indexes_are_reported(ops):
    from quantized_prefill_gemm_mmq_gb300._lib import MMQError
    lens, N = [100, 50], 20
    cache = make_cache(ops, lens, 2, 64, 16)
    q = queries(cache, lens, N, 2).cuda()
    want = ops.attn_prefill(cache, q)

    def reported(text):
        with pytest.raises(MMQError, match=text) as e:
            ops.check_status()
        assert e.value.status == -11

    cache.table[0, 2] = 1 << 20
    got = ops.attn_prefill(cache, q)
    reported("prompt or tree attention: a page id")
    assert torch.equal(got[N:], want[N:])
    cache.table[0, 2] = 0
    cache.lens[0] = 1 << 30
    got = ops.attn_prefill(cache, q)
    reported("length")
    assert torch.equal(got[N:], want[N:]) and bool((got[:N] == 0).all())
    cache.lens[0] = 7                                    # fewer entries than new tokens
    got = ops.attn_prefill(cache, q)
    reported("length")
    assert torch.equal(got[N:], want[N:]) and bool((got[:N] == 0).all())
    cache.lens[0] = 100
    ops.attn_prefill(cache, q, new=dev([-1, 21]))
    reported("count")
    ops.kv_keep(cache, dev([[2, 2], [0, 20]]), None, N)
    reported("keeping a path: a kept node")
    ops.kv_keep(cache, dev([[2, 3], [0, 1]]), dev([3, -1]), N)
    reported("count")
    ops.check_status()


def test_refusals(ops):
    cache = make_cache(ops, [100, 50], 2, 64, 16)
    q = queries(cache, [100, 50], 4, 2).cuda()
    bad = [dict(q=q.float()), dict(q=q[:7]), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q.cpu()), dict(slopes=torch.ones(3).cuda()),
           dict(prefix=torch.zeros(2).cuda()), dict(first=torch.zeros(2, dtype=torch.int32).cuda()), dict(out_dtype=BF16),
           dict(out=torch.zeros(8, 4, 64).cuda(), out_dtype=F16), dict(new=torch.zeros(2, dtype=torch.int64).cuda()),
           dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))]
    for kw in bad:
        with pytest.raises(ValueError):
            ops.attn_prefill(cache, **{"q": q, **kw})
    from quantized_prefill_gemm_mmq_gb300._lib import MMQError
    for kw in (dict(cap=-1.0), dict(cap=1025.0), dict(cap=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(out=q)):
        with pytest.raises(MMQError):
            ops.attn_prefill(cache, q, **kw)
    tree = ops.tree_words([[-1, 0, 1, 2]] * 2)
    for kw in (dict(tree=tree.int()), dict(tree=tree[:1]), dict(q=q[:2])):
        with pytest.raises(ValueError):
            ops.attn_tree(cache, **{"q": q, "tree": tree, **kw})
    big = queries(cache, [100, 50], 65, 1).cuda()
    with pytest.raises(ValueError):
        ops.attn_tree(cache, big, torch.zeros((2, 65), dtype=torch.int64).cuda())
    for p in ([[0]], [[-1, 1]], [[-2]], [[-1] * 65]):
        with pytest.raises(ValueError):
            ops.tree_words(p)


# ------------------------------------------------------------ normed rotary append ---

@pytest.mark.parametrize("B,N,Hq,H,dim,rot,inter,dtype,page,layout,sections,out,norms", [
    (1, 1, 4, 4, 128, 128, False, F16, 16, "hnd", None, F32, "qk"),
    (1, 1, 1, 1, 8, 8, True, BF16, 1, "hnd", [2, 2], BF16, "qk"),
    (3, 5, 8, 2, 128, 64, True, BF16, 7, "nhd", [8, 12, 12], BF16, "q"),
    (2, 70, 6, 3, 80, 40, False, F16, 24, "nhd", [20], F32, "k"),
    (1, 33, 2, 1, 256, 256, False, F16, 64, "hnd", [32, 48, 48], F16, "qk"),
    (2, 3, 4, 2, 72, 36, False, F16, 5, "hnd", [6, 6, 6], F16, "qk"),        # pairs that no 16-byte access fits
    (2, 3, 4, 2, 72, 70, True, BF16, 5, "hnd", None, F32, "qk"),
    (2, 9, 3, 1, 24, 2, False, F16, 5, "hnd", None, F16, "qk"),
    (1, 700, 32, 8, 128, 128, False, BF16, 64, "hnd", [16, 24, 24], BF16, "qk"),
    (2, 4, 5, 5, 192, 192, True, F16, 32, "nhd", [96, 0], F32, ""),
])
def test_norm_rope_append(ops, B, N, Hq, H, dim, rot, inter, dtype, page, layout, sections, out, norms):
    g = torch.Generator().manual_seed(B * N + dim)
    new = [N] + [max(0, N - 2 * b) for b in range(1, B)]
    lens = [N + 3 + 11 * b for b in range(B)]
    cache = make_cache(ops, lens, H, dim, page, dtype, layout)
    before = [t.cpu().clone() for t in (cache.k, cache.v, cache.weight, cache.pos)]
    row = torch.randn((B * N, (Hq + 2 * H) * dim), generator=g) * torch.exp(2 * torch.randn((B * N, 1), generator=g))
    axes = 1 if sections is None else len(sections)
    pos = torch.randint(0, 40000, (axes, B * N), generator=g, dtype=torch.int32)
    pos[-1, 0] = 1 << 30
    table = ops.rope_table(rot, scaling="by_parts", factor=4.0, context=512, sections=sections, alternate=B == 3)
    inv, mag = ops.rope_frequencies(rot, 10000.0, "by_parts", 4.0, 512)
    axis = None if sections is None else ops.rope_axes(rot, sections, alternate=B == 3)
    qw, kw = (torch.randn(dim, generator=g) for _ in range(2))
    d = row.cuda()
    q, k, v = (d[:, a * dim:b * dim].view(B * N, b - a, dim) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    got = ops.norm_rope_append(cache, table, q, k, v, (pos[0] if sections is None else pos).cuda(), q_norm=qw.cuda() if "q" in norms else None,
                               k_norm=kw.cuda() if "k" in norms else None, eps=1e-5, interleaved=inter, new=dev(new) if B > 1 else None,
                               out_dtype=out)
    ops.check_status()
    fixed = ops.rope_fixed(inv)
    live = torch.tensor([t < new[b] for b in range(B) for t in range(N)])
    want, tol = ref.norm_rope(q.cpu(), qw if "q" in norms else None, 1e-5, pos, axis, fixed, rot, mag, inter)
    want[~live] = 0
    half = 0.0 if out == F32 else ref.HALF[out] * 1.01
    assert got.dtype == out
    assert bool(((got.cpu().double() - want).abs() <= tol + want.abs() * half + 2.0 ** -25).all())
    kw64, kt = ref.norm_rope(k.cpu(), kw if "k" in norms else None, 1e-5, pos, axis, fixed, rot, mag, inter)
    half = ref.HALF[dtype]
    got_k, got_v, got_w, got_p = (t.cpu() for t in (cache.k, cache.v, cache.weight, cache.pos))
    tab, vc = cache.table.cpu(), v.cpu()
    touched = torch.zeros(got_w.shape[0], got_w.shape[2], dtype=torch.bool)
    for b in range(B):
        for t in range(new[b]):
            pg, off = serve_ref.slot_place(tab, page, b, lens[b] - new[b] + t)
            r = b * N + t
            assert bool(((got_k[pg, :, off].double() - kw64[r]).abs() <= kt[r] + kw64[r].abs() * half * 1.01 + 2.0 ** -25).all())
            assert torch.equal(got_v[pg, :, off], vc[r].to(dtype))
            assert bool((got_w[pg, :, off] == 0).all()) and bool((got_p[pg, :, off] == pos[0, r]).all())
            touched[pg, off] = True
    for x, was in zip((got_k, got_v, got_w, got_p), before):             # nothing else is written
        same = (x == was) if x.dim() == 3 else (x == was).all(-1)
        assert bool((same | touched[:, None]).all())


def test_norm_rope_without_norms_is_rope_append(ops):
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((2, h, 64), generator=g).cuda() for h in (4, 2, 2))
    pos, table = dev([8, 39]), ops.rope_table(64)
    a, b = make_cache(ops, [9, 40], 2, 64, 16), make_cache(ops, [9, 40], 2, 64, 16, track=False)
    want = ops.rope_append(a, table, q, k, v, pos)
    got = ops.norm_rope_append(b, table, q, k, v, pos, out=q)            # in place
    ops.check_status()
    assert got is q
    assert float((got - want).abs().max()) <= 2.0 ** -21 and float((a.k - b.k).abs().max()) <= 2.0 ** -9 and torch.equal(a.v, b.v)


@pytest.mark.parametrize("dim,rot,inter,page", [(64, 32, False, 16), (128, 64, True, 7), (80, 40, True, 16), (72, 36, False, 5), (72, 34, True, 16)])
def test_values_past_the_rotated_ones_are_left_alone(ops, dim, rot, inter, page):
    """NaN, infinities and -0 in values that do not turn: without a norm they come out as they are, and no other value
    changes; with one, a head of finite values beside them is what it was."""
    g = torch.Generator().manual_seed(dim + rot)
    q, k, v = (torch.randn((2, h, dim), generator=g) for h in (4, 2, 2))
    for x in (q, k):
        x[0, 0, rot + 1], x[0, 1, rot], x[1, 0, dim - 1] = float("nan"), float("inf"), float("-inf")
        x[1, 1, rot::2] = -0.0
    pos, table = dev([8, 39]), ops.rope_table(rot)
    caches = [make_cache(ops, [9, 40], 2, dim, page) for _ in range(2)]
    want = ops.rope_append(caches[0], table, q.cuda(), k.cuda(), v.cuda(), pos, interleaved=inter)
    got = ops.norm_rope_append(caches[1], table, q.cuda(), k.cuda(), v.cuda(), pos, interleaved=inter)
    ops.check_status()

    def bits(x):                                             # of NaNs there are many: a product with 1 may give another one
        x = torch.where(torch.isnan(x), torch.full_like(x, float("nan")), x).contiguous()
        return x.view(torch.int32 if x.dtype == F32 else torch.int16)
    assert torch.equal(bits(got[..., rot:]), bits(want[..., rot:])) and torch.equal(bits(got[..., rot:].cpu()), bits(q[..., rot:]))
    assert float((got[..., :rot] - want[..., :rot]).abs().max()) <= 2.0 ** -21 * 8
    for b in range(2):
        pg, off = serve_ref.slot_place(caches[0].table.cpu(), page, b, [8, 39][b])
        a, c = (x.k[pg, :, off] for x in caches)
        assert torch.equal(bits(a[:, rot:]), bits(c[:, rot:])) and torch.equal(bits(c[:, rot:].cpu()), bits(k[b, :, rot:].to(F16)))
    w = torch.ones(dim).cuda()
    normed = ops.norm_rope_append(caches[1], table, q.cuda(), k.cuda(), v.cuda(), pos, q_norm=w, k_norm=w, interleaved=inter)
    clean = ops.norm_rope_append(caches[1], table, torch.nan_to_num(q, 1.0, 1.0, 1.0).cuda(), k.cuda(), v.cuda(), pos, q_norm=w, k_norm=w,
                                 interleaved=inter)
    ops.check_status()
    finite = torch.isfinite(q).all(-1).cuda()
    assert torch.equal(normed[finite], clean[finite]) and bool(torch.isfinite(normed[finite]).all())


def test_norm_of_zeros_and_huge_rows(ops):
    cache = make_cache(ops, [3], 1, 64, 16, BF16)
    q = torch.zeros((3, 1, 64))
    q[1] = 1e15
    q[2, 0, 5] = 3e-20
    k = torch.ones((3, 1, 64))
    got = ops.norm_rope_append(cache, ops.rope_table(64), q.cuda(), k.cuda(), k.cuda(), dev([0, 0, 0]), q_norm=torch.ones(64).cuda(), eps=1e-6).cpu()
    ops.check_status()
    assert bool((got[0] == 0).all()) and torch.allclose(got[1], torch.ones(1, 64), rtol=1e-6)
    assert abs(float(got[2, 0, 5]) / 3e-17 - 1) < 1e-6


def test_norm_rope_refusals(ops):
    from quantized_prefill_gemm_mmq_gb300._lib import MMQError
    cache = make_cache(ops, [9, 40], 2, 64, 16)
    q, k, v = (torch.zeros((2, h, 64)).cuda() for h in (4, 2, 2))
    pos, one, three = dev([8, 39]), ops.rope_table(64), ops.rope_table(64, sections=[8, 12, 12])
    ok = dict(cache=cache, rope=one, q=q, k=k, v=v, pos=pos)
    for kw in (dict(rope=three), dict(q_norm=torch.ones(32).cuda()), dict(k_norm=torch.ones(64, dtype=F16).cuda()), dict(out_dtype=BF16),
               dict(out=torch.zeros(2, 4, 64, dtype=F16).cuda(), out_dtype=F32), dict(pos=pos.long()), dict(k=k[:, :1])):
        with pytest.raises(ValueError):
            ops.norm_rope_append(**{**ok, **kw})
    with pytest.raises(MMQError):
        ops.norm_rope_append(**ok, eps=-1.0)
    with pytest.raises(ValueError):
        ops.rope_append(cache, three, q, k, v, pos)
    for bad in ([8, 12], [40, -8], [], [1] * 32):
        with pytest.raises(ValueError):
            ops.rope_axes(64, bad)
    three.axis[5] = 3
    ops.norm_rope_append(cache, three, q, k, v, torch.zeros((3, 2), dtype=torch.int32).cuda())
    with pytest.raises(MMQError, match="an axis"):
        ops.check_status()


# ---------------------------------------------------------------- keeping a path ---

@pytest.mark.parametrize("dtype,dim,H,page,layout,N,width,new,count,track", [
    (F16, 128, 4, 16, "hnd", 16, 5, None, None, True),
    (BF16, 8, 1, 1, "nhd", 64, 64, None, [64, 10, 0], True),
    (F16, 72, 3, 7, "nhd", 40, 12, [40, 13, 12], [12, 3, 12], False),
    (BF16, 256, 33, 64, "hnd", 63, 20, None, [20, 1, 7], True),
    (F16, 64, 2, 16, "hnd", 1, 1, None, None, True),
])
def test_keep(ops, dtype, dim, H, page, layout, N, width, new, count, track):
    lens = [N + 5, 2 * N + 33, N]
    cache = make_cache(ops, lens, H, dim, page, dtype, layout, track=track)
    if track:
        cache.pos.copy_(torch.randint(0, 1000, tuple(cache.pos.shape), generator=torch.Generator().manual_seed(1)))
    counts = new if new is not None else [N] * 3
    g = torch.Generator().manual_seed(2)
    path = torch.zeros((3, width), dtype=torch.int32)
    for b in range(3):
        m = min(width, counts[b])
        path[b, :m] = torch.randperm(counts[b], generator=g)[:m].sort().values.to(torch.int32)
    kept = count if count is not None else [width] * 3
    pools = [x.cpu().clone() for x in ((cache.k, cache.v, cache.weight, cache.pos) if track else (cache.k, cache.v))]
    ref.keep(pools, cache.table.cpu(), lens, counts, page, path, kept)
    ops.kv_keep(cache, path.cuda(), dev(count), N, new=dev(new))
    ops.check_status()
    for x, want in zip((cache.k, cache.v, cache.weight, cache.pos), pools):
        assert torch.equal(x.cpu(), want)


def test_keep_refusals(ops):
    cache = make_cache(ops, [90, 90], 1, 64, 16)
    for keep, nodes in ((torch.zeros((2, 3)).cuda(), 4), (dev([[0, 1, 2]]), 4), (dev([[0, 1, 2]] * 2), 2), (dev([[0]] * 2), 65), (dev([0, 1]), 4)):
        with pytest.raises(ValueError):
            ops.kv_keep(cache, keep, None, nodes)
    before = cache.k.clone()
    ops.kv_keep(cache, torch.zeros((2, 0), dtype=torch.int32).cuda(), None, 4)
    ops.check_status()
    assert torch.equal(before, cache.k)


# --------------------------------------------------------------------- together ---

@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompt_in_chunks_then_trees(ops, dtype):
    """A prompt at once and in chunks gives the same cache; a tree's accepted path, kept, gives the rows that the same tokens
    give as a chain (the attention's rounding apart: two roundings of p and one of the output either way)."""
    H, G, dim, cap = 2, 2, 64, 20.0
    total = 150
    g = torch.Generator().manual_seed(9)
    rows = torch.randn((total + 12, (G + 2) * H * dim), generator=g).cuda()
    qw, kw = (1 + 0.1 * torch.randn(dim, generator=g).cuda() for _ in range(2))
    table = ops.rope_table(dim, sections=[8, 12, 12])
    at = torch.stack([torch.arange(total + 12), torch.arange(total + 12) // 7, torch.arange(total + 12) % 7]).to(torch.int32).cuda()

    def step(cache, idx, pos):
        d = rows[idx]
        q, k, v = (d[:, a * dim:b * dim].view(len(idx), b - a, dim) for a, b in ((0, G * H), (G * H, G * H + H), (G * H + H, (G + 2) * H)))
        cache.lens.add_(len(idx))
        return ops.norm_rope_append(cache, table, q, k, v, at[:, pos].contiguous(), qw, kw, out_dtype=dtype)

    def new_cache():
        return ops.KVCache.allocate(1, 12, H, dim, 16, dtype)

    once, chunks, chain = new_cache(), new_cache(), new_cache()
    everything = list(range(total))
    whole = ops.attn_prefill(once, step(once, everything, everything), cap=cap)
    parts = [ops.attn_prefill(chunks, step(chunks, everything[i:i + 64], everything[i:i + 64]), cap=cap) for i in range(0, total, 64)]
    step(chain, everything, everything)
    ops.check_status()
    assert torch.equal(once.k, chunks.k) and torch.equal(once.v, chunks.v) and torch.equal(once.pos, chunks.pos)
    tol = 4 * ref.HALF[dtype] * float(once.v.float().abs().max())
    assert float((whole - torch.cat(parts)).abs().max()) <= tol
    # a tree of eight drafts; nodes 0, 2, 5, 7 are accepted; a node's position goes by its depth
    parents = [-1, 0, 0, 1, 1, 2, 2, 5]
    depth = [0, 1, 1, 2, 2, 2, 2, 3]
    nodes, path = [total + i for i in range(8)], [0, 2, 5, 7]
    q = step(once, nodes, [total + d for d in depth])
    tree = ops.attn_tree(once, q, ops.tree_words([parents]), cap=cap)
    ops.kv_keep(once, dev([path]), None, 8)
    once.lens.sub_(4)
    want = ops.attn_prefill(chain, step(chain, [nodes[i] for i in path], [total + depth[i] for i in path]), cap=cap)
    ops.check_status()
    assert float((tree[path] - want).abs().max()) <= tol
    live = total + 4
    for a, b in ((once.k, chain.k), (once.v, chain.v)):
        a, b = (x[once.table[0].long()].transpose(1, 2).flatten(0, 1)[:live] for x in (a, b))
        assert torch.equal(a, b)
    # and a single token on top of either
    last = [ops.attn_prefill(c, step(c, [total + 9], [total + 4]), cap=cap) for c in (once, chain)]
    ops.check_status()
    assert torch.equal(*last)


def test_capped_scores_that_are_not_finite(ops):
    """A K entry that is NaN or infinite under a cap: NaN makes the rows that see it NaN and leaves the others, also where
    they share everything but that entry; an infinite score counts as the cap."""
    lens, N, dim = [300], 200, 64
    for bad in (float("nan"), float("inf")):
        cache = make_cache(ops, lens, 1, dim, 16, BF16)
        q = queries(cache, lens, N, 1)
        q[:, :, 0] = 1.0
        want = ops.attn_prefill(cache, q.cuda(), cap=10.0)
        pg, off = serve_ref.slot_place(cache.table.cpu(), 16, 0, 250)
        cache.k[pg, 0, off, 0] = bad
        got = ops.attn_prefill(cache, q.cuda(), cap=10.0)
        ops.check_status()
        assert torch.equal(got[:150], want[:150])
        if bad != bad:
            assert bool(torch.isnan(got[150:]).all())
        else:
            cache.k[pg, 0, off, 0] = 3e4                     # as good as infinite: tanh is 1 either way
            cache.k[pg, 0, off, 1:] = 0
            assert torch.equal(got, ops.attn_prefill(cache, q.cuda(), cap=10.0))


@pytest.mark.parametrize("lens,H,group,dim,page", [([5000], 8, 1, 128, 7), ([5000], 8, 1, 128, 16), ([3000, 100], 8, 4, 128, 64), ([4000], 4, 2, 256, 24)])
def test_many_calls_in_a_row_agree(ops, lens, H, group, dim, page):
    """Few rows and cut units, back to back: whatever the warps' timing, the same bits."""
    cache = make_cache(ops, lens, H, dim, page, BF16)
    q = queries(cache, lens, 1, group).cuda()
    want = check(ops, cache, queries(cache, lens, 1, group), lens)
    work = ops.prefill_workspace(cache, H * group, 1)
    outs = torch.stack([ops.attn_prefill(cache, q, workspace=work) for _ in range(600)])
    ops.check_status()
    assert bool((outs == want).all())


def test_units_taken_over_in_graphs_and_on_two_streams(ops):
    """Calls with more units than the device has multiprocessors (CTAs take over units of those that have not started):
    captured and replayed, and two at once on streams of their own."""
    lens, N = [900, 950], 900
    caches = [make_cache(ops, lens, 32, 64, 16, dt) for dt in (BF16, F16)]
    qs = [queries(c, lens, N, 2).cuda() for c in caches]
    want = [ops.attn_prefill(c, q, window=300) for c, q in zip(caches, qs)]
    out = [torch.empty_like(w) for w in want]
    work = [ops.prefill_workspace(c, 64, N) for c in caches]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for i in range(2):
            ops.attn_prefill(caches[i], qs[i], window=300, out=out[i], workspace=work[i])
    for _ in range(5):
        for o in out:
            o.fill_(3)
        g.replay()
        assert all(torch.equal(o, w) for o, w in zip(out, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for o in out:
        o.fill_(3)
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                ops.attn_prefill(caches[i], qs[i], window=300, out=out[i], workspace=work[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(out, want))
    ops.check_status()


def test_layouts_without_tensor_copies(ops):
    """Heads that share one key-value row (a stride of 0), and a cache of one page: the same as laid out plainly."""
    g = torch.Generator().manual_seed(8)
    one = torch.randn((2, 6, 1, 16, 64), generator=g).to(BF16).cuda()
    table, lens = torch.arange(6, dtype=torch.int32).view(1, 6).cuda(), dev([90])
    shared = ops.KVCache(*(x.expand(6, 3, 16, 64) for x in one), table, lens)
    plain = ops.KVCache(*(x.expand(6, 3, 16, 64).contiguous() for x in one), table, lens)
    q = queries(plain, [90], 20, 2).cuda()
    assert torch.equal(ops.attn_prefill(shared, q), ops.attn_prefill(plain, q))
    single = ops.KVCache(*(x[:1].expand(1, 3, 16, 64).contiguous() for x in one), table[:, :1].contiguous(), dev([13]))
    check(ops, single, queries(single, [13], 5, 2), [13])


def test_many_ragged_sequences(ops):
    """More sequences than a warp looks at in one go, empty ones among them, in caches long enough to be cut up."""
    g = torch.Generator().manual_seed(12)
    lens = torch.randint(0, 60, (75,), generator=g).tolist()
    lens[3], lens[40], lens[74], lens[0] = 0, 1500, 900, 0
    new = [min(n, 2) for n in lens]
    cache = make_cache(ops, lens, 2, 64, 16, BF16)
    got = check(ops, cache, queries(cache, lens, 2, 3), lens, new=new)
    assert bool((got.view(75, 2, -1)[3] == 0).all())
    parents, words = trees(75, 2)
    check(ops, cache, queries(cache, lens, 2, 3), lens, new=new, tree=words)


@pytest.mark.parametrize("H,group,N,dim", [(1, 128, 1, 64), (1, 128, 3, 128), (2, 96, 2, 160), (1, 5, 60, 184)])
def test_wide_groups(ops, H, group, N, dim):
    lens = [700, 90]
    cache = make_cache(ops, lens, H, dim, 24, F16)
    check(ops, cache, queries(cache, lens, N, group), lens)


def test_limits_of_what_rows_see(ops):
    """Prefixes past the length or negative, documents that begin before the cache, windows longer than anything."""
    lens, N = [300, 64], 64
    cache = make_cache(ops, lens, 1, 64, 16)
    q = queries(cache, lens, N, 2)
    check(ops, cache, q, lens, prefix=[1 << 30, -5], first=[[-3] * N, [t - 10 for t in range(N)]], window=(1 << 31) - 1)


@pytest.mark.parametrize("out_dtype,offset", [(F32, 4), (BF16, 8)])
def test_outputs_that_begin_on_16_bytes(ops, out_dtype, offset):
    lens, N = [1100], 20
    cache = make_cache(ops, lens, 2, 128, 16, BF16)
    q = queries(cache, lens, N, 2).cuda()
    want = ops.attn_prefill(cache, q, out_dtype=out_dtype)
    buf = torch.full((N * 4 * 128 + 64,), 7.0, dtype=out_dtype).cuda()
    out = buf[offset:offset + N * 4 * 128].view(N, 4, 128)
    ops.attn_prefill(cache, q, out=out)
    ops.check_status()
    assert torch.equal(out, want) and bool((buf[:offset] == 7).all()) and bool((buf[offset + N * 4 * 128:] == 7).all())


def test_keep_nothing_and_everything(ops):
    cache = make_cache(ops, [40, 30], 2, 64, 16)
    before = [x.clone() for x in (cache.k, cache.v, cache.weight)]
    ops.kv_keep(cache, dev([[0, 1, 2, 3]] * 2), None, 4)                 # already in place
    ops.kv_keep(cache, dev([[2, 3]] * 2), dev([0, 0]), 4)                # nothing stays
    ops.kv_keep(cache, dev([[2, 3]] * 2), None, 4, new=dev([0, 0]))      # no nodes: indexes past them are reported
    with pytest.raises(RuntimeError, match="a kept node"):
        ops.check_status()
    assert all(torch.equal(a, b) for a, b in zip((cache.k, cache.v, cache.weight), before))


@pytest.mark.parametrize("window", [1 << 31, (1 << 32) + 5, -(1 << 32) + 5])
def test_windows_that_no_int32_holds(ops, window):
    """Refused; the last two would be windows of five entries, cut to 32 bits."""
    cache = make_cache(ops, [40], 1, 64, 16)
    with pytest.raises(ValueError, match="window"):
        ops.attn_prefill(cache, queries(cache, [40], 4, 2).cuda(), window=window)


@pytest.mark.parametrize("dtype,dim,group", [(BF16, 128, 1), (F16, 64, 4), (BF16, 192, 2)])
def test_values_that_are_not_finite_in_tiles_that_two_halves_share(ops, dtype, dim, group):
    """Every tile is seen in part and holds V entries that are not finite, in units whose two halves both look for them: rows
    that see none are the same bit for bit in every one of many calls, the others not finite."""
    lens, N, window = [900], 600, 40
    cache = make_cache(ops, lens, 2, dim, 16, dtype)
    q = queries(cache, lens, N, group).cuda()
    want = ops.attn_prefill(cache, q, window=window)
    where = [s for s in range(0, 900, 57)]
    for i, s in enumerate(where):
        pg, off = serve_ref.slot_place(cache.table.cpu(), 16, 0, s)
        cache.v[pg, :, off, (i * 37) % dim] = (float("nan"), float("inf"), float("-inf"))[i % 3]
    hit = torch.tensor([any(i - window < s <= i for s in where) for i in range(300, 900)]).cuda()
    assert 100 < int(hit.sum()) < 500
    outs = [ops.attn_prefill(cache, q, window=window) for _ in range(100)]
    ops.check_status()
    for got in outs:
        assert torch.equal(got[~hit], want[~hit])
        assert not bool(torch.isfinite(got[hit]).all(-1).any())


@pytest.mark.parametrize("N,group,dim,page", [(40, 4, 128, 16), (40, 4, 128, 7), (40, 2, 256, 16)])
def test_rows_that_are_not_there_may_hold_anything(ops, N, group, dim, page):
    """q rows past the counts that are not finite: the others are the same bit for bit."""
    lens, new = [300, 200], [25, 7]
    cache = make_cache(ops, lens, 2, dim, page, BF16)
    q = queries(cache, lens, N, group)
    want = ops.attn_prefill(cache, q.cuda(), new=dev(new))
    want_cap = ops.attn_prefill(cache, q.cuda(), new=dev(new), cap=5.0, window=100)
    bad = q.view(2, N, 2 * group, dim).clone()
    for b, n in enumerate(new):
        bad[b, n:] = float("nan")
        bad[b, n + 1::2] = float("inf")
    bad = bad.view_as(q).cuda()
    assert torch.equal(ops.attn_prefill(cache, bad, new=dev(new)), want)
    assert torch.equal(ops.attn_prefill(cache, bad, new=dev(new), cap=5.0, window=100), want_cap)
    ops.check_status()


@pytest.mark.parametrize("cap", [1e-30, 1e-39, 1e-44])
def test_the_smallest_caps(ops, cap):
    """Scores of a cap that is next to nothing are equal, those of 0 among them: means of the values."""
    cache = make_cache(ops, [70], 1, 64, 16, BF16)
    pg, off = serve_ref.slot_place(cache.table.cpu(), 16, 0, 3)
    cache.k[pg, 0, off] = 0
    q = queries(cache, [70], 20, 2)
    got = check(ops, cache, q, [70], cap=cap, out_dtype=F32)
    assert bool(torch.isfinite(got).all())
    check(ops, cache, q, [70], cap=cap, scale=-1.0, out_dtype=F32)
