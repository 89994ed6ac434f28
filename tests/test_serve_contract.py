"""GPU tests of what the decode-side operators promise beside their values:
outputs that are the caller's alone, rows that are not finite staying so
wherever their parts are joined, scores of any size, limits, errors and rows
from odd places.

Tolerances are those of test_serve_ops.py, or equality."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import serve_ref as ref  # noqa: E402
from tests.test_serve_ops import check_attention, make_cache, ops  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------- attention ---

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("qscale", [3e6, 1e8, 1e12])
@pytest.mark.parametrize("dim,group,N", [(64, 1, 1), (128, 4, 1), (128, 2, 3), (64, 8, 4), (256, 3, 1)])
def test_attn_large_scores(ops, dim, group, N, qscale, dtype):
    """Scores far past 2^24, where f32 no longer tells neighbouring whole numbers apart.  An output is still a mean of the
    values that its row sees; where the largest score leads by more than four times what a score may be off (2^-20 of
    scale sum|q||k|) and 64 besides, it is that entry's value (the others' share is below 2^-64), to 2^-19.
    Weights lie between 0 and the number of rows that add to them, and such an entry gets all of its row's."""
    lens, page, scale = [300, 9000], 64, 4.0
    cache = make_cache(ops, lens, 2, dim, page, dtype)
    q = torch.randn((2 * N, 2 * group, dim), generator=torch.Generator().manual_seed(11)) * qscale
    cache.weight.zero_()
    got = ops.attn_decode(cache, q.cuda(), scale=scale, accumulate=True)
    assert torch.equal(got, ops.attn_decode(cache, q.cuda(), scale=scale))
    ops.check_status()
    got, weight = got.cpu().double(), cache.weight.cpu().double()
    assert bool(torch.isfinite(got).all())
    assert bool(((weight >= 0) & (weight <= N * group * (1 + 2.0 ** -18))).all())
    tab, kp, vp, clear = cache.table.cpu(), cache.k.cpu(), cache.v.cpu(), 0
    for b, n in enumerate(lens):
        pages = tab[b, :-(-n // page)].long()
        for h in range(2):
            k, v = (x[pages, h].reshape(-1, dim)[:n].double() for x in (kp, vp))
            won = torch.zeros(n)
            for t in range(N):
                m = n - N + t + 1
                lo, hi, slack = v[:m].amin(0), v[:m].amax(0), 2.0 ** -18 * v[:m].abs().max()
                for j in range(h * group, (h + 1) * group):
                    row = q[b * N + t, j].double()
                    out, s = got[b * N + t, j], k[:m] @ row * scale
                    assert bool(((out >= lo - slack) & (out <= hi + slack)).all())
                    best, at = s.topk(2)
                    off = 2.0 ** -20 * scale * float((k[:m].abs() @ row.abs()).max())
                    if float(best[0] - best[1]) > 4 * off + 64:
                        assert float((out - v[at[0]]).abs().max()) <= 2.0 ** -19 * float(v[at[0]].abs().max())
                        won[at[0]] += 1
                        clear += 1
            assert bool((weight[pages, h].reshape(-1)[:n] >= won * (1 - 2.0 ** -18)).all())
    assert clear > 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,dim,group,N", [(torch.float16, 64, 1, 1), (torch.bfloat16, 128, 4, 1), (torch.bfloat16, 64, 3, 3),
                                               (torch.float16, 128, 8, 4), (torch.float16, 256, 2, 1)])
def test_attn_queries_that_are_not_finite(ops, bad, dtype, dim, group, N):
    """A row of q that is not finite gives a row that is not, in one CTA's segments and in split ones; the other rows
    do not change."""
    cache = make_cache(ops, [20000, 40], 2, dim, 64, dtype)
    q = torch.randn((2 * N, 2 * group, dim), generator=torch.Generator().manual_seed(7)).cuda()
    want = ops.attn_decode(cache, q)
    rows = [(0, 0), (2 * N - 1, 2 * group - 1)]         # of the long sequence and of the short one
    for r, h in rows:
        q[r, h, 3] = bad
    got = ops.attn_decode(cache, q)
    ops.check_status()
    same = torch.ones((2 * N, 2 * group), dtype=torch.bool)
    for r, h in rows:
        assert not bool(torch.isfinite(got[r, h]).any())
        same[r, h] = False
    assert torch.equal(got[same.cuda()], want[same.cuda()])


@pytest.mark.parametrize("dtype,dim,group", [(torch.float16, 64, 1), (torch.bfloat16, 128, 4), (torch.float16, 128, 8), (torch.float16, 256, 2)])
def test_attn_runs_of_entries_that_are_not_finite(ops, dtype, dim, group):
    """Keys that are NaN over a run that fills whole parts of a split sequence, or infinite values where the scores are
    so low that their probability is 0: every row sees them, so no row is finite."""
    n, page = 20000, 64
    g = torch.Generator().manual_seed(8)
    q = torch.randn((1, group, dim), generator=g).cuda()
    for which in ("k", "v"):
        cache = make_cache(ops, [n], 1, dim, page, dtype)
        pages = cache.table[0, 100:200].long()           # entries 6400 .. 12799
        if which == "k":
            cache.k[pages] = float("nan")
        else:
            cache.v[pages] = float("inf")
            cache.k[pages] = 0                           # scores of 0; each row has an entry of score 4000 besides
            cache.k[cache.table[0, 0].long(), :, :group] = (q[0] * (4000.0 / q[0].square().sum(-1, keepdim=True))).to(dtype)
        got = ops.attn_decode(cache, q, scale=1.0)
        ops.check_status()
        assert not bool(torch.isfinite(got).any()), which


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attn_split_rows_that_see_nothing_are_zero(ops, dtype):
    """Rows that are not there, over parts that hold Inf values: 0, also where the parts of a long sequence are joined."""
    N, group, dim = 3, 2, 64
    cache = make_cache(ops, [20000], 2, dim, 64, dtype)
    cache.v[cache.table[0].long(), :, 5] = float("inf")
    q = torch.randn((N, 2 * group, dim), generator=torch.Generator().manual_seed(6)).cuda()
    got = ops.attn_decode(cache, q, new=torch.tensor([1], dtype=torch.int32).cuda())
    ops.check_status()
    assert not bool(torch.isfinite(got[0]).any()) and bool((got[1:] == 0).all())


# ---------------------------------------------------------------- outputs ---

def output_calls(ops, dim):
    """name -> call returning new output tensors; shapes that depend on dim."""
    cache = make_cache(ops, [30], 2, dim, 16)
    q, k, v = (torch.randn((1, h, dim), generator=torch.Generator().manual_seed(h)).cuda() for h in (4, 2, 2))
    table, pos = ops.rope_table(dim), torch.full((1,), 29, dtype=torch.int32).cuda()
    target = torch.softmax(torch.randn((dim, 3, 50), generator=torch.Generator().manual_seed(9)), -1).cuda()
    drafted, uniform = torch.zeros((dim, 2), dtype=torch.int32).cuda(), torch.full((dim, 3), 0.5).cuda()
    return {"attn": lambda: [ops.attn_decode(cache, q)], "rope": lambda: [ops.rope_append(cache, table, q, k, v, pos)],
            "verify": lambda: list(ops.spec_verify(target, None, drafted, uniform))}


@pytest.mark.parametrize("name", ["attn", "rope", "verify"])
def test_outputs_own_their_storage(ops, name):
    call = output_calls(ops, 40)[name]
    outs = [o for _ in range(6) for o in call()]
    for o in outs:
        assert o.untyped_storage().nbytes() == o.numel() * o.element_size() and o.storage_offset() == 0
    kept = [o.clone() for o in outs]
    for i, o in enumerate(outs):                        # growing one output leaves every other one alone
        o.resize_((3 * o.shape[0],) + tuple(o.shape[1:])).fill_(-5)
        assert all(torch.equal(a, b) for a, b in zip(outs[i + 1:], kept[i + 1:]))
        assert all(bool((a == -5).all()) for a in outs[:i + 1])


@pytest.mark.parametrize("name,dim", [("attn", 48), ("rope", 56), ("verify", 24)])
def test_outputs_after_a_call_in_inference_mode(ops, name, dim):
    call = output_calls(ops, dim)[name]
    with torch.inference_mode():
        call()
    for o in call():
        assert not o.is_inference()
        o.add_(1)
        if o.is_floating_point():                        # and autograd may keep it
            w = torch.ones((), device="cuda", requires_grad=True)
            (o * w).sum().backward()
            assert bool(torch.isfinite(w.grad))


# ----------------------------------------------------------------- errors ---

CHECKS = """
import time, torch
from quantized_prefill_gemm_mmq_gb300 import ops

def check():
    best = 1e9
    for _ in range(30):
        t = time.perf_counter()
        for _ in range(50):
            ops.check_status()
        best = min(best, time.perf_counter() - t)
    return best

ops.quantize_q8_1(torch.randn((4, 512), device="cuda"))
before = check()
target = torch.full((1, 2, 4), 0.25, device="cuda")
ops.spec_verify(target, None, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros((1, 2), device="cuda"))
print(before / check())
"""


def test_status_checks_of_programs_without_these_operators(ops):
    """A process that has launched none of them does not pay for their status word: it is a second copy from the device,
    about a third of a check's time."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHECKS], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert float(r.stdout) < 0.85


def test_index_errors_say_what_they_are(ops):
    from quantized_prefill_gemm_mmq_gb300._lib import MMQError
    cache = make_cache(ops, [100, 50], 2, 64, 16)
    q = torch.randn((2, 4, 64)).cuda()
    cache.table[0, 2] = -1
    ops.attn_decode(cache, q)
    with pytest.raises(MMQError, match="attention: a page id") as e:
        ops.check_status()
    assert e.value.status == -11 and "barrier" not in str(e.value)
    ops.check_status()


def test_pending_errors_are_reported_together(ops):
    """A product's wait that ran out and an attention call's bad page, both before the check: one error names both, and
    the next check is clean."""
    from quantized_prefill_gemm_mmq_gb300 import _lib, synth
    lib = _lib.load()
    cache = make_cache(ops, [100, 50], 2, 64, 16)
    rows = torch.randn((2, 4, 64)).cuda()
    w = torch.from_numpy(synth.make_weights("q4_K", 512, 1024, 81)).cuda()
    x = torch.from_numpy(synth.make_x(256, 1024, 82, outliers=True)).cuda()
    _, ds, _, xa = ops.quantize_q8_1(x, want_qs=False, want_xh=False)
    ops.check_status()
    try:
        assert lib.mmq_debug_fault_inject(1, 1000) == 0  # withhold a copy; the wait for it gives up after 1 ms
        ops.gemm("q4_K", w, xa, ds, 512)
        torch.cuda.synchronize()
    finally:
        assert lib.mmq_debug_fault_inject(0, 0) == 0
    cache.table[0, 2] = -1
    ops.attn_decode(cache, rows)
    with pytest.raises(_lib.MMQError) as e:
        ops.check_status()
    assert e.value.status == -5 and "barrier" in str(e.value) and "attention: a page id" in str(e.value)
    ops.check_status()


def test_evict_more_than_65535_rows(ops):
    """Eviction of 2100 sequences of 32 heads: what evict_workspace sizes, kv_evict takes."""
    B, H, page, dim, n, budget = 2100, 32, 4, 8, 4, 3
    g = torch.Generator().manual_seed(13)
    k = torch.randn((B, H, page, dim), generator=g).half().cuda()
    v = torch.randn((B, H, page, dim), generator=g).half().cuda()
    table = torch.randperm(B, generator=g).to(torch.int32).view(B, 1).cuda()
    w = torch.stack([torch.randperm(page, generator=g) for _ in range(B * H)]).view(B, H, page).float().cuda()
    pos = torch.arange(page, dtype=torch.int32).expand(B, H, page).contiguous().cuda()
    cache = ops.KVCache(k, v, table, torch.full((B,), n, dtype=torch.int32).cuda(), w, pos)
    want, gone = {}, w == 0
    for name, x in (("k", k), ("v", v), ("w", w), ("pos", pos)):
        want[name] = x.clone()                           # one entry goes per page and head: the last takes its place
        want[name][gone] = x[:, :, page - 1:].expand(x.shape[:3] + x.shape[3:])[gone]
    wo, po = torch.zeros_like(w), torch.zeros_like(pos)
    ops.kv_evict(cache, budget, torch.full((B,), n, dtype=torch.int32).cuda(), wo, po, workspace=ops.evict_workspace(cache, budget))
    ops.check_status()
    for got, name in ((k, "k"), (v, "v"), (wo, "w"), (po, "pos")):
        assert torch.equal(got[:, :, :budget], want[name][:, :, :budget])


def test_one_row_of_a_product_of_odd_width(ops):
    """The distance between rows does not matter where there is one: a slice of a row of any width is taken."""
    cache = make_cache(ops, [30], 2, 64, 16)
    wide = torch.randn((1, 8 * 64 + 3)).cuda()
    q, k, v = (wide[:, a * 64:b * 64].view(1, b - a, 64) for a, b in ((0, 4), (4, 6), (6, 8)))
    pos, table = torch.full((1,), 29, dtype=torch.int32).cuda(), ops.rope_table(64)
    want = ops.rope_append(cache, table, q.contiguous(), k.contiguous(), v.contiguous(), pos)
    assert torch.equal(ops.rope_append(cache, table, q, k, v, pos), want)
    assert torch.equal(ops.attn_decode(cache, q), ops.attn_decode(cache, q.contiguous()))
    ops.check_status()


# ----------------------------------------------- further sizes and ranges ---

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [72, 80])
@pytest.mark.parametrize("group,N", [(20, 1), (8, 5), (35, 2), (13, 6)])
def test_attn_many_rows_of_80(ops, dtype, dim, group, N):
    """Two and four warps along 20 to 78 rows of heads of 72 and 80."""
    for accumulate in (False, True):
        check_attention(ops, [150, N, 129], N, group, 1, dim, 16, dtype, new=[N, N, N - 1], accumulate=accumulate,
                        seed=group, fill=float("inf"))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [1, 20])
def test_attn_long_split_of_80(ops, dtype, group):
    check_attention(ops, [20000, 40], 1, group, 1, 80, 64, dtype, seed=9)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,group", [(torch.float16, 1), (torch.bfloat16, 5), (torch.float16, 12)])
def test_attn_masked_entries_do_not_reach_earlier_rows_of_80(ops, bad, dtype, group):
    N, lens = 4, [67, 131]
    cache = make_cache(ops, lens, 2, 80, 16, dtype)
    q = torch.randn((8, 2 * group, 80), generator=torch.Generator().manual_seed(5)).cuda()
    want = ops.attn_decode(cache, q)
    tab = cache.table.cpu()
    for b, n in enumerate(lens):                         # the last new entry is not finite
        pg, off = ref.slot_place(tab, 16, b, n - 1)
        cache.v[pg, :, off] = bad
        cache.k[pg, :, off] = bad
    got = ops.attn_decode(cache, q)
    ops.check_status()
    for b in range(2):
        a, w = got[b * N:b * N + 3], want[b * N:b * N + 3]
        assert float((a - w).abs().max()) <= 2.0 ** -18 * float(w.abs().max())
        assert not bool(torch.isfinite(got[b * N + 3]).any())


def verify_counts(target, draft, n):
    """How often each token comes first, over the n x n pairs of midpoint uniforms: [drafted][token], in whole numbers."""
    u = (np.arange(n) + 0.5) / n
    V, counts = len(target), np.zeros((len(target), len(target)), np.int64)
    whole = lambda x: [round(float(min(max(y, np.float32(0)), np.float32(1))) * 2 ** 40) for y in x]  # noqa: E731
    rest = whole(target - draft)
    cum = np.cumsum(np.array(rest, dtype=object))
    redraw = np.zeros(V, np.int64)
    for x in u:
        r = cum[-1] * int(x * 2 ** 24) >> 24
        redraw[next(j for j in range(V) if cum[j] > r)] += 1
    for x in range(V):
        accepted = int((u.astype(np.float32) * draft[x] < target[x]).sum())
        counts[x] = (n - accepted) * redraw
        counts[x, x] += n * accepted
    return counts


def test_verify_counts(ops):
    """Accepted or redrawn, the first token over a grid of 2^16 pairs of uniforms: the counts themselves, which follow
    the target to within the grid's steps."""
    n = 1 << 8
    target = np.array([0.3, 0.25, 0.2, 0.1, 0.05, 0.05, 0.03, 0.02], np.float32)
    draft = np.array([0.1, 0.1, 0.1, 0.1, 0.15, 0.15, 0.15, 0.15], np.float32)
    counts = verify_counts(target, draft, n)
    u = (torch.arange(n) + 0.5) / n
    pairs = torch.stack((u.repeat_interleave(n), u.repeat(n)), 1)
    t, d = torch.from_numpy(target).cuda(), torch.from_numpy(draft).cuda()
    for x in range(8):
        got = torch.zeros(8, dtype=torch.int64)
        for part in pairs.split(n * n // 4):
            B = part.shape[0]
            tokens, _ = ops.spec_verify(t.expand(B, 2, 8).contiguous(), d.expand(B, 1, 8).contiguous(),
                                        torch.full((B, 1), x, dtype=torch.int32).cuda(), part.contiguous().cuda())
            got += torch.bincount(tokens[:, 0].cpu().long(), minlength=8)
        assert got.tolist() == counts[x].tolist()
    # an acceptance threshold and both ends of a redrawn token's interval lie within half a step of their place, so a
    # token is off by at most a step of 1/n for its own acceptance, and the redrawn share (below 1) by one of 1/n more
    total = (draft[:, None].astype(np.float64) * counts).sum(0) / n ** 2
    assert float(np.abs(total - target).max()) <= 2 / n


@pytest.mark.parametrize("bad", [81, 1 << 29, -1])
def test_bad_lengths_write_nothing(ops, bad):
    """A sequence whose length is out of range is taken as empty: the table entries past its real length, which may hold
    another's pages, are not followed."""
    from quantized_prefill_gemm_mmq_gb300._lib import MMQError
    rows = [torch.randn((2, h, 64), generator=torch.Generator().manual_seed(h)).cuda() for h in (4, 2, 2)]
    pos, table = torch.full((2,), 39, dtype=torch.int32).cuda(), ops.rope_table(64)
    results = []
    for first in (0, bad):
        cache = make_cache(ops, [40, 40], 2, 64, 16, extra=40)         # five pages: 80 entries
        cache.table[0, 2:] = cache.table[1, :3]
        before = [t.clone() for t in (cache.k, cache.v, cache.weight, cache.pos)]
        cache.lens[0] = first
        ops.rope_append(cache, table, *rows, pos)
        with pytest.raises(MMQError) as e:                             # one new token does not fit no entries either
            ops.check_status()
        assert e.value.status == -11
        out = ops.attn_decode(cache, rows[0], accumulate=True)
        assert bool((out[0] == 0).all())
        wo, po = torch.full_like(cache.weight, -7.0), torch.full_like(cache.pos, -7)
        ops.kv_evict(cache, 39, torch.tensor([0, 30], dtype=torch.int32).cuda(), wo, po)
        if first == 0:
            ops.check_status()
        else:
            with pytest.raises(MMQError) as e:
                ops.check_status()
            assert e.value.status == -11
        own = sorted(set(cache.table[1].tolist()))
        others = [p for p in range(cache.k.shape[0]) if p not in own]
        for got, was in zip((cache.k, cache.v, cache.weight, cache.pos), before):
            assert torch.equal(got[others], was[others])
        assert bool((wo[others] == -7).all()) and bool((po[others] == -7).all())
        results.append([t.cpu() for t in (cache.k, cache.v, cache.weight, cache.pos, wo, po, out)])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("qscale,scale", [(1e36, 1e-36), (1e-37, 1e36)])
@pytest.mark.parametrize("group,N", [(1, 1), (4, 3)])
def test_attn_queries_at_the_ends_of_f32(ops, group, N, qscale, scale, dtype):
    check_attention(ops, [300, 20], N, 2 * group, 2, 128, 16, dtype, qscale=qscale, scale=scale)
