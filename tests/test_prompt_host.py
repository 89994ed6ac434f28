"""CPU checks of the host side of the operators for prompts and trees of drafts: refusals at the C boundary before a GPU is
touched, workspace sizes, axes of rotation tables."""
from __future__ import annotations

import ctypes
import os

import pytest

from quantized_prefill_gemm_mmq_gb300 import _lib
from tests.test_serve_host import BAD_CACHE, Args

needs_lib = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmmq.so not built (run __graft_entry__.build())")


@pytest.fixture(scope="module")
def a():
    return Args()


def prefill(a, cache=None, q="p", ldq=256, out="other", out_dtype=0, qh=4, new=1, scale=0.1, cap=0.0, window=0, work="p"):
    at = {"p": a.p, "odd": a.odd, "null": a.null, "other": ctypes.c_void_p(a.p.value + 2048)}
    return _lib.load().mmq_attn_prefill(cache if cache is not None else a.cache(), at[q], ldq, a.null, a.null, a.null, a.null, at[out], out_dtype,
                                        qh, new, scale, cap, window, at[work], a.null)


@needs_lib
@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches(a, kw, status):
    lib, c, p, n = _lib.load(), a.cache(**kw), a.p, a.null
    assert prefill(a, cache=c) == status
    assert lib.mmq_attn_tree(c, p, 256, p, n, n, a.odd, 0, 4, 1, 0.1, 0.0, p, n) == status
    assert lib.mmq_kv_keep(c, p, n, n, 2, 4, n) == status
    assert lib.mmq_norm_rope_append(c, p, n, 64, 1.0, 0, n, n, 1e-6, p, 256, p, 128, p, 128, p, 1, n, p, 256, 2, 4, 1, n) == status
    assert lib.mmq_prefill_sizes(c, 4, 1, ctypes.byref(ctypes.c_int64())) == status


@needs_lib
def test_prefill_refusals(a):
    assert prefill(a, qh=3) == prefill(a, qh=0) == prefill(a, new=0) == prefill(a, ldq=248) == prefill(a, qh=258) == -1
    nan, inf = float("nan"), float("inf")
    assert prefill(a, scale=nan) == prefill(a, scale=inf) == prefill(a, cap=nan) == prefill(a, cap=-1.0) == prefill(a, cap=1025.0) == -1
    assert prefill(a, window=-1) == prefill(a, out_dtype=1) == prefill(a, out_dtype=3) == prefill(a, out="p") == -1
    assert prefill(a, q="null") == prefill(a, out="null") == prefill(a, work="null") == -6
    assert prefill(a, q="odd") == prefill(a, out="odd") == prefill(a, work="odd") == prefill(a, ldq=260) == -2
    assert prefill(a, cache=a.cache(seqs=0)) == 0


@needs_lib
def test_scales_that_overflow_in_powers_of_two(a):
    """Finite in f32, but not times log2(e): every score of 0 would be NaN."""
    assert prefill(a, scale=3e38) == prefill(a, scale=-3e38) == prefill(a, scale=3e38, cap=5.0) == -1
    assert prefill(a, scale=2e38, work="odd") == -2          # as far as the alignment


@needs_lib
def test_tree_refusals(a):
    lib, c, p, n = _lib.load(), a.cache(), a.p, a.null
    call = lambda tree=p, new=1, cache=c, qh=4: lib.mmq_attn_tree(cache, p, 256, tree, n, n, a.odd, 0, qh, new, 0.1, 0.0, p, n)  # noqa: E731
    assert call(new=65) == -1 and call(new=0) == -1 and call(qh=5) == -1 and call(tree=n) == -6
    assert call() == -2 and call(cache=a.cache(seqs=0), tree=n) == 0


@needs_lib
def test_sizes(a):
    lib, nf = _lib.load(), ctypes.c_int64()
    assert lib.mmq_prefill_sizes(a.cache(), 4, 1, None) == -6
    for kw, qh, new, ok in ((dict(), 4, 1, True), (dict(), 5, 1, False), (dict(), 4, 0, False), (dict(), 258, 1, False),
                            (dict(seqs=65535, heads=32767, cols=8), 32767, 1, True),        # one tile each
                            (dict(seqs=65535, heads=32768, cols=16), 32768, 1, False),
                            (dict(seqs=65535), 2, 32769, False), (dict(heads=1), 128, 1 << 24, False)):
        assert lib.mmq_prefill_sizes(a.cache(**kw), qh, new, ctypes.byref(nf)) == (0 if ok else -1)
        if ok:
            assert 4 <= nf.value <= 24 << 20
    assert lib.mmq_prefill_sizes(a.cache(dim=256), 256, 100, ctypes.byref(nf)) == 0 and 0 < nf.value <= 24 << 20


@needs_lib
def test_norm_rope_refusals(a):
    lib, p, n = _lib.load(), a.p, a.null

    def call(cache=None, freq=p, axis=p, rot=64, qn=p, eps=1e-6, q=p, ldq=256, k=p, ldk=128, pos=p, axes=2, out=a.odd, ldo=256, dt=2, qh=4, new=1):
        return lib.mmq_norm_rope_append(cache if cache is not None else a.cache(), freq, axis, rot, 1.0, 0, qn, n, eps, q, ldq, k, ldk, p, 128, pos,
                                        axes, n, out, ldo, dt, qh, new, n)
    assert call(rot=0) == call(rot=63) == call(rot=66) == call(qh=0) == call(new=-1) == call(ldq=252) == call(ldk=64) == call(ldo=252) == -1
    assert call(axes=0) == call(axes=9) == call(eps=-1.0) == call(eps=float("nan")) == call(dt=1) == call(dt=3) == -1
    assert call(out=p, ldo=260) == call(out=p, dt=0) == -1                   # in place with two strides, or of another type
    assert call(new=0) == call(cache=a.cache(seqs=0)) == 0
    assert call(q=n) == call(freq=n) == call(pos=n) == call(out=n) == call(axis=n) == -6
    assert call(k=a.odd) == call(ldk=130) == call() == call(qn=a.odd, out=p) == call(out=ctypes.c_void_p(p.value + 1024), ldo=260, dt=0) == -2


@needs_lib
def test_keep_refusals(a):
    lib, p, n = _lib.load(), a.p, a.null
    call = lambda keep=p, width=2, nodes=4, cache=a.cache(): lib.mmq_kv_keep(cache, keep, n, n, width, nodes, n)  # noqa: E731
    assert call(width=5) == -1 and call(width=-1) == -1 and call(nodes=65) == -1 and call(nodes=-1) == -1
    assert call(keep=n) == -6 and call(width=0) == 0 and call(cache=a.cache(seqs=0)) == 0


def test_axes():
    pytest.importorskip("torch")
    from quantized_prefill_gemm_mmq_gb300 import ops
    assert ops.rope_axes(12, [2, 3, 1]) == [0, 0, 1, 1, 1, 2]
    assert ops.rope_axes(16, [4, 2, 2], alternate=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert ops.rope_axes(8, [4]) == [0, 0, 0, 0]
    for rot, bad in ((12, [2, 3]), (12, [7, -1]), (12, []), (18, [1] * 9)):
        with pytest.raises(ValueError):
            ops.rope_axes(rot, bad)


def test_axes_that_alternate_as_far_as_the_pairs_reach():
    """Against axes written out: sections that the order cannot give in full, and one that it can."""
    pytest.importorskip("torch")
    from quantized_prefill_gemm_mmq_gb300 import ops
    # axis 1 has 1, 4, .. 31, axis 2 has 2, 5, .. 29
    pairs = [0, 1, 2] * 10 + [0, 1]
    assert ops.rope_axes(64, [8, 12, 12], alternate=True) == pairs
    assert [pairs.count(a) for a in range(3)] == [11, 11, 10]
    assert ops.rope_axes(16, [0, 4, 4], alternate=True) == [0, 1, 2, 0, 1, 2, 0, 1]
    assert ops.rope_axes(16, [6, 0, 2], alternate=True) == [0, 0, 2, 0, 0, 2, 0, 0]
    # one that fits: 11 pairs of axis 1 end at 31, 10 of axis 2 at 29
    assert ops.rope_axes(64, [11, 11, 10], alternate=True) == pairs
