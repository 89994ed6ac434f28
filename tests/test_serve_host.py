"""CPU checks of the decode-side operators' host side: argument refusals at the
C boundary before a GPU is touched, workspace sizes, rotation tables."""
from __future__ import annotations

import ctypes
import math
import os

import pytest

from quantized_prefill_gemm_mmq_gb300 import _lib

needs_lib = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmmq.so not built (run __graft_entry__.build())")


class Args:
    def __init__(self):
        self.buf = ctypes.create_string_buffer(4096)
        self.p = ctypes.c_void_p((ctypes.addressof(self.buf) + 15) & ~15)
        self.odd = ctypes.c_void_p(self.p.value + 4)
        self.null = ctypes.c_void_p(0)

    def cache(self, **kw):
        f = dict(k=self.p, v=self.p, weight=self.p, pos=self.p, table=self.p, len=self.p, k_page=2 * 16 * 64, k_head=16 * 64, k_slot=64,
                 v_page=2 * 16 * 64, v_head=16 * 64, v_slot=64, pages=8, dtype=0, heads=2, dim=64, page_size=16, seqs=1, cols=8)
        f.update(kw)
        return ctypes.byref(_lib.KVCacheC(**f))


@pytest.fixture(scope="module")
def a():
    return Args()


BAD_CACHE = [(dict(dtype=2), -1), (dict(heads=0), -1), (dict(dim=0), -1), (dict(dim=60), -1), (dict(dim=264), -1), (dict(page_size=0), -1),
             (dict(seqs=-1), -1), (dict(seqs=65536), -1), (dict(cols=0), -1), (dict(pages=0), -1), (dict(pages=1 << 31), -1),
             (dict(cols=1 << 27), -1), (dict(k_page=-8), -1), (dict(k_slot=68), -2), (dict(v_head=4), -2), (dict(k=None), -6), (dict(table=None), -6),
             (dict(len=None), -6)]


@needs_lib
@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches(a, kw, status):
    lib = _lib.load()
    c, p, n = a.cache(**kw), a.p, a.null
    assert lib.mmq_rope_append(c, p, 64, 1.0, 0, p, 256, p, 128, p, 128, p, n, p, 256, 4, 1, n) == status
    assert lib.mmq_attn_decode(c, p, 4 * 512, n, p, 4, 1, 0.1, 0, p, n) == status
    assert lib.mmq_kv_evict(c, 4, p, a.odd, a.odd, p, n) == status


@needs_lib
def test_rope_refusals(a):
    lib, c, p, n = _lib.load(), a.cache(), a.p, a.null
    call = lambda rot=64, q=p, ldq=256, k=p, ldk=128, pos=p, out=p, ldo=256, qh=4, new=1, freq=p, cache=c: lib.mmq_rope_append(  # noqa: E731
        cache, freq, rot, 1.0, 0, q, ldq, k, ldk, p, 128, pos, n, out, ldo, qh, new, n)
    assert call(rot=0) == -1 and call(rot=63) == -1 and call(rot=66) == -1
    assert call(qh=0) == -1 and call(new=-1) == -1 and call(ldq=252) == -1 and call(ldk=64) == -1
    assert call(ldq=256, ldo=260) == -1                       # in place with two strides
    assert call(new=0) == 0 and call(cache=a.cache(seqs=0)) == 0
    assert call(q=n) == -6 and call(freq=n) == -6 and call(pos=n) == -6
    assert call(k=a.odd) == -2 and call(ldk=130) == -2 and call(out=a.odd) == -2
    assert call(cache=ctypes.c_void_p(0)) == -6


@needs_lib
def test_attn_refusals(a):
    lib, c, p, n = _lib.load(), a.cache(), a.p, a.null
    other = ctypes.c_void_p(p.value + 2048)
    call = lambda q=p, ldq=256, out=other, qh=4, new=1, scale=0.1, acc=0, work=p, cache=c: lib.mmq_attn_decode(  # noqa: E731
        cache, q, ldq, n, out, qh, new, scale, acc, work, n)
    assert call(qh=3) == -1 and call(qh=0) == -1 and call(new=0) == -1 and call(new=17) == -1 and call(ldq=255) == -1
    assert call(scale=float("nan")) == -1 and call(scale=float("inf")) == -1
    assert call(q=n) == -6 and call(out=n) == -6 and call(work=n) == -6
    assert call(acc=1, cache=a.cache(weight=None)) == -6 and call(out=p) == -1           # q is read while out is written
    assert call(q=a.odd) == -2 and call(ldq=258) == -2 and call(work=a.odd) == -2
    assert call(cache=a.cache(seqs=0)) == 0
    nf = ctypes.c_int64()
    assert lib.mmq_attn_sizes(c, 4, 1, 0, None) == -6
    assert lib.mmq_attn_sizes(c, 5, 1, 0, ctypes.byref(nf)) == -1
    assert lib.mmq_attn_sizes(c, 258, 1, 0, ctypes.byref(nf)) == -1       # 129 query heads for each
    assert lib.mmq_attn_sizes(c, 4, 1, 0, ctypes.byref(nf)) == 0
    plain = nf.value
    assert plain > 0
    assert lib.mmq_attn_sizes(c, 4, 1, 1, ctypes.byref(nf)) == 0
    assert nf.value >= plain + 2 * 2 * 128                     # a score for every row and slot besides


@needs_lib
def test_evict_refusals(a):
    lib, p, n = _lib.load(), a.p, a.null
    other = a.odd
    call = lambda budget=4, keep=p, wo=other, po=other, work=p, cache=a.cache(): lib.mmq_kv_evict(cache, budget, keep, wo, po, work, n)  # noqa: E731
    assert call(budget=0) == -1 and call(cache=a.cache(cols=16385)) == -1
    assert call(wo=p) == -1 and call(po=p) == -1              # in place
    assert call(keep=n) == -6 and call(work=n) == -6 and call(cache=a.cache(weight=None)) == -6 and call(cache=a.cache(pos=None)) == -6
    assert call(cache=a.cache(seqs=0)) == 0
    ni = ctypes.c_int64()
    assert lib.mmq_evict_sizes(a.cache(), 0, ctypes.byref(ni)) == -1
    assert lib.mmq_evict_sizes(a.cache(), 100, ctypes.byref(ni)) == 0 and ni.value >= 2 * 2 * 28


@needs_lib
def test_verify_refusals(a):
    lib, p, n = _lib.load(), a.p, a.null
    call = lambda target=p, draft=p, dtype=2, tokens=p, uni=p, out=p, acc=p, seqs=1, drafts=2, vocab=10: lib.mmq_spec_verify(  # noqa: E731
        target, draft, dtype, tokens, uni, n, out, acc, seqs, drafts, vocab, n)
    for kw in (dict(seqs=-1), dict(seqs=65536), dict(drafts=0), dict(drafts=65), dict(vocab=0), dict(vocab=(1 << 20) + 1), dict(dtype=3)):
        assert call(**kw) == -1
    for kw in (dict(target=n), dict(tokens=n), dict(uni=n), dict(out=n), dict(acc=n)):
        assert call(**kw) == -6
    assert call(target=a.odd) == -2 and call(seqs=0) == 0


@needs_lib
def test_index_status_has_a_name():
    assert b"out of range" in _lib.load().mmq_status_str(-11)


def test_rope_frequencies():
    torch = pytest.importorskip("torch")  # noqa: F841
    from quantized_prefill_gemm_mmq_gb300 import ops
    inv, mag = ops.rope_frequencies(128)
    assert mag == 1.0 and inv[0] == 1.0 and len(inv) == 64 and math.isclose(inv[-1], 10000 ** (-126 / 128))
    lin, _ = ops.rope_frequencies(128, scaling="linear", factor=4.0)
    assert all(math.isclose(a, b / 4) for a, b in zip(lin, inv))
    base, _ = ops.rope_frequencies(128, scaling="base", factor=4.0)
    assert base[0] == 1.0 and math.isclose(base[-1], inv[-1] / 4)
    parts, mag = ops.rope_frequencies(128, scaling="by_parts", factor=8.0, context=4096)
    assert math.isclose(mag, 1 + 0.1 * math.log(8.0)) and parts[0] == inv[0] and math.isclose(parts[-1], inv[-1] / 8)
    assert all(b / 8 <= a <= b for a, b in zip(parts, inv))
    for f, x in zip(inv, ops.rope_fixed(inv)):                # 64-bit fractions of a turn: exact to f64's 53 bits
        turns = 123457 * f / (2 * math.pi)
        got = ((123457 * x) % (1 << 64)) / 2.0 ** 64
        assert abs((got - turns + 0.5) % 1.0 - 0.5) < 1e-10
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, factor=0.5, scaling="linear"), dict(rot=8, scaling="other"), dict(rot=8, fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            ops.rope_frequencies(**bad)


@needs_lib
def test_evict_sizes_refuses_what_evict_does(a):
    lib, p, n = _lib.load(), a.p, a.null
    ni = ctypes.c_int64()
    for kw, ok in ((dict(seqs=2048, heads=32), True), (dict(seqs=65535, heads=4096), True), (dict(seqs=65535, heads=4097), False),
                   (dict(seqs=65535, heads=65535), False), (dict(cols=16385), False)):
        assert lib.mmq_evict_sizes(a.cache(**kw), 100, ctypes.byref(ni)) == (0 if ok else -1)
        # nothing is launched: with `work` missing, a cache that fits is refused for that alone
        assert lib.mmq_kv_evict(a.cache(**kw), 100, p, a.odd, a.odd, n, n) == (-6 if ok else -1)


@needs_lib
def test_attn_sizes_refuses_what_attention_does(a):
    lib, p, n = _lib.load(), a.p, a.null
    other, nf = ctypes.c_void_p(p.value + 2048), ctypes.c_int64()
    for kw, new, acc, ok in ((dict(seqs=65535, heads=16384, cols=8), 1, 1, True),
                             (dict(seqs=65535, heads=16384, cols=8), 2, 0, True),
                             (dict(seqs=65535, heads=16384, cols=8), 2, 1, False),      # three blocks: two rows, one of entries
                             (dict(seqs=65535, heads=16384, cols=8), 3, 0, False),
                             (dict(seqs=65535, heads=16384, cols=24), 1, 0, False)):    # three tiles
        heads = kw["heads"]
        c = a.cache(**kw)
        assert lib.mmq_attn_sizes(c, heads, new, acc, ctypes.byref(nf)) == (0 if ok else -1)
        if not ok:                                            # never launched
            assert lib.mmq_attn_decode(c, p, heads * 64, n, other, heads, new, 0.1, acc, p, n) < 0
