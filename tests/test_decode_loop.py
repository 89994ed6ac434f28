"""The decode example end to end on the GPU: rows, cache, attention, eviction
and verification together."""
from __future__ import annotations

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("decode_loop", os.path.join(ROOT, "examples", "decode_loop.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


SMALL = dict(layers=2, hidden=512, heads=8, kv_heads=2, dim=64, ffn=512, vocab=1000, room=400)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_chunks_and_single_tokens_agree(ex, dtype):
    """A prompt in chunks of 16 and token by token: the same logits at its end.  The products' f32 sums differ in
    order by T, which can move a q8_1 code by one step of 1/127 of its block's largest value, in each of some
    fourteen products: a few parts in a thousand of the logits."""
    tokens = torch.randint(0, 1000, (45,), generator=torch.Generator().manual_seed(2)).tolist()
    a, b = ex.Decoder(cache_dtype=dtype, **SMALL), ex.Decoder(cache_dtype=dtype, **SMALL)
    for i in range(0, 45, 16):
        la = a.forward(tokens[i:i + 16])
    for t in tokens:
        lb = b.forward([t])
    ex.ops.check_status()
    scale = float(lb.abs().max())
    assert float((la[-1] - lb[-1]).abs().max()) <= 2e-2 * scale
    for ca, cb in zip(a.caches, b.caches):
        assert torch.equal(ca.pos, cb.pos)
        # every one of the 45 rows of each head hands out one unit of weight per query head
        total = ca.weight.sum((0, 2))
        assert torch.allclose(total, torch.full_like(total, 45 * 4.0), rtol=1e-4)


def test_dropped_drafts_leave_no_trace_in_the_logits(ex):
    tokens = list(range(20))
    a, b = ex.Decoder(**SMALL), ex.Decoder(**SMALL)
    for m in (a, b):
        m.forward(tokens[:16])
    a.forward([16, 900, 901])                                  # two drafts, both rejected
    a.drop(2)
    b.forward([16])
    la, lb = a.forward([17]), b.forward([17])
    assert float((la - lb).abs().max()) <= 2e-2 * float(lb.abs().max())


def test_generate_with_eviction(ex):
    prompt = torch.randint(0, 50, (90,), generator=torch.Generator().manual_seed(4)).tolist()
    m = ex.Decoder(**SMALL)
    out, (drafted, accepted, evictions) = ex.generate(m, prompt, steps=30, budget=48)
    again, _ = ex.generate(ex.Decoder(**SMALL), prompt, steps=30, budget=48)
    assert out == again                                        # nothing depends on timing
    assert len(out) == 30 + accepted and drafted > 0 and evictions >= 2
    assert m.entries == int(m.lens[0]) <= 48 + 32
    assert m.next_pos == len(prompt) - 1 + len(out)
    for c in m.caches:                                         # the newest quarter of the budget is always there
        ps = c.page_size
        pos = torch.stack([c.pos[c.table[0, s // ps].long(), :, s % ps] for s in range(m.entries)])
        for h in range(pos.shape[1]):
            have = set(pos[:, h].tolist())
            assert len(have) == m.entries and all(x in have for x in range(m.next_pos - 12, m.next_pos))


def live_weights(m, cache):
    """[heads][entries]"""
    return cache.weight[cache.table[0].long()].transpose(0, 1).flatten(1)[:, :m.entries]


def test_dropped_drafts_leave_no_trace_in_the_weights(ex):
    """What eviction goes by: every row that stayed hands out one unit per query head, a rejected draft's row nothing."""
    tokens = list(range(20))
    a, b = ex.Decoder(**SMALL), ex.Decoder(**SMALL)
    for m in (a, b):
        m.forward(tokens[:16])
    a.forward([16, 17, 900, 901], drafts=3)                    # three drafts, the first accepted
    a.drop(2)
    b.forward([16])
    b.forward([17])
    for m in (a, b):
        m.forward([18])
    for ca, cb in zip(a.caches, b.caches):
        wa, wb = live_weights(a, ca), live_weights(b, cb)
        assert wa.shape == wb.shape == (2, 19)
        assert torch.allclose(wa.sum(1), torch.full_like(wa.sum(1), 19 * 4.0), rtol=1e-4)
        assert float((wa - wb).abs().max()) <= 2e-2 * float(wb.max())


def test_generate_counts_no_rejected_rows(ex):
    prompt = torch.randint(0, 50, (90,), generator=torch.Generator().manual_seed(4)).tolist()
    m = ex.Decoder(**{**SMALL, "vocab": 60})
    _, (drafted, accepted, evictions) = ex.generate(m, prompt, steps=30, budget=1000, temperature=2.0)
    assert drafted > accepted > 0 and evictions == 0           # warm enough that drafts are turned down
    for c in m.caches:
        total = live_weights(m, c).sum(1)
        assert torch.allclose(total, torch.full_like(total, m.entries * 4.0), rtol=1e-4)
