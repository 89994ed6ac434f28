"""GPU tests of what the decode-side operators promise beside their values:
outputs that are the caller's alone, rows that are not finite staying so
wherever their parts are joined, scores of any size, limits, errors and rows
from odd places.

Tolerances are those of test_serve_ops.py, or equality."""
from __future__ import annotations

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
