"""The bounded waits of prompt and tree attention, exercised without a fault: the test-only knob lowers the wait limit to 1 ms
and withholds the last K tile of every run of tiles, so the waits for it run out.  The kernel must record MMQ_ERR_TIMEOUT,
wait for the copies that it has under way, free its tensor memory and return, and the next launches must give what the ones
before gave, bit for bit.  Nothing faults, traps or hangs: every wait gives up by itself."""
from __future__ import annotations

import ctypes
import time

import pytest

torch = pytest.importorskip("torch")

from tests.test_prompt_ops import queries  # noqa: E402
from tests.test_serve_ops import make_cache, ops  # noqa: E402, F401

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("lens,N,H,group,dim,page,dtype", [
    ([900, 700], 600, 48, 1, 64, 16, BF16),              # whole units, taken over from CTAs that have not started; two halves
    ([700], 1, 4, 1, 128, 16, F16),                      # whole units of few rows
    ([9000, 300], 40, 2, 4, 128, 64, F16),               # cut units, joined; two halves
    ([9000], 1, 8, 4, 128, 64, BF16),                    # cut units of few rows
    ([3000], 20, 2, 2, 256, 32, F16),                    # the largest heads
    ([2000], 150, 2, 2, 192, 16, BF16),
    ([5000], 30, 2, 2, 128, 7, BF16),                    # pages that are copied row by row
])
def test_waits_run_out_and_the_next_call_is_clean(ops, lens, N, H, group, dim, page, dtype):
    from quantized_prefill_gemm_mmq_gb300 import _lib
    lib = _lib.load()
    cache = make_cache(ops, lens, H, dim, page, dtype)
    q = queries(cache, lens, N, group).cuda()
    work = ops.prefill_workspace(cache, H * group, N)
    clean = ops.attn_prefill(cache, q, workspace=work)
    ops.check_status()
    try:
        assert lib.mmq_debug_fault_inject(1, 1000) == 0
        t0 = time.perf_counter()
        ops.attn_prefill(cache, q, workspace=work)
        with pytest.raises(_lib.MMQError) as e:
            ops.check_status()
        assert time.perf_counter() - t0 < 10.0           # it gave up on its own
        assert e.value.status == -5                      # MMQ_ERR_TIMEOUT
        info = (ctypes.c_int * 4)()
        assert lib.mmq_last_failure_info(info) == 0 and info[0] >= 1000      # waited the 1 ms (us)
        ops.attn_prefill(cache, q, workspace=work)
        detail = (ctypes.c_int * 4)()
        assert lib.mmq_check_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), detail) == -5
        assert detail[1] == 36 and 1 <= detail[2] <= 13  # this kernel, one of its waits
    finally:
        assert lib.mmq_debug_fault_inject(0, 0) == 0
    ops.check_status()                                   # nothing is left in the status words
    for _ in range(3):
        assert torch.equal(ops.attn_prefill(cache, q, workspace=work), clean)
    ops.check_status()


def test_trees_and_captured_calls_after_a_wait_ran_out(ops):
    from quantized_prefill_gemm_mmq_gb300 import _lib
    lib = _lib.load()
    lens, N = [5000, 400], 33
    cache = make_cache(ops, lens, 2, 64, 16, BF16)
    q = queries(cache, lens, N, 4).cuda()
    tree = ops.tree_words([list(range(-1, N - 1))] * 2)
    work = ops.prefill_workspace(cache, 8, N)
    clean = ops.attn_tree(cache, q, tree, workspace=work)
    out = torch.empty_like(clean)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ops.attn_tree(cache, q, tree, out=out, workspace=work)
    try:
        assert lib.mmq_debug_fault_inject(1, 1000) == 0
        ops.attn_tree(cache, q, tree, workspace=work)
        with pytest.raises(_lib.MMQError) as e:
            ops.check_status()
        assert e.value.status == -5
    finally:
        assert lib.mmq_debug_fault_inject(0, 0) == 0
    for _ in range(3):
        out.fill_(7)
        g.replay()
        ops.check_status()
        assert torch.equal(out, clean)
