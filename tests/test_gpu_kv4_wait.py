"""The attention over a paged 4-bit cache bounds its waits by a count of tries:
one that runs out is reported with the kernel and the wait, and the context stays
usable.  The self-test waits, through the kernels' own wait, on a barrier nothing
completes."""
import time

import numpy as np
import pytest

from block_diffusion_sparse_gb300 import herald as H

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("tries", [1, 500, 25000])
def test_a_kv4_wait_that_runs_out_is_reported(tries):
    import kv4_ref as ref
    from test_gpu_kv4 import check, make_cache, run_attn
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    H.herald_selftest_kv4_wait(tries, ws)
    code = H.herald_workspace_error(ws)  # synchronises
    elapsed = time.perf_counter() - t0
    # a copy wait (1) of kernel 10, its wait for a full stage (2): the wait on the
    # completed barrier before it (1) left no trace
    assert code == 1 | 10 << 8 | 2 << 16
    assert elapsed < 0.05 + 10 * tries * 4e-6  # 250000 tries, the kernels' count: seconds at most
    assert H.herald_workspace_error(ws) == 0
    rng = np.random.default_rng(1)
    for B in (1, 32):
        c = make_cache(rng, 1, 2, 64, 16, [200])
        q = ref.bf16(rng.standard_normal((1, B, 8, 64)))
        want, tol = ref.attention(q, c, [200])
        check(run_attn(c, q, [200], B, 200), want, tol, "after a wait ran out")


@pytest.mark.parametrize("tries,ws", [(0, 1 << 12), (250001, 1 << 12), (-1, 1 << 12), (1, 0), (1, 8)])
def test_kv4_wait_self_test_refusals(tries, ws):
    """Host-side: launches nothing."""
    with pytest.raises(H.HeraldError) as e:
        H.herald_selftest_kv4_wait(tries, ws)
    assert e.value.status == 1
