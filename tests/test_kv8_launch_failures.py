"""A launch that fails inside a call on the paged 8-bit cache, whichever of the call's launches it
is: HERALD_ERR_CUDA with the call's launch named, nothing left armed, and the next call does the
whole work.  (The failing launch does not happen; nothing faults.)"""
import numpy as np
import pytest

import test_kv8_cpu as cpu
from block_diffusion_sparse_gb300 import herald as H

torch = pytest.importorskip("torch")
LAUNCH_FAILURE = 719  # cudaErrorLaunchFailure, and no error a missing GPU gives


@pytest.mark.parametrize("call,name", [
    (cpu.append, "kv8 append launch"),
    (lambda: H.herald_kv8_gather(cpu.dims(), 0x6000, 0x7000, 8, cpu.Raw().s, 0x8000, None), "kv8 gather launch")],
    ids=["append", "gather"])
def test_the_first_launch(call, name):
    """These two reach their first launch without a GPU too."""
    H.herald_inject_launch_failure(0, LAUNCH_FAILURE)
    try:
        with pytest.raises(H.HeraldError) as e:
            call()
    finally:
        H.herald_inject_launch_failure(-1)
    assert e.value.status == 4
    assert name in str(e.value) and "cudaErrorLaunchFailure" in str(e.value)


def failing(after, call, name):
    H.herald_inject_launch_failure(after, LAUNCH_FAILURE)
    try:
        with pytest.raises(H.HeraldError) as e:
            call()
    finally:
        H.herald_inject_launch_failure(-1)
    assert e.value.status == 4
    assert name in str(e.value) and "cudaErrorLaunchFailure" in str(e.value)
    torch.cuda.synchronize()  # the context is usable


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 8, 20])
@pytest.mark.parametrize("after", [0, 1])  # the attention kernel, the join
def test_attention(after, B):
    import kv4_ref
    from test_gpu_kv8 import OnGpu, bits, check, dev, make_cache, ref
    rng = np.random.default_rng(B)
    L, d = 700, 64
    c = make_cache(rng, 1, 2, d, 32, 16, [L])
    g = OnGpu(c)
    q, (bk, bv) = kv4_ref.bf16(rng.standard_normal((1, B, 8, d))), kv4_ref.bf16(rng.standard_normal((2, 1, B, 2, d)))
    dm = H.dims(1, 8, 2, d, B, L)
    ws = torch.zeros(H.herald_workspace_size_kv8(dm), dtype=torch.uint8, device="cuda")
    out = torch.zeros((1, B, 8, d), dtype=torch.int16, device="cuda")
    ctx = torch.tensor([L], dtype=torch.int32, device="cuda")
    args = dm, dev(q), g.kv8, ctx, dev(bk), dev(bv), out
    failing(after, lambda: H.herald_kv8_attn(*args, ws=ws), "kv8 attention launch")
    assert (out == 0).all()  # the join writes it
    H.herald_kv8_attn(*args, ws=ws)
    torch.cuda.synchronize()
    assert H.herald_workspace_error(ws) == 0
    want, tol = ref.attention(q, c, [L], bk, bv)
    check(kv4_ref.f64(bits(out)), want, tol, "after a failed launch")


@pytest.mark.gpu
@pytest.mark.parametrize("after", [0, 1, 2])  # the append, its block means, its advance
def test_append(after):
    import kv4_ref
    from test_gpu_kv8 import OnGpu, dev, ref
    rng = np.random.default_rng(after)
    N, Hkv, d, T, Bk = 2, 2, 128, 9, 16
    c = ref.Cache(rng, N, Hkv, d, 16, 16, [T + 3] * N)
    g = OnGpu(c)
    k, v = kv4_ref.bf16(rng.standard_normal((2, N, T, Hkv, d)))
    ctx = torch.zeros(N, dtype=torch.int32, device="cuda")
    pooled = torch.full((N, Hkv, 1, d), 9.0, device="cuda")
    dk, dv = dev(k), dev(v)

    def call():
        H.herald_kv8_append(H.dims(N, 4, Hkv, d, 1, T + 3), T, None, dk, dv, ctx, g.kv8, None, None,
                            pooled=pooled, Bk=Bk, flags=H.HERALD_KV8_ADVANCE)

    failing(after, call, "kv8 append launch")
    assert ctx.tolist() == [0] * N  # the lengths advance last
    if after < 2:
        assert (pooled == 9).all()
    if after == 0:
        assert np.array_equal(g.codes.cpu().numpy(), c.codes)
    call()  # the same call again: the same rows, once
    torch.cuda.synchronize()
    for n in range(N):
        c.write(n, 0, kv4_ref.f64(k[n]), kv4_ref.f64(v[n]))
    assert np.array_equal(g.codes.cpu().numpy(), c.codes) and np.array_equal(g.scales.cpu().numpy(), c.scales)
    assert ctx.tolist() == [T] * N
    want = np.stack([c.rows(0, n, np.arange(T)).mean(1) for n in range(N)])[:, :, None]
    # fp32 sums of 9 values below 16, one division
    assert np.abs(pooled.cpu().numpy() - want).max() <= (T + 2) * 2.0 ** -24 * 16
