"""Attention over the paged 8-bit cache with the block's own keys at softmax scales and query sizes
near the ends of fp32: keys of the cache and of the block are weighed on one scale."""
import numpy as np
import pytest

import kv4_ref
import kv8_ref as ref
from test_gpu_kv8 import bf, check, run_attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,G", [(64, 4), (128, 2)])
@pytest.mark.parametrize("B", [1, 4, 8, 40])
def test_far_scales_with_block_keys(B, d, G):
    """Scores of 2^80 to 2^116: a row is the mean of the keys that fp32 does not tell apart from the
    largest score, be they in the cache or in the block."""
    rng = np.random.default_rng(B + d)
    L, own, rows = 200, 0, 0
    for e_scale, e_q, e_k in ((80, 0, 0), (94, 0, 0), (104, 0, 0), (114, 0, 0), (40, 60, 0), (126, -30, 0),
                              (126, 0, -28), (126, 5, -24), (100, 20, -20), (60, 30, 14)):
        scale = 2.0 ** e_scale
        k, v = rng.standard_normal((2, L, 1, d))
        c = ref.Cache(rng, 1, 1, d, 16, 16, [L])
        c.write(0, 0, bf(k * 2.0 ** e_k), bf(v))
        q = kv4_ref.bf16(rng.standard_normal((1, B, G, d)) * 2.0 ** e_q)
        bk = kv4_ref.bf16(2.0 * rng.standard_normal((1, B, 1, d)) * 2.0 ** e_k)
        bv = kv4_ref.bf16(rng.standard_normal((1, B, 1, d)))
        got = run_attn(c, q, [L], B, L, bk, bv, scale=scale)
        assert np.isfinite(got).all(), (e_scale, e_q, e_k)
        x = np.concatenate((c.rows(0, 0, np.arange(L))[0], kv4_ref.f64(bk[0, :, 0])))
        held = np.concatenate((c.rows(1, 0, np.arange(L))[0], kv4_ref.f64(bv[0, :, 0])))
        qf = kv4_ref.f64(q)[0]
        s = np.einsum("bhd,jd->bhj", qf, x)
        # Of a score: fp32 sums of d products and a few roundings, (d + 16) 2^-24 of sum |q k|, and
        # queries as two e4m3 numbers, 2^-17 of the row's largest times sum |k|; of two scores twice
        # that.  Beside that a key weighs nothing: scores are 2^80 and more.
        err = (d + 16) * 2.0 ** -23 * np.einsum("bhd,jd->bhj", np.abs(qf), np.abs(x)).max(-1) \
            + 2.0 ** -16 * np.abs(qf).max(-1) * np.abs(x).sum(-1).max()
        near = s >= (s.max(-1) - err)[..., None]
        rows += B * G
        for b in range(B):
            for h in range(G):
                y = held[near[b, h]]
                own += bool(near[b, h, L:].any() and not near[b, h, :L].any())
                lo, hi = y.min(0), y.max(0)
                off = np.maximum(np.maximum(lo - got[0, b, h], got[0, b, h] - hi), 0)
                # half a bf16 step of the output, and the weights' rounding (fp16: 2^-11)
                assert (off <= (2.0 ** -8 + 2.0 ** -10) * np.abs(y).max(0)).all(), (e_scale, e_q, e_k, b, h)
    assert 0 < own < rows  # keys of the block and of the cache, both win rows


@pytest.mark.parametrize("B", [1, 4, 8, 40])
def test_small_queries_with_a_large_scale(B):
    """Ordinary scores out of tiny queries and a huge scale, and of huge queries and a tiny one."""
    rng = np.random.default_rng(B)
    d, G, L = 64, 4, 300
    c = ref.Cache(rng, 1, 1, d, 32, 16, [L])
    k, v = rng.standard_normal((2, L, 1, d))
    c.write(0, 0, bf(k), bf(v))
    bk, bv = (kv4_ref.bf16(rng.standard_normal((1, B, 1, d))) for _ in range(2))
    for e in (-100, -60, 60, 100):
        q = kv4_ref.bf16(rng.standard_normal((1, B, G, d)) * 2.0 ** e)
        scale = 2.0 ** (-3 - e)
        want, tol = ref.attention(q, c, [L], bk, bv, scale=scale)
        check(run_attn(c, q, [L], B, L, bk, bv, scale=scale), want, tol, f"queries of 2^{e}")
