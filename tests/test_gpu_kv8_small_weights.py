"""Attention over the paged 8-bit cache where one key has nearly all of the weight and no value
(an attention sink), and many small weights make the output."""
import numpy as np
import pytest

import kv4_ref
import kv8_ref as ref
from test_gpu_kv8 import bf, check, run_attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [1, 4, 8, 32])  # 4, 16, 32 and 128 query rows a KV head
def test_small_weights_beside_a_sink(B, d):
    """Keys 2^-24 to 2^-27 below a sink that shares their scales and their CTA: with few rows a
    weight is held down to 2^-24 and with many (fp16) to 2^-24 too, where the row's largest is 2^4
    at least, so each is off by at most half a step, 2^-29 of the largest weight."""
    rng = np.random.default_rng(B + d)
    Hkv, G, L = 4, 4, 2048
    N = -(-torch.cuda.get_device_properties(0).multi_processor_count // Hkv)  # a segment a CTA, or nearly
    c = ref.Cache(rng, 1, Hkv, d, 64, 64, [L])
    k, v = 0.1 * rng.standard_normal((2, L, Hkv, d))
    v += 1.0
    k[:, :, 0] = 0
    k[5, :, 0], v[5] = 9.0, 0
    c.write(0, 0, bf(k), bf(v))
    c.N, c.table = N, np.repeat(c.table, N, 0)
    q = 0.1 * rng.standard_normal((N, B, Hkv * G, d))
    for below in (24, 26, 27):
        q[..., 0] = below * np.log(2) * np.sqrt(d) / 9.0
        qb = kv4_ref.bf16(q)
        got = run_attn(c, qb, [L] * N, B, L)
        for n in (0, 1, N // 2, N - 1):
            want, tol = ref.attention(qb[n:n + 1], c, [L])
            # ref.attention's bound allows 2^-26 a key (times what a value's scale lies under the
            # head's largest) for weights below a step: 2^-29 instead
            e, held = c.exps(1, n, np.arange(L)), np.abs(c.rows(1, n, np.arange(L)))
            floor = (2.0 ** (e.max(1, keepdims=True) - e)[..., None] * held).sum(1)  # [Hkv, d]
            tol = tol[0] - (2.0 ** -26 - 2.0 ** -29) * np.repeat(floor, G, 0)
            check(got[n], want[0], tol, f"2^-{below}, sequence {n}")
