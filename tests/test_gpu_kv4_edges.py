"""The paged 4-bit cache's attention where its keys have holes or NaN: missing
pages beside block keys and NaN scales, in every kernel variant (query rows per
KV head up to 8, 16, 128, 256)."""
import numpy as np
import pytest

import kv4_ref as ref
from test_gpu_kv4 import check, make_cache, run_attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# query tokens of 4 heads a group: 4, 16, 128 and 256 rows per KV head
BLOCKS = [1, 4, 32, 64]


@pytest.mark.parametrize("B", BLOCKS)
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("block", [False, True])
def test_missing_pages(B, page, block):
    """Table entries without a page are masked: single pages, whole 128-key tiles,
    a sequence's first and last, and sequences that have none at all."""
    rng = np.random.default_rng(page + B)
    N, Hq, Hkv, d = 4, 8, 2, 128
    lengths = [1000, 900, 640, 257]
    c = make_cache(rng, N, Hkv, d, page, lengths)
    per = 128 // page
    c.table[0, per:2 * per] = -1             # the second tile of 128 keys
    c.table[0, 4 * per] = c.n_pages          # past the arrays
    c.table[0, 5 * per + per // 2] = 2 ** 31 - 1
    c.table[1, 0] = -1
    c.table[1, -(-900 // page) - 1] = -7     # the page that holds the last keys
    c.table[2, :] = -5
    c.table[3, ::2] = -1
    q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
    bk = bv = None
    if block:
        bk, bv = (ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    r = ref.Cache.__new__(ref.Cache)         # (the reference wants -1 for a missing page)
    r.__dict__.update(c.__dict__, table=np.where((c.table < 0) | (c.table >= c.n_pages), -1, c.table))
    want, tol = ref.attention(q, r, lengths, bk, bv)
    got = run_attn(c, q, lengths, B, 1000, bk, bv)
    check(got, want, tol, f"B {B} page {page}")
    if not block:
        assert (got[2] == 0).all()


@pytest.mark.parametrize("B", BLOCKS)
@pytest.mark.parametrize("kv", [0, 1])
def test_nan_scales_reach_their_head_only(B, kv):
    """A NaN scale of a held key makes its head's rows NaN, of a held value that
    group's 16 channels of them; one behind the length, nothing."""
    rng = np.random.default_rng(20 + kv)
    N, Hq, Hkv, d, L = 2, 8, 2, 128, 300
    c = make_cache(rng, N, Hkv, d, 64, [L, L])
    pos, group = 131, 5
    c.scales[kv, c.table[0, pos // 64], 1, pos % 64, group] = 0x7F
    c.scales[kv, c.table[1, 4], :, L - 256:] = 0x7F  # rows past the length
    q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
    got = run_attn(c, q, [L, L], B, L)
    bad = np.zeros(got.shape, bool)
    bad[0, :, 4:, 16 * group:16 * group + 16] = True
    if kv == 0:
        bad[0, :, 4:] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
