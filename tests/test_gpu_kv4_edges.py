"""The paged 4-bit cache's attention where its numbers are extreme or its keys
have holes: scores past what fp32 resolves, NaN values, missing pages beside
block keys, and every kernel variant (query rows per KV head up to 8, 16, 128,
256)."""
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


def rows_of_sign(rng, L, Hkv, d, top, high):
    """Keys c w per position (w of +-1 per head): c = 6 at the positions `top`
    (of 1/4 where not `high`), else one of 1 to 4.  Returns keys [L, Hkv, d] and w."""
    w = rng.choice([-1.0, 1.0], (Hkv, d)).astype(np.float32)
    c = rng.integers(1, 5, L).astype(np.float32)
    c[top] = 6 if high else 0.25
    return c[:, None, None] * w, w


@pytest.mark.parametrize("B", BLOCKS)
@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** 22, 2.0 ** 28, 2.0 ** 34])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_past_what_fp32_resolves(B, size, sign):
    """Scores up to 2^41, whose fp32 steps are 2^17: two equal keys far above all
    others, in different tiles, share the weight; rows of ordinary queries beside
    them and the sign of the scores change nothing.  The others' weights are zero
    (the next score is at least 0.3 of the largest below it); the two have bitwise
    equal scores, so that the result is the mean of their values: off by its own
    rounding (2^-8), P's in fp16 against the row sum (2^-11) and fp32 sums (2^-13)."""
    rng = np.random.default_rng(int(np.log2(size)) + B)
    N, Hq, Hkv, d, L = 2, 8, 2, 128, 1500
    top = [77, 1203]
    c = ref.Cache(rng, N, Hkv, d, 64, [L, L])
    v = rng.standard_normal((N, L, Hkv, d)).astype(np.float32)
    ws = []
    for n in range(N):
        k, w = rows_of_sign(rng, L, Hkv, d, top, sign > 0)
        c.write(n, np.arange(L), k, v[n])
        ws.append(w)
    q = rng.standard_normal((N, B, Hq, d)).astype(np.float32)
    huge = rng.random((N, B, Hq)) < 0.5
    huge[0, 0, 0], huge[1, -1, -1] = True, False
    far = np.repeat(np.stack(ws), Hq // Hkv, 1)[:, None] * np.float32(sign * size)
    q = np.where(huge[..., None], far, q)
    q = ref.bf16(q)
    want, tol = ref.attention(q, c, [L, L])
    for n in range(N):
        rows = c.rows(1, n, top)              # [Hkv, 2, d]
        mean = np.repeat(rows.mean(1), Hq // Hkv, 0)
        mag = np.repeat(np.abs(rows).mean(1), Hq // Hkv, 0)
        for h in range(Hq):
            at = huge[n, :, h]
            want[n, at, h] = mean[h]
            tol[n, at, h] = 2.0 ** -8 * np.abs(mean[h]) + (2.0 ** -11 + 2.0 ** -13) * mag[h]
    check(run_attn(c, q, [L, L], B, L), want, tol, f"size {size} sign {sign}")


@pytest.mark.parametrize("B", BLOCKS)
@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** 24, 2.0 ** 30])
def test_block_scores_past_what_fp32_resolves(B, size):
    """The same where a key of the block stands above all others."""
    rng = np.random.default_rng(int(np.log2(size)) + B)
    N, Hq, Hkv, d, L = 2, 8, 2, 128, 700
    c = ref.Cache(rng, N, Hkv, d, 64, [L, L], v_scale=0.25)
    q = np.zeros((N, B, Hq, d), np.float32)
    bk, bv = np.zeros((N, B, Hkv, d), np.float32), rng.standard_normal((N, B, Hkv, d))
    at = B // 2
    for n in range(N):
        k, w = rows_of_sign(rng, L, Hkv, d, [], True)
        c.write(n, np.arange(L), k, rng.standard_normal((L, Hkv, d)).astype(np.float32))
        q[n] = np.repeat(w, Hq // Hkv, 0) * np.float32(size)
        bk[n] = w * rng.integers(1, 5, B)[:, None, None]
        bk[n, at] = w * 8
    bv = ref.bf16(bv)
    got = run_attn(c, ref.bf16(q), [L, L], B, L, ref.bf16(bk), bv)
    want = np.broadcast_to(np.repeat(ref.f64(bv)[:, at], Hq // Hkv, 1)[:, None], got.shape)
    # its own rounding; P in bf16 (2^-8) against the row sum
    check(got, want, (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -13) * np.abs(want), f"size {size}")


@pytest.mark.parametrize("B", BLOCKS)
def test_scale_and_cache_factor_past_fp32_together(B):
    """The softmax scale times the cache's factor is past fp32's largest number, the
    scores are ordinary."""
    rng = np.random.default_rng(50 + B)
    N, Hq, Hkv, d, L = 1, 8, 2, 128, 500
    c = ref.Cache(rng, N, Hkv, d, 64, [L], k_scale=2.0 ** 60)
    k = rng.standard_normal((L, Hkv, d)) * 2.0 ** 53
    c.write(0, np.arange(L), k.astype(np.float32), rng.standard_normal((L, Hkv, d)).astype(np.float32))
    q = ref.bf16((rng.standard_normal((N, B, Hq, d)) * 2.0 ** -124).astype(np.float32))
    want, tol = ref.attention(q, c, [L], scale=2.0 ** 69)
    assert np.abs(want - c.rows(1, 0, np.arange(L)).mean(1).repeat(4, 0)).max() > 0.1  # not uniform
    check(run_attn(c, q, [L], B, L, scale=2.0 ** 69), want, tol, "scales")


@pytest.mark.parametrize("B", BLOCKS)
@pytest.mark.parametrize("lengths", [[0, 1], [128, 7]], ids=str)
def test_weights_of_the_blocks_keys_keep_16_bits(B, lengths):
    """Short contexts, where the block's own keys carry most of the weight: their
    weights are held as precisely as the cache's, not in bf16's 8 bits.  The bound
    is ref.attention's with 2^-16 A_b (a weight as the sum of two bf16 numbers) in
    the place of 2^-8 A_b, and 2^-23 A_b for the product with 1/v_scale."""
    rng = np.random.default_rng(60 + B + sum(lengths))
    N, Hq, Hkv, d = 2, 8, 2, 128
    c = make_cache(rng, N, Hkv, d, 64, lengths, v_scale=0.3)
    q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
    bk, bv = (ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    want, tol = ref.attention(q, c, lengths, bk, bv)
    for n in range(N):
        at = np.arange(lengths[n])
        for h in range(Hq):
            keys = np.concatenate((c.rows(0, n, at)[h // 4], ref.f64(bk)[n, :, h // 4]))
            s = ref.f64(q)[n, :, h] @ keys.T / np.sqrt(d)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            Ab = p[:, lengths[n]:] @ np.abs(ref.f64(bv)[n, :, h // 4])
            tol[n, :, h] -= (2.0 ** -8 - 2.0 ** -16 - 2.0 ** -23) * Ab
    check(run_attn(c, q, lengths, B, max(lengths), bk, bv), want, tol, f"B {B} {lengths}")
