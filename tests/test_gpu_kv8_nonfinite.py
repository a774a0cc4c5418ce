"""Attention over the paged 8-bit cache where the block's own keys or values hold infinities and
NaNs: what the formula gives, in every form of the join (up to four block keys, more, more than
64; groups of threads and whole rows)."""
import numpy as np
import pytest

import kv4_ref
import kv8_ref as ref
from test_gpu_kv8 import make_cache, run_attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF, NAN = 0x7F80, 0x7FC0

# (N, Hkv, G, d, B): rows a KV head, and few or many of them beside the CTAs there are
SHAPES = [(1, 1, 4, 64, 1), (2, 2, 4, 128, 4), (70, 8, 2, 128, 3), (1, 2, 4, 128, 5), (3, 2, 4, 64, 16),
          (4, 8, 2, 128, 17), (2, 4, 7, 128, 32), (2, 8, 2, 64, 33), (40, 4, 2, 64, 8), (1, 3, 1, 128, 130),
          (1, 1, 2, 64, 128)]


def inputs(shape, length, seed):
    N, Hkv, G, d, B = shape
    rng = np.random.default_rng(seed)
    lengths = [length] * N
    c = make_cache(rng, N, Hkv, d, 32, 16, lengths)
    q = kv4_ref.bf16(rng.standard_normal((N, B, Hkv * G, d)))
    bk, bv = (kv4_ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    return rng, lengths, c, q, bk, bv


def compare(got, want, tol, what):
    """want: numbers, infinities of a sign, NaN; tol for the finite ones."""
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN elsewhere"
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), f"{what}: infinities"
    assert (np.abs(got[fin] - want[fin]) <= tol[fin]).all(), f"{what}: finite ones"


@pytest.mark.parametrize("length", [0, 300])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_infinite_block_values(shape, length):
    """An infinity among a channel's block values is that channel's output, two of different signs
    or a NaN make a NaN; other channels do not see them."""
    N, Hkv, G, d, B = shape
    rng, lengths, c, q, bk, bv = inputs(shape, length, B)
    clean = bv.copy()
    # which channels of sequence 0's heads: one or more +inf, -inf, both, NaN, NaN and inf
    want_at = {}
    for g in range(Hkv):
        for ch, vals in ((1, [INF]), (2, [INF | 0x8000]), (9, [INF] * min(B, 3)), (d - 1, [NAN]),
                         (d // 2, [INF, NAN] if B > 1 else [NAN]),
                         (17, [INF, INF | 0x8000] if B > 1 else [INF])):
            for x, at in zip(vals, rng.permutation(B)):
                bv[0, at, g, ch] = x
                clean[0, at, g, ch] = 0
            f = kv4_ref.f64(np.array(vals, np.uint16))
            with np.errstate(invalid="ignore"):
                want_at[g, ch] = f.sum()  # (weights are positive)
    want, tol = ref.attention(q, c, lengths, bk, clean)
    for (g, ch), x in want_at.items():
        want[0, :, g * G:(g + 1) * G, ch] = x
    # (scores of these queries and keys lie within 2^7 of one another: no weight is 0)
    compare(run_attn(c, q, lengths, B, max(1, length), bk, bv), want, tol, str(shape))


@pytest.mark.parametrize("length", [0, 300])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_infinite_block_keys(shape, length):
    """An infinite key value scores +inf or -inf by the query's sign: a +inf makes the row NaN
    (inf - inf), a -inf leaves the key without weight; a NaN key makes its head's rows NaN."""
    N, Hkv, G, d, B = shape
    rng, lengths, c, q, bk, bv = inputs(shape, length, B + 1)
    at = int(rng.integers(0, B))
    bk[0, at, 0, 5] = INF
    if N > 1:
        bk[1, B - 1, Hkv - 1, 0] = NAN
    gone = bk.copy()
    gone[0, at, 0, 5] = 0
    if N > 1:
        gone[1, B - 1, Hkv - 1, 0] = 0
    # the same without that key, for the rows that give it -inf
    want, tol = ref.attention(q, c, lengths, gone, bv)
    keep = [b for b in range(B) if b != at]
    some = kv4_ref.f64(q[0, :, :G, 5]) > 0
    if keep or length:
        x = np.concatenate((c.rows(0, 0, np.arange(length))[0], kv4_ref.f64(bk[0, keep, 0])))
        v = np.concatenate((c.rows(1, 0, np.arange(length))[0], kv4_ref.f64(bv[0, keep, 0])))
        s = kv4_ref.f64(q[0, :, :G]) @ x.T / np.sqrt(d)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        want[0, :, :G] = p @ v
        # the bound of the same rows with a finite key there: its terms are means of |v| under the
        # weights, here those of the other keys
        tol[0, :, :G] = 2.0 ** -8 * np.abs(want[0, :, :G]) + 2.0 ** -10 * (p @ np.abs(v))
    else:
        want[0, :, :G], tol[0, :, :G] = 0, 0
    want[0, :, :G][some] = np.nan
    if N > 1:
        want[1, :, (Hkv - 1) * G:] = np.nan
    compare(run_attn(c, q, lengths, B, max(1, length), bk, bv), want, tol, str(shape))
