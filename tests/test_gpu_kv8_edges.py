"""The paged 8-bit cache's attention over its kernels' variants (query rows per KV head up to
8, 16, 32, 128, 256; both head sizes), pages and blocks: keys with holes, bytes behind the
lengths, pieces of every kind, and random cases."""
import random

import numpy as np
import pytest

import kv4_ref
import kv8_ref as ref
from helpers import dev
from test_gpu_kv8 import OnGpu, _h, bits, check, make_cache, run_attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# query tokens of 4 heads a group: 4, 16, 32, 128 and 256 rows per KV head
TOKENS = [1, 4, 8, 32, 64]


@pytest.mark.parametrize("B", TOKENS)
@pytest.mark.parametrize("page,block", [(16, 16), (64, 32), (128, 128)])
@pytest.mark.parametrize("d", [64, 128])
def test_missing_pages(B, page, block, d):
    """Table entries without a page are masked: single pages, whole 128-key tiles, a sequence's
    first and last, and sequences that have none at all."""
    rng = np.random.default_rng(page + B)
    N, Hq, Hkv = 4, 8, 2
    lengths = [1000, 900, 640, 257]
    c = make_cache(rng, N, Hkv, d, page, block, lengths)
    per = 128 // page
    c.table[0, per:2 * per] = -1             # the second tile of 128 keys
    c.table[0, 4 * per] = c.n_pages          # past the arrays
    c.table[0, 5 * per + per // 2] = 2 ** 31 - 1
    c.table[1, 0] = -1
    c.table[1, -(-900 // page) - 1] = -7     # the page that holds the last keys
    c.table[2, :] = -5
    c.table[3, ::2] = -1
    q = kv4_ref.bf16(rng.standard_normal((N, B, Hq, d)))
    r = ref.Cache.__new__(ref.Cache)         # (the reference wants -1 for a missing page)
    r.__dict__.update(c.__dict__, table=np.where((c.table < 0) | (c.table >= c.n_pages), -1, c.table))
    want, tol = ref.attention(q, r, lengths)
    got = run_attn(c, q, lengths, B, 1000)
    check(got, want, tol, f"B {B} page {page}")
    assert (got[2] == 0).all()


@pytest.mark.parametrize("B", TOKENS)
def test_bytes_behind_the_lengths(B):
    """NaN codes and any scales behind a length, inside its block and page, change nothing."""
    rng = np.random.default_rng(50)
    N, Hq, Hkv, d, page = 3, 8, 2, 128, 64
    lengths = [65, 127, 300]
    c = make_cache(rng, N, Hkv, d, page, 16, lengths)
    for n, L in enumerate(lengths):
        ph, r = c.table[n, L // page], L % page
        c.codes[:, ph, :, r:] = 0x7F
        c.scales[:, ph, :, -(-r // 16):] = 255
    q = kv4_ref.bf16(rng.standard_normal((N, B, Hq, d)))
    want, tol = ref.attention(q, c, lengths)
    check(run_attn(c, q, lengths, B, 300), want, tol, "behind")


@pytest.mark.parametrize("seed", range(24))
def test_random_cases(seed):
    r = random.Random(seed)
    rng = np.random.default_rng(seed)
    d, Hkv, G = r.choice((64, 128)), r.choice((1, 2, 3, 8)), r.choice((1, 2, 3, 5, 7, 8))
    page = r.choice((16, 32, 64, 128))
    block = r.choice([b for b in (16, 32, 64, 128) if b <= page])
    B = r.choice((1, 1, 2, 3, 4, r.randint(1, 256 // G)))
    top = r.choice((1, 130, 1000, 5000))
    N = r.randint(1, max(1, min(24, 60000 // (top * Hkv))))
    lengths = [r.choice((0, 1, top, r.randint(0, top))) for _ in range(N)]
    c = make_cache(rng, N, Hkv, d, page, block, lengths)
    q = kv4_ref.bf16(rng.standard_normal((N, B, Hkv * G, d)))
    bk = bv = None
    if r.random() < 0.5:
        bk, bv = (kv4_ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    want, tol = ref.attention(q, c, lengths, bk, bv)
    what = f"N {N} Hkv {Hkv} G {G} d {d} B {B} page {page} block {block} top {top} own {bk is not None}"
    check(run_attn(c, q, lengths, B, max(1, max(lengths)), bk, bv), want, tol, what)


@pytest.mark.parametrize("B", TOKENS)
def test_one_sequence_of_every_length(B):
    """Lengths around tiles, pages and blocks."""
    rng = np.random.default_rng(51)
    for L in (1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 511, 513, 640):
        c = make_cache(rng, 1, 1, 128, 16, 16, [L])
        q = kv4_ref.bf16(rng.standard_normal((1, B, 4, 128)))
        want, tol = ref.attention(q, c, [L])
        check(run_attn(c, q, [L], B, L), want, tol, f"length {L}")


@pytest.mark.parametrize("d,P,values,shift", [(128, 5003, False, 0), (64, 9001, False, 8), (128, 77, True, 8),
                                              (64, 33, True, 16)])
def test_gather_layouts(d, P, values, shift):
    """Launches of more than one wave (two rows a thread), and pools aligned to 16 bytes but not
    to 32; the whole cache and more: the last rows repeat."""
    H = _h()
    rng = np.random.default_rng(P)
    N, Hkv, page, block = 2, 4, 64, 16
    lengths = [P - 2, P // 2 + 1]
    c = make_cache(rng, N, Hkv, d, page, block, lengths)
    g = OnGpu(c)
    idx = np.zeros((N, Hkv, P), np.int32)
    n_sel = np.full((N, Hkv), P, np.int32)
    for n, L in enumerate(lengths):
        idx[n] = np.minimum(np.arange(P), L - 1)
    n_sel[1, 1] = P // 3
    pools = []
    for _ in range(2):
        flat = torch.full((N * Hkv * P * d + shift,), 7, dtype=torch.int16, device="cuda")
        pools.append(flat[shift:].view(N, Hkv, P, d))
    H.herald_kv8_gather(H.dims(N, Hkv, Hkv, d, 1, P), dev(idx), dev(n_sel), P, g.kv8, pools[0],
                        pools[1] if values else None)
    for i in range(2 if values else 1):
        want = np.stack([c.rows(i, n, idx[n, 0]) for n in range(N)])
        want[1, 1, P // 3:] = 0
        assert np.array_equal(kv4_ref.f64(bits(pools[i])), want)
    if not values:
        assert (pools[1] == 7).all()


@pytest.mark.parametrize("d,B", [(128, 1), (64, 4), (128, 9), (64, 40)])
@pytest.mark.parametrize("shift", [0, 16])
def test_workspace_of_16_bytes_alignment(d, B, shift):
    """A workspace of exactly the size asked for, aligned to 16 bytes only: the same results, and
    nothing beside it is written."""
    H = _h()
    rng = np.random.default_rng(d + B)
    N, Hq, Hkv, page = 3, 8, 2, 64
    lengths = [3000, 0, 700]
    c = make_cache(rng, N, Hkv, d, page, 32, lengths)
    q = kv4_ref.bf16(rng.standard_normal((N, B, Hq, d)))
    bk, bv = (kv4_ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    size = H.herald_workspace_size_kv8(H.dims(N, Hq, Hkv, d, B, 3000))
    room = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = room[16 + shift:16 + shift + size]
    ws[:4] = 0  # (the error word)
    got = run_attn(c, q, lengths, B, 3000, bk, bv, ws=ws)
    want, tol = ref.attention(q, c, lengths, bk, bv)
    check(got, want, tol, "16-byte workspace")
    assert (room[:16 + shift] == 0x5A).all() and (room[16 + shift + size:] == 0x5A).all()
    assert np.array_equal(got, run_attn(c, q, lengths, B, 3000, bk, bv))
