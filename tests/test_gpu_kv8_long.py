"""Attention over the paged 8-bit cache in steady state: every CTA has a piece of 40 tiles of 128
keys and more, so that rings, scale groups and look-aheads of the page table wrap several times
inside a piece.  Many sequences share a few dozen pages; the fp64 reference is taken for some."""
import numpy as np
import pytest

import kv4_ref
import kv8_ref as ref
from test_gpu_kv8 import bf, check, run_attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def shared_cache(rng, N, Hkv, d, page, block, length, pool, hot):
    """N sequences of `length` positions over `pool` ordinary pages and, at hot[n] (a list of
    positions), one whose keys reach far along channel 0.  Value and key scales differ by block."""
    c = ref.Cache(rng, 1, Hkv, d, page, block, [(pool + 1) * page])
    rows = (pool + 1) * page
    k, v = rng.standard_normal((2, rows, Hkv, d))
    k[:, :, 0] = 0.5 * np.abs(k[:, :, 0])
    k *= 2.0 ** rng.integers(-1, 2, rows // 16).repeat(16)[:, None, None]
    k[pool * page:, :, 0] = 12.0
    v *= 2.0 ** rng.integers(-3, 4, rows // 16).repeat(16)[:, None, None]
    c.write(0, 0, bf(k), bf(v))
    mine = c.table[0]
    c.N, c.max_pages = N, -(-length // page)
    c.table = np.stack([np.concatenate([rng.permutation(mine[:pool]) for _ in range(-(-c.max_pages // pool))])
                        [: c.max_pages] for _ in range(N)]).astype(np.int32)
    for n, places in hot.items():
        for p in places:
            c.table[n, p // page] = mine[pool]
    return c


# (tokens, d, page, block, pool, block keys): 4, 16, 32 and 128 query rows a KV head
CASES = [(B, d, page, block, own) for B, own in ((1, True), (4, False), (8, True), (32, True))
         for d, page, block in ((128, 64, 16), (64, 16, 16), (128, 128, 128), (64, 128, 32))]


@pytest.mark.parametrize("B,d,page,block,own", CASES, ids=str)
def test_pieces_of_many_tiles(B, d, page, block, own):
    rng = np.random.default_rng(1000 * B + d + page)
    Hkv, G, length = 4, 4, 8192
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    N = -(-ctas * 90 // (Hkv * (length // 128)))  # 90 tiles a CTA of segments of 64
    lengths = [length] * N
    lengths[1], lengths[2], lengths[-1] = length - 1, length - 77, length - 127
    hot = {0: [23 * 128], 1: [128, 30 * 128], 2: [50 * 128, 61 * 128]}
    c = shared_cache(rng, N, Hkv, d, page, block, length, max(3, 2048 // page), hot)
    per = -(-128 // page)
    c.table[0, 40 * per], c.table[0, 47 * per: 49 * per] = -1, -1  # holes: a page, two whole tiles
    c.table[1, (length - 1) // page] = c.n_pages                   # the last keys' page
    c.table[2, :per], c.table[2, 33 * per] = -9, -1
    q = rng.standard_normal((N, B, Hkv * G, d))
    q[..., 0] = 8.0
    q = kv4_ref.bf16(q)
    bk = bv = None
    if own:
        bk, bv = (kv4_ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    got = run_attn(c, q, lengths, B, length, bk, bv)
    for n in (0, 1, 2, N // 2, N - 1):
        r = ref.Cache.__new__(ref.Cache)
        t = np.where((c.table[n:n + 1] < 0) | (c.table[n:n + 1] >= c.n_pages), -1, c.table[n:n + 1])
        r.__dict__.update(c.__dict__, table=t, N=1)
        want, tol = ref.attention(q[n:n + 1], r, lengths[n:n + 1],
                                  *(None if x is None else x[n:n + 1] for x in (bk, bv)))
        check(got[n:n + 1], want, tol, f"sequence {n}")
