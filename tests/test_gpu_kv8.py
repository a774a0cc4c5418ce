"""The paged 8-bit cache on the GPU against the plain reference (kv8_ref.py): held bytes bit
by bit, gathered rows bit by bit, attention within a bound derived from its roundings."""
import numpy as np
import pytest

import kv4_ref
import kv8_ref as ref
from helpers import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _h():
    from block_diffusion_sparse_gb300 import herald as H
    return H


class OnGpu:
    def __init__(self, c):
        self.table = dev(c.table)
        self.codes, self.scales = dev(c.codes), dev(c.scales)
        self.kv8 = _h().kv8(c.page, c.block, self.table, self.codes[0], self.scales[0], self.codes[1],
                            self.scales[1])


def bits(t):
    return t.cpu().numpy().view(np.uint16)


def bf(x):
    return kv4_ref.f64(kv4_ref.bf16(x))


def make_cache(rng, N, Hkv, d, page, block, lengths, k_size=1.0, v_size=1.0):
    """Normal keys and values, a few keys and channels larger, block sizes apart by up to 2^4."""
    c = ref.Cache(rng, N, Hkv, d, page, block, lengths)
    for n, L in enumerate(lengths):
        L = min(int(L), int((c.table[n] >= 0).sum()) * page)
        if L:
            k, v = rng.standard_normal((2, L, Hkv, d))
            k[rng.random(L) < 0.02] *= 3
            k[..., 3] *= 4
            v *= 2.0 ** rng.integers(-2, 3, (L // 16 + 1)).repeat(16)[:L, None, None]
            c.write(n, 0, bf(k_size * k), bf(v_size * v))
    return c


def run_attn(c, q, lengths, B, L_max, bk=None, bv=None, scale=0.0, ws=None, stream=None):
    H = _h()
    N, _, Hq, d = q.shape
    dm = H.dims(N, Hq, c.Hkv, d, B, L_max)
    g = OnGpu(c)
    if ws is None:
        ws = torch.zeros(H.herald_workspace_size_kv8(dm), dtype=torch.uint8, device="cuda")
    out = torch.full((N, B, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    ctx = torch.tensor([int(x) for x in lengths], dtype=torch.int32, device="cuda")
    H.herald_kv8_attn(dm, dev(q), g.kv8, ctx, None if bk is None else dev(bk),
                      None if bv is None else dev(bv), out, scale, ws, stream=stream)
    torch.cuda.synchronize()
    assert H.herald_workspace_error(ws) == 0
    return kv4_ref.f64(bits(out.view(torch.int16)))


def check(got, want, tol, what):
    assert np.isfinite(got).all(), what
    over = np.abs(got - want) - tol
    assert (over <= 0).all(), f"{what}: off by {np.abs(got - want).max()}, {over.max()} past the bound"


# (N, Hq, Hkv, d, B, page, block, lengths, block keys)
ATTN = [
    (1, 4, 1, 64, 1, 16, 16, [1], False),
    (1, 4, 1, 64, 1, 16, 16, [0], True),          # only the block
    (3, 4, 2, 64, 1, 16, 16, [0, 17, 0], False),  # rows without any key
    (2, 8, 1, 128, 1, 32, 16, [15, 33], True),
    (1, 7, 1, 128, 1, 64, 64, [4099], True),      # split over many CTAs
    (5, 28, 4, 128, 1, 16, 16, [1, 2000, 0, 300, 64], True),
    (9, 16, 8, 128, 1, 128, 32, [200, 0, 0, 1000, 5, 129, 128, 127, 0], False),
    (2, 8, 2, 64, 3, 64, 32, [700, 65], True),    # 12 rows
    (2, 14, 2, 128, 2, 32, 32, [999, 31], False),  # 14 rows
    (2, 14, 2, 64, 3, 128, 64, [999, 131], True),  # 21 rows
    (2, 8, 1, 128, 4, 64, 16, [1300, 7], True),   # 32 rows
    (1, 2, 2, 128, 16, 16, 16, [513], True),
    (2, 28, 4, 128, 5, 64, 32, [1500, 40], True),  # 35 rows
    (2, 2, 2, 64, 33, 32, 16, [260, 0], False),   # 33 rows
    (1, 28, 4, 128, 32, 64, 64, [3001], True),     # 224 rows
    (2, 8, 1, 64, 32, 128, 128, [1025, 3], True),  # 256 rows
    (3, 16, 4, 128, 32, 16, 16, [0, 1, 2047], False),  # 128 rows
    (1, 5, 5, 64, 256, 32, 32, [77], True),        # one head a group, 256 tokens
    (40, 2, 1, 64, 2, 16, 16, list(range(40)), True),
    (1, 32, 8, 128, 17, 64, 32, [130], True),     # 68 rows
    # several tiles and segments per CTA
    (8, 32, 8, 128, 32, 128, 128, [1024, 0, 900, 1, 128, 1000, 640, 777], True),
    (8, 32, 8, 128, 4, 128, 64, [1024, 0, 900, 1, 128, 1000, 640, 777], False),
    (6, 28, 4, 128, 32, 64, 16, [1600, 0, 1200, 1, 1500, 1111], True),
    (9, 16, 8, 64, 20, 16, 16, [1000, 0, 900, 1, 128, 1000, 640, 777, 130], True),
    (2, 8, 8, 128, 200, 32, 32, [2000, 1300], True),
    (30, 40, 8, 64, 8, 32, 16, [int(x) for x in range(0, 1500, 50)], True),
    (30, 40, 8, 64, 1, 32, 16, [int(x) for x in range(0, 1500, 50)], True),
]


@pytest.mark.parametrize("case", ATTN, ids=str)
def test_attention(case):
    N, Hq, Hkv, d, B, page, block, lengths, block_keys = case
    rng = np.random.default_rng(sum(lengths) + 7 * Hq + B)
    c = make_cache(rng, N, Hkv, d, page, block, lengths, 0.75, 0.5)
    q = kv4_ref.bf16(rng.standard_normal((N, B, Hq, d)))
    bk = bv = None
    if block_keys:
        bk, bv = (kv4_ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    want, tol = ref.attention(q, c, lengths, bk, bv)
    got = run_attn(c, q, lengths, B, max(1, max(lengths)), bk, bv)
    check(got, want, tol, str(case))
    if not block_keys:
        for n, L in enumerate(lengths):
            assert L or (got[n] == 0).all()


ROWS = [1, 4, 8, 32]  # tokens at four heads a group: 4, 16, 32 and 128 rows


@pytest.mark.parametrize("B", ROWS)
def test_attention_extremes(B):
    """Queries of very different sizes, one dominating key, equal scores, an all-zero query,
    and a scale of its own."""
    rng = np.random.default_rng(5)
    N, Hq, Hkv, d, L = 1, 8, 2, 128, 777
    c = make_cache(rng, N, Hkv, d, 32, 16, [L])
    q = rng.standard_normal((N, B, Hq, d)).astype(np.float32)
    q[0, 0, 0] *= 1e-30
    q[0, 0, 1] *= 30.0
    q[0, 0, 2] = 0
    q[0, 0, 3, ::2] *= 1e-6
    q[0, 0, 4] *= 1e-38
    if B > 1:
        q[0, 1] *= 8.0
        q[0, B - 1, 1] = 0
    q = kv4_ref.bf16(q)
    for scale in (0.0, 0.3):
        want, tol = ref.attention(q, c, [L], scale=scale or None)
        check(run_attn(c, q, [L], B, L, scale=scale), want, tol, f"scale {scale}")


@pytest.mark.parametrize("B", ROWS)
@pytest.mark.parametrize("size", [1e-6, 3e4])
def test_attention_sizes(B, size):
    """Keys and values far from 1, the softmax scale the other way."""
    rng = np.random.default_rng(15)
    L = 300
    c = make_cache(rng, 1, 2, 64, 64, 32, [L], size, size)
    q = kv4_ref.bf16(rng.standard_normal((1, B, 8, 64)))
    scale = float(np.float32(0.125 / size))
    want, tol = ref.attention(q, c, [L], scale=scale)
    check(run_attn(c, q, [L], B, L, scale=scale), want, tol, "sizes")


@pytest.mark.parametrize("B", ROWS)
def test_attention_value_scales_apart(B):
    """Blocks of values whose scales lie far apart, in rising and falling order, zeros among them,
    and the weight on small ones."""
    rng = np.random.default_rng(16)
    d, L = 128, 640
    for order in (1, -1):
        c = ref.Cache(rng, 1, 1, d, 32, 16, [L])
        k, v = rng.standard_normal((2, L, 1, d))
        steps = np.repeat(np.arange(L // 16) // 2 - 10, 16)[::order]
        v *= 2.0 ** steps[:, None, None]
        v[64:80] = 0
        k[:, 0, 0] -= 0.6 * steps  # the smaller the values, the larger the weight
        c.write(0, 0, bf(k), bf(v))
        q = rng.standard_normal((1, B, 4, d))
        q[..., 0] = 8.0
        q = kv4_ref.bf16(q)
        want, tol = ref.attention(q, c, [L])
        check(run_attn(c, q, [L], B, L), want, tol, f"scales apart {order}")


@pytest.mark.parametrize("B", ROWS)
def test_attention_sink(B):
    """One key takes nearly all of the weight, its value small; the rest share what is left."""
    rng = np.random.default_rng(17)
    d, L = 64, 5000
    c = ref.Cache(rng, 1, 1, d, 16, 16, [L])
    k, v = 0.1 * rng.standard_normal((2, L, 1, d))
    k[0, 0, 0], v[:16] = 9.0, v[:16] * 2.0 ** -10
    v[16:] += 1.0
    c.write(0, 0, bf(k), bf(v))
    q = 0.1 * rng.standard_normal((1, B, 4, d))
    for lead in (4.0, 8.0, 14.0):
        q[..., 0] = lead
        qb = kv4_ref.bf16(q)
        want, tol = ref.attention(qb, c, [L])
        check(run_attn(c, qb, [L], B, L), want, tol, f"sink {lead}")


@pytest.mark.parametrize("B", ROWS)
def test_attention_rising_scores(B):
    """Scores that grow along the cache: the exponent base has to move often."""
    rng = np.random.default_rng(6)
    d, L = 64, 900
    w = rng.standard_normal(d)
    k = np.linspace(0, 6, L)[:, None, None] * w + 0.1 * rng.standard_normal((L, 1, d))
    q = kv4_ref.bf16(np.broadcast_to(w, (1, B, 4, d)) * np.float32(0.6))
    for rows in (k, k[::-1]):
        c = ref.Cache(rng, 1, 1, d, 16, 16, [L])
        c.write(0, 0, bf(rows), bf(rng.standard_normal((L, 1, d))))
        want, tol = ref.attention(q, c, [L])
        check(run_attn(c, q, [L], B, L), want, tol, "rising, then falling")


@pytest.mark.parametrize("B", ROWS)
@pytest.mark.parametrize("block_keys", [False, True])
def test_attention_missing_pages(B, block_keys):
    """Table entries without a page are masked, wherever they stand."""
    rng = np.random.default_rng(8)
    N, Hq, Hkv, d, page = 3, 8, 2, 128, 16
    lengths = [333, 64, 40]
    c = make_cache(rng, N, Hkv, d, page, 16, lengths)
    c.table[0, 3:5] = -1
    c.table[0, 8:16] = -7              # a whole tile of 128
    c.table[0, 17] = c.n_pages         # past the arrays
    c.table[0, 20] = 2 ** 31 - 1
    c.table[1, :] = -5                 # a whole sequence without pages
    c.table[2, 0] = -1
    q = kv4_ref.bf16(rng.standard_normal((N, B, Hq, d)))
    bk = bv = None
    if block_keys:
        bk, bv = (kv4_ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    r = ref.Cache.__new__(ref.Cache)   # the reference wants -1 for a missing page
    r.__dict__.update(c.__dict__, table=np.where((c.table < 0) | (c.table >= c.n_pages), -1, c.table))
    want, tol = ref.attention(q, r, lengths, bk, bv)
    got = run_attn(c, q, lengths, B, 333, bk, bv)
    check(got, want, tol, "missing pages")
    assert block_keys or (got[1] == 0).all()


@pytest.mark.parametrize("B", ROWS)
def test_attention_lengths_are_clamped(B):
    rng = np.random.default_rng(9)
    c = make_cache(rng, 3, 2, 64, 32, 16, [100, 100, 100])
    q = kv4_ref.bf16(rng.standard_normal((3, B, 8, 64)))
    want, tol = ref.attention(q, c, [0, 70, 70])
    check(run_attn(c, q, [-3, 70, 1000], B, 70), want, tol, "clamped")


@pytest.mark.parametrize("B", ROWS)
def test_attention_scale_bytes_are_clamped(B):
    rng = np.random.default_rng(19)
    c = make_cache(rng, 1, 2, 64, 32, 16, [100], 1e-8, 1e-8)
    c.scales[0, c.table[0, 0], 0, 0] = 3
    c.scales[1, c.table[0, 1], 0, 1] = 0
    c.scales[1, c.table[0, 2], 1, 0] = 255
    q = kv4_ref.bf16(rng.standard_normal((1, B, 8, 64)))
    want, tol = ref.attention(q, c, [100])
    check(run_attn(c, q, [100], B, 100), want, tol, "scale bytes")


@pytest.mark.parametrize("B", ROWS)
def test_attention_nan_and_inf(B):
    """A NaN key or value reaches its head's rows and no others; a NaN query its own row; an
    infinite query value makes a NaN row, as inf - inf does."""
    rng = np.random.default_rng(10)
    N, Hq, Hkv, d, L = 3, 8, 2, 128, 200
    c = make_cache(rng, N, Hkv, d, 64, 32, [L] * N)
    c.codes[0, c.table[0, 1], 1, 3, 2] = 0x7F   # K of sequence 0, head 1, position 67
    c.codes[1, c.table[2, 2], 0, 9, 5] = 0xFF   # V of sequence 2, head 0, position 137, channel 5
    q = kv4_ref.bf16(rng.standard_normal((N, B, Hq, d)))
    q[1, 0, 2, 5] = 0x7FC0
    q[1, 0, 7, 5] = 0x7F80
    got = run_attn(c, q, [L] * N, B, L)
    bad = np.zeros((N, B, Hq, d), bool)
    bad[0, :, 4:] = True
    bad[1, 0, 2] = bad[1, 0, 7] = True
    bad[2, :, :4, 5] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


@pytest.mark.parametrize("B", ROWS)
def test_attention_far_scores(B):
    """Scores so large that fp32 holds them to whole units and more: the largest one's key, or an
    even share of keys that it does not tell apart from it; no NaN, no infinity."""
    rng = np.random.default_rng(18)
    d, L = 64, 200
    k = rng.standard_normal((L, 1, d))
    v = rng.standard_normal((L, 1, d))
    for size in (2.0 ** 16, 2.0 ** 22, 2.0 ** 30, 2.0 ** 40):
        c = ref.Cache(rng, 1, 1, d, 16, 16, [L])
        c.write(0, 0, bf(k), bf(v))
        q = kv4_ref.bf16(rng.standard_normal((1, B, 4, d)))
        got = run_attn(c, q, [L], B, L, scale=float(size))
        rows, held = c.rows(0, 0, np.arange(L))[0], c.rows(1, 0, np.arange(L))[0]
        s = np.einsum("bhd,jd->bhj", kv4_ref.f64(q)[0], rows)
        # fp32 sums of d products, then a few roundings of the score: keys within this of the
        # largest score may share the weight
        band = (d + 16) * 2.0 ** -22 * np.einsum("bhd,jd->bhj", np.abs(kv4_ref.f64(q)[0]), np.abs(rows)).max(-1)
        near = s >= (s.max(-1) - band - 64 / size)[..., None]
        assert np.isfinite(got).all()
        for b in range(B):
            for h in range(4):
                x = held[near[b, h]]
                lo, hi = x.min(0), x.max(0)
                off = np.maximum(np.maximum(lo - got[0, b, h], got[0, b, h] - hi), 0)
                # half a bf16 step, and weights' 11 bits
                assert (off <= (2.0 ** -8 + 2.0 ** -10) * np.abs(x).max(0)).all(), (size, b, h)


def test_attention_on_another_stream_and_in_a_graph():
    H = _h()
    rng = np.random.default_rng(11)
    N, Hq, Hkv, d = 2, 8, 2, 128
    lengths = [600, 31]
    c = make_cache(rng, N, Hkv, d, 64, 32, [700, 700])
    for B in ROWS:
        g = OnGpu(c)
        q = kv4_ref.bf16(rng.standard_normal((N, B, Hq, d)))
        dm = H.dims(N, Hq, Hkv, d, B, 700)
        ws = torch.zeros(H.herald_workspace_size_kv8(dm), dtype=torch.uint8, device="cuda")
        qd, out = dev(q), torch.zeros((N, B, Hq, d), dtype=torch.bfloat16, device="cuda")
        ctx = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            H.herald_kv8_attn(dm, qd, g.kv8, ctx, None, None, out, ws=ws, stream=st)
        st.synchronize()
        want, tol = ref.attention(q, c, lengths)
        check(kv4_ref.f64(bits(out.view(torch.int16))), want, tol, "stream")
        first = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            H.herald_kv8_attn(dm, qd, g.kv8, ctx, None, None, out, ws=ws,
                              stream=torch.cuda.current_stream())
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)  # bit for bit
        ctx.copy_(torch.tensor([77, 700], dtype=torch.int32))  # the graph reads the lengths anew
        graph.replay()
        torch.cuda.synchronize()
        want, tol = ref.attention(q, c, [77, 700])
        check(kv4_ref.f64(bits(out.view(torch.int16))), want, tol, "replayed")


def test_attention_is_deterministic_and_ignores_the_workspace():
    rng = np.random.default_rng(12)
    H = _h()
    for B in ROWS:
        c = make_cache(rng, 2, 2, 128, 64, 32, [3000, 1234])
        q = kv4_ref.bf16(rng.standard_normal((2, B, 8, 128)))
        dm = H.dims(2, 8, 2, 128, B, 3000)
        size = H.herald_workspace_size_kv8(dm)
        outs = []
        for fill in (0, 0xFF, 0x7F):
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            ws[:16] = 0  # the error word
            outs.append(run_attn(c, q, [3000, 1234], B, 3000, ws=ws))
        assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


# ----------------------------------------------------------------- append

# (N, Hq, Hkv, d, T, page, block, ctx, n_tok, rot, interleaved, fused, Bk)
APPEND = [
    (1, 4, 1, 64, 1, 16, 16, [0], None, 64, 0, False, 0),
    (3, 4, 2, 64, 1, 16, 16, [15, 16, 0], [1, 1, 0], 64, 1, True, 16),
    (2, 28, 4, 128, 32, 64, 32, [37, 100], None, 128, 0, False, 64),
    (2, 28, 4, 128, 32, 64, 64, [37, 100], [32, 5], 128, 1, True, 32),
    (3, 8, 8, 128, 77, 32, 16, [0, 1, 200], [77, 0, 50], 64, 0, True, 7),
    (1, 8, 2, 128, 130, 128, 128, [5], None, 96, 0, False, 64),
    (2, 8, 2, 64, 40, 16, 16, [3, 0], [-4, 99], 32, 0, True, 0),
    (2, 16, 2, 128, 9, 16, 16, [3, 55], None, 0, 0, False, 64),
    (2, 8, 2, 128, 600, 64, 64, [0, 33], [600, 590], 128, 0, True, 64),
    (1, 8, 1, 128, 20, 16, 16, [90], None, 128, 0, False, 64),  # runs into L_max = 100
    (2, 4, 2, 64, 5, 16, 16, [3, 10], [5, 2], 64, 0, True, 64),  # one block longer than the cache
    (2, 6, 3, 64, 70, 128, 128, [100, 127], None, 32, 1, False, 0),
    (5, 8, 2, 64, 3, 128, 32, [31, 30, 29, 95, 32], [1, 2, 3, 1, 3], 64, 0, False, 0),
    (1, 16, 16, 128, 2000, 64, 16, [11], None, 128, 1, True, 0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(case, in_place):
    H = _h()
    N, Hq, Hkv, d, T, page, block, ctx, n_tok, rot, inter, fused, Bk = case
    if in_place and fused:
        pytest.skip("in place needs dense inputs")
    rng = np.random.default_rng(T + rot)
    L_max = 100 if ctx == [90] else max(ctx) + T
    c = ref.Cache(rng, N, Hkv, d, page, block, [min(x + T, L_max) for x in ctx])
    for n, x in enumerate(ctx):  # older rows, smaller than what comes in half of the heads
        small = np.where(np.arange(Hkv) % 2, 0.1, 3.0)[:, None]
        c.write(n, 0, *(bf(rng.standard_normal((x, Hkv, d)) * small) for _ in range(2)))
    g = OnGpu(c)
    q, k, v = (kv4_ref.bf16(rng.standard_normal((N, T, h, d))) for h in (Hq, Hkv, Hkv))
    v[:, ::7, :, 3] = kv4_ref.bf16(1e-4)
    k[:, T // 2:, 0] = 0                         # blocks of zeros
    tq, tk, tv = dev(q), dev(k), dev(v)
    if fused:
        qkv = torch.cat((tq, tk, tv), 2).contiguous()
        tq, tk, tv = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    q_rot = tq if in_place else torch.full((N, T, Hq, d), -1, dtype=torch.int16, device="cuda")
    k_rot = tk if in_place else torch.full((N, T, Hkv, d), -1, dtype=torch.int16, device="cuda")
    q_was, k_was = bits(q_rot).copy(), bits(k_rot).copy()
    cs = kv4_ref.angles(L_max + 3, rot) if rot else None
    rope = H.rope(dev(cs), rot, inter) if rot else None
    dctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    dn = None if n_tok is None else torch.tensor(n_tok, dtype=torch.int32, device="cuda")
    pooled = torch.full((N, Hkv, -(-L_max // Bk), d), 9.0, device="cuda") if Bk else None
    dm = H.dims(N, Hq, Hkv, d, 1, L_max)
    H.herald_kv8_append(dm, T, tq, tk, tv, dctx, g.kv8, q_rot, k_rot, rope, dn, pooled, Bk,
                        H.HERALD_KV8_ADVANCE)
    torch.cuda.synchronize()
    # the reference, row by row
    want_pool = np.full((N, Hkv, -(-L_max // Bk), d), 9.0) if Bk else None
    ends = []
    for n in range(N):
        m = min(T if n_tok is None else min(max(n_tok[n], 0), T), L_max - ctx[n])
        ends.append(ctx[n] + m)
        pos = ctx[n] + np.arange(m)
        rq = kv4_ref.rotate32(kv4_ref.f64(q[n, :m]), cs, pos, rot, inter)
        rk = kv4_ref.bf16(kv4_ref.rotate32(kv4_ref.f64(k[n, :m]), cs, pos, rot, inter))
        q_was[n, :m], k_was[n, :m] = kv4_ref.bf16(rq), rk
        if m:
            c.write(n, ctx[n], kv4_ref.f64(rk), kv4_ref.f64(v[n, :m]))
        if Bk and m:
            for b in range(ctx[n] // Bk, -(-ends[n] // Bk)):
                at = np.arange(b * Bk, min(ends[n], (b + 1) * Bk))
                want_pool[n, :, b] = c.rows(0, n, at).mean(1)
    assert np.array_equal(bits(q_rot), q_was) and np.array_equal(bits(k_rot), k_was)
    assert np.array_equal(g.scales.cpu().numpy(), c.scales), "scales"
    assert np.array_equal(g.codes.cpu().numpy(), c.codes), "codes"
    assert dctx.tolist() == ends
    if Bk:
        got = pooled.cpu().numpy().astype(np.float64)
        # fp32 sums of up to Bk values of at most 15, one division
        assert np.abs(got - want_pool).max() <= (Bk + 2) * 2.0 ** -24 * 16


def test_append_token_by_token():
    """One token a call: a block's scale grows with its rows, and a new block starts anew; the
    cache is the reference's after every token, also where lengths go back (rejected drafts)."""
    H = _h()
    rng = np.random.default_rng(21)
    N, Hq, Hkv, d, page, block, L = 2, 4, 2, 64, 32, 32, 70
    c = ref.Cache(rng, N, Hkv, d, page, block, [L, L])
    g = OnGpu(c)
    dm = H.dims(N, Hq, Hkv, d, 1, L)
    ctx = torch.zeros(N, dtype=torch.int32, device="cuda")
    k_rot = torch.empty((N, 1, Hkv, d), dtype=torch.int16, device="cuda")
    lengths = [0, 0]
    for step in range(60):
        if step == 40:
            lengths = [37, 3]
            ctx.copy_(torch.tensor(lengths, dtype=torch.int32))
        size = 2.0 ** rng.integers(-6, 7)
        k, v = (kv4_ref.bf16(size * rng.standard_normal((N, 1, Hkv, d))) for _ in range(2))
        H.herald_kv8_append(dm, 1, None, dev(k), dev(v), ctx, g.kv8, None, k_rot,
                            flags=H.HERALD_KV8_ADVANCE)
        for n in range(N):
            c.write(n, lengths[n], kv4_ref.f64(k[n]), kv4_ref.f64(v[n]))
            lengths[n] += 1
        assert np.array_equal(g.scales.cpu().numpy(), c.scales), step
        assert np.array_equal(g.codes.cpu().numpy(), c.codes), step
    assert ctx.tolist() == lengths


def test_append_extremes():
    """Infinities saturate and NaNs stay alone, neither moving the scale; values past both ends
    of the scales; negative zeros."""
    H = _h()
    rng = np.random.default_rng(22)
    N, Hkv, d, T = 1, 3, 128, 40
    c = ref.Cache(rng, N, Hkv, d, 16, 16, [T])
    g = OnGpu(c)
    x = rng.standard_normal((2, N, T, Hkv, d)).astype(np.float32)
    x[:, 0, 5, 0, 7], x[:, 0, 6, 0, 8], x[:, 0, 7, 1, 0] = np.inf, -np.inf, np.nan
    x[0, 0, 20:, 1] *= 1e30
    x[1, 0, 20:, 1] *= 1e-30
    x[:, 0, 3, 2] = -0.0
    x[:, 0, 16:32, 2] = np.inf
    x[0, 0, 33:35, 0] = 448.0
    x[0, 0, 36, 0, 1] = 3.38e38
    k, v = kv4_ref.bf16(x[0]), kv4_ref.bf16(x[1])
    ctx = torch.zeros(N, dtype=torch.int32, device="cuda")
    H.herald_kv8_append(H.dims(N, Hkv, Hkv, d, 1, T), T, None, dev(k), dev(v), ctx, g.kv8, None, None)
    c.write(0, 0, kv4_ref.f64(k[0]), kv4_ref.f64(v[0]))
    assert np.array_equal(g.scales.cpu().numpy(), c.scales)
    assert np.array_equal(g.codes.cpu().numpy(), c.codes)


def test_append_missing_pages_and_rotation_alone():
    H = _h()
    rng = np.random.default_rng(23)
    N, Hq, Hkv, d, T, page = 2, 4, 2, 64, 50, 16
    c = ref.Cache(rng, N, Hkv, d, page, 16, [T + 9, T + 9])
    c.table[0, 1], c.table[1, 0] = -1, -3
    was = (c.codes.copy(), c.scales.copy())
    g = OnGpu(c)
    q, k, v = (kv4_ref.bf16(rng.standard_normal((N, T, h, d))) for h in (Hq, Hkv, Hkv))
    cs = kv4_ref.angles(T + 9, d)
    rope = H.rope(dev(cs), d)
    dm, ctx = H.dims(N, Hq, Hkv, d, 1, T + 9), torch.tensor([9, 0], dtype=torch.int32, device="cuda")
    outs = [torch.zeros((N, T, h, d), dtype=torch.int16, device="cuda") for h in (Hq, Hkv, Hq, Hkv)]
    H.herald_kv8_append(dm, T, dev(q), dev(k), None, ctx, None, outs[0], outs[1], rope)
    assert np.array_equal(g.codes.cpu().numpy(), was[0])
    H.herald_kv8_append(dm, T, dev(q), dev(k), dev(v), ctx, g.kv8, outs[2], outs[3], rope)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    c.scales[0, c.table[0, 0], :, 0] = was[1][0, c.table[0, 0], :, 0]
    r = ref.Cache.__new__(ref.Cache)
    r.__dict__.update(c.__dict__)
    for n, at in ((0, 9), (1, 0)):
        r.write(n, at, kv4_ref.f64(bits(outs[3])[n]), kv4_ref.f64(v[n]))
    assert np.array_equal(g.scales.cpu().numpy(), r.scales)
    assert np.array_equal(g.codes.cpu().numpy(), r.codes)


# ----------------------------------------------------------------- gather

@pytest.mark.parametrize("case", [(2, 3, 128, 64, 32, [900, 5], 77, True), (1, 2, 64, 16, 16, [33], 40, False),
                                  (3, 1, 64, 128, 128, [129, 0, 4000], 513, True),
                                  (4, 8, 128, 32, 16, [5000, 1, 700, 64], 3000, True)], ids=str)
def test_gather(case):
    H = _h()
    N, Hkv, d, page, block, lengths, P, values = case
    rng = np.random.default_rng(P)
    c = make_cache(rng, N, Hkv, d, page, block, lengths)
    L_max = max(lengths)
    idx = np.full((N, Hkv, P), -1, np.int32)
    n_sel = np.zeros((N, Hkv), np.int32)
    for n, L in enumerate(lengths):
        for h in range(Hkv):
            m = min(P, L, P if h == 0 else int(rng.integers(0, P + 1)))
            idx[n, h, :m] = np.sort(rng.permutation(L)[:m])
            n_sel[n, h] = m
    idx[0, 0, 1] = L_max + 7            # outside the cache: a zero row
    idx[0, 0, 2] = -5
    if (c.table[0] >= 0).sum() > 3:
        c.table[0, 2] = -1
    g = OnGpu(c)
    pk = torch.full((N, Hkv, P, d), 7, dtype=torch.int16, device="cuda")
    pv = torch.full((N, Hkv, P, d), 7, dtype=torch.int16, device="cuda")
    H.herald_kv8_gather(H.dims(N, Hkv, Hkv, d, 1, L_max), dev(idx), dev(n_sel), P, g.kv8, pk,
                        pv if values else None)
    want = np.zeros((2, N, Hkv, P, d))
    for n in range(N):
        for h in range(Hkv):
            for s in range(n_sel[n, h]):
                p = idx[n, h, s]
                if 0 <= p < L_max and c.table[n, p // page] >= 0:
                    for i in range(2):
                        want[i, n, h, s] = c.rows(i, n, [p])[h, 0]
    got = [kv4_ref.f64(bits(x)) for x in (pk, pv)]
    assert np.array_equal(got[0], want[0])
    assert np.array_equal(got[1], want[1]) if values else (pv == 7).all()
