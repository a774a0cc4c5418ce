"""The paged 4-bit cache on the GPU against the plain reference (kv4_ref.py):
held bytes bit by bit, gathered rows bit by bit, attention within a bound
derived from its roundings."""
import numpy as np
import pytest

import kv4_ref as ref
from helpers import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _h():
    from block_diffusion_sparse_gb300 import herald as H
    return H


class OnGpu:
    def __init__(self, c):
        H = _h()
        self.table = dev(c.table)
        self.codes, self.scales = dev(c.codes), dev(c.scales)
        self.kv4 = H.kv4(c.page, self.table, self.codes[0], self.scales[0], self.codes[1],
                         self.scales[1], c.k_scale, c.v_scale)


def bits(t):
    return t.cpu().numpy().view(np.uint16)


def make_cache(rng, N, Hkv, d, page, lengths, **kw):
    c = ref.Cache(rng, N, Hkv, d, page, lengths, **kw)
    for n, L in enumerate(lengths):
        L = min(int(L), int((c.table[n] >= 0).sum()) * page)
        k = rng.standard_normal((L, Hkv, d)).astype(np.float32) * c.k_scale
        v = rng.standard_normal((L, Hkv, d)).astype(np.float32) * c.v_scale
        hot = rng.random(L) < 0.02
        k[hot] *= 3
        if L:
            c.write(n, np.arange(L), k, v)
    return c


def run_attn(c, q, lengths, B, L_max, bk=None, bv=None, scale=0.0, ws=None, stream=None):
    H = _h()
    N, _, Hq, d = q.shape
    dm = H.dims(N, Hq, c.Hkv, d, B, L_max)
    g = OnGpu(c)
    if ws is None:
        ws = torch.zeros(H.herald_workspace_size_kv4(dm), dtype=torch.uint8, device="cuda")
    out = torch.full((N, B, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    ctx = torch.tensor([int(x) for x in lengths], dtype=torch.int32, device="cuda")
    H.herald_kv4_attn(dm, dev(q), g.kv4, ctx, None if bk is None else dev(bk),
                      None if bv is None else dev(bv), out, scale, ws, stream=stream)
    torch.cuda.synchronize()
    assert H.herald_workspace_error(ws) == 0
    return ref.f64(bits(out.view(torch.int16)))


def check(got, want, tol, what):
    assert np.isfinite(got).all(), what
    over = np.abs(got - want) - tol
    assert (over <= 0).all(), f"{what}: off by {np.abs(got - want).max()}, {over.max()} past the bound"


# (N, Hq, Hkv, d, B, page, lengths, block)
ATTN = [
    (1, 4, 1, 64, 1, 16, [1], False),
    (1, 4, 1, 64, 1, 16, [0], True),          # only the block
    (3, 4, 2, 64, 1, 16, [0, 17, 0], False),  # rows without any key
    (2, 8, 1, 128, 1, 32, [15, 33], True),
    (1, 7, 1, 128, 1, 64, [4099], True),      # split over many CTAs
    (5, 28, 4, 128, 1, 16, [1, 2000, 0, 300, 64], True),
    (9, 16, 8, 128, 1, 128, [200, 0, 0, 1000, 5, 129, 128, 127, 0], False),
    (2, 8, 2, 64, 3, 64, [700, 65], True),    # 12 rows
    (2, 14, 2, 128, 2, 32, [999, 31], False),  # 14 rows
    (1, 2, 2, 128, 16, 16, [513], True),
    (2, 28, 4, 128, 5, 64, [1500, 40], True),  # 35 rows
    (1, 28, 4, 128, 32, 64, [3001], True),     # 224 rows
    (2, 8, 1, 64, 32, 128, [1025, 3], True),   # 256 rows
    (3, 16, 4, 128, 32, 16, [0, 1, 2047], False),  # 128 rows
    (1, 5, 5, 64, 256, 32, [77], True),        # one head a group, 256 tokens
    (40, 2, 1, 64, 2, 16, list(range(40)), True),
    (1, 32, 8, 128, 17, 64, [130], True),     # 68 rows
    # several tiles and segments per CTA of the tensor-core kernel
    (8, 32, 8, 128, 32, 128, [1024, 0, 900, 1, 128, 1000, 640, 777], True),
    (8, 32, 8, 128, 32, 128, [1024, 0, 900, 1, 128, 1000, 640, 777], False),
    (6, 28, 4, 128, 32, 64, [1600, 0, 1200, 1, 1500, 1111], True),
    (9, 16, 8, 64, 20, 16, [1000, 0, 900, 1, 128, 1000, 640, 777, 130], True),
    (2, 8, 8, 128, 200, 32, [2000, 1300], True),  # two block tiles
    (30, 40, 8, 64, 8, 32, [int(x) for x in range(0, 1500, 50)], True),
]


@pytest.mark.parametrize("case", ATTN, ids=str)
def test_attention(case):
    N, Hq, Hkv, d, B, page, lengths, block = case
    rng = np.random.default_rng(sum(lengths) + 7 * Hq + B)
    c = make_cache(rng, N, Hkv, d, page, lengths, k_scale=0.75, v_scale=0.5)
    q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
    bk = bv = None
    if block:
        bk, bv = (ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    want, tol = ref.attention(q, c, lengths, bk, bv)
    got = run_attn(c, q, lengths, B, max(1, max(lengths)), bk, bv)
    check(got, want, tol, str(case))
    if not block:
        for n, L in enumerate(lengths):
            assert L or (got[n] == 0).all()


@pytest.mark.parametrize("B", [1, 32])
def test_attention_extremes(B):
    """Queries of very different sizes, one dominating key, equal scores, an
    all-zero query, and a scale of its own."""
    rng = np.random.default_rng(5)
    N, Hq, Hkv, d, L = 1, 8, 2, 128, 777
    c = make_cache(rng, N, Hkv, d, 32, [L])
    q = rng.standard_normal((N, B, Hq, d)).astype(np.float32)
    q[0, 0, 0] *= 1e-30
    q[0, 0, 1] *= 30.0
    q[0, 0, 2] = 0
    q[0, 0, 3, ::2] *= 1e-6
    q[0, 0, 4] *= 1e-38
    if B > 1:
        q[0, 1] *= 8.0
        q[0, 5, 1] = 0
    q = ref.bf16(q)
    for scale in (0.0, 0.3):
        want, tol = ref.attention(q, c, [L], scale=scale or None)
        check(run_attn(c, q, [L], B, L, scale=scale), want, tol, f"scale {scale}")


@pytest.mark.parametrize("B", [1, 4, 32])
def test_attention_rising_scores(B):
    """Scores that grow along the cache: the exponent base has to move often."""
    rng = np.random.default_rng(6)
    d, L = 64, 900
    c = ref.Cache(rng, 1, 1, d, 16, [L])
    w = rng.standard_normal(d).astype(np.float32)
    k = (np.linspace(0, 6, L)[:, None, None] * w + 0.1 * rng.standard_normal((L, 1, d)))
    c.write(0, np.arange(L), k.astype(np.float32), rng.standard_normal((L, 1, d)).astype(np.float32))
    q = ref.bf16(np.broadcast_to(w, (1, B, 4, d)) * np.float32(0.6))
    want, tol = ref.attention(q, c, [L])
    check(run_attn(c, q, [L], B, L), want, tol, "rising")
    # and falling: later units far below the base
    c2 = ref.Cache(rng, 1, 1, d, 16, [L])
    c2.write(0, np.arange(L), k[::-1].astype(np.float32),
             rng.standard_normal((L, 1, d)).astype(np.float32))
    want, tol = ref.attention(q, c2, [L])
    check(run_attn(c2, q, [L], B, L), want, tol, "falling")


@pytest.mark.parametrize("B", [1, 32])
def test_attention_missing_pages(B):
    """Table entries without a page are masked, wherever they stand."""
    rng = np.random.default_rng(8)
    N, Hq, Hkv, d, page = 3, 8, 2, 128, 16
    lengths = [333, 64, 40]
    c = make_cache(rng, N, Hkv, d, page, lengths)
    c.table[0, 3:5] = -1
    c.table[0, 9] = c.n_pages          # past the arrays
    c.table[0, 20] = 2 ** 31 - 1
    c.table[1, :] = -5                  # a whole sequence without pages
    c.table[2, 0] = -1
    q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
    # the reference wants -1 for a missing page
    r = ref.Cache.__new__(ref.Cache)
    r.__dict__.update(c.__dict__, table=np.where((c.table < 0) | (c.table >= c.n_pages), -1, c.table))
    want, tol = ref.attention(q, r, lengths)
    got = run_attn(c, q, lengths, B, 333)
    check(got, want, tol, "missing pages")
    assert (got[1] == 0).all()


@pytest.mark.parametrize("B", [1, 32])
def test_attention_lengths_are_clamped(B):
    rng = np.random.default_rng(9)
    c = make_cache(rng, 3, 2, 64, 32, [100, 100, 100])
    q = ref.bf16(rng.standard_normal((3, B, 8, 64)))
    want, tol = ref.attention(q, c, [0, 70, 70])
    check(run_attn(c, q, [-3, 70, 1000], B, 70), want, tol, "clamped")


@pytest.mark.parametrize("B", [1, 32])
def test_attention_nan_and_inf(B):
    """A NaN key or value reaches its head's rows and no others; a NaN query
    its own row; an infinite query value makes a NaN row, as inf - inf does."""
    rng = np.random.default_rng(10)
    N, Hq, Hkv, d, L = 2, 8, 2, 128, 200
    c = make_cache(rng, N, Hkv, d, 64, [L, L])
    ph = c.table[0, 1]
    c.scales[0, ph, 1, 3, 2] = 0x7F     # K of sequence 0, head 1, position 67
    q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
    q[1, 0, 2, 5] = 0x7FC0
    q[1, 0, 7, 5] = 0x7F80
    got = run_attn(c, q, [L, L], B, L)
    bad = np.zeros((N, B, Hq), bool)
    bad[0, :, 4:] = True
    bad[1, 0, 2] = bad[1, 0, 7] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


def test_attention_on_another_stream_and_in_a_graph():
    H = _h()
    rng = np.random.default_rng(11)
    N, Hq, Hkv, d, B = 2, 8, 2, 128, 1
    lengths = [600, 31]
    c = make_cache(rng, N, Hkv, d, 64, [700, 700])
    g = OnGpu(c)
    q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
    dm = H.dims(N, Hq, Hkv, d, B, 700)
    ws = torch.zeros(H.herald_workspace_size_kv4(dm), dtype=torch.uint8, device="cuda")
    qd, out = dev(q), torch.zeros((N, B, Hq, d), dtype=torch.bfloat16, device="cuda")
    ctx = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        H.herald_kv4_attn(dm, qd, g.kv4, ctx, None, None, out, ws=ws, stream=st)
    st.synchronize()
    want, tol = ref.attention(q, c, lengths)
    check(ref.f64(bits(out.view(torch.int16))), want, tol, "stream")
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H.herald_kv4_attn(dm, qd, g.kv4, ctx, None, None, out, ws=ws,
                          stream=torch.cuda.current_stream())
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)  # bit for bit
    ctx.copy_(torch.tensor([77, 700], dtype=torch.int32))  # the graph reads the lengths anew
    graph.replay()
    torch.cuda.synchronize()
    want, tol = ref.attention(q, c, [77, 700])
    check(ref.f64(bits(out.view(torch.int16))), want, tol, "replayed")


def test_attention_is_deterministic_and_ignores_the_workspace():
    rng = np.random.default_rng(12)
    H = _h()
    for B in (1, 4, 32):
        c = make_cache(rng, 2, 2, 128, 64, [3000, 1234])
        q = ref.bf16(rng.standard_normal((2, B, 14, 128)))
        dm = H.dims(2, 14, 2, 128, B, 3000)
        size = H.herald_workspace_size_kv4(dm)
        outs = []
        for fill in (0, 0xFF, 0x7F):
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            ws[:16] = 0  # the error word
            outs.append(run_attn(c, q, [3000, 1234], B, 3000, ws=ws))
        assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


# ----------------------------------------------------------------- append

# (N, Hq, Hkv, d, T, page, ctx, n_tok, rot, interleaved, fused, Bk)
APPEND = [
    (1, 4, 1, 64, 1, 16, [0], None, 64, 0, False, 0),
    (3, 4, 2, 64, 1, 16, [15, 16, 0], [1, 1, 0], 64, 1, True, 16),
    (2, 28, 4, 128, 32, 64, [37, 100], None, 128, 0, False, 64),
    (2, 28, 4, 128, 32, 64, [37, 100], [32, 5], 128, 1, True, 32),
    (3, 8, 8, 128, 77, 32, [0, 1, 200], [77, 0, 50], 64, 0, True, 7),
    (1, 8, 2, 128, 130, 128, [5], None, 96, 0, False, 64),
    (2, 8, 2, 64, 40, 16, [3, 0], [-4, 99], 32, 0, True, 0),
    (2, 16, 2, 128, 9, 16, [3, 55], None, 0, 0, False, 64),
    (2, 8, 2, 128, 600, 64, [0, 33], [600, 590], 128, 0, True, 64),
    (1, 8, 1, 128, 20, 16, [90], None, 128, 0, False, 64),  # runs into L_max = 100
    (2, 4, 2, 64, 5, 16, [3, 10], [5, 2], 64, 0, True, 64),  # one block longer than the cache
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(case, in_place):
    H = _h()
    N, Hq, Hkv, d, T, page, ctx, n_tok, rot, inter, fused, Bk = case
    if in_place and fused:
        pytest.skip("in place needs dense inputs")
    rng = np.random.default_rng(T + rot)
    L_max = 100 if ctx == [90] else max(ctx) + T
    c = make_cache(rng, N, Hkv, d, page, [min(x + T, L_max) for x in ctx], k_scale=0.5, v_scale=0.3)
    g = OnGpu(c)
    q, k, v = (ref.bf16(3 * rng.standard_normal((N, T, h, d))) for h in (Hq, Hkv, Hkv))
    k[:, ::5, :, :16] = 0                        # groups of zeros
    v[:, ::7, :, 3] = ref.bf16(1e-4)
    tq, tk, tv = dev(q), dev(k), dev(v)
    if fused:
        qkv = torch.cat((tq, tk, tv), 2).contiguous()
        tq, tk, tv = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    q_rot = tq if in_place else torch.full((N, T, Hq, d), -1, dtype=torch.int16, device="cuda")
    k_rot = tk if in_place else torch.full((N, T, Hkv, d), -1, dtype=torch.int16, device="cuda")
    q_was, k_was = bits(q_rot).copy(), bits(k_rot).copy()
    cs = ref.angles(L_max + 3, rot) if rot else None
    rope = H.rope(dev(cs), rot, inter) if rot else None
    dctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    dn = None if n_tok is None else torch.tensor(n_tok, dtype=torch.int32, device="cuda")
    pooled = torch.full((N, Hkv, -(-L_max // Bk), d), 9.0, device="cuda") if Bk else None
    dm = H.dims(N, Hq, Hkv, d, 1, L_max)
    H.herald_kv4_append(dm, T, tq, tk, tv, dctx, g.kv4, q_rot, k_rot, rope, dn, pooled, Bk,
                        H.HERALD_KV4_ADVANCE)
    torch.cuda.synchronize()
    # the reference, row by row
    codes0, scales0 = c.codes.copy(), c.scales.copy()
    want_pool = np.full((N, Hkv, -(-L_max // Bk), d), 9.0) if Bk else None
    ends = []
    for n in range(N):
        m = min(T if n_tok is None else min(max(n_tok[n], 0), T), L_max - ctx[n])
        ends.append(ctx[n] + m)
        pos = ctx[n] + np.arange(m)
        rq = ref.rotate32(ref.f64(q[n, :m]), cs, pos, rot, inter)
        rk = ref.rotate32(ref.f64(k[n, :m]), cs, pos, rot, inter)
        q_was[n, :m], k_was[n, :m] = ref.bf16(rq), ref.bf16(rk)
        if m:
            c.write(n, pos, rk, ref.f64(v[n, :m]).astype(np.float32))
        if Bk and m:
            for b in range(ctx[n] // Bk, -(-ends[n] // Bk)):
                at = np.arange(b * Bk, min(ends[n], (b + 1) * Bk))
                want_pool[n, :, b] = c.rows(0, n, at).mean(1)
    assert np.array_equal(bits(q_rot), q_was) and np.array_equal(bits(k_rot), k_was)
    assert np.array_equal(g.codes.cpu().numpy(), c.codes), "codes"
    assert np.array_equal(g.scales.cpu().numpy(), c.scales), "scales"
    assert dctx.tolist() == ends
    assert not np.array_equal(codes0, c.codes) or sum(ends) == sum(ctx)
    del scales0
    if Bk:
        got = pooled.cpu().numpy().astype(np.float64)
        # fp32 sums of up to Bk values of at most 3 k_scale 4.5 sigma, one product, one division
        assert np.abs(got - want_pool).max() <= (Bk + 2) * 2.0 ** -24 * 40


def test_rotation_alone():
    """Without a cache only q_rot and k_rot are written; far positions turn by
    the table's angles; q alone is enough."""
    H = _h()
    rng = np.random.default_rng(3)
    N, Hq, Hkv, d, T, L_max = 2, 8, 2, 128, 16, 140000
    cs = ref.angles(L_max, d)
    rope = H.rope(dev(cs), d, False)
    q, k = (ref.bf16(rng.standard_normal((N, T, h, d))) for h in (Hq, Hkv))
    ctx = [131071, 5]
    dm = H.dims(N, Hq, Hkv, d, 1, L_max)
    dctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    for keys in (True, False):
        q_rot = torch.zeros((N, T, Hq, d), dtype=torch.int16, device="cuda")
        k_rot = torch.zeros((N, T, Hkv, d), dtype=torch.int16, device="cuda")
        H.herald_kv4_append(dm, T, dev(q), dev(k) if keys else None, None, dctx, None, q_rot,
                            k_rot if keys else None, rope)
        torch.cuda.synchronize()
        assert dctx.tolist() == ctx
        for n in range(N):
            pos = ctx[n] + np.arange(T)
            assert np.array_equal(bits(q_rot)[n], ref.bf16(ref.rotate32(ref.f64(q[n]), cs, pos, d, 0)))
            # against the angles in 64 bits: the table's rounding, three fp32
            # roundings and the one to bf16
            z = ref.f64(q[n])
            a = pos[:, None, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
            x, y = z[..., :d // 2], z[..., d // 2:]
            w = np.concatenate((x * np.cos(a) - y * np.sin(a), y * np.cos(a) + x * np.sin(a)), -1)
            mag = np.concatenate((np.abs(x) + np.abs(y),) * 2, -1)
            assert (np.abs(ref.f64(bits(q_rot)[n]) - w) <= 2.0 ** -8 * np.abs(w) + 2.0 ** -22 * mag).all()
            if keys:
                assert np.array_equal(bits(k_rot)[n],
                                      ref.bf16(ref.rotate32(ref.f64(k[n]), cs, pos, d, 0)))
            else:
                assert (bits(k_rot) == 0).all()


@pytest.mark.parametrize("scale0", [1.0, 0.3, 2.0 ** -14, 7e17, 1e-18, 2.0 ** 60, 2.0 ** -60])
@pytest.mark.parametrize("inter", [0, 1])
def test_append_codes_to_the_bit(scale0, inter):
    """Codes, their zeros' signs and scales over every magnitude, quotients at the
    midpoints of two codes among them."""
    H = _h()
    rng = np.random.default_rng(17)
    N, Hkv, d, page, T = 1, 2, 64, 64, 1024
    c = make_cache(rng, N, Hkv, d, page, [T], k_scale=scale0, v_scale=scale0)
    g = OnGpu(c)
    unit = np.exp2(rng.integers(-12, 10, (2, N, T, Hkv, d // 16, 1)))
    x = rng.standard_normal((2, N, T, Hkv, d // 16, 16)) * np.exp2(rng.integers(-3, 1, (16,)))
    at_mids = rng.choice([0, -0.0, .25, .5, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -1.25, -5, 6], x.shape)
    x = np.where(np.arange(T)[:, None, None, None] % 2 == 0, at_mids, x) * unit
    with np.errstate(over="ignore"):
        x = np.clip(x * np.float64(np.float32(scale0)), -3e38, 3e38)
    x[0, 0, 0] = np.where(rng.random(x[0, 0, 0].shape) < 0.5, -0.0, 0.0)
    x[1, 0, 1, :, :, 5] = 3e38                   # past the largest scale
    k, v = ref.bf16(x.astype(np.float32).reshape(2, N, T, Hkv, d))
    cs = ref.angles(T, d)
    dctx = torch.tensor([0], dtype=torch.int32, device="cuda")
    H.herald_kv4_append(H.dims(N, Hkv, Hkv, d, 1, T), T, None, dev(k), dev(v), dctx, g.kv4, None, None,
                        H.rope(dev(cs), d, inter))
    torch.cuda.synchronize()
    rk = ref.rotate32(ref.f64(k[0]), cs, np.arange(T), d, inter)
    c.write(0, np.arange(T), rk, ref.f64(v[0]).astype(np.float32))
    assert np.array_equal(g.scales.cpu().numpy(), c.scales)
    assert np.array_equal(g.codes.cpu().numpy(), c.codes)


def test_append_odd_values():
    """Infinities saturate, a NaN makes its group NaN, tiny groups become zeros,
    tokens without a page are dropped; neighbours stay as they were."""
    H = _h()
    rng = np.random.default_rng(4)
    N, Hkv, d, page, T = 1, 1, 64, 16, 20
    c = make_cache(rng, N, Hkv, d, page, [32])
    c.table[0, 1] = -1
    g = OnGpu(c)
    k = rng.standard_normal((N, T, Hkv, d)).astype(np.float32)
    k[0, 0, 0, 3] = np.inf
    k[0, 1, 0, 20] = -np.inf
    k[0, 2, 0, 40] = np.nan
    k[0, 3] = 1e-6
    k[0, 4] = 3e38
    k[0, 5] *= -0.0
    kb = ref.bf16(k)
    dctx = torch.tensor([0], dtype=torch.int32, device="cuda")
    dm = H.dims(N, 1, Hkv, d, 1, 32)
    H.herald_kv4_append(dm, T, None, dev(kb), dev(kb), dctx, g.kv4, None, None)
    torch.cuda.synchronize()
    c.write(0, np.arange(T), ref.f64(kb[0]).astype(np.float32), ref.f64(kb[0]).astype(np.float32))
    ph = c.table[0, 0]
    got = ref.values(g.codes[0, ph, 0].cpu().numpy(), g.scales[0, ph, 0].cpu().numpy(), 1.0)
    want = c.rows(0, 0, np.arange(16))[0]
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got[2, 32:48]).all()
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))
    assert got[0, 3] == 2688 and got[1, 20] == -2688 and (got[3] == 0).all() and (got[4] == 2688).all()
    others = np.arange(c.n_pages) != ph
    assert np.array_equal(g.codes.cpu().numpy()[:, others], c.codes[:, others])
    assert dctx.tolist() == [0]  # not advanced without the flag


# ----------------------------------------------------------------- gather

@pytest.mark.parametrize("case", [(1, 1, 64, 16, [40], 17), (3, 4, 128, 64, [700, 0, 65], 300),
                                  (2, 2, 128, 128, [129, 1000], 1), (2, 8, 64, 32, [64, 5], 100)],
                         ids=str)
@pytest.mark.parametrize("with_v", [True, False])
def test_gather(case, with_v):
    H = _h()
    N, Hkv, d, page, lengths, P = case
    rng = np.random.default_rng(P)
    c = make_cache(rng, N, Hkv, d, page, lengths, k_scale=0.7, v_scale=1.3)
    g = OnGpu(c)
    L_max = max(lengths)
    idx = np.full((N, Hkv, P), -1, np.int32)
    ns = np.zeros((N, Hkv), np.int32)
    for n in range(N):
        for h in range(Hkv):
            m = min(lengths[n], P - h % 2 if P > 1 else P)
            idx[n, h, :m] = np.sort(rng.permutation(lengths[n])[:m])
            ns[n, h] = m
    if ns[0, 0] > 3:  # the same row twice, rows outside the cache
        idx[0, 0, 1] = idx[0, 0, 2]
        idx[0, 0, 0] = -7
        idx[0, 0, 3] = L_max
    if N > 1 and lengths[1] == 1000:
        ns[1, 0] = 99     # past P: clamped
    dm = H.dims(N, Hkv, Hkv, d, 1, L_max)
    pk = torch.full((N, Hkv, P, d), -1, dtype=torch.int16, device="cuda")
    pv = torch.full_like(pk, -1)
    H.herald_kv4_gather(dm, dev(idx), dev(ns), P, g.kv4, pk, pv if with_v else None)
    torch.cuda.synchronize()
    for i, p in ((0, pk), (1, pv)):
        want = np.zeros((N, Hkv, P, d), np.uint16)
        for n in range(N):
            for h in range(Hkv):
                for r in range(min(ns[n, h], P)):
                    if 0 <= idx[n, h, r] < L_max:
                        want[n, h, r] = ref.bf16(c.rows(i, n, [idx[n, h, r]])[h, 0].astype(np.float32))
        if i and not with_v:
            want[:] = 0xFFFF
        # (code * scale is exact, times k_scale one fp32 rounding: the reference's
        # fp64 product rounded to fp32 is the same number)
        assert np.array_equal(bits(p), want)


# ------------------------------------------------------- a run of them all

def test_blocks_decoded_over_the_cache():
    """Prompts are appended, then two blocks are decoded: rotation for each
    denoising step, block-granular stage 1 over the means the append keeps,
    stage 2 over candidate rows gathered from the cache, the pool gathered
    from it, sparse attention, and the append.  With a budget that covers the
    context the sparse step equals full attention over the cache."""
    H = _h()
    rng = np.random.default_rng(21)
    N, Hq, Hkv, d, B, Bk, page = 2, 8, 2, 128, 16, 32, 64
    prompt = [300, 211]
    L_max = 512
    C_blocks = 12
    Cn, S, W = C_blocks * Bk, 8, 16
    K = Cn
    P = K + S + W
    dm = H.dims(N, Hq, Hkv, d, B, L_max)
    c = ref.Cache(rng, N, Hkv, d, page, [L_max] * N)
    g = OnGpu(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    i16 = dict(dtype=torch.int16, device="cuda")
    rope = H.rope(dev(ref.angles(L_max, d)), d, False)
    ctx = torch.zeros(N, **i32)
    pooled = torch.zeros((N, Hkv, L_max // Bk, d), device="cuda")
    T0 = max(prompt)
    k0, v0 = (dev(ref.bf16(rng.standard_normal((N, T0, Hkv, d)))) for _ in range(2))
    H.herald_kv4_append(dm, T0, None, k0, v0, ctx, g.kv4, None, None, rope,
                        torch.tensor(prompt, **i32), pooled, Bk, H.HERALD_KV4_ADVANCE)
    ws = torch.zeros(H.herald_workspace_size(dm, Cn, P), dtype=torch.uint8, device="cuda")
    ws4 = torch.zeros(H.herald_workspace_size_kv4(dm), dtype=torch.uint8, device="cuda")
    cand, n_cand = torch.zeros((N, Hkv, Cn), **i32), torch.zeros((N, Hkv), **i32)
    idx, n_sel = torch.zeros((N, Hkv, P), **i32), torch.zeros((N, Hkv), **i32)
    staged = torch.zeros((N, Hkv, Cn, d), **i16)
    pk, pv = torch.zeros((N, Hkv, P, d), **i16), torch.zeros((N, Hkv, P, d), **i16)
    out, full = torch.zeros((N, B, Hq, d), **i16), torch.zeros((N, B, Hq, d), **i16)
    q_rot, k_rot = torch.zeros((N, B, Hq, d), **i16), torch.zeros((N, B, Hkv, d), **i16)
    for block in range(2):
        for step in range(2):
            qkv = dev(ref.bf16(rng.standard_normal((N, B, Hq + 2 * Hkv, d))))
            q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
            last = step == 1
            if not last:
                H.herald_kv4_append(dm, B, q, k, None, ctx, None, q_rot, k_rot, rope)
                H.herald_select_stage1_blocks(dm, q_rot, pooled, ctx, Bk, C_blocks, cand, n_cand, ws)
                H.herald_kv4_gather(dm, cand, n_cand, Cn, g.kv4, staged)
                H.herald_select_stage2_staged(dm, q_rot, staged, ctx, cand, n_cand, Cn, K, S, W, P,
                                              idx, n_sel, ws)
                H.herald_kv4_gather(dm, idx, n_sel, P, g.kv4, pk, pv)
            else:
                # the step's rotation and, after the attention, the append of
                # its keys: here one call first, the context not yet advanced
                H.herald_kv4_append(dm, B, q, k, v, ctx, g.kv4, q_rot, k_rot, rope)
            vv = v.contiguous()
            H.herald_denoise_attn(dm, q_rot, pk, pv, n_sel, P, k_rot, vv, out, 0.0, ws)
            H.herald_kv4_attn(dm, q_rot, g.kv4, ctx, k_rot, vv, full, ws=ws4)
            torch.cuda.synchronize()
            L = ctx.tolist()
            assert n_sel.tolist() == [[x] * Hkv for x in L]
            c.codes, c.scales = g.codes.cpu().numpy(), g.scales.cpu().numpy()
            want, tol = ref.attention(bits(q_rot), c, L, bits(k_rot), bits(vv))
            check(ref.f64(bits(full)), want, tol, f"block {block} step {step}: full")
            # the sparse step reads the same rows rounded to bf16 (exact here:
            # 6 significant bits, scales of 1)
            check(ref.f64(bits(out)), want, 2e-2, f"block {block} step {step}: sparse")
        H.herald_kv4_append(dm, B, None, k, v, ctx, g.kv4, None, None, rope, None, pooled, Bk,
                            H.HERALD_KV4_ADVANCE)
        torch.cuda.synchronize()
        assert ctx.tolist() == [x + B * (block + 1) for x in prompt]
        # the means equal those of the rows as held
        c.codes, c.scales = g.codes.cpu().numpy(), g.scales.cpu().numpy()
        for n, L in enumerate(ctx.tolist()):
            rows = c.rows(0, n, np.arange(L))
            for b in range(-(-L // Bk)):
                mean = rows[:, b * Bk:min(L, (b + 1) * Bk)].mean(1)
                assert np.abs(pooled[n, :, b].cpu().numpy() - mean).max() <= 40 * 2.0 ** -24 * Bk
    assert H.herald_workspace_error(ws) == 0
