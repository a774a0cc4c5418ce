"""The paged 4-bit cache as a server would use it: a decoding loop captured once
and replayed, two calls at once, pages shared by sequences, a cache past 2^32
bytes, many sequences, and the debug build's device checks."""
import os
import subprocess
import sys

import numpy as np
import pytest

import kv4_ref as ref
from helpers import dev
from test_gpu_kv4 import OnGpu, _h, bits, check, make_cache, run_attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
BAD_INDEX, BAD_COUNT = 0x10, 0x20


def test_a_captured_decoding_loop():
    """One token a step: rotation, append, advance and attention in one graph,
    replayed; a sequence that has reached L_max stays there."""
    H = _h()
    rng = np.random.default_rng(31)
    N, Hq, Hkv, d, page, steps = 3, 8, 2, 64, 16, 21
    start, L_max = [0, 14, 40], 50
    c = make_cache(rng, N, Hkv, d, page, [L_max] * N)
    g = OnGpu(c)
    cs = ref.angles(L_max, d)
    rope = H.rope(dev(cs), d, True)
    qkv = ref.bf16(rng.standard_normal((steps, N, 1, Hq + 2 * Hkv, d)))
    x = dev(qkv[0])
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    ctx = torch.tensor(start, dtype=torch.int32, device="cuda")
    q_rot = torch.zeros((N, 1, Hq, d), dtype=torch.int16, device="cuda")
    k_rot = torch.zeros((N, 1, Hkv, d), dtype=torch.int16, device="cuda")
    out = torch.zeros((N, 1, Hq, d), dtype=torch.int16, device="cuda")
    dm = H.dims(N, Hq, Hkv, d, 1, L_max)
    ws = torch.zeros(H.herald_workspace_size_kv4(dm), dtype=torch.uint8, device="cuda")

    def step():
        st = torch.cuda.current_stream()
        H.herald_kv4_append(dm, 1, q, k, v, ctx, g.kv4, q_rot, k_rot, rope,
                            flags=H.HERALD_KV4_ADVANCE, stream=st)
        H.herald_kv4_attn(dm, q_rot, g.kv4, ctx, None, None, out, ws=ws, stream=st)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert ctx.tolist() == start  # captured, not run
    L = list(start)
    for s in range(steps):
        x.copy_(dev(qkv[s]))
        graph.replay()
        torch.cuda.synchronize()
        for n in range(N):
            if L[n] < L_max:
                rows = ref.rotate32(ref.f64(qkv[s, n, :, Hq:Hq + Hkv]), cs, np.array([L[n]]), d, True)
                c.write(n, [L[n]], rows, ref.f64(qkv[s, n, :, Hq + Hkv:]).astype(np.float32))
                L[n] += 1
        assert ctx.tolist() == L
        assert np.array_equal(g.codes.cpu().numpy(), c.codes)
        assert np.array_equal(g.scales.cpu().numpy(), c.scales)
        want, tol = ref.attention(bits(q_rot), c, L)
        check(ref.f64(bits(out)), want, tol, f"step {s}")
    assert H.herald_workspace_error(ws) == 0


@pytest.mark.parametrize("B", [1, 32])
def test_two_calls_at_once(B):
    """Two streams, a workspace each, the same cache: each result is what the
    call gives alone, bit for bit."""
    H = _h()
    rng = np.random.default_rng(32)
    N, Hq, Hkv, d, L = 2, 16, 4, 128, 3000
    c = make_cache(rng, N, Hkv, d, 64, [L, 1234])
    g = OnGpu(c)
    dm = H.dims(N, Hq, Hkv, d, B, L)
    ctx = torch.tensor([L, 1234], dtype=torch.int32, device="cuda")
    qs = [dev(ref.bf16(rng.standard_normal((N, B, Hq, d)))) for _ in range(2)]
    ws = [torch.zeros(H.herald_workspace_size_kv4(dm), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    alone = [torch.zeros((N, B, Hq, d), dtype=torch.int16, device="cuda") for _ in range(2)]
    for i in range(2):
        H.herald_kv4_attn(dm, qs[i], g.kv4, ctx, None, None, alone[i], ws=ws[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(alone[0]) for _ in range(6)] for _ in range(2)]
    torch.cuda.synchronize()
    for r in range(6):
        for i in range(2):
            H.herald_kv4_attn(dm, qs[i], g.kv4, ctx, None, None, outs[i][r], ws=ws[i],
                              stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert H.herald_workspace_error(ws[i]) == 0
        for o in outs[i]:
            assert torch.equal(o, alone[i])


@pytest.mark.parametrize("B", [1, 8])
def test_sequences_may_share_pages(B):
    """A prefix held once: several tables name its pages."""
    rng = np.random.default_rng(33)
    N, Hq, Hkv, d, page = 3, 8, 2, 128, 32
    c = make_cache(rng, N, Hkv, d, page, [400, 400, 400])
    c.table[1, :6] = c.table[0, :6]
    c.table[2, :6] = c.table[0, :6]
    q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
    lengths = [400, 190, 333]
    want, tol = ref.attention(q, c, lengths)
    check(run_attn(c, q, lengths, B, 400), want, tol, "shared")


@pytest.mark.parametrize("case", [(70, 8, 2, 64, 8, 16, 90), (33, 16, 4, 128, 4, 32, 200),
                                  (65, 6, 6, 64, 17, 128, 257)], ids=str)
def test_attention_of_many_sequences(case):
    """More sequences than a warp has lanes; lengths that end inside a tile."""
    N, Hq, Hkv, d, B, page, top = case
    rng = np.random.default_rng(N)
    lengths = [int(x) for x in rng.integers(0, top, N)]
    lengths[3] = lengths[-2] = 0
    c = make_cache(rng, N, Hkv, d, page, lengths)
    q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
    bk, bv = (ref.bf16(rng.standard_normal((N, B, Hkv, d))) for _ in range(2))
    for b in (None, 1):
        want, tol = ref.attention(q, c, lengths, bk if b else None, bv if b else None)
        got = run_attn(c, q, lengths, B, max(lengths), bk if b else None, bv if b else None)
        check(got, want, tol, f"{case}, block {b}")


def test_offsets_past_32_bits():
    """Pages at the end of arrays of more than 2^32 bytes: append, attention with
    few and with many rows, gather."""
    H = _h()
    rng = np.random.default_rng(34)
    N, Hq, Hkv, d, page, pages = 1, 8, 8, 128, 128, 70000
    T, P = 200, 64
    need = pages * Hkv * page * (d // 2 + d // 16) * 2 + (1 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("needs 11 GB")
    c = ref.Cache(rng, N, Hkv, d, page, [T])
    codes = torch.zeros((2, pages, Hkv, page, d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, pages, Hkv, page, d // 16), dtype=torch.uint8, device="cuda")
    assert codes[0].numel() > 1 << 32
    table = dev((pages - 1 - c.table).astype(np.int32))
    kv4 = H.kv4(page, table, codes[0], scales[0], codes[1], scales[1], 1.0, 1.0)
    k, v = (ref.bf16(rng.standard_normal((N, T, Hkv, d))) for _ in range(2))
    ctx = torch.zeros(N, dtype=torch.int32, device="cuda")
    H.herald_kv4_append(H.dims(N, Hq, Hkv, d, 1, T), T, None, dev(k), dev(v), ctx, kv4, None, None,
                        flags=H.HERALD_KV4_ADVANCE)
    c.write(0, np.arange(T), ref.f64(k[0]).astype(np.float32), ref.f64(v[0]).astype(np.float32))
    for j, ph in enumerate(c.table[0]):
        rows = min(page, T - j * page)
        held = codes[:, pages - 1 - int(ph), :, :rows].cpu().numpy()
        assert np.array_equal(held, c.codes[:, ph, :, :rows])
    for B in (1, 32):
        dm = H.dims(N, Hq, Hkv, d, B, T)
        q = ref.bf16(rng.standard_normal((N, B, Hq, d)))
        ws = torch.zeros(H.herald_workspace_size_kv4(dm), dtype=torch.uint8, device="cuda")
        out = torch.zeros((N, B, Hq, d), dtype=torch.int16, device="cuda")
        H.herald_kv4_attn(dm, dev(q), kv4, ctx, None, None, out, ws=ws)
        want, tol = ref.attention(q, c, [T])
        check(ref.f64(bits(out)), want, tol, f"B {B}")
        assert H.herald_workspace_error(ws) == 0
    idx = rng.integers(0, T, (N, Hkv, P)).astype(np.int32)
    n_sel = torch.full((N, Hkv), P, dtype=torch.int32, device="cuda")
    pk = torch.zeros((N, Hkv, P, d), dtype=torch.int16, device="cuda")
    pv = torch.zeros_like(pk)
    H.herald_kv4_gather(H.dims(N, Hq, Hkv, d, 1, T), dev(idx), n_sel, P, kv4, pk, pv)
    torch.cuda.synchronize()
    for i, t in enumerate((pk, pv)):
        for h in range(Hkv):
            assert np.array_equal(bits(t)[0, h], ref.bf16(c.rows(i, 0, idx[0, h])[h]))


def run_debug(out_path):
    """In the debug library: valid calls, then a position without a page, a length
    past L_max, a count past T and a selected row without a page, all inside their
    allocations; saves the check word after each."""
    H = _h()
    rng = np.random.default_rng(35)
    N, Hq, Hkv, d, page, L = 2, 8, 2, 128, 32, 300
    c = make_cache(rng, N, Hkv, d, page, [L, L])
    g = OnGpu(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx = torch.tensor([L - 40, 100], **i32)
    words = {"debug": int(H.herald_debug_build())}

    def attn(B, name):
        dm = H.dims(N, Hq, Hkv, d, B, L)
        q = torch.zeros((N, B, Hq, d), dtype=torch.int16, device="cuda")
        ws = torch.zeros(H.herald_workspace_size_kv4(dm), dtype=torch.uint8, device="cuda")
        H.herald_kv4_attn(dm, q, g.kv4, ctx, None, None, torch.zeros_like(q), ws=ws)
        torch.cuda.synchronize()
        words[f"{name}_{B}"] = H.herald_debug_status()

    def append(n_tok, name):
        x = torch.zeros((N, 8, Hkv, d), dtype=torch.int16, device="cuda")
        pooled = torch.zeros((N, Hkv, -(-L // 32), d), device="cuda")
        H.herald_kv4_append(H.dims(N, Hq, Hkv, d, 1, L), 8, None, x, x, ctx, g.kv4, None, None,
                            n_tok=n_tok, pooled=pooled, Bk=32)
        torch.cuda.synchronize()
        words[name] = H.herald_debug_status()

    def gather(name):
        idx = torch.arange(64, **i32).repeat(N * Hkv).view(N, Hkv, 64)
        n_sel = torch.full((N, Hkv), 64, **i32)
        pk = torch.zeros((N, Hkv, 64, d), dtype=torch.int16, device="cuda")
        H.herald_kv4_gather(H.dims(N, Hq, Hkv, d, 1, L), idx, n_sel, 64, g.kv4, pk)
        torch.cuda.synchronize()
        words[name] = H.herald_debug_status()

    H.herald_debug_status()
    attn(1, "valid"), attn(32, "valid")
    append(None, "append_valid"), gather("gather_valid")
    append(torch.tensor([9, 3], **i32), "count")
    ctx.copy_(torch.tensor([L + 5, 100], **i32))
    attn(1, "length"), attn(32, "length")
    ctx.copy_(torch.tensor([L - 40, 100], **i32))
    g.table[0, 1] = -1
    attn(1, "page"), attn(32, "page")
    gather("gather_page")
    ctx.copy_(torch.tensor([30, 100], **i32))
    append(None, "append_page")
    np.savez(out_path, **{k: np.int64(v) for k, v in words.items()})


def test_debug_build_checks(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_diffusion_sparse_gb300 import build
    assert os.path.exists(build.DEBUG_LIB), "the debug build is made by __graft_entry__.build()"
    out = str(tmp_path / "kv4.npz")
    code = (f"import sys; sys.path[:0] = [{HERE!r}, {ROOT!r}]; "
            f"import test_gpu_kv4_use as t; t.run_debug({out!r})")
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, HERALD_LIB="debug"),
                       cwd=HERE, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    w = {k: int(v) for k, v in np.load(out).items()}
    assert w["debug"] == 1
    for k in ("valid_1", "valid_32", "append_valid", "gather_valid"):
        assert w[k] == 0, f"{k}: {w[k]:#x}"
    assert w["count"] & BAD_COUNT
    assert w["length_1"] & BAD_COUNT and w["length_32"] & BAD_COUNT
    for k in ("page_1", "page_32", "gather_page", "append_page"):
        assert w[k] & BAD_INDEX, k
