"""The 8-bit cache's reference against itself and torch, and the calls' refusals (no GPU)."""
import ctypes as C

import numpy as np
import pytest

import kv4_ref
import kv8_ref as ref
from block_diffusion_sparse_gb300 import herald as H

torch = pytest.importorskip("torch")


def test_codes_against_torch():
    x = np.concatenate([np.linspace(-460, 460, 9001), np.geomspace(1e-5, 500, 4000),
                        ref._MIDS, -ref._MIDS, [0.0, -0.0]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3(x), want)
    assert ref.e4m3(np.nan) == 0x7F and ref.e4m3(np.inf) == 0x7E and ref.e4m3(-np.inf) == 0xFE


@pytest.mark.parametrize("top,e", [(448.0, 0), (449.0, 1), (0.0, -32), (1.75, -8), (1.76, -7),
                                   (1e30, 32), (1e-30, -32), (224.5, 0), (224.0, -1)])
def test_exponent(top, e):
    assert ref.need([0.0, -top]) == e
    assert ref.need([top, np.inf, np.nan]) == e


def test_older_rows_follow_a_growing_scale():
    rng = np.random.default_rng(0)
    c = ref.Cache(rng, 1, 1, 64, 32, 32, [32])
    a = kv4_ref.f64(kv4_ref.bf16(rng.standard_normal((5, 1, 64))))
    c.write(0, 0, a, a)
    before, e0 = c.rows(0, 0, range(5)), c.exps(0, 0, [0])[0, 0]
    c.write(0, 5, 100 * a[:1], a[:1])
    e1 = c.exps(0, 0, [0])[0, 0]
    assert e1 > e0 and c.exps(1, 0, [0])[0, 0] == e0
    step = 2.0 ** (e1 - 9)  # e4m3's subnormals under the new scale
    assert np.abs(c.rows(0, 0, range(5)) - before).max() <= step / 2
    assert np.array_equal(c.rows(1, 0, range(5)), before)
    # a block begins anew with its first row
    c.write(0, 0, 1e-3 * a, a)
    assert c.exps(0, 0, [0])[0, 0] < e0


# ------------------------------------------------------------- refusals, by address

class Raw:
    """A cache struct of plain addresses: the checks come before any of them is used."""

    def __init__(self, **kw):
        f = dict(page=64, block=32, n_pages=4, max_pages=16, table=0x1000, k_codes=0x2000, k_scales=0x3000,
                 v_codes=0x4000, v_scales=0x5000)
        f.update(kw)
        self.s = H.Kv8(*f.values())


def dims(**kw):
    f = dict(N=2, Hq=8, Hkv=2, d=128, B=1, L_max=1024)
    f.update(kw)
    return H.dims(**f)


def attn(cache=None, d=None, scale=0.0, ws_bytes=1 << 40, bk=0x7000, bv=0x8000, q=0x6000, out=0x9000):
    H.herald_kv8_attn(d or dims(), q, (cache or Raw()).s, 0xA000, bk, bv, out, scale, 0xB000, ws_bytes)


def append(cache=None, d=None, T=3, q=0x100000, k=0x200000, v=0x300000, q_rot=0x400000,
           k_rot=0x500000, **kw):
    c = Raw().s if cache is None else cache.s if isinstance(cache, Raw) else None
    H.herald_kv8_append(d or dims(), T, q, k, v, 0xA000, c, q_rot, k_rot, **kw)


BAD_CACHES = [(dict(page=48), 2), (dict(page=8), 2), (dict(page=256), 2), (dict(block=8), 2),
              (dict(block=128), 2), (dict(block=48), 2), (dict(block=0), 2), (dict(page=16), 2),
              (dict(n_pages=0), 1), (dict(max_pages=15), 1), (dict(max_pages=0), 1),
              (dict(table=None), 1), (dict(k_codes=0x2008), 1), (dict(v_scales=None), 1),
              (dict(k_scales=None), 1), (dict(v_codes=None), 1)]


@pytest.mark.parametrize("bad,status", BAD_CACHES, ids=str)
def test_refused_caches(bad, status):
    for call in (lambda: attn(Raw(**bad)), lambda: append(Raw(**bad)),
                 lambda: H.herald_kv8_gather(dims(), 0x6000, 0x7000, 8, Raw(**bad).s, 0x8000, None)):
        with pytest.raises(H.HeraldError) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("kw,status", [
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(ws_bytes=1000), 3), (dict(bk=None), 1), (dict(bv=None), 1), (dict(q=0x6002), 1),
    (dict(out=None), 1), (dict(out=0x6000), 1), (dict(out=0x6ff0), 1), (dict(out=0x7000), 1),
    (dict(out=0x8010), 1), (dict(bk=0x7008), 1), (dict(d=dims(d=96)), 2), (dict(d=dims(B=65)), 2),
    (dict(d=dims(N=32768)), 2), (dict(d=dims(L_max=(1 << 30) + 1, N=1, Hkv=1)), 2)], ids=str)
def test_refused_attention(kw, status):
    with pytest.raises(H.HeraldError) as e:
        attn(**kw)
    assert e.value.status == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(q=None, k=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(q_rot=None), 1), (dict(flags=2), 1), (dict(q_ld=1020), 1), (dict(k_ld=252), 1),
    (dict(v_ld=8), 1), (dict(pooled=0x600000, Bk=0), 1), (dict(cache=0, flags=1), 1),
    (dict(cache=0, k_rot=None), 1), (dict(cache=0, pooled=0x600000, Bk=64), 1),
    (dict(k_rot=0x300000), 1), (dict(q_rot=0x200000), 1), (dict(q_rot=0x100000, q_ld=2048), 1),
    (dict(T=(1 << 30) + 1), 2), (dict(rope=H.Rope(0x700000, 1024, 48, 0)), 2),
    (dict(rope=H.Rope(0x700000, 1023, 64, 0)), 1), (dict(rope=H.Rope(0x700000, 1024, 64, 2)), 1),
    (dict(rope=H.Rope(None, 1024, 64, 0)), 1)], ids=str)
def test_refused_appends(kw, status):
    with pytest.raises(H.HeraldError) as e:
        append(**kw)
    assert e.value.status == status


def test_workspace_size():
    assert H.herald_workspace_size_kv8(dims(d=96)) == 0
    assert H.herald_workspace_size_kv8(dims()) > 0
    assert H.herald_workspace_size_kv8(dims(B=64)) > H.herald_workspace_size_kv8(dims())


def test_binding_checks_the_cache():
    u8 = dict(dtype=torch.uint8)
    table = torch.zeros((2, 4), dtype=torch.int32)
    codes, scales = torch.zeros((2, 8, 2, 64, 128), **u8), torch.zeros((2, 8, 2, 2), **u8)
    c = H.kv8(64, 32, table, codes[0], scales[0], codes[1], scales[1])
    assert (c.page, c.block, c.n_pages, c.max_pages) == (64, 32, 8, 4)
    bad = [(64, 16, table, codes[0], scales[0], codes[1], scales[1]),
           (32, 32, table, codes[0], scales[0], codes[1], scales[1]),
           (64, 32, table.long(), codes[0], scales[0], codes[1], scales[1]),
           (64, 32, table, codes[0].transpose(0, 1), scales[0], codes[1], scales[1]),
           (64, 32, table, codes[0], scales[0], codes[1][:4], scales[1]),
           (64, 32, table, codes[0], scales[0][:, :1].contiguous(), codes[1], scales[1]),
           (64, 32, table, codes[0].int(), scales[0], codes[1], scales[1])]
    for args in bad:
        with pytest.raises(ValueError):
            H.kv8(*args)
    q = torch.zeros((2, 1, 8, 128), dtype=torch.bfloat16)
    for other in (dims(Hkv=4), dims(d=64), dims(N=3)):  # a cache of another shape
        with pytest.raises(ValueError):
            H.herald_kv8_attn(other, 0x6000, c, 0xA000, None, None, 0x9000, ws=0xB000, ws_bytes=1 << 40)
    with pytest.raises(ValueError):  # queries of another shape
        H.herald_kv8_attn(dims(), q[:, :, :4], c, 0xA000, None, None, q, ws=0xB000, ws_bytes=1 << 40)
    with pytest.raises(ValueError):  # two sequences' lengths are wanted
        H.herald_kv8_attn(dims(), q, c, torch.zeros(1, dtype=torch.int32), None, None, q, ws=0xB000,
                          ws_bytes=1 << 40)
    with pytest.raises(C.ArgumentError):  # a 4-bit cache
        H.herald_kv8_gather(dims(), 0x6000, 0x7000, 8, H.Kv4(), 0x8000)
    with pytest.raises(C.ArgumentError):
        H.herald_kv4_gather(dims(), 0x6000, 0x7000, 8, c, 0x8000)


def test_launch_failures_are_reported():
    for fn, name in ((attn, "kv8 attention launch"), (append, "kv8 append launch"),
                     (lambda: H.herald_kv8_gather(dims(), 0x6000, 0x7000, 8, Raw().s, 0x8000, None),
                      "kv8 gather launch")):
        H.herald_inject_launch_failure(0)
        with pytest.raises(H.HeraldError) as e:
            fn()
        H.herald_inject_launch_failure(-1)
        assert e.value.status == 4
        assert name in str(e.value) or not torch.cuda.is_available()
