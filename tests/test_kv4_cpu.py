"""The paged 4-bit cache on the host: its reference's number formats, and the
refusals of the calls (each returns before any CUDA call)."""
import ctypes as C
import os

import numpy as np
import pytest

import kv4_ref as ref
from block_diffusion_sparse_gb300 import herald as H

OK = 1 << 12  # an aligned address that these paths never follow


def _built():
    if not os.path.exists(H.LIB_PATH):
        from block_diffusion_sparse_gb300 import build
        build.build()
    return H.lib()


def _cache(**over):
    a = dict(page=64, n_pages=40, max_pages=32, table=OK, k_codes=OK, k_scales=OK, v_codes=OK,
             v_scales=OK, k_scale=1.0, v_scale=1.0)
    a.update(over)
    return H.Kv4(*a.values())


def test_reference_formats():
    torch = pytest.importorskip("torch")
    b = torch.arange(256, dtype=torch.uint8)
    want = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(want), np.isnan(ref.E4M3))
    assert np.array_equal(np.nan_to_num(want), np.nan_to_num(ref.E4M3))
    # every midpoint of two codes goes to the even one; past 6 saturates
    x = np.zeros(16, np.float32)
    x[:12] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -5, -.25, .26, 4.99]
    c, s = ref.quantise(x, 1.0)
    assert ref.values(c, s, 1.0)[:12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4, 0, .5, 4]
    # the scale of a group is its largest magnitude / 6
    c, s = ref.quantise(np.full(16, 3.0, np.float32), 1.0)
    assert ref.E4M3[s[0]] == 0.5 and (ref.values(c, s, 1.0) == 3).all()


CACHE_FAULTS = [(dict(page=48), 2), (dict(page=256), 2), (dict(n_pages=0), 1),
                (dict(max_pages=31), 1), (dict(table=0), 1), (dict(k_codes=OK + 8), 1),
                (dict(v_scales=0), 1), (dict(k_scale=0.0), 1), (dict(v_scale=float("nan")), 1),
                (dict(v_scale=2.0 ** 61), 1)]


@pytest.mark.parametrize("over,status", CACHE_FAULTS)
def test_bad_caches_rejected(over, status):
    _built()
    d = H.dims(2, 8, 2, 128, 4, 2048)
    c = _cache(**over)
    ws = H.herald_workspace_size_kv4(d)
    for call in (lambda: H.herald_kv4_attn(d, OK, c, OK, OK, OK, OK, ws=OK, ws_bytes=ws),
                 lambda: H.herald_kv4_gather(d, OK, OK, 64, c, OK, OK),
                 lambda: H.herald_kv4_append(d, 4, OK, OK, OK, OK, c, OK, OK)):
        with pytest.raises(H.HeraldError) as e:
            call()
        assert e.value.status == status, e.value
        assert H.lib().herald_last_error().decode()


@pytest.mark.parametrize("over,status", [
    (dict(q=0), 1), (dict(cache=None), 1), (dict(ctx=OK + 4), 1), (dict(bk=None), 1),
    (dict(bv=None), 1), (dict(bk=OK + 2), 1), (dict(out=0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(ws=0), 1),
    (dict(ws_bytes=-1), 3)])
def test_attention_refusals(over, status):
    _built()
    d = H.dims(2, 8, 2, 128, 4, 2048)
    need = H.herald_workspace_size_kv4(d)
    assert need > 0
    a = dict(q=OK, cache=_cache(), ctx=OK, bk=OK, bv=OK, out=OK, scale=0.0, ws=OK, ws_bytes=0)
    a.update(over)
    with pytest.raises(H.HeraldError) as e:
        H.herald_kv4_attn(d, a["q"], a["cache"], a["ctx"], a["bk"], a["bv"], a["out"], a["scale"],
                          a["ws"], need + a["ws_bytes"])
    assert e.value.status == status, e.value


@pytest.mark.parametrize("bad,status", [(dict(d=96), 2), (dict(Hq=9), 2), (dict(Hq=18), 2),
                                        (dict(B=65), 2), (dict(N=0), 1),
                                        (dict(N=40000, L_max=8), 2),
                                        (dict(N=1, Hq=1, Hkv=1, L_max=(1 << 30) + 1), 2)])
def test_shapes_rejected(bad, status):
    _built()
    a = dict(N=2, Hq=8, Hkv=2, d=128, B=4, L_max=2048)
    a.update(bad)
    d = H.dims(**a)
    assert H.herald_workspace_size_kv4(d) == 0
    with pytest.raises(H.HeraldError) as e:
        H.herald_kv4_attn(d, OK, _cache(), OK, OK, OK, OK, ws=OK, ws_bytes=1 << 40)
    assert e.value.status == status


@pytest.mark.parametrize("over,status", [
    (dict(T=0), 1), (dict(T=1 << 30), 2), (dict(q=None, k=None), 1), (dict(q=OK + 8), 1),
    (dict(q_rot=None), 1), (dict(cache=None, k_rot=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(ctx=None), 1), (dict(n_tok=OK + 4), 1), (dict(flags=2), 1),
    (dict(cache=None, flags=1), 1), (dict(cache=None, pooled=OK, Bk=64), 1),
    (dict(pooled=OK, Bk=0), 1), (dict(pooled=OK, Bk=(1 << 30) + 1), 1), (dict(pooled=OK + 8, Bk=64), 1),
    (dict(q_ld=1000), 1), (dict(k_ld=257), 1), (dict(v_ld=-8), 1),
    (dict(q=OK, q_rot=OK, q_ld=2048), 1), (dict(k=OK, k_rot=OK, k_ld=2048), 1),
    (dict(rope=dict(cos_sin=0)), 1), (dict(rope=dict(rot=48)), 2), (dict(rope=dict(rot=0)), 2),
    (dict(rope=dict(rot=160)), 2), (dict(rope=dict(n_pos=2047)), 1),
    (dict(rope=dict(interleaved=2)), 1)])
def test_append_refusals(over, status):
    _built()
    d = H.dims(2, 8, 2, 128, 4, 2048)
    a = dict(T=4, q=OK, k=OK * 2, v=OK * 3, ctx=OK, cache=_cache(), q_rot=OK * 4, k_rot=OK * 5,
             n_tok=None, pooled=None, Bk=0, flags=0, q_ld=0, k_ld=0, v_ld=0, rope=None)
    a.update(over)
    if isinstance(a["rope"], dict):
        r = dict(cos_sin=OK, n_pos=2048, rot=64, interleaved=0)
        r.update(a["rope"])
        a["rope"] = H.Rope(*r.values())
    with pytest.raises(H.HeraldError) as e:
        H.herald_kv4_append(d, a["T"], a["q"], a["k"], a["v"], a["ctx"], a["cache"], a["q_rot"],
                            a["k_rot"], a["rope"], a["n_tok"], a["pooled"], a["Bk"], a["flags"],
                            a["q_ld"], a["k_ld"], a["v_ld"])
    assert e.value.status == status, e.value


@pytest.mark.parametrize("over", [dict(q_rot=2), dict(q_rot=3), dict(q_rot=5), dict(k_rot=1),
                                  dict(k_rot=3)])
def test_append_outputs_over_other_inputs_rejected(over):
    """A rotated output may lie over its own input, not over one that others still read."""
    _built()
    d = H.dims(2, 8, 2, 128, 4, 2048)
    a = dict(q=1, k=2, v=3, q_rot=4, k_rot=5)
    a.update(over)
    q, k, v, q_rot, k_rot = (OK * x for x in a.values())
    with pytest.raises(H.HeraldError) as e:
        H.herald_kv4_append(d, 4, q, k, v, OK * 7, _cache(), q_rot, k_rot)
    assert e.value.status == 1, e.value


def test_append_counts_rejected():
    """Token positions and head counts that launches or 32-bit positions do not hold."""
    _built()
    c = _cache(max_pages=1 << 25)
    for d, T in ((H.dims(1, 1, 1, 64, 1, 1 << 30), (1 << 30) + 1),
                 (H.dims(1, 8 * 7000, 7000, 64, 1, 16), 4)):
        with pytest.raises(H.HeraldError) as e:
            H.herald_kv4_append(d, T, OK, OK * 2, OK * 3, OK, c, OK * 4, OK * 5)
        assert e.value.status == 2, e.value


@pytest.mark.parametrize("over,status", [(dict(idx=0), 1), (dict(n_sel=OK + 4), 1), (dict(P=0), 1),
                                         (dict(P=1 << 30), 2), (dict(pk=None), 1),
                                         (dict(pv=OK + 2), 1), (dict(cache=None), 1)])
def test_gather_refusals(over, status):
    _built()
    a = dict(idx=OK, n_sel=OK, P=64, cache=_cache(), pk=OK, pv=OK)
    a.update(over)
    with pytest.raises(H.HeraldError) as e:
        H.herald_kv4_gather(H.dims(2, 8, 2, 128, 4, 2048), a["idx"], a["n_sel"], a["P"],
                            a["cache"], a["pk"], a["pv"])
    assert e.value.status == status, e.value


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    u8 = dict(dtype=torch.uint8)
    c, s = torch.zeros(5, 2, 16, 64, **u8), torch.zeros(5, 2, 16, 8, **u8)
    t = torch.zeros(3, 4, dtype=torch.int32)
    k = H.kv4(16, t, c, s, c, s, 1.0, 0.5)
    assert (k.n_pages, k.max_pages, k.page) == (5, 4, 16) and k.v_scale == 0.5
    for bad in ((32, t, c, s, c, s), (16, t, c, c, c, s), (16, t, c, s, c[:4], s),
                (16, t.long(), c, s, c, s), (16, t, c.transpose(0, 1), s, c, s)):
        with pytest.raises(ValueError):
            H.kv4(*bad)
    with pytest.raises(ValueError):
        H.rope(torch.zeros(10, 16, 2), 64)
    qkv = torch.zeros(2, 3, 6, 128, dtype=torch.bfloat16)
    assert H._token_ld(qkv[:, :, :4], None, "q") == 6 * 128
    assert H._token_ld(qkv[:, :, :4].contiguous(), None, "q") == 4 * 128
    assert H._token_ld(qkv[:, :1, 4:], None, "k") == 3 * 6 * 128
    assert H._token_ld(qkv[:1, :1, 4:], None, "k") == 2 * 128
    for bad in (qkv[..., ::2], qkv[:, :, ::2], qkv[:, :2, :4]):
        with pytest.raises(ValueError):
            H._token_ld(bad, None, "q")


def test_binding_checks_token_counts():
    """Tensors of another N or T than the call's would be read at wrong strides."""
    torch = pytest.importorskip("torch")
    _built()
    d = H.dims(2, 4, 2, 64, 1, 64)
    x = torch.zeros(2, 6, 2, 64, dtype=torch.bfloat16)
    cache = _cache(max_pages=4, page=16)
    for T, k in ((5, x), (7, x), (6, x[:1])):
        with pytest.raises(ValueError):
            H.herald_kv4_append(d, T, None, k, k, OK, cache, None, None)
    one = H.dims(1, 4, 2, 64, 1, 64)
    with pytest.raises(ValueError):
        H.herald_kv4_append(one, 7, None, x[:1], x[:1], OK, cache, None, None)


@pytest.mark.gpu
def test_launch_failures_are_reported():
    torch = pytest.importorskip("torch")
    d = H.dims(1, 4, 1, 64, 1, 32)
    u8 = dict(dtype=torch.uint8, device="cuda")
    c, s = torch.zeros(2, 1, 16, 32, **u8), torch.zeros(2, 1, 16, 4, **u8)
    kv = H.kv4(16, torch.arange(2, dtype=torch.int32, device="cuda")[None], c, s, c.clone(), s.clone())
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(H.herald_workspace_size_kv4(d), **u8)
    for after in (0, 1):
        H.herald_inject_launch_failure(after)
        with pytest.raises(H.HeraldError) as e:
            H.herald_kv4_attn(d, q, kv, ctx, None, None, out, ws=ws)
        assert e.value.status == 4 and "kv4 attention" in str(e.value)
    H.herald_kv4_attn(d, q, kv, ctx, None, None, out, ws=ws)
    torch.cuda.synchronize()
    assert (out == 0).all()
