"""What the binding of the paged 4-bit cache's calls refuses before any of
them reaches the library: tensors that would be read or written elsewhere than
where they lie."""
import os

import pytest

from block_diffusion_sparse_gb300 import herald as H

torch = pytest.importorskip("torch")

OK = 1 << 12  # an aligned address that these paths never follow


@pytest.mark.parametrize("shape", [(3, 1, 2, 64), (3, 4, 2, 64), (1, 9, 2, 64)], ids=str)
def test_broadcast_tokens_are_refused(shape):
    """A token stride of 0 means dense to the call: a broadcast view would be
    read past its only row."""
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16).expand(*shape)
    N, T = shape[:2]
    d = H.dims(N, 2, 2, 64, 1, 64)
    with pytest.raises(ValueError, match="broadcast"):
        H.herald_kv4_append(d, T, None, x, x, OK, None, None, OK)
    with pytest.raises(ValueError, match="broadcast"):
        H.herald_kv4_append(d, T, x, None, None, OK, None, OK, None)


def test_overlapping_tokens_are_refused():
    x = torch.zeros(4096, dtype=torch.bfloat16).as_strided((1, 4, 2, 64), (512, 64, 64, 1))
    with pytest.raises(ValueError, match="overlap"):
        H.herald_kv4_append(H.dims(1, 2, 2, 64, 1, 64), 4, x, None, None, OK, None, OK, None)


def test_addresses_cross_without_a_failed_look_up():
    """Raw addresses and streams are taken as they are: looking for a tensor's
    attribute on each made a call of a dozen addresses 5 us longer."""
    class Address(int):
        def __getattr__(self, name):
            raise AssertionError(f"looked for {name}")

    assert H._p(Address(OK)) == OK and H._s(Address(7)) == 7 and H._s(None) is None
    for f in (H._p, H._s):
        with pytest.raises(TypeError):
            f(1.5)


def _cache(N=2, Hkv=2, d=64, page=16, max_pages=4):
    u8 = dict(dtype=torch.uint8)
    c, s = torch.zeros(3, Hkv, page, d // 2, **u8), torch.zeros(3, Hkv, page, d // 16, **u8)
    return H.kv4(page, torch.zeros(N, max_pages, dtype=torch.int32), c, s, c.clone(), s.clone())


@pytest.mark.parametrize("other", [dict(Hkv=4), dict(Hkv=1), dict(d=128), dict(N=3)], ids=str)
def test_caches_of_another_shape_are_refused(other):
    """A cache of fewer heads, channels or sequences than the call's would be
    reached past its end; one of more would be read at wrong rows."""
    a = dict(N=2, Hq=8, Hkv=2, d=64, B=1, L_max=64)
    a.update(other)
    d, c = H.dims(**a), _cache()
    for call in (lambda: H.herald_kv4_append(d, 4, OK, OK * 9, OK * 17, OK, c, OK * 25, OK * 33),
                 lambda: H.herald_kv4_attn(d, OK, c, OK, None, None, OK, ws=OK, ws_bytes=1 << 40),
                 lambda: H.herald_kv4_gather(d, OK, OK, 8, c, OK)):
        with pytest.raises(ValueError, match="cache"):
            call()


def _bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _attn(**over):
    d = H.dims(2, 8, 2, 64, 3, 64)
    a = dict(q=_bf16(2, 3, 8, 64), ctx=_i32(2), bk=_bf16(2, 3, 2, 64), bv=_bf16(2, 3, 2, 64),
             out=_bf16(2, 3, 8, 64))
    a.update(over)
    # (no workspace: what passes the binding is refused by the library)
    H.herald_kv4_attn(d, a["q"], _cache(), a["ctx"], a["bk"], a["bv"], a["out"], ws=0, ws_bytes=0)


def _gather(**over):
    a = dict(idx=_i32(2, 2, 5), n_sel=_i32(2, 2), pk=_bf16(2, 2, 5, 64), pv=_bf16(2, 2, 5, 64))
    a.update(over)
    H.herald_kv4_gather(H.dims(2, 8, 2, 64, 1, 1 << 20), a["idx"], a["n_sel"], 5, _cache(), a["pk"], a["pv"])


def _append(**over):
    a = dict(q=_bf16(2, 3, 8, 64), k=_bf16(2, 3, 2, 64), v=_bf16(2, 3, 2, 64), ctx=_i32(2),
             n_tok=_i32(2), q_rot=_bf16(2, 3, 8, 64), k_rot=_bf16(2, 3, 2, 64),
             pooled=torch.zeros(2, 2, 4, 64))
    a.update(over)
    H.herald_kv4_append(H.dims(2, 8, 2, 64, 1, 64), 3, a["q"], a["k"], a["v"], a["ctx"], _cache(),
                        a["q_rot"], a["k_rot"], None, a["n_tok"], a["pooled"], 16, flags=1 << 9)


_qkv = _bf16(2, 3, 12, 64)  # a fused projection's output
MISFITS = [
    (_attn, dict(q=_qkv[:, :, :8])), (_attn, dict(bv=_qkv[:, :, 10:])),
    (_attn, dict(bk=_qkv[:, :, 8:10])), (_attn, dict(q=_bf16(2, 8, 3, 64))),
    (_attn, dict(q=_bf16(2, 3, 8, 64).float())), (_attn, dict(out=_bf16(2, 3, 4, 64))),
    (_attn, dict(bk=_bf16(2, 1, 2, 64).expand(2, 3, 2, 64))), (_attn, dict(ctx=_i32(1))),
    (_attn, dict(ctx=_i32(2).long())), (_attn, dict(out=_bf16(2, 8, 3, 64).transpose(1, 2))),
    (_gather, dict(idx=_i32(2, 2, 4))), (_gather, dict(idx=_i32(2, 2, 6))),
    (_gather, dict(n_sel=_i32(2))), (_gather, dict(pk=_bf16(2, 2, 5, 128))),
    (_gather, dict(pv=_bf16(2, 2, 10, 64)[:, :, ::2])), (_gather, dict(idx=_i32(2, 2, 5).long())),
    (_append, dict(q_rot=_qkv[:, :, :8])), (_append, dict(k_rot=_bf16(2, 2, 3, 64))),
    (_append, dict(q=_qkv[:, :, :7])), (_append, dict(k=_qkv[:, :, 8:])),
    (_append, dict(v=_bf16(2, 3, 2, 64).float())), (_append, dict(n_tok=_i32(1))),
    (_append, dict(ctx=_i32(1))), (_append, dict(pooled=torch.zeros(2, 2, 3, 64))),
    (_append, dict(pooled=_bf16(2, 2, 4, 64))), (_append, dict(q_rot=_bf16(2, 2, 8, 64))),
]


@pytest.mark.parametrize("call,over", MISFITS,
                         ids=[f"{c.__name__}-{next(iter(o))}-{i}" for i, (c, o) in enumerate(MISFITS)])
def test_tensors_of_another_layout_are_refused(call, over):
    """The kernels take dense arrays of the call's shape; anything else would be
    read or written elsewhere than where it lies."""
    with pytest.raises(ValueError, match=next(iter(over)).replace("bk", "block_k").replace("bv", "block_v")
                       .replace("pk", "pool_k").replace("pv", "pool_v")):
        call(**over)


@pytest.mark.parametrize("call,over", [
    (_attn, {}), (_gather, {}), (_append, {}), (_attn, dict(q=OK, bk=OK, bv=OK, out=OK, ctx=OK)),
    (_attn, dict(q=_bf16(6, 8, 64), out=_bf16(2, 3, 2, 4, 64))),   # axes merged, axes split
    (_attn, dict(q=_bf16(5000), ctx=_i32(7))),                     # flat and longer
    (_attn, dict(out=_bf16(3, 3, 8, 64), bk=None, bv=None)),       # more sequences behind
    (_gather, dict(pv=None, n_sel=_i32(4))),
    (_append, dict(q=_qkv[:, :, :8], k=_qkv[:, :, 8:10], v=_qkv[:, :, 10:], n_tok=None, pooled=None)),
], ids=str)
def test_dense_tensors_and_addresses_reach_the_library(call, over):
    """What has the call's layout passes the binding; the library then refuses the
    missing workspace, the short table or the unknown flag."""
    if not os.path.exists(H.LIB_PATH):
        from block_diffusion_sparse_gb300 import build
        build.build()
    with pytest.raises(H.HeraldError) as e:
        call(**over)
    assert e.value.status == 1 and any(w in str(e.value) for w in ("ws", "max_pages", "flags")), e.value


@pytest.mark.parametrize("over", [
    dict(q_rot=lambda a: a["q"] + 256), dict(q_rot=lambda a: a["q"] - 256),
    dict(q_rot=lambda a: a["k"] + 256), dict(q_rot=lambda a: a["v"] - 16),
    dict(k_rot=lambda a: a["k"] + 16), dict(k_rot=lambda a: a["q"] + 512),
    dict(k_rot=lambda a: a["v"] - 16), dict(q_rot=lambda a: a["k_rot"] - 16),
    dict(q_rot=lambda a: a["k_rot"] + 16),
    # slices of one buffer: queries of the last token end behind the first keys
    dict(k=lambda a: a["q"] + 2048, v=lambda a: a["q"] + 2560, q_ld=1536, k_ld=1536, v_ld=1536,
         k_rot=lambda a: a["q"] + 4096)], ids=lambda o: "-".join(o))
def test_append_outputs_partly_over_other_arrays_are_refused(over):
    """Not only equal addresses: a rotated output that begins inside an array the
    call reads would change rows before they are read."""
    a = dict(q=1 << 20, k=2 << 20, v=3 << 20, q_rot=4 << 20, k_rot=5 << 20, q_ld=0, k_ld=0, v_ld=0)
    for name, at in over.items():
        a[name] = at(a) if callable(at) else at
    cache = H.Kv4(64, 40, 32, OK, OK, OK, OK, OK, 1.0, 1.0)
    with pytest.raises(H.HeraldError, match="q_rot and k_rot") as e:
        H.herald_kv4_append(H.dims(2, 8, 2, 128, 4, 2048), 4, a["q"], a["k"], a["v"], OK, cache,
                            a["q_rot"], a["k_rot"], q_ld=a["q_ld"], k_ld=a["k_ld"], v_ld=a["v_ld"])
    assert e.value.status == 1


def test_scales_without_a_finite_base_2_form_are_refused():
    d = H.dims(2, 8, 2, 128, 4, 2048)
    cache = H.Kv4(64, 40, 32, OK, OK, OK, OK, OK, 1.0, 1.0)
    with pytest.raises(H.HeraldError, match="scale") as e:
        H.herald_kv4_attn(d, OK, cache, OK, None, None, OK, 3e38, OK, H.herald_workspace_size_kv4(d))
    assert e.value.status == 1
