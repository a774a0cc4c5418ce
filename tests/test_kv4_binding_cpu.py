"""What the binding of the paged 4-bit cache's calls refuses before any of
them reaches the library: tensors that would be read or written elsewhere than
where they lie."""
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
