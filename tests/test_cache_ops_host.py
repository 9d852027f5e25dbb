"""Refusals of the shared-prefix attention, the attention mass and the eviction: every bad argument is turned down on
the host, before anything is launched.  No call here reaches a kernel (the pointers are made up)."""
import pytest

from test_abi_host import _lib_path

P, ST = 1 << 20, 1 << 21  # aligned made-up addresses


@pytest.fixture(scope="module")
def abi():
    _lib_path()
    from ar_lm_decoding_b200 import abi
    return abi


def _status(abi, fn, *args):
    try:
        fn(*args, stream=0)
    except abi.TidarError as e:
        return e.status
    raise AssertionError("accepted")


def _shared(abi, **kw):
    a = dict(q=P, kn=P, vn=P, ks=P, vs=P, sl=P, S_max=256, kc=P, vc=P, pl=P, B=2, Hq=4, Hkv=2, D=64, k=2, R=8,
             P_max=128, scale=0.125, mode=0, out=P, lse=P, ws=P, ws_bytes=1 << 40, st=ST)
    a.update(kw)
    return _status(abi, abi.tidar_attn_step_shared, *a.values())


def _shared_paged(abi, **kw):
    a = dict(q=P, kn=P, vn=P, kp=P, vp=P, sht=P, msp=4, sl=P, bt=P, mp=2, npg=64, pl=P, B=2, Hq=4, Hkv=2, D=64, k=2,
             R=8, scale=0.125, mode=0, out=P, lse=P, ws=P, ws_bytes=1 << 40, st=ST)
    a.update(kw)
    return _status(abi, abi.tidar_attn_step_shared_paged, *a.values())


def _mass(abi, **kw):
    a = dict(qs=P, lses=P, kc=P, m=P, bt=None, mp=0, npg=0, pl=P, rc=P, L=2, B=2, Hq=4, Hkv=2, D=64, R=8, P_max=128,
             scale=0.125, decay=1.0, st=ST)
    a.update(kw)
    return _status(abi, abi.tidar_attn_mass, *a.values())


def _evict(abi, **kw):
    a = dict(kc=P, vc=P, m=P, bt=None, mp=0, npg=0, pl=P, L=2, B=2, Hkv=2, D=64, P_max=128, budget=64, sink=4,
             recent=8, st=ST)
    a.update(kw)
    return _status(abi, abi.tidar_kv_evict, *a.values())


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.mark.parametrize("kw", [dict(q=None), dict(kn=None), dict(vn=None), dict(ks=None), dict(vs=None), dict(sl=None),
                                dict(kc=None), dict(vc=None), dict(pl=None), dict(out=None), dict(st=None), dict(q=P + 8),
                                dict(ks=P + 2), dict(vc=P + 4), dict(out=P + 8), dict(lse=P + 2), dict(B=0), dict(Hq=0),
                                dict(Hkv=0), dict(R=0), dict(k=0), dict(R=9), dict(S_max=-1), dict(P_max=-1),
                                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                                dict(mode=2), dict(mode=-1)], ids=str)
def test_shared_invalid(abi, kw):
    assert _shared(abi, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Hq=3), dict(D=96), dict(D=32), dict(k=17, R=17 * 19), dict(B=1025), dict(Hq=258, Hkv=2),
                                dict(mode=1, R=4097), dict(Hkv=2, S_max=1 << 30), dict(B=1024, Hkv=2, P_max=1 << 20),
                                dict(B=1024, Hq=1024, Hkv=8, mode=1, R=4096)], ids=str)
def test_shared_unsupported(abi, kw):
    assert _shared(abi, **kw) == UNSUPPORTED


def test_shared_workspace(abi):
    need = abi.tidar_attn_shared_workspace_size(2, 4, 2, 64, 8, 256, 128)
    if need > 0:
        assert _shared(abi, ws_bytes=need - 1) == WORKSPACE
        assert _shared(abi, ws=None) == INVALID
        assert _shared(abi, ws=P + 128) == INVALID
    for bad in ((0, 4, 2, 64, 8, 256, 128), (2, 3, 2, 64, 8, 256, 128), (2, 4, 2, 80, 8, 256, 128),
                (2, 4, 2, 64, 0, 256, 128), (2, 4, 2, 64, 8, -1, 128)):
        assert abi.tidar_attn_shared_workspace_size(*bad) == 0


def test_shared_workspace_sizes(abi):
    """Every size that one of the two calls takes needs room; no size that both reject has any."""
    size = abi.tidar_attn_shared_workspace_size
    small = size(1, 1, 1, 64, 1, 0, 0)
    assert small > 0
    assert size(2, 4, 2, 64, 8, 256, 128) > small
    assert size(1024, 8, 2, 128, 1, 4096 * 64, 65536) > size(1, 8, 2, 128, 1, 4096 * 64, 65536)
    # too many rows for contiguous caches, not for pages: the contiguous call says so, the paged one takes the sizes
    assert size(1024, 64, 32, 64, 1, 0, 65536) > 0
    assert _shared(abi, B=1024, Hq=64, Hkv=32, mode=1, R=1, S_max=0, P_max=65536) == UNSUPPORTED
    assert _shared_paged(abi, B=1024, Hq=64, Hkv=32, mode=1, R=1, msp=0, sht=None, mp=1024, ws_bytes=0) == WORKSPACE
    for bad in ((1, 129, 1, 64, 1, 0, 0), (1, 1, 1, 64, 4097, 0, 0), (1025, 1, 1, 64, 1, 0, 0), (1, 1, 1, 64, 1, 0, -1),
                (1, 0, 1, 64, 1, 0, 0), (1, 1, 0, 64, 1, 0, 0), (2, 4, 2, 64, 8, 1 << 30, 128),
                (1024, 4, 2, 64, 8, 0, 1 << 20),
                (1024, 1024, 8, 64, 4096, 0, 0)):
        assert size(*bad) == 0, bad


def test_limits_at_their_edges(abi):
    """Sizes at a documented limit are taken, as the next check (a pointer that is missing) shows; one more is not."""
    assert _evict(abi, L=1 << 17, B=1 << 5, Hkv=1 << 5, st=None) == INVALID
    assert _evict(abi, L=(1 << 17) + 1, B=1 << 5, Hkv=1 << 5, st=None) == UNSUPPORTED
    assert _evict(abi, P_max=65536, st=None) == INVALID and _evict(abi, bt=P, mp=1024, npg=4, st=None) == INVALID
    assert _mass(abi, P_max=1 << 22, st=None) == INVALID and _mass(abi, bt=P, mp=1024, npg=4, st=None) == INVALID
    assert _mass(abi, R=(1 << 29) - 1, st=None) == INVALID and _mass(abi, R=1 << 29, st=None) == UNSUPPORTED
    assert _shared_paged(abi, npg=(1 << 24) - 1, kp=None) == INVALID and _shared_paged(abi, npg=1 << 24, kp=None) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(kp=None), dict(vp=None), dict(sht=None), dict(bt=None), dict(mp=0), dict(npg=0),
                                dict(msp=-1), dict(R=7), dict(st=None)], ids=str)
def test_shared_paged_invalid(abi, kw):
    assert _shared_paged(abi, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(mp=1025), dict(msp=4097), dict(npg=1 << 25), dict(D=80), dict(B=1025)], ids=str)
def test_shared_paged_unsupported(abi, kw):
    assert _shared_paged(abi, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(qs=None), dict(lses=None), dict(kc=None), dict(m=None), dict(pl=None), dict(st=None),
                                dict(L=0), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(R=0), dict(P_max=-1),
                                dict(bt=P), dict(bt=P, mp=2), dict(scale=0.0), dict(scale=float("inf")),
                                dict(decay=-0.5), dict(decay=float("nan")), dict(decay=float("inf"))], ids=str)
def test_mass_invalid(abi, kw):
    assert _mass(abi, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Hq=5), dict(D=256), dict(B=1025), dict(P_max=(1 << 22) + 1), dict(bt=P, mp=1025, npg=9),
                                dict(R=1 << 30, Hq=4)], ids=str)
def test_mass_unsupported(abi, kw):
    assert _mass(abi, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(kc=None), dict(vc=None), dict(m=None), dict(pl=None), dict(st=None), dict(L=0),
                                dict(B=0), dict(Hkv=0), dict(P_max=-1), dict(budget=-1), dict(sink=-1), dict(recent=-1),
                                dict(sink=60), dict(sink=2**31 - 1, recent=2**31 - 1), dict(bt=P), dict(bt=P, npg=4)], ids=str)
def test_evict_invalid(abi, kw):
    assert _evict(abi, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(D=80), dict(P_max=65537), dict(bt=P, mp=1025, npg=4), dict(L=1 << 20, B=1 << 10)], ids=str)
def test_evict_unsupported(abi, kw):
    assert _evict(abi, **kw) == UNSUPPORTED


def test_stalled_hooks_invalid(abi):
    assert _status(abi, abi.tidar_testing_attn_step_shared_stalled, P, P, P, P, P, P, 256, P, P, P, 2, 4, 2, 64, 2, 8, 128,
                   0.125, 0, P, P, P, 1 << 40, ST, 0) == INVALID
    assert _status(abi, abi.tidar_testing_attn_mass_stalled, P, P, P, P, None, 0, 0, P, P, 2, 2, 4, 2, 64, 8, 128, 0.125,
                   1.0, ST, 0) == INVALID
