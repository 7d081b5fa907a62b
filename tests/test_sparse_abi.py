"""Host-side argument checks of the operators that decode over part of a paged
cache: every call below fails a check, or has nothing to do, before the library
would reach CUDA."""
import ctypes

import pytest

from pagedattention_paged_kv_02_b200 import build as pa_build

FAKE = ctypes.c_void_p(0x10000)     # aligned, never dereferenced
ODD4 = ctypes.c_void_p(0x10004)
ODD2 = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def pa():
    pa_build.build()
    from pagedattention_paged_kv_02_b200 import pa as _pa
    return _pa


def refusals(pa, fn, args, cases):
    f = getattr(pa.lib(), fn)
    for change, status in cases:
        a = dict(args)
        a.update(change)
        assert f(*a.values(), None) == status, (fn, change)


SHAPE = dict(D=128, bs=16, NB=64, MB=8)


def common_cases(pa):
    return [(dict(D=96), pa.PA_ERR_UNSUPPORTED), (dict(bs=8), pa.PA_ERR_UNSUPPORTED),
            (dict(dtype=7), pa.PA_ERR_INVALID_ARG), (dict(B=-1), pa.PA_ERR_INVALID_ARG),
            (dict(Hkv=0), pa.PA_ERR_INVALID_ARG), (dict(NB=0), pa.PA_ERR_INVALID_ARG),
            (dict(MB=0), pa.PA_ERR_INVALID_ARG), (dict(B=65536), pa.PA_ERR_UNSUPPORTED),
            (dict(Hkv=65536, Hq=65536), pa.PA_ERR_UNSUPPORTED),
            (dict(MB=1 << 28), pa.PA_ERR_UNSUPPORTED),
            (dict(tables=None), pa.PA_ERR_INVALID_ARG), (dict(lens=ODD2), pa.PA_ERR_INVALID_ARG),
            (dict(B=0), pa.PA_OK)]


def test_update_key_bounds_host_checks(pa):
    args = dict(bounds=FAKE, k=FAKE, tables=FAKE, lens=FAKE, new=FAKE, B=4, max_new=1, Hkv=2,
                **SHAPE, dtype=1)
    cases = [c for c in common_cases(pa) if "Hq" not in c[0]]
    refusals(pa, "pa_update_key_bounds", args, cases + [
        (dict(bounds=None), pa.PA_ERR_INVALID_ARG), (dict(k=ODD4), pa.PA_ERR_INVALID_ARG),
        (dict(new=None), pa.PA_ERR_INVALID_ARG), (dict(max_new=-1), pa.PA_ERR_INVALID_ARG),
        (dict(max_new=129), pa.PA_ERR_INVALID_ARG), (dict(max_new=0), pa.PA_OK)])


def test_select_blocks_host_checks(pa):
    args = dict(sel=FAKE, q=FAKE, bounds=FAKE, tables=FAKE, lens=FAKE, K=4, first=1, last=1, B=4,
                Hq=8, Hkv=2, **SHAPE, max_ctx=128, dtype=1)
    refusals(pa, "pa_select_blocks", args, common_cases(pa) + [
        (dict(Hq=7), pa.PA_ERR_UNSUPPORTED), (dict(K=0), pa.PA_ERR_INVALID_ARG),
        (dict(first=-1), pa.PA_ERR_INVALID_ARG), (dict(last=4), pa.PA_ERR_INVALID_ARG),
        (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), pa.PA_ERR_INVALID_ARG),
        (dict(max_ctx=129), pa.PA_ERR_INVALID_ARG), (dict(max_ctx=-1), pa.PA_ERR_INVALID_ARG),
        (dict(sel=ODD2), pa.PA_ERR_INVALID_ARG), (dict(q=None), pa.PA_ERR_INVALID_ARG),
        (dict(MB=196609, max_ctx=196609 * 16), pa.PA_ERR_UNSUPPORTED)])
