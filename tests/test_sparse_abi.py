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
    need = pa.pa_select_blocks_workspace_size(4, 2, 16, 127)
    assert need == 4 * 2 * 8 * 8
    f = pa.pa_select_blocks_workspace_size
    assert f(0, 2, 16, 128) == 0 and f(4, 2, 16, 0) == 0 and f(4, 0, 16, 128) == 0
    assert f(65535, 8, 16, 1 << 20) == 65535 * 8 * 65536 * 8
    args = dict(sel=FAKE, q=FAKE, bounds=FAKE, tables=FAKE, lens=FAKE, K=4, first=1, last=1, B=4,
                Hq=8, Hkv=2, **SHAPE, max_ctx=128, ws=FAKE, ws_bytes=0, dtype=1)
    refusals(pa, "pa_select_blocks", args, common_cases(pa) + [
        (dict(Hq=7), pa.PA_ERR_UNSUPPORTED), (dict(K=0), pa.PA_ERR_INVALID_ARG),
        (dict(first=-1), pa.PA_ERR_INVALID_ARG), (dict(last=4), pa.PA_ERR_INVALID_ARG),
        (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), pa.PA_ERR_INVALID_ARG),
        (dict(max_ctx=129), pa.PA_ERR_INVALID_ARG), (dict(max_ctx=-1), pa.PA_ERR_INVALID_ARG),
        (dict(sel=ODD2), pa.PA_ERR_INVALID_ARG), (dict(q=None), pa.PA_ERR_INVALID_ARG),
        (dict(), pa.PA_ERR_WORKSPACE), (dict(ws_bytes=need - 1), pa.PA_ERR_WORKSPACE),
        (dict(K=(1 << 30) + 1), pa.PA_ERR_UNSUPPORTED),
        (dict(ws=None, ws_bytes=need), pa.PA_ERR_WORKSPACE),
        (dict(ws=ctypes.c_void_p(0x10010), ws_bytes=need), pa.PA_ERR_WORKSPACE)])


def test_decode_selected_blocks_host_checks(pa):
    args = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, tables=FAKE, lens=FAKE, sel=FAKE, K=4, B=4,
                Hq=8, Hkv=2, **SHAPE, scale=0.1, part=0, ws=None, ws_bytes=0, dtype=1)
    need = pa.pa_decode_selected_blocks_workspace_size(4, 8, 2, 128, 16, 9, 16)
    o, l_ = 4 * 8 * 9 * 128 * 4, 4 * 8 * 9 * 4
    assert need == o + -(-l_ // 256) * 256
    # up to eight partitions are merged inside a cluster
    assert pa.pa_decode_selected_blocks_workspace_size(4, 8, 2, 128, 16, 8, 16) == 0
    # one partition needs none; invalid sizes report none
    f = pa.pa_decode_selected_blocks_workspace_size
    assert f(4, 8, 2, 128, 16, 4, -1) == 0 and f(4, 8, 2, 128, 16, 0) == 0
    assert f(4, 7, 2, 128, 16, 4) == 0 and f(4, 8, 2, 128, 16, 4, 24) == 0
    refusals(pa, "pa_decode_selected_blocks", args, common_cases(pa) + [
        (dict(Hq=7), pa.PA_ERR_UNSUPPORTED), (dict(K=0), pa.PA_ERR_INVALID_ARG),
        (dict(scale=float("nan")), pa.PA_ERR_INVALID_ARG), (dict(sel=None), pa.PA_ERR_INVALID_ARG),
        (dict(sel=ODD2), pa.PA_ERR_INVALID_ARG), (dict(out=ODD4), pa.PA_ERR_INVALID_ARG),
        (dict(part=24), pa.PA_ERR_INVALID_ARG), (dict(part=32768), pa.PA_ERR_INVALID_ARG),
        (dict(part=-1, K=1025), pa.PA_ERR_UNSUPPORTED), (dict(K=1 << 28), pa.PA_ERR_UNSUPPORTED),
        # listed tokens past 2^30, whatever the partition
        (dict(K=(1 << 26) + 1), pa.PA_ERR_UNSUPPORTED),
        (dict(K=(1 << 26) + 1, part=16), pa.PA_ERR_UNSUPPORTED),
        (dict(part=16, K=9), pa.PA_ERR_WORKSPACE),
        (dict(part=16, K=9, ws=FAKE, ws_bytes=need - 1), pa.PA_ERR_WORKSPACE),
        (dict(part=16, K=9, ws=ctypes.c_void_p(0x10010), ws_bytes=need), pa.PA_ERR_WORKSPACE)])


def test_decode_accumulate_weights_host_checks(pa):
    args = dict(out=FAKE, wo=FAKE, wi=None, q=FAKE, k=FAKE, v=FAKE, tables=FAKE, lens=FAKE, B=4,
                Hq=8, Hkv=2, **SHAPE, max_ctx=128, stride=128, scale=0.1, part=0, ws=FAKE,
                ws_bytes=0, dtype=1)
    f = pa.pa_decode_accumulate_weights_workspace_size
    # two statistics per (row, head, partition) and a score per position
    need = f(4, 8, 128, 128)
    assert need == 2 * 256 + 4 * 8 * 128 * 4
    assert f(4, 8, 128, 100, 16) == pa.pa_decode_workspace_size(4, 8, 128, 100, 16) + \
        2 * 1024 + 4 * 8 * 112 * 4
    assert f(0, 8, 128, 128) == 0 and f(4, 8, 128, 0) == 0 and f(4, 8, 128, 128, 24) == 0
    assert f(1, 8, 128, (1 << 30) + 1) == 0
    long = dict(MB=(1 << 26) + 1, max_ctx=(1 << 30) + 1, stride=(1 << 30) + 1)
    near = ctypes.c_void_p(0x10000 + 64)
    refusals(pa, "pa_decode_accumulate_weights", args, common_cases(pa) + [
        (dict(Hq=7), pa.PA_ERR_UNSUPPORTED), (dict(max_ctx=129, stride=256), pa.PA_ERR_INVALID_ARG),
        (dict(max_ctx=-1), pa.PA_ERR_INVALID_ARG), (dict(stride=127), pa.PA_ERR_INVALID_ARG),
        (dict(scale=float("inf")), pa.PA_ERR_INVALID_ARG), (dict(wo=None), pa.PA_ERR_INVALID_ARG),
        (dict(wo=ODD2), pa.PA_ERR_INVALID_ARG), (dict(wi=ODD2), pa.PA_ERR_INVALID_ARG),
        (dict(wi=near), pa.PA_ERR_INVALID_ARG), (dict(part=24), pa.PA_ERR_INVALID_ARG),
        (long, pa.PA_ERR_UNSUPPORTED),
        (dict(), pa.PA_ERR_WORKSPACE), (dict(ws=None, ws_bytes=need), pa.PA_ERR_WORKSPACE),
        (dict(ws=ctypes.c_void_p(0x10010), ws_bytes=need), pa.PA_ERR_WORKSPACE)])


def test_evict_tokens_host_checks(pa):
    far = ctypes.c_void_p(0x40000)
    args = dict(k=FAKE, v=FAKE, wo=FAKE, wi=FAKE, kept=FAKE, new=far, tables=FAKE, dst=FAKE,
                lens=FAKE, budget=64, first=4, last=8, B=4, Hkv=2, **SHAPE, dst_MB=4, max_ctx=128,
                stride=128, dtype=1)
    cases = [c for c in common_cases(pa) if "Hq" not in c[0]]
    refusals(pa, "pa_evict_tokens", args, cases + [
        (dict(budget=0), pa.PA_ERR_INVALID_ARG), (dict(first=60, last=5), pa.PA_ERR_INVALID_ARG),
        (dict(first=-1), pa.PA_ERR_INVALID_ARG),
        (dict(budget=(1 << 30) + 1, dst_MB=8), pa.PA_ERR_UNSUPPORTED),
        (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), pa.PA_ERR_INVALID_ARG),
        (dict(dst_MB=0), pa.PA_ERR_INVALID_ARG), (dict(dst_MB=3), pa.PA_ERR_INVALID_ARG),
        (dict(max_ctx=129, stride=200), pa.PA_ERR_INVALID_ARG),
        (dict(max_ctx=-1), pa.PA_ERR_INVALID_ARG), (dict(stride=127), pa.PA_ERR_INVALID_ARG),
        (dict(MB=(1 << 26) + 1, max_ctx=(1 << 30) + 1, stride=(1 << 30) + 1),
         pa.PA_ERR_UNSUPPORTED),
        (dict(new=FAKE), pa.PA_ERR_INVALID_ARG), (dict(new=ODD4), pa.PA_ERR_INVALID_ARG),
        (dict(wi=ctypes.c_void_p(0x10040)), pa.PA_ERR_INVALID_ARG),
        (dict(wi=None), pa.PA_ERR_INVALID_ARG), (dict(kept=None), pa.PA_ERR_INVALID_ARG),
        (dict(dst=ODD2), pa.PA_ERR_INVALID_ARG), (dict(k=ODD4), pa.PA_ERR_INVALID_ARG)])
