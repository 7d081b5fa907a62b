"""Calls of two host threads, each on a stream of its own, whose launches of one
kernel need very different amounts of shared memory: none is refused, and each
result is the one that a single thread gets."""
import sys
import threading

import pytest
import torch

from helpers import bits
from pagedattention_paged_kv_02_b200 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
CALLS = 1500


@pytest.fixture(scope="module")
def pa():
    from pagedattention_paged_kv_02_b200 import build, pa as _pa
    build.build()
    torch.cuda.init()
    return _pa


@pytest.fixture(autouse=True)
def clean_error_word(pa):
    pa.pa_device_error(clear=True)
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    yield
    sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    pa.pa_device_error(clear=True)


def pool(heads, blocks, bs, D, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(blocks, heads, bs, D, generator=g, device=DEV).to(dtype)


def select_call(pa, dtype, blocks, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kb = torch.randn(blocks, 1, 2, 64, generator=g, device=DEV).sort(dim=2).values.to(dtype)
    q = torch.randn(1, 1, 64, generator=g, device=DEV).to(dtype)
    table = torch.arange(blocks, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([blocks * 16], dtype=torch.int32, device=DEV)
    out = torch.empty(1, 1, 20, dtype=torch.int32, device=DEV)
    ws = torch.empty(pa.pa_select_blocks_workspace_size(1, 1, 16, blocks * 16), dtype=torch.uint8,
                     device=DEV)
    return pa.prepare_select_blocks(out, q, kb, table, lens, blocks * 16, 16, 1, 1, ws), out


def evict_call(pa, dtype, n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    k = pool(1, 4, 64, 64, dtype, seed)
    w = torch.rand(1, 1, n, generator=g, device=DEV)
    src = torch.zeros(1, -(-n // 64), dtype=torch.int32, device=DEV)
    dst = torch.ones(1, 1, dtype=torch.int32, device=DEV)
    kept = torch.empty(1, 1, 30, dtype=torch.int32, device=DEV)
    new = torch.empty(1, dtype=torch.int32, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    return pa.prepare_evict_tokens(k, k.clone(), torch.empty_like(w), w, kept, new, src, dst, lens,
                                   n, 30, 1, 1), kept


def decode_call(pa, kind, dtype, part, seed):
    batch = W.decode_batch([1000], 4, 1, 128, 16, 70, dtype, seed=seed)
    d = batch.to(DEV)
    out = torch.empty_like(d.q)
    head = (out, d.q, d.k_cache, d.v_cache, d.block_tables, d.context_lens)
    new_ws = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    if kind == "selected":
        sel = torch.arange(63, dtype=torch.int32, device=DEV)[None, None].contiguous()
        n = pa.pa_decode_selected_blocks_workspace_size(1, 4, 1, 128, 16, 63, part)
        return pa.prepare_decode_selected_blocks(*head, sel, batch.scale, part, new_ws(n)), out
    if kind == "weights":
        w = torch.empty(1, 1, 1000, device=DEV)
        n = pa.pa_decode_accumulate_weights_workspace_size(1, 4, 128, 1000, part)
        return pa.prepare_decode_accumulate_weights(out, w, None, *head[1:], 1000, batch.scale,
                                                    part, new_ws(n)), out
    n = pa.pa_decode_workspace_size(1, 4, 128, 1000, part)
    ws = new_ws(n)
    call = pa.prepare_decode(*head, 1000, batch.scale, part, ws)
    call.kept = (d, ws)
    return call, out


def make(pa, kind, dtype, large):
    if kind == "select":       # both with the threads of a CTA that long rows get
        return select_call(pa, dtype, 24000 if large else 2100, 701)
    if kind == "evict":        # likewise, a CTA to a row
        return evict_call(pa, dtype, 4000 if large else 100, 702)
    return decode_call(pa, kind, dtype, 16384 if large else 16, 703)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("kind", ["select", "evict", "selected", "weights", "decode"])
def test_small_and_large_calls_from_two_threads(pa, kind, dtype):
    pairs = [make(pa, kind, dtype, large) for large in (False, True)]
    for call, _ in pairs:
        call()
    torch.cuda.synchronize()
    want = [out.clone() for _, out in pairs]
    for _, out in pairs:
        out.zero_()
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(2)

    def issue(call):
        s = torch.cuda.Stream()
        start.wait()
        try:
            for i in range(CALLS):
                call(stream=s)
                if i % 100 == 99:
                    s.synchronize()
        except Exception as e:      # noqa: BLE001 (reported below, in the test's own thread)
            errors.append(e)
        s.synchronize()

    threads = [threading.Thread(target=issue, args=(call,)) for call, _ in pairs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for (_, out), w in zip(pairs, want):
        assert torch.equal(bits(out), bits(w))
    assert pa.pa_device_error() == 0
