"""A host thread whose first CUDA call is a launch of this library: every form
that describes its caches to the TMA engine runs there as it does elsewhere."""
import threading

import pytest
import torch

from helpers import bits, oracle_after_append
from pagedattention_paged_kv_02_b200 import workloads as W
from test_gpu_prefill import mixed_chunks

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def pa():
    from pagedattention_paged_kv_02_b200 import build, pa as _pa
    build.build()
    torch.cuda.init()
    return _pa


@pytest.fixture(autouse=True)
def clean_error_word(pa):
    pa.pa_device_error(clear=True)
    yield
    torch.cuda.synchronize()
    pa.pa_device_error(clear=True)


def workspace(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)


def make(pa, kind):
    """A prepared call, its output and what it needs alive."""
    if kind == "prefill":
        batch = mixed_chunks([100, 0], [40, 70], 8, 2, 16, seed=801)
        batch.k_cache, batch.v_cache = oracle_after_append(batch)
        d = batch.to(DEV)
        out = torch.zeros_like(d.prefill_q)
        return pa.prepare_prefill_chunk(out, d.prefill_q, d.k_cache, d.v_cache,
                                        d.prefill_block_tables, d.prefill_context_lens,
                                        d.query_start_loc, 70, batch.scale), out, d
    batch = W.decode_batch([700, 33, 300], 8, 2, 128, 16, 80, BF16, seed=802)
    batch.k_cache, batch.v_cache = oracle_after_append(batch)
    if kind in ("fp8", "int8"):
        batch = (W.to_fp8 if kind == "fp8" else W.to_int8)(batch)
    d = batch.to(DEV)
    out = torch.zeros_like(d.q)
    head = (out, d.q, d.k_cache, d.v_cache)
    rows = (d.block_tables, d.context_lens)
    if kind in ("fp8", "int8"):
        ws = workspace(pa.pa_decode_workspace_size(3, 8, 128, 700, 0))
        call = pa.prepare_decode_fp8(*head, d.k_scale, d.v_scale, *rows, 700, batch.scale, 0, ws)
    elif kind == "selected":
        sel = torch.arange(44, dtype=torch.int32).repeat(3, 2, 1)
        sel = torch.where(sel * 16 < batch.context_lens[:, None, None], sel, -1).to(DEV)
        ws = workspace(pa.pa_decode_selected_blocks_workspace_size(3, 8, 2, 128, 16, 44))
        call = pa.prepare_decode_selected_blocks(*head, *rows, sel, batch.scale, 0, ws)
    elif kind == "weights":
        w = torch.zeros(3, 2, 700, device=DEV)
        ws = workspace(pa.pa_decode_accumulate_weights_workspace_size(3, 8, 128, 700))
        call = pa.prepare_decode_accumulate_weights(out, w, None, *head[1:], *rows, 700,
                                                    batch.scale, 0, ws)
    else:
        ws = workspace(pa.pa_decode_workspace_size(3, 8, 128, 700, 0))
        call = pa.prepare_decode(*head, *rows, 700, batch.scale, 0, ws)
    return call, out, (d, ws)


@pytest.mark.parametrize("kind", ["decode", "prefill", "fp8", "int8", "selected", "weights"])
def test_first_call_of_a_host_thread(pa, kind):
    call, out, kept = make(pa, kind)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    errors = []

    def issue():
        try:
            call(stream=s)
        except Exception as e:      # noqa: BLE001 (reported below, in the test's own thread)
            errors.append(e)

    t = threading.Thread(target=issue)
    t.start()
    t.join()
    s.synchronize()
    assert not errors, errors
    assert torch.equal(bits(out), bits(want)) and bool((want.float().abs() > 0).any())
    assert pa.pa_device_error() == 0
