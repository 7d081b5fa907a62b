"""A NaN that a row attends shows in its output, however the row is split and
merged: a NaN query or key makes the rows that use it NaN in every dimension (and
their weights), a NaN value one dimension, and all other rows keep their bits."""
import pytest
import torch

from helpers import bits, oracle_after_append
from pagedattention_paged_kv_02_b200 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
CTX, HQ, HKV, D, BS = [700, 33, 600], 8, 2, 128, 16


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


def make(dtype):
    batch = W.decode_batch(CTX, HQ, HKV, D, BS, 100, dtype, seed=901)
    batch.k_cache, batch.v_cache = oracle_after_append(batch)
    return batch


def run(pa, batch, form, part):
    """Outputs, and the weights where there are any."""
    d = batch.to(DEV)
    out, w = torch.full_like(d.q, 5.0), None
    head = (d.q, d.k_cache, d.v_cache, d.block_tables, d.context_lens)
    ws = lambda n: torch.full((max(n, 1),), 255, dtype=torch.uint8, device=DEV)
    if form == "selected":
        sel = torch.arange(44, dtype=torch.int32).repeat(3, HKV, 1)
        sel = torch.where(sel * BS < batch.context_lens[:, None, None], sel, -1).to(DEV)
        n = pa.pa_decode_selected_blocks_workspace_size(3, HQ, HKV, D, BS, 44, part)
        pa.pa_decode_selected_blocks(out, *head, sel, batch.scale, part, ws(n))
    elif form == "weights":
        w = torch.zeros(3, HKV, max(CTX), device=DEV)
        n = pa.pa_decode_accumulate_weights_workspace_size(3, HQ, D, max(CTX), part)
        pa.pa_decode_accumulate_weights(out, w, None, *head, max(CTX), batch.scale, part, ws(n))
    else:
        n = pa.pa_decode_workspace_size(3, HQ, D, max(CTX), part)
        pa.pa_decode(out, *head, max(CTX), batch.scale, part, ws(n))
    torch.cuda.synchronize()
    return out.cpu(), None if w is None else w.cpu()


# one partition; a cluster of three (256 tokens); merges of 15 and of 44 partials
@pytest.mark.parametrize("part", [-1, 256, 48, 16])
@pytest.mark.parametrize("form", ["selected", "weights", "decode"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_nan_shows_where_it_is_attended(pa, dtype, form, part):
    nan = float("nan")
    group = HQ // HKV
    clean, clean_w = run(pa, make(dtype), form, part)
    assert not bool(torch.isnan(clean).any())

    def check(batch, rows, dims=slice(None), weights=True):
        got, w = run(pa, batch, form, part)
        want = clean.clone()
        for b, heads in rows:
            want[b, heads, dims] = nan
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(bits(got.nan_to_num(3.0)), bits(want.nan_to_num(3.0)))
        if w is not None:
            for b, ctx in enumerate(CTX):
                for h in range(HKV):
                    heads = set(range(h * group, (h + 1) * group))
                    bad = weights and any(r == b and heads & set(range(HQ)[hs]) for r, hs in rows)
                    if bad:
                        assert bool(torch.isnan(w[b, h, :ctx]).all())
                    else:
                        assert torch.equal(w[b, h], clean_w[b, h])

    batch = make(dtype)                                # a query, of one head
    batch.q[0, 5, 77] = nan
    check(batch, [(0, slice(5, 6))])
    for pos in (0, 300, 699):                          # a key, first, inside, last
        batch = make(dtype)
        batch.k_cache[batch.block_tables[0, pos // BS], 1, pos % BS, 3] = nan
        check(batch, [(0, slice(group, HQ))])
    batch = make(dtype)                                # every key of one K/V head
    blocks = batch.block_tables[2, :-(-CTX[2] // BS)].long()
    batch.k_cache[blocks, 0] = nan
    check(batch, [(2, slice(0, group))])
    batch = make(dtype)                                # a value: its dimension only
    batch.v_cache[batch.block_tables[1, 1], 1, 4, 9] = nan
    check(batch, [(1, slice(group, HQ))], dims=9, weights=False)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("part", [0, 128])
def test_nan_in_a_shared_prefix(pa, part):
    """The prefix partition that holds it hands it to every member's merge."""
    from test_gpu_shared_prefix import _grouped, shared_decode
    ctxs = [300, 280, 410, 90]
    batch = _grouped(ctxs, [0, 0, 0, -1], 200, 8, 2, 128, 16, seed=902)
    d = batch.to(DEV)
    pa.pa_reshape_and_cache(d.key, d.value, d.k_cache, d.v_cache, d.slot_mapping)
    clean = shared_decode(pa, batch, d, part)
    d.k_cache[d.block_tables[0, 4].long(), 1, 3, 50] = float("nan")
    got = shared_decode(pa, batch, d, part)
    torch.cuda.synchronize()
    rows = torch.zeros(4, 8, dtype=torch.bool)
    rows[:3, 4:] = True
    assert torch.equal(torch.isnan(got).all(-1).cpu(), rows)
    assert torch.equal(bits(got.nan_to_num(3.0))[~rows.to(DEV)], bits(clean)[~rows.to(DEV)])
    assert pa.pa_device_error() == 0
