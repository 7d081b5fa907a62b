"""pa_decode_selected_blocks on the GPU against the 64-bit form, on lists of
every shape: empty, padded in the middle, unordered, with repeats, of blocks
that are partly filled, longer than the row; and against pa_decode where the
list names every block. Caches are poisoned with NaN past each row's length and
in blocks no list names."""
import pytest
import torch

import sparse_reference as R
from helpers import assert_close, bits, oracle_after_append
from pagedattention_paged_kv_02_b200 import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


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


def appended(ctxs, hq, hkv, D, bs, dtype, seed):
    nb = sum(-(-c // bs) for c in ctxs) + 4
    batch = W.decode_batch(ctxs, hq, hkv, D, bs, nb, dtype, seed=seed)
    batch.k_cache, batch.v_cache = oracle_after_append(batch)
    return batch


def run(pa, batch, selected, part=0, scale=None):
    d = batch.to(DEV)
    B, H_q, D = d.q.shape
    n = pa.pa_decode_selected_blocks_workspace_size(B, H_q, batch.num_kv_heads, D,
                                                    batch.block_size, selected.shape[2], part)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None
    out = torch.full_like(d.q, float("nan"))
    pa.pa_decode_selected_blocks(out, d.q, d.k_cache, d.v_cache, d.block_tables, d.context_lens,
                                 selected.to(DEV), batch.scale, part, ws)
    torch.cuda.synchronize()
    return out


def reference(batch, selected):
    return R.decode_selected(batch.q, batch.k_cache, batch.v_cache, batch.block_tables,
                             batch.context_lens, selected, batch.scale)


def random_lists(batch, count, seed, keep=0.7):
    """Distinct blocks of each row in random order, padding in between."""
    g = torch.Generator().manual_seed(seed)
    B, H = batch.num_seqs, batch.num_kv_heads
    sel = torch.full((B, H, count), -1, dtype=torch.int32)
    for b, ctx in enumerate(batch.context_lens.tolist()):
        n = -(-ctx // batch.block_size)
        for h in range(H):
            at = torch.randperm(count, generator=g)[:min(n, int(count * keep) + 1)]
            sel[b, h, at] = torch.randperm(n, generator=g)[:len(at)].int()
    return sel


SHAPES = [
    ([5, 17, 33, 40, 0], 4, 4, 64, 16, F32),
    ([1, 130, 515], 16, 2, 128, 16, F32),
    ([5, 63, 64, 65, 200, 0], 8, 2, 128, 16, BF16),
    ([1, 31, 32, 33, 300], 6, 2, 64, 32, BF16),
    ([2, 64, 129, 1500], 20, 1, 128, 64, BF16),
    ([700, 1400], 40, 2, 64, 16, BF16),
]


@pytest.mark.parametrize("part", [0, -1, 16, 48, 256])
@pytest.mark.parametrize("count", [1, 3, 40])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_lists_against_the_64_bit_form(pa, shape, count, part):
    batch = appended(*shape, 301)
    sel = random_lists(batch, count, 302 + count)
    got = run(pa, batch, sel, part)
    assert_close(got, reference(batch, sel), f"{shape} {count} {part}")
    assert torch.all(got[batch.context_lens == 0] == 0)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_all_padding_gives_zero(pa, dtype):
    batch = appended([100, 40], 8, 2, 128, 16, dtype, 303)
    for count in (1, 200):
        sel = torch.full((2, 2, count), -1, dtype=torch.int32)
        sel[1, 0, 0] = -2 ** 31
        assert torch.all(run(pa, batch, sel) == 0)
    # one head of one row attends, the others do not
    sel[0, 1, 77] = 6
    got = run(pa, batch, sel)
    assert_close(got, reference(batch, sel), "one block")
    assert torch.all(got[1] == 0) and torch.all(got[0, :4] == 0)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_repeated_block_counts_twice(pa, dtype):
    batch = appended([100], 4, 2, 64, 16, dtype, 304)
    sel = torch.tensor([[[3, 3, 6], [5, 0, 5]]], dtype=torch.int32)
    assert_close(run(pa, batch, sel), reference(batch, sel), "repeats")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_block_is_plain_decode(pa, dtype):
    batch = appended([1, 500, 333, 1024], 8, 2, 128, 16, dtype, 305)
    d = batch.to(DEV)
    sel = torch.arange(64, dtype=torch.int32).repeat(4, 2, 1)
    for b, ctx in enumerate(batch.context_lens.tolist()):
        sel[b, :, -(-ctx // 16):] = -1
    want = torch.empty_like(d.q)
    ws = torch.empty(pa.pa_decode_workspace_size(4, 8, 128, 1024, 256), dtype=torch.uint8,
                     device=DEV)
    pa.pa_decode(want, d.q, d.k_cache, d.v_cache, d.block_tables, d.context_lens, 1024,
                 batch.scale, 256, ws)
    assert_close(run(pa, batch, sel, 256), want.double().cpu(), "every block")


def test_bad_entries_are_skipped_and_recorded(pa):
    batch = appended([100, 40], 8, 2, 128, 16, BF16, 306)
    sel = torch.tensor([[[0, 2, 6], [1, 3, 5]], [[0, 1, 2], [2, 1, 0]]], dtype=torch.int32)
    good = sel.clone()
    good[0, 1, 1] = -1
    for bad in (7, 2 ** 31 - 1):     # at and far past ceil(100 / 16)
        sel[0, 1, 1] = bad
        got = run(pa, batch, sel)
        assert_close(got, reference(batch, good), f"entry {bad}")
        assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE
    # a block id outside the pool
    for bad in (-1, batch.num_blocks):
        broken = appended([100, 40], 8, 2, 128, 16, BF16, 306)
        broken.block_tables[0, 3] = bad
        sel[0, 1, 1] = 3
        assert_close(run(pa, broken, sel), reference(batch, good), f"id {bad}")
        assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE
    # a length the table cannot hold is clamped to what it can
    long = appended([112, 40], 8, 2, 128, 16, BF16, 307)
    sel[0, 1, 1] = 6
    want = reference(long, sel)
    long.context_lens[0] = 10 ** 6
    assert_close(run(pa, long, sel), want, "length")
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE


def test_select_then_decode_a_step(pa):
    """A decode step over selected blocks, as an engine runs it: append, refresh
    the bounds, select, attend."""
    batch = W.decode_batch([700, 33, 1300, 64, 1], 16, 2, 128, 16, 200, BF16, seed=308)
    d = batch.to(DEV)
    host_k, host_v = oracle_after_append(batch)
    B, H_q, D = d.q.shape
    NB, H, bs, _ = d.k_cache.shape
    bounds = torch.zeros(NB, H, 2, D, dtype=BF16, device=DEV)
    old = d.context_lens - 1
    pa.pa_update_key_bounds(bounds, d.k_cache, d.block_tables, old, old, 1300)
    pa.pa_reshape_and_cache(d.key, d.value, d.k_cache, d.v_cache, d.slot_mapping)
    ones = torch.ones_like(d.context_lens)
    pa.pa_update_key_bounds(bounds, d.k_cache, d.block_tables, d.context_lens, ones, 1)
    sel = torch.empty(B, H, 12, dtype=torch.int32, device=DEV)
    pa.pa_select_blocks(sel, d.q, bounds, d.block_tables, d.context_lens, 1300, bs, 1, 2)
    n = pa.pa_decode_selected_blocks_workspace_size(B, H_q, H, D, bs, 12)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(d.q)
    pa.pa_decode_selected_blocks(out, d.q, d.k_cache, d.v_cache, d.block_tables, d.context_lens,
                                 sel, batch.scale, 0, ws)
    torch.cuda.synchronize()
    kb = R.update_key_bounds(torch.zeros(NB, H, 2, D, dtype=BF16), host_k, batch.block_tables,
                             batch.context_lens, batch.context_lens)
    want = R.select_blocks(batch.q, kb, batch.block_tables, batch.context_lens, bs, 12, 1, 2)
    assert torch.equal(sel.cpu(), want)
    ref = R.decode_selected(batch.q, host_k, host_v, batch.block_tables, batch.context_lens, want,
                            batch.scale)
    assert_close(out, ref, "step")
    assert pa.pa_device_error() == 0


def test_two_graphs_on_two_streams(pa):
    """Captured once, replayed from two streams at once with a workspace each:
    the same bits as the eager call, also after the inputs change in place."""
    batch = appended([1500, 40, 700, 2047], 16, 2, 128, 16, BF16, 309)
    d = batch.to(DEV)
    sel = random_lists(batch, 60, 310).to(DEV)
    n = pa.pa_decode_selected_blocks_workspace_size(4, 16, 2, 128, 16, 60, 64)
    assert n > 0
    runs = []
    for _ in range(2):
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(d.q)
        call = pa.prepare_decode_selected_blocks(out, d.q, d.k_cache, d.v_cache, d.block_tables,
                                                 d.context_lens, sel, batch.scale, 64, ws)
        call()
        torch.cuda.synchronize()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            call(stream=s)
        runs.append((g, s, out, call))
    eager = runs[0][2].clone()
    assert torch.equal(bits(eager), bits(runs[1][2]))
    for _ in range(20):
        for g, s, out, _ in runs:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
        torch.cuda.synchronize()
        for _, _, out, _ in runs:
            assert torch.equal(bits(out), bits(eager))
    d.q.mul_(-1.0)
    runs[0][0].replay()
    torch.cuda.synchronize()
    again = runs[0][2].clone()
    runs[1][3]()
    torch.cuda.synchronize()
    assert torch.equal(bits(again), bits(runs[1][2])) and not torch.equal(bits(again), bits(eager))


def test_binding_refuses_mismatched_tensors(pa):
    batch = appended([100, 40], 8, 2, 128, 16, BF16, 311)
    d = batch.to(DEV)
    sel = torch.full((2, 2, 20), -1, dtype=torch.int32, device=DEV)
    base = dict(out=torch.empty_like(d.q), q=d.q, k=d.k_cache, v=d.v_cache, t=d.block_tables,
                n=d.context_lens, s=sel, scale=0.1, part=0, ws=None)
    call = lambda **k: pa.pa_decode_selected_blocks(*{**base, **k}.values())
    call()
    for bad, err in ((dict(s=sel.long()), TypeError), (dict(s=sel[:1]), ValueError),
                     (dict(q=d.q.float()), ValueError), (dict(v=d.v_cache[:-1]), ValueError),
                     (dict(n=d.context_lens[:1]), ValueError), (dict(k=d.k_cache.cpu()), ValueError),
                     (dict(part=24), pa.PAError), (dict(part=16), pa.PAError),
                     (dict(scale=float("inf")), pa.PAError)):
        with pytest.raises(err):
            call(**bad)
    torch.cuda.synchronize()
