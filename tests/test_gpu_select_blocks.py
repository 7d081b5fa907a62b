"""pa_update_key_bounds and pa_select_blocks on the GPU: the bounds equal the
minimum and maximum of each touched block's valid keys bit for bit and nothing
else changes; the selection equals the one by 64-bit scores index for index,
ties and NaN included. The keys are poisoned with NaN past each row's length,
so a bound over an invalid token shows."""
import pytest
import torch

import sparse_reference as R
from helpers import bits, oracle_after_append
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


def appended(ctxs, hq, hkv, D, bs, dtype, seed, **kw):
    nb = sum(-(-c // bs) for c in ctxs) + 4
    batch = W.decode_batch(ctxs, hq, hkv, D, bs, nb, dtype, seed=seed, **kw)
    batch.k_cache, batch.v_cache = oracle_after_append(batch)
    return batch


def new_bounds(batch, value=7.0):
    NB, H, _, D = batch.k_cache.shape
    return torch.full((NB, H, 2, D), value, dtype=batch.k_cache.dtype)


SHAPES = [  # ctxs, q heads, kv heads, D, block, dtype
    ([1, 16, 17, 40, 0], 4, 4, 64, 16, F32),
    ([5, 63, 64, 65, 200], 8, 2, 128, 16, BF16),
    ([1, 31, 32, 33, 300], 6, 2, 64, 32, BF16),
    ([2, 64, 129, 500], 16, 1, 128, 64, BF16),
    ([7, 190], 3, 3, 128, 64, F32),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bounds_of_whole_rows(pa, shape):
    ctxs, hq, hkv, D, bs, dtype = shape
    batch = appended(ctxs, hq, hkv, D, bs, dtype, 201)
    want = R.update_key_bounds(new_bounds(batch), batch.k_cache, batch.block_tables,
                               batch.context_lens, batch.context_lens)
    d = batch.to(DEV)
    got = new_bounds(batch).to(DEV)
    pa.pa_update_key_bounds(got, d.k_cache, d.block_tables, d.context_lens, d.context_lens,
                            max(ctxs))
    assert torch.equal(bits(got.cpu()), bits(want))
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("new", [1, 2, 16, 17, 33])
def test_bounds_step_by_step(pa, new):
    """Only the blocks of the last ``new`` tokens change; the others keep what
    they held, and rows with nothing new keep everything."""
    ctxs = [new, new + 1, 50 + new, 64, 65 + new, 130 + new]
    batch = appended(ctxs, 8, 2, 128, 16, BF16, 202)
    new_lens = torch.tensor([min(new, c) for c in ctxs], dtype=torch.int32)
    new_lens[2] = 0
    want = R.update_key_bounds(new_bounds(batch), batch.k_cache, batch.block_tables,
                               batch.context_lens, new_lens)
    d = batch.to(DEV)
    got = new_bounds(batch).to(DEV)
    pa.pa_update_key_bounds(got, d.k_cache, d.block_tables, d.context_lens, new_lens.to(DEV), new)
    assert torch.equal(bits(got.cpu()), bits(want))
    assert pa.pa_device_error() == 0


def test_bounds_of_special_values(pa):
    """NaN spreads to its dimension only; infinities are ordinary extremes."""
    for dtype in (BF16, F32):
        batch = appended([20], 2, 2, 64, 16, dtype, 203)
        t = batch.block_tables
        batch.k_cache[t[0, 0], 0, 3, 5] = float("nan")
        batch.k_cache[t[0, 0], 1, 4, 6] = float("inf")
        batch.k_cache[t[0, 1], 1, 2, 7] = float("-inf")
        d = batch.to(DEV)
        got = new_bounds(batch).to(DEV)
        pa.pa_update_key_bounds(got, d.k_cache, d.block_tables, d.context_lens, d.context_lens, 20)
        g = got.cpu()
        want = R.update_key_bounds(new_bounds(batch), batch.k_cache, t, batch.context_lens,
                                   batch.context_lens)
        assert torch.equal(torch.isnan(g), torch.isnan(want))
        assert torch.equal(g.nan_to_num(3.0), want.nan_to_num(3.0))
        assert torch.isnan(g[t[0, 0], 0, :, 5]).all() and int(torch.isnan(g).sum()) == 2
    assert pa.pa_device_error() == 0


def test_bounds_bad_rows_are_clamped_and_recorded(pa):
    batch = appended([40, 50, 30], 4, 2, 64, 16, BF16, 204)
    d = batch.to(DEV)
    # a block id outside the pool: that block is skipped
    d.block_tables[1, 1] = batch.num_blocks
    new = torch.tensor([40, 50, 30], dtype=torch.int32)
    want = new_bounds(batch)
    R.update_key_bounds(want, batch.k_cache, batch.block_tables, batch.context_lens, new)
    want[batch.block_tables[1, 1].long()] = 7.0
    got = new_bounds(batch).to(DEV)
    pa.pa_update_key_bounds(got, d.k_cache, d.block_tables, d.context_lens, new.to(DEV), 64)
    assert torch.equal(bits(got.cpu()), bits(want))
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE
    # more new tokens than the host's bound, or than the row has; a negative count
    d = batch.to(DEV)
    for bad, use in (([41, 1, 1], [40, 1, 1]), ([1, 48, 1], [1, 40, 1]), ([1, -3, 1], [1, 0, 1])):
        want = R.update_key_bounds(new_bounds(batch), batch.k_cache, batch.block_tables,
                                   batch.context_lens, torch.tensor(use))
        got = new_bounds(batch).to(DEV)
        pa.pa_update_key_bounds(got, d.k_cache, d.block_tables, d.context_lens,
                                torch.tensor(bad, dtype=torch.int32, device=DEV), 40)
        assert torch.equal(bits(got.cpu()), bits(want)), bad
        assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE, bad


# ---------------------------------------------------------------- selection
def run_select(pa, q, bounds, tables, lens, max_ctx, bs, count, first, last):
    B, H = q.shape[0], bounds.shape[1]
    got = torch.full((B, H, count), -7, dtype=torch.int32, device=DEV)
    pa.pa_select_blocks(got, q.to(DEV), bounds.to(DEV), tables.to(DEV), lens.to(DEV), max_ctx, bs,
                        first, last)
    return got.cpu()


def bounds_case(ctxs, hq, hkv, D, bs, dtype, seed):
    """q, bounds, tables and lengths without the cache behind them."""
    g = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-c // bs) for c in ctxs))
    NB = len(ctxs) * width + 3
    a = torch.randn(NB, hkv, D, generator=g)
    b = torch.randn(NB, hkv, D, generator=g)
    bounds = torch.stack((torch.minimum(a, b) - 1, torch.maximum(a, b) + 1), 2).to(dtype)
    tables = torch.randperm(NB, generator=g)[:len(ctxs) * width].reshape(-1, width).int()
    q = torch.randn(len(ctxs), hq, D, generator=g).to(dtype)
    return q, bounds, tables, torch.tensor(ctxs, dtype=torch.int32)


@pytest.mark.parametrize("count,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (4, 1, 1),
                                              (7, 0, 2), (8, 4, 4), (16, 2, 0), (64, 1, 2)])
@pytest.mark.parametrize("shape", [
    ([0, 1, 16, 17, 100, 255, 256, 257], 4, 4, 64, 16, F32),
    ([1000, 31, 0, 999, 1024], 8, 2, 128, 16, BF16),
    ([3000, 64, 65, 2048], 3, 1, 64, 64, BF16),
    ([2000, 500], 40, 2, 128, 32, BF16),
    ([777], 16, 2, 128, 16, F32),
], ids=str)
def test_selection_equals_the_64_bit_one(pa, shape, count, first, last):
    ctxs, hq, hkv, D, bs, dtype = shape
    q, bounds, tables, lens = bounds_case(ctxs, hq, hkv, D, bs, dtype, 205 + count)
    want = R.select_blocks(q, bounds, tables, lens, bs, count, first, last)
    got = run_select(pa, q, bounds, tables, lens, max(ctxs), bs, count, first, last)
    assert torch.equal(got, want)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("batch", [1, 3, 40])
def test_selection_of_long_rows(pa, batch):
    """Rows of thousands of blocks, at every cluster size the batch leads to."""
    ctxs = [40000 - 701 * (i % 7) for i in range(batch)]
    q, bounds, tables, lens = bounds_case(ctxs, 8, 2, 64, 16, BF16, 206)
    want = R.select_blocks(q, bounds, tables, lens, 16, 200, 3, 5)
    got = run_select(pa, q, bounds, tables, lens, max(ctxs), 16, 200, 3, 5)
    assert torch.equal(got, want)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (64, F32), (128, F32)])
def test_selection_of_many_short_rows(pa, D, dtype):
    ctxs = [1 + (37 * i) % 700 for i in range(320)]
    q, bounds, tables, lens = bounds_case(ctxs, 4, 2, D, 16, dtype, 220)
    bounds[tables[5].long()] = bounds[tables[5, 0].long()].clone()   # a row of equal blocks
    want = R.select_blocks(q, bounds, tables, lens, 16, 9, 1, 1)
    assert torch.equal(run_select(pa, q, bounds, tables, lens, 700, 16, 9, 1, 1), want)
    assert pa.pa_device_error() == 0


def test_equal_scores_go_to_the_lowest_index(pa):
    for dtype in (BF16, F32):
        q, bounds, tables, lens = bounds_case([1600, 3200], 8, 2, 128, 16, dtype, 207)
        bounds[:] = bounds[0]            # every block the same
        want = R.select_blocks(q, bounds, tables, lens, 16, 20, 2, 3)
        assert want[0, 0].tolist() == list(range(17)) + [97, 98, 99]
        assert torch.equal(run_select(pa, q, bounds, tables, lens, 3200, 16, 20, 2, 3), want)
        # a zero query: every score is zero, of either sign
        q[0] = 0.0
        q[1] = -0.0
        assert torch.equal(run_select(pa, q, bounds, tables, lens, 3200, 16, 20, 2, 3), want)
        # a few values only: many ties around the border
        q, bounds, tables, lens = bounds_case([1600, 3200], 4, 2, 64, 16, dtype, 208)
        q[:] = 0
        q[:, :, 0] = 1
        bounds[:, :, :, 0] = bounds[:, :, :, 0].round()
        want = R.select_blocks(q, bounds, tables, lens, 16, 33, 1, 1)
        assert torch.equal(run_select(pa, q, bounds, tables, lens, 3200, 16, 33, 1, 1), want)


def test_scores_that_agree_to_32_bits(pa):
    """Blocks whose scores differ by less than 32 bits resolve: large terms that
    cancel in the sum leave the difference of two small ones."""
    for dtype, big in ((BF16, 2.0 ** 12), (F32, 2.0 ** 12)):
        q, bounds, tables, lens = bounds_case([1600], 4, 2, 128, 16, dtype, 209)
        q.abs_().clamp_(min=0.25)
        q[:, :, 0] = 1.0
        q[:, :, 1] = 1.0
        bounds[:] = 0.0
        bounds[:, :, 1, 0] = big
        bounds[:, :, 1, 1] = -big
        bounds[:, :, 0, 1] = -big
        g = torch.Generator().manual_seed(210)
        tiny = torch.randint(1, 1 << 7, bounds[:, :, 1, 2].shape, generator=g).float() * 2.0 ** -18
        bounds[:, :, 1, 2] = tiny.to(dtype)
        want = R.select_blocks(q, bounds, tables, lens, 16, 10, 0, 0)
        assert torch.equal(run_select(pa, q, bounds, tables, lens, 1600, 16, 10, 0, 0), want)


@pytest.mark.parametrize("near", [2, 30, 256, 257, 1500])
@pytest.mark.parametrize("batch", [1, 20])
def test_many_scores_near_the_border(pa, near, batch):
    """``near`` blocks whose scores differ in the last bits only, with clear
    winners and clear losers around them and equal ones among them."""
    n = 2000
    q, bounds, tables, lens = bounds_case([n * 16] * batch, 8, 2, 128, 16, BF16, 216)
    g = torch.Generator().manual_seed(217)
    q.abs_().clamp_(min=0.25)
    q[:, :, :3] = 1.0
    bounds[:] = 0.0
    bounds[:, :, 1, 0] = 2.0 ** 10
    bounds[:, :, :, 1] = -2.0 ** 10
    # all blocks far down, then `near` of them at the border, then 20 far up
    bounds[:, :, 1, 3] = -3.0 - torch.rand(bounds[:, :, 1, 3].shape, generator=g).to(BF16)
    for b in range(batch):
        order = tables[b, torch.randperm(n, generator=g)].long()
        bounds[order[:near], :, 1, 3] = 0.0
        tiny = torch.randint(0, 1 << 7, (near, 2), generator=g).float() * 2.0 ** -18
        bounds[order[:near], :, 1, 2] = tiny.to(BF16)
        bounds[order[near:near + 20], :, 1, 2] = 5.0
        bounds[order[near:near + 20], :, 1, 3] = 0.0
    for count in (20 + near // 2, 21, 19 + near):
        want = R.select_blocks(q, bounds, tables, lens, 16, count, 0, 0)
        got = run_select(pa, q, bounds, tables, lens, n * 16, 16, count, 0, 0)
        assert torch.equal(got, want), count
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("group", [1, 8, 9, 33, 64, 65])
@pytest.mark.parametrize("D", [64, 128])
def test_group_sizes(pa, group, D):
    q, bounds, tables, lens = bounds_case([3000, 1700], 2 * group, 2, D, 16, BF16, 218)
    want = R.select_blocks(q, bounds, tables, lens, 16, 30, 1, 1)
    assert torch.equal(run_select(pa, q, bounds, tables, lens, 3000, 16, 30, 1, 1), want)


def test_fewer_good_blocks_than_places(pa):
    """Most of a row's ids are outside the pool: the good ones, then the lowest."""
    q, bounds, tables, lens = bounds_case([1600], 4, 2, 64, 16, BF16, 219)
    bad = torch.full_like(tables, -1)
    good = [90, 7, 33]
    bad[0, good] = tables[0, good]
    got = run_select(pa, q, bounds, bad, lens, 1600, 16, 8, 0, 1)
    assert got[0, 0].tolist() == [0, 1, 2, 3, 7, 33, 90, 99]
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE


def test_nan_and_infinite_scores(pa):
    """NaN ranks first, then +inf, ..., then -inf."""
    for dtype in (BF16, F32):
        q, bounds, tables, lens = bounds_case([1600], 2, 2, 64, 16, dtype, 211)
        q[:, :, 0] = 1.0
        t = tables[0].long()
        bounds[t[50], 0, 1, 3] = float("nan")
        bounds[t[60], 0, 1, 0] = float("inf")
        bounds[t[70], 0, 1, 0] = float("-inf")
        bounds[t[70], 0, 0, 0] = float("-inf")
        q[:, :, 3] = 0.5
        for count in (1, 2, 3, 99):
            want = R.select_blocks(q, bounds, tables, lens, 16, count, 0, 0)
            got = run_select(pa, q, bounds, tables, lens, 1600, 16, count, 0, 0)
            assert torch.equal(got, want), count
        # a NaN query makes every score NaN: the lowest indices
        q[0, 0, 9] = float("nan")
        got = run_select(pa, q, bounds, tables, lens, 1600, 16, 12, 1, 1)
        assert got[0, 0].tolist() == list(range(11)) + [99]
    # products beyond the 32-bit range are finite in 64 bits
    q, bounds, tables, lens = bounds_case([800], 2, 2, 64, 16, BF16, 212)
    want = R.select_blocks(q * 1e30, bounds * 1e30, tables, lens, 16, 9, 0, 0)
    got = run_select(pa, q * 1e30, bounds * 1e30, tables, lens, 800, 16, 9, 0, 0)
    assert torch.equal(got, want)


def test_selection_with_bad_tables_and_lengths(pa):
    q, bounds, tables, lens = bounds_case([1600, 1600], 4, 2, 64, 16, BF16, 213)
    want = R.select_blocks(q, bounds, tables, lens, 16, 10, 1, 1)
    best = int(want[0, 0, 4])
    bad = tables.clone()
    bad[0, best] = -1
    got = run_select(pa, q, bounds, bad, lens, 1600, 16, 10, 1, 1)
    assert best not in got[0, 0].tolist()
    assert torch.equal(got[1], want[1])
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE
    lens[1] = 5000  # clamped to max_context_len
    got = run_select(pa, q, bounds, tables, lens, 1600, 16, 10, 1, 1)
    assert torch.equal(got, want)
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE
    lens[1] = -5
    got = run_select(pa, q, bounds, tables, lens, 1600, 16, 10, 1, 1)
    assert torch.equal(got[0], want[0]) and torch.all(got[1] == -1)
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE


def test_empty_calls(pa):
    q, bounds, tables, lens = bounds_case([100], 4, 2, 64, 16, BF16, 214)
    sel = torch.empty(0, 2, 4, dtype=torch.int32, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    pa.pa_select_blocks(sel, q[:0].to(DEV), bounds.to(DEV), tables[:0].to(DEV), none, 100, 16)
    k = torch.zeros(bounds.shape[0], 2, 16, 64, dtype=BF16, device=DEV)
    pa.pa_update_key_bounds(bounds.to(DEV), k, tables[:0].to(DEV), none, none, 4)
    torch.cuda.synchronize()
    assert pa.pa_device_error() == 0


def test_binding_refuses_mismatched_tensors(pa):
    q, bounds, tables, lens = (t.to(DEV) for t in bounds_case([100], 4, 2, 64, 16, BF16, 215))
    sel = torch.empty(1, 2, 4, dtype=torch.int32, device=DEV)
    call = lambda **k: pa.pa_select_blocks(*[{**dict(
        selected=sel, q=q, b=bounds, t=tables, n=lens, m=100, bs=16), **k}[x]
        for x in ("selected", "q", "b", "t", "n", "m", "bs")])
    call()
    for bad, err in ((dict(q=q.float()), TypeError), (dict(q=q[:, :, :32]), ValueError),
                     (dict(selected=sel.long()), TypeError), (dict(selected=sel[:, :1]), ValueError),
                     (dict(n=lens.long()), TypeError), (dict(t=tables[0]), ValueError),
                     (dict(q=q.cpu()), ValueError), (dict(b=bounds[:, :, 0]), ValueError),
                     (dict(t=tables.t().contiguous().t()[:, ::2]), ValueError),
                     (dict(m=10 ** 6), pa.PAError), (dict(bs=8), pa.PAError)):
        with pytest.raises(err):
            call(**bad)
    torch.cuda.synchronize()
