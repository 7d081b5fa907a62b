"""pa_select_blocks where scores reach the ends of the 32-bit range: rows of
equal, or nearly equal, lowest and largest values. The lists lie inside a larger
buffer whose other entries have to keep their value."""
import pytest
import torch

import sparse_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
MAX = torch.finfo(F32).max


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


def guarded_select(pa, q, bounds, tables, lens, bs, count, first, last):
    """The lists, and whether the buffer around them is as it was."""
    B, H, max_ctx = q.shape[0], bounds.shape[1], int(lens.max())
    pad = -(-max_ctx // bs) + 64
    buf = torch.full((2 * pad + B * H * count,), -77, dtype=torch.int32, device=DEV)
    sel = buf[pad:pad + B * H * count].view(B, H, count)
    pa.pa_select_blocks(sel, q.to(DEV), bounds.to(DEV), tables.to(DEV), lens.to(DEV), max_ctx, bs,
                        first, last)
    torch.cuda.synchronize()
    around = torch.cat((buf[:pad], buf[pad + B * H * count:]))
    return sel.cpu(), bool((around == -77).all())


def extreme_case(ctxs, dtype, D, value, seed):
    """One-hot queries (bf16: two ones) against bounds that make every score
    ``value`` up to a rounding."""
    g = torch.Generator().manual_seed(seed)
    H, bs = 2, 16
    width = max(-(-c // bs) for c in ctxs)
    NB = len(ctxs) * width
    tables = torch.randperm(NB, generator=g).reshape(len(ctxs), width).int()
    q = torch.zeros(len(ctxs), 3 * H, D, dtype=dtype)
    bounds = torch.zeros(NB, H, 2, D, dtype=dtype)
    q[:, :, 7] = 1.0
    bounds[..., 7] = value                     # (bf16: rounds past the range, see below)
    if dtype == BF16:
        most = torch.finfo(BF16).max
        sign = 1.0 if value > 0 else -1.0
        bounds[..., 7] = sign * most
        q[:, :, 40] = 1.0
        bounds[..., 40] = sign * (abs(value) - most)
    return q, bounds, tables, torch.tensor(ctxs, dtype=torch.int32)


@pytest.mark.parametrize("count,first,last", [(8, 1, 1), (1, 0, 0), (40, 3, 0)])
@pytest.mark.parametrize("ctxs", [[1600, 33, 1599], [48000, 47000]], ids=str)
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 128), (BF16, 64), (BF16, 128)])
def test_equal_scores_at_the_end_of_the_range(pa, dtype, D, sign, ctxs, count, first, last):
    """s - 2e (or s + 2e) is not a number of 32 bits: fp32 from 3.40281e38 on,
    bf16 from 3.40272e38 on."""
    value = sign * (MAX if dtype == F32 else 3.40275e38)
    q, bounds, tables, lens = extreme_case(ctxs, dtype, D, value, 611)
    s = R.block_scores(q[0], bounds, tables[0], 4, 0, 3)
    assert bool((s.abs() > 3.4027e38).all() and (s.abs() <= MAX).all())
    want = R.select_blocks(q, bounds, tables, lens, 16, count, first, last)
    got, kept = guarded_select(pa, q, bounds, tables, lens, 16, count, first, last)
    assert kept and torch.equal(got, want)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nearly_equal_scores_at_the_end_of_the_range(pa, dtype, sign):
    """Some blocks one unit in the last place nearer to zero, some of another
    size altogether, and one row of ordinary scores beside them."""
    q, bounds, tables, lens = extreme_case([1600, 1600, 1600], dtype, 128,
                                           sign * (MAX if dtype == F32 else 3.40275e38), 612)
    g = torch.Generator().manual_seed(613)
    few = tables[0, torch.randperm(100, generator=g)[:9]].long()
    at = 7 if dtype == F32 else 40
    bits = bounds[..., at].clone().view(torch.int32 if dtype == F32 else torch.int16)
    bits[few] -= 1
    bounds[..., at] = bits.view(dtype)
    far = tables[1, torch.randperm(100, generator=g)[:30]].long()
    bounds[far, :, :, 7] = torch.randn(30, 2, 2, generator=g).to(dtype)
    bounds[far, :, :, 40] = 0.0
    t = tables[2].long()
    bounds[t, :, :, 7] = torch.randn(100, 2, 2, generator=g).to(dtype)
    bounds[t, :, :, 40] = 0.0
    for count, first, last in ((1, 0, 0), (5, 0, 0), (20, 2, 3), (60, 1, 1), (98, 0, 1)):
        want = R.select_blocks(q, bounds, tables, lens, 16, count, first, last)
        got, kept = guarded_select(pa, q, bounds, tables, lens, 16, count, first, last)
        assert kept and torch.equal(got, want), (count, first, last)
    assert pa.pa_device_error() == 0


def test_lowest_values_as_a_mask(pa):
    """Blocks masked by finfo.min in every dimension, all of them or all but a
    few: the others come first, then the masked ones from the lowest index on."""
    for dtype in (F32, BF16):
        g = torch.Generator().manual_seed(614)
        q = torch.zeros(2, 4, 64, dtype=dtype)
        q[:, :, 5] = 1.0
        bounds = torch.full((200, 2, 2, 64), torch.finfo(dtype).min, dtype=dtype)
        tables = torch.arange(200, dtype=torch.int32).reshape(2, 100)
        bounds[[120, 150, 190]] = torch.randn(3, 2, 2, 64, generator=g).to(dtype)
        lens = torch.tensor([1600, 1600], dtype=torch.int32)
        want = R.select_blocks(q, bounds, tables, lens, 16, 9, 1, 1)
        assert want[0, 0].tolist() == list(range(8)) + [99]
        assert want[1, 0].tolist() == [0, 1, 2, 3, 4, 20, 50, 90, 99]
        got, kept = guarded_select(pa, q, bounds, tables, lens, 16, 9, 1, 1)
        assert kept and torch.equal(got, want)
    assert pa.pa_device_error() == 0
