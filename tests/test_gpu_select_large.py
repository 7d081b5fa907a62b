"""pa_select_blocks where one scoring warp takes several tiles of a row, and
float32 rows of thousands of blocks: index for index against 64-bit scores that
the GPU computes from the formula, with ragged rows that end inside a later
stride, ids outside the pool there, and scores that 32 bits do not tell apart."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
BS = 16


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


def tiles_per_warp(B, H, n, dtype):
    """The library's rule: the tiles of a row (16 blocks in bf16, 4 in fp32) that a
    warp scores one behind the other."""
    tiles = -(-n // (16 if dtype == BF16 else 4))
    steps = 1
    while steps < 4 and B * H * tiles > 8 * 148 * 4 * 4 * steps:
        steps *= 2
    return steps


def make(B, H, group, n, D, dtype, seed, NB=5000):
    """Rows of up to n blocks out of one pool of NB, on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    bounds = torch.randn(NB, H, 2, D, generator=g, device=DEV).sort(dim=2).values.to(dtype)
    q = torch.randn(B, H * group, D, generator=g, device=DEV).to(dtype)
    tables = torch.stack([torch.randperm(NB, generator=g, device=DEV)[:n] for _ in range(B)]).int()
    return q, bounds, tables


def reference(q, bounds, tables, blocks, count, first, last):
    """Lists by a stable sort of 64-bit scores; ids outside the pool rank last."""
    B, n = tables.shape
    NB, H, _, D = bounds.shape
    out = torch.full((B, H, count), -1, dtype=torch.int32)
    for b, m in enumerate(blocks):
        if m <= count:
            out[b, :, :m] = torch.arange(m, dtype=torch.int32)
            continue
        ids = tables[b, :m].long()
        bad = (ids < 0) | (ids >= NB)
        kb = bounds[ids.clamp(0, NB - 1)].double()
        s = None
        for x in q[b].double().view(H, -1, D).unbind(1):
            one = (x.clamp(min=0) * kb[:, :, 1] + x.clamp(max=0) * kb[:, :, 0]).sum(-1)
            s = one if s is None else torch.maximum(s, one)
        s = s.masked_fill(bad[:, None], -float("inf")).t()          # [H, m]
        order = s[:, first:m - last].sort(dim=-1, descending=True, stable=True).indices
        mid = order[:, :count - first - last].sort(dim=-1).values + first
        out[b, :, :first] = torch.arange(first, dtype=torch.int32)
        out[b, :, first:count - last] = mid.int().cpu()
        out[b, :, count - last:] = torch.arange(m - last, m, dtype=torch.int32)
    return out


def select(pa, q, bounds, tables, lens, count, first, last):
    sel = torch.full((q.shape[0], bounds.shape[1], count), -7, dtype=torch.int32, device=DEV)
    pa.pa_select_blocks(sel, q, bounds, tables, lens, tables.shape[1] * BS, BS, first, last)
    torch.cuda.synchronize()
    return sel.cpu()


def ragged(B, n, tiles_at_once):
    """Lengths in blocks around the strides' ends, long and short ones between."""
    at = [n, n - 1, tiles_at_once, tiles_at_once + 1, tiles_at_once - 1, 2 * tiles_at_once + 5,
          3 * tiles_at_once - 7, 50, 1, 0]
    return [min(n, max(0, at[i % len(at)] - (i // len(at)) % 3)) for i in range(B)]


# rows, K/V heads, group, blocks, D, type, tiles of a warp
@pytest.mark.parametrize("B,H,group,n,D,dtype,steps", [
    (40, 8, 1, 900, 64, BF16, 1), (40, 8, 3, 1000, 64, BF16, 2), (48, 8, 1, 2003, 128, BF16, 4),
    (700, 2, 9, 450, 64, BF16, 4), (8, 8, 2, 900, 64, F32, 1), (12, 8, 2, 1001, 64, F32, 2),
    (30, 4, 1, 2100, 128, F32, 4), (200, 2, 5, 600, 64, F32, 4)], ids=str)
def test_several_tiles_to_a_warp(pa, B, H, group, n, D, dtype, steps):
    assert tiles_per_warp(B, H, n, dtype) == steps
    q, bounds, tables = make(B, H, group, n, D, dtype, 641)
    tile = 16 if dtype == BF16 else 4
    stride = -(-(-(-n // tile)) // steps) * tile       # blocks between a warp's tiles
    blocks = ragged(B, n, stride)
    lens = torch.tensor([max(0, m * BS - (i * 5) % BS) for i, m in enumerate(blocks)],
                        dtype=torch.int32, device=DEV)
    for count, first, last in ((60, 2, 3), (1, 0, 0), (200, 0, 7)):
        want = reference(q, bounds, tables, blocks, count, first, last)
        assert torch.equal(select(pa, q, bounds, tables, lens, count, first, last), want)
    assert pa.pa_device_error() == 0
    # ids outside the pool in every stride of a row: they are not chosen
    g = torch.Generator().manual_seed(642)
    for b in range(0, B, 3):
        for s in range(0, blocks[b], stride):
            width = min(stride, blocks[b] - s)
            tables[b, s + torch.randint(width, (1 + width // 9,), generator=g)] = \
                -1 if b % 2 else bounds.shape[0]
    want = reference(q, bounds, tables, blocks, 60, 2, 3)
    assert torch.equal(select(pa, q, bounds, tables, lens, 60, 2, 3), want)
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE


@pytest.mark.parametrize("n", [2049, 5000, 24576, 24577, 40000])
@pytest.mark.parametrize("D", [64, 128])
def test_long_rows_in_fp32(pa, D, n):
    """More than 2048 blocks, and more than a CTA's shared memory holds."""
    q, bounds, tables = make(2, 2, 3, n, D, F32, 643, NB=n)
    blocks = [n, n - 17]
    lens = torch.tensor([m * BS for m in blocks], dtype=torch.int32, device=DEV)
    for count, first, last in ((700, 3, 4), (1, 0, 0), (n - 20, 1, 1)):
        want = reference(q, bounds, tables, blocks, count, first, last)
        assert torch.equal(select(pa, q, bounds, tables, lens, count, first, last), want)
    # three kinds of blocks: no bin narrows the border down
    g = torch.Generator(device=DEV).manual_seed(644)
    bounds[1:] = bounds[torch.randint(0, 3, (n - 1,), generator=g, device=DEV)].clone()
    want = reference(q, bounds, tables, blocks, 700, 3, 4)
    assert torch.equal(select(pa, q, bounds, tables, lens, 700, 3, 4), want)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("near", [2, 30, 256, 257, 1500])
@pytest.mark.parametrize("n", [2000, 2500])
def test_many_fp32_scores_near_the_border(pa, n, near):
    """``near`` blocks whose scores differ by less than 32 bits hold of their
    terms, clear winners and losers around them and equal ones among them. All
    terms are multiples of 2^-18 below 2^12: sums in 64 bits are exact."""
    q, bounds, tables = make(2, 2, 2, n, 128, F32, 645, NB=2 * n)
    g = torch.Generator(device=DEV).manual_seed(646)
    q[:] = 0.0
    q[:, :, :4] = 1.0
    bounds[:] = 0.0
    bounds[:, :, 1, 0] = 2.0 ** 10
    bounds[:, :, :, 1] = -2.0 ** 10
    far = torch.rand(bounds[:, :, 1, 3].shape, generator=g, device=DEV)
    bounds[:, :, 1, 3] = -3.0 - (far * 64).floor() / 64
    tables = torch.randperm(2 * n, generator=g, device=DEV).int().view(2, n)
    for b in range(2):
        order = tables[b, torch.randperm(n, generator=g, device=DEV)].long()
        bounds[order[:near], :, 1, 3] = 0.0
        tiny = torch.randint(0, 1 << 7, (near, 2), generator=g, device=DEV).float() * 2.0 ** -18
        bounds[order[:near], :, 1, 2] = tiny
        bounds[order[near:near + 20], :, 1, 2] = 5.0
        bounds[order[near:near + 20], :, 1, 3] = 0.0
    lens = torch.full((2,), n * BS, dtype=torch.int32, device=DEV)
    for count in (20 + near // 2, 21, 19 + near):
        want = reference(q, bounds, tables, [n, n], count, 0, 0)
        assert torch.equal(select(pa, q, bounds, tables, lens, count, 0, 0), want), count
    assert pa.pa_device_error() == 0
