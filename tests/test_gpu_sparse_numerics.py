"""How far the numbers behind the operators over part of a cache may be from
the 64-bit ones: decode outputs element by element, with the rounding of the
attention weights to bf16 counted in."""
import pytest
import torch

import sparse_reference as R
from helpers import oracle_after_append
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


def output_tolerance(batch):
    """An output's exact value, and how far off it may be, float64 [B, H_q, D].

    bf16, u = 2^-8 the largest relative rounding to it. The weights p become
    p (1 + d), |d| <= u, in numerator and denominator: 2 u / (1 - u) sum p |V|.
    A score is a sum of D products in steps of 16, each step off by at most
    18 * 2^-23 of what has been added up (D / 16 <= 8 steps: 2^-15 sum |q K|),
    and the weights by twice that times the scale, the exponential's own error
    (2^-20 at most) beside it. The sums of P V: at most 32 steps of 16 tokens in
    each of four warps, 32 * 18 * 2^-23 < 2^-13 sum p |V|. Then the output is
    rounded: u of it. fp32: u = 2^-24; sums of up to 2048 terms in 32 bits,
    2048 * 2^-24 = 2^-13 of sum p |V| at most."""
    u = 2.0 ** -8 if batch.q.dtype == BF16 else 2.0 ** -24
    B, H_q, D = batch.q.shape
    G = H_q // batch.num_kv_heads
    exact = torch.zeros(B, H_q, D, dtype=torch.float64)
    off = torch.zeros_like(exact)
    for b, ctx in enumerate(batch.context_lens.tolist()):
        for h in range(batch.num_kv_heads):
            k = R.tokens(batch.k_cache, batch.block_tables[b], ctx, h)
            v = R.tokens(batch.v_cache, batch.block_tables[b], ctx, h)
            rows = slice(h * G, (h + 1) * G)
            q = batch.q[b, rows].double()
            o, p = R.attend(q, k, v, batch.scale)
            score = 2 * batch.scale * 2.0 ** -15 * (q.abs() @ k.abs().T).amax(-1, keepdim=True)
            mass = p @ v.abs()
            exact[b, rows] = o
            off[b, rows] = (2 * u / (1 - u) + 2 * score + 2.0 ** -20 + 2.0 ** -13) * mass + u * o.abs()
    return exact, off * (1 + u)


@pytest.mark.parametrize("shape", [([40, 1500, 777, 2000], 8, 2, 128, 16, BF16),
                                   ([1, 2048, 130], 5, 1, 64, 32, BF16),
                                   ([300, 2000], 16, 8, 128, 64, F32)], ids=str)
def test_outputs_element_by_element(pa, shape):
    ctxs, hq, hkv, D, bs, dtype = shape
    nb = sum(-(-c // bs) for c in ctxs) + 4
    batch = W.decode_batch(ctxs, hq, hkv, D, bs, nb, dtype, seed=601)
    batch.k_cache, batch.v_cache = oracle_after_append(batch)
    exact, off = output_tolerance(batch)
    d = batch.to(DEV)
    B, width = d.block_tables.shape
    sel = torch.arange(width, dtype=torch.int32, device=DEV).repeat(B, hkv, 1)
    sel = torch.where(sel * bs < d.context_lens[:, None, None], sel, -1).contiguous()
    outs = {}
    for part in (0, 256):
        n = pa.pa_decode_selected_blocks_workspace_size(B, hq, hkv, D, bs, width, part)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
        outs["selected", part] = torch.empty_like(d.q)
        pa.pa_decode_selected_blocks(outs["selected", part], d.q, d.k_cache, d.v_cache,
                                     d.block_tables, d.context_lens, sel, batch.scale, part, ws)
        n = pa.pa_decode_accumulate_weights_workspace_size(B, hq, D, max(ctxs), part)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        outs["weights", part] = torch.empty_like(d.q)
        w = torch.empty(B, hkv, max(ctxs), device=DEV)
        pa.pa_decode_accumulate_weights(outs["weights", part], w, None, d.q, d.k_cache, d.v_cache,
                                        d.block_tables, d.context_lens, max(ctxs), batch.scale,
                                        part, ws)
    torch.cuda.synchronize()
    for name, out in outs.items():
        err = (out.cpu().double() - exact).abs()
        assert bool((err <= off).all()), (name, (err / off).max().item())
    assert pa.pa_device_error() == 0


# ---------------------------------------------------------------- block scores
def score_inputs(kind, dtype, D, group, seed):
    """q [B, H_q, D], bounds [NB, H, 2, D] and tables whose scores have terms of
    the given kind."""
    g = torch.Generator().manual_seed(seed)
    B, H, n = 2, 2, 700
    NB = B * n
    rand = lambda *s: torch.randn(*s, generator=g)
    q, bounds = rand(B, H * group, D), rand(NB, H, 2, D)
    if kind == "cancelling":         # pairs of large terms that leave a small sum
        q = q.abs() + 0.5
        q[..., 1::2] = q[..., ::2]
        bounds *= 2.0 ** -9
        big = 2.0 ** torch.randint(0, 12, (NB, H, 1, D // 2), generator=g).float()
        bounds[..., ::2] += big
        bounds[..., 1::2] -= big
    elif kind == "wide":             # exponents over 2^-60 .. 2^60 in one sum
        q *= 2.0 ** torch.randint(-30, 31, q.shape, generator=g).float()
        bounds *= 2.0 ** torch.randint(-30, 31, bounds.shape, generator=g).float()
    elif kind == "cut":              # few large terms, the rest just at what a sum keeps beside them
        q[:] = 1.0
        small = 1.0 + torch.rand(NB, H, 2, D, generator=g)
        bounds = small * 2.0 ** torch.randint(-26, -20, bounds.shape, generator=g).float()
        bounds[..., ::16] = 1.0 + torch.rand(NB, H, 2, D // 16, generator=g)
        bounds[NB // 2:, ..., 16:32] *= -1.0
    elif kind == "tiny":             # products below the smallest number of 32 bits
        q *= 2.0 ** -70
        bounds *= 2.0 ** torch.randint(-80, -60, bounds.shape, generator=g).float()
    elif kind == "subnormal":        # operands below 2^-126, and products that are not
        q *= 2.0 ** 100
        bounds *= 2.0 ** torch.randint(-132, -125, bounds.shape, generator=g).float()
    elif kind == "large":            # sums near the end of the range
        q *= 2.0 ** 60
        bounds *= 2.0 ** 59
    tables = torch.randperm(NB, generator=g).reshape(B, n).int()
    return q.to(dtype), bounds.to(dtype), tables


@pytest.mark.parametrize("kind", ["normal", "cancelling", "wide", "cut", "tiny", "subnormal",
                                  "large"])
@pytest.mark.parametrize("group", [1, 5, 16])
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
def test_scores_are_within_their_error_bounds(pa, dtype, D, group, kind):
    """The workspace holds a 32-bit score and its error bound for every contested
    block; the 64-bit score lies within. (The 64-bit one is itself off by less
    than 2 D * 2^-53 of its terms' sum, 2^-28 of the least bound here.)"""
    bs, count, first, last = 16, 30, 2, 1
    q, bounds, tables = score_inputs(kind, dtype, D, group, 620 + group)
    B, n = tables.shape
    H = bounds.shape[1]
    lens = torch.full((B,), n * bs, dtype=torch.int32)
    size = pa.pa_select_blocks_workspace_size(B, H, bs, n * bs)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    sel = torch.empty(B, H, count, dtype=torch.int32, device=DEV)
    pa.pa_select_blocks(sel, q.to(DEV), bounds.to(DEV), tables.to(DEV), lens.to(DEV), n * bs, bs,
                        first, last, ws)
    torch.cuda.synchronize()
    middle = n - first - last
    entry = ws.cpu().view(torch.int64).view(B, H, n)[..., :middle]
    key = (entry >> 32) & 0xffffffff
    pattern = torch.where(key >= 1 << 31, key & 0x7fffffff, key ^ 0xffffffff)
    low = lambda x: torch.where(x >= 1 << 31, x - (1 << 32), x).int().view(torch.float32).double()
    score, off = low(pattern), low(entry & 0xffffffff)
    exact = torch.stack([torch.stack([R.block_scores(q[b], bounds, tables[b], n, h, group)
                                      for h in range(H)]) for b in range(B)])
    exact = exact[..., first:n - last]
    bounded = torch.isfinite(off)
    assert bool(bounded.all()) or kind == "large"
    assert int(bounded.sum()) > 0
    ratio = ((score - exact).abs() / off)[bounded].max().item()
    print(f"{kind} {dtype} D {D} group {group}: {ratio:.3f} of the bound")
    assert ratio <= 1.0
    # and what is selected by them is the 64-bit choice
    want = R.select_blocks(q, bounds, tables, lens, bs, count, first, last)
    assert torch.equal(sel.cpu(), want)
    assert pa.pa_device_error() == 0
