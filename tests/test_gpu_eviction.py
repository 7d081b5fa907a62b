"""pa_decode_accumulate_weights and pa_evict_tokens on the GPU.

The weights are compared with the 64-bit form. Their tolerance: a score in base
2 is a sum of D products, rounded (or truncated, on the tensor cores) to 32
bits at most D + 8 times relative to A = scale * log2(e) * sum_d |q_d k_d|, an
absolute error of (D + 8) * 2^-23 * A; numerator and denominator of a weight
both carry it, as a relative error of ln 2 times that; exp2 and the sums add a
few units of 2^-23, and the addition to the old weight one."""
import math

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


def appended(ctxs, hq, hkv, D, bs, dtype, seed, extra=4, **kw):
    nb = sum(-(-c // bs) for c in ctxs) + extra
    batch = W.decode_batch(ctxs, hq, hkv, D, bs, nb, dtype, seed=seed, **kw)
    batch.k_cache, batch.v_cache = oracle_after_append(batch)
    return batch


# ------------------------------------------------------------------- weights
def run_weights(pa, d, part, weights_out, weights_in, max_ctx=None):
    B, H_q, D = d.q.shape
    max_ctx = max_ctx or d.max_context_len
    n = pa.pa_decode_accumulate_weights_workspace_size(B, H_q, D, max_ctx, part)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device=DEV)
    out = torch.full_like(d.q, float("nan"))
    pa.pa_decode_accumulate_weights(out, weights_out, weights_in, d.q, d.k_cache, d.v_cache,
                                    d.block_tables, d.context_lens, max_ctx, d.scale, part, ws)
    torch.cuda.synchronize()
    return out


def check_weights(batch, got, before, want):
    """got: new weights; before: what the buffer held; want: NaN past each row."""
    H, bs = batch.num_kv_heads, batch.block_size
    G, D = batch.num_q_heads // H, batch.head_dim
    got = got.cpu().double()
    for b, ctx in enumerate(batch.context_lens.tolist()):
        assert torch.equal(got[b, :, ctx:].nan_to_num(-3), before[b, :, ctx:].double().cpu()
                           .nan_to_num(-3)), "positions past the row were written"
        for h in range(H):
            if ctx == 0:
                continue
            k = R.tokens(batch.k_cache, batch.block_tables[b], ctx, h)
            q = batch.q[b, h * G:(h + 1) * G].double()
            A = batch.scale * math.log2(math.e) * (q.abs() @ k.abs().T).max().item()
            p = torch.softmax(batch.scale * (q @ k.T), -1).sum(0)
            tol = p * (2 * math.log(2) * (D + 8) * 2.0 ** -23 * A + 8 * 2.0 ** -23)
            tol = tol + 2.0 ** -23 * want[b, h, :ctx].abs()
            err = (got[b, h, :ctx] - want[b, h, :ctx]).abs()
            assert torch.all(err <= tol), (b, h, (err / tol).max().item())


SHAPES = [
    ([5, 17, 33, 40, 0], 4, 4, 64, 16, F32),
    ([1, 130, 515], 16, 2, 128, 16, F32),
    ([5, 63, 64, 65, 200, 0], 8, 2, 128, 16, BF16),
    ([1, 31, 32, 33, 300], 6, 2, 64, 32, BF16),
    ([2, 64, 129, 1500, 1025], 20, 1, 128, 64, BF16),
    ([70, 1100], 140, 2, 64, 16, BF16),
]


@pytest.mark.parametrize("part", [0, -1, 16, 64])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_weights_against_the_64_bit_form(pa, shape, part):
    batch = appended(*shape, 401)
    d = batch.to(DEV)
    B, H = batch.num_seqs, batch.num_kv_heads
    for stride in (max(shape[0]), max(shape[0]) + 3):   # odd strides too
        g = torch.Generator().manual_seed(402)
        old = torch.rand(B, H, stride, generator=g)
        for b, ctx in enumerate(shape[0]):
            old[b, :, ctx:] = float("nan")  # never read
        ref, want = R.decode_weights(batch.q, batch.k_cache, batch.v_cache, batch.block_tables,
                                     batch.context_lens, batch.scale, old, stride)
        new = torch.full((B, H, stride), 5.0, device=DEV)
        out = run_weights(pa, d, part, new, old.to(DEV))
        assert_close(out, ref, f"out {shape} {part}")
        check_weights(batch, new, torch.full((B, H, stride), 5.0), want)
        # in place, and from nothing
        same = old.to(DEV)
        run_weights(pa, d, part, same, same)
        assert torch.equal(same.cpu().nan_to_num(-1)[:, :, :1], new.cpu()[:, :, :1]
                           .where(batch.context_lens[:, None, None] > 0, torch.tensor(-1.0)))
        check_weights(batch, same, old, want)
        zero = torch.full((B, H, stride), 5.0, device=DEV)
        run_weights(pa, d, part, zero, None)
        check_weights(batch, zero, torch.full((B, H, stride), 5.0), want - old.double())
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("part", [-1, 64])
def test_out_is_that_of_pa_decode(pa, dtype, part):
    batch = appended([1, 500, 333, 1024, 0], 8, 2, 128, 16, dtype, 403)
    d = batch.to(DEV)
    n = pa.pa_decode_workspace_size(5, 8, 128, 1024, part)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    want = torch.empty_like(d.q)
    pa.pa_decode(want, d.q, d.k_cache, d.v_cache, d.block_tables, d.context_lens, 1024,
                 batch.scale, part, ws)
    w = torch.zeros(5, 2, 1024, device=DEV)
    out = run_weights(pa, d, part, w, w)
    if dtype == BF16:
        assert torch.equal(bits(out), bits(want))
    else:  # the same sums in another order
        assert_close(out, want.double().cpu(), "out")
    # each query head hands out a weight of one
    total = w.double().sum(-1).cpu()
    assert torch.allclose(total[:4], torch.full((4, 2), 4.0, dtype=torch.float64), atol=1e-4)
    assert torch.all(total[4] == 0)


def test_weights_with_a_block_outside_the_pool(pa):
    """Its tokens have no weight, and the others' sum to one."""
    for dtype in (BF16, F32):
        batch = appended([100, 64], 4, 2, 64, 16, dtype, 404)
        d = batch.to(DEV)
        d.block_tables[0, 2] = batch.num_blocks + 5
        d.block_tables[1, :4] = -1
        w = torch.full((2, 2, 112), 9.0, device=DEV)
        out = run_weights(pa, d, 0, w, None)
        assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE
        w = w.cpu()
        assert torch.all(w[0, :, 32:48] == 0) and torch.all(w[0, :, 100:] == 9)
        assert torch.allclose(w[0, :, :100].sum(-1), torch.tensor(2.0), atol=1e-5)
        assert torch.all(w[1, :, :64] == 0) and torch.all(out[1] == 0)


def test_weights_longer_than_the_bound_are_clamped(pa):
    batch = appended([100, 40], 4, 2, 64, 16, BF16, 405)
    d = batch.to(DEV)
    w = torch.full((2, 2, 112), 9.0, device=DEV)
    run_weights(pa, d, 0, w, None, max_ctx=48)
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE
    assert torch.all(w[0, :, 48:] == 9) and torch.all(w[1, :, 40:] == 9)
    assert torch.allclose(w[0, :, :48].sum(-1), torch.tensor(2.0, device=DEV), atol=1e-5)


# ------------------------------------------------------------------ eviction
def evict_case(ctxs, hkv, D, bs, dtype, budget, seed, stride=None):
    """A poisoned batch, weights with ties and zeros, and fresh blocks to move
    into (a permutation of block ids the rows do not use)."""
    fresh = -(-budget // bs)
    batch = appended(ctxs, hkv, hkv, D, bs, dtype, seed, extra=4 + len(ctxs) * fresh)
    g = torch.Generator().manual_seed(seed + 1)
    stride = stride or max(ctxs)
    w = torch.rand(len(ctxs), hkv, stride, generator=g)
    w = torch.where(torch.rand(w.shape, generator=g) < 0.3, (w * 4).round() / 4, w)
    for b, c in enumerate(ctxs):
        w[b, :, c:] = float("nan")
    used = set(batch.block_tables.flatten().tolist())
    free = [i for i in range(batch.num_blocks) if i not in used]
    dst = torch.tensor(free[:len(ctxs) * fresh], dtype=torch.int32).reshape(len(ctxs), fresh)
    return batch, w, dst


def run_evict(pa, d, w_out, w_in, dst, budget, first, last, max_ctx=None):
    B, H = w_in.shape[:2]
    kept = torch.full((B, H, budget), -9, dtype=torch.int32, device=DEV)
    lens = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    pa.pa_evict_tokens(d.k_cache, d.v_cache, w_out, w_in, kept, lens, d.block_tables, dst,
                       d.context_lens, max_ctx or max(1, d.max_context_len), budget, first, last)
    torch.cuda.synchronize()
    return kept.cpu(), lens.cpu()


def check_evict(batch, w, dst, budget, first, last, d, w_out, w_before, kept, lens):
    """Everything the call leaves, the untouched parts of the pools included."""
    want = R.evict(w, batch.context_lens, budget, first, last)
    bs = batch.block_size
    k, v = batch.k_cache.clone(), batch.v_cache.clone()
    new_w = w_before.clone()
    for b, n in enumerate(batch.context_lens.tolist()):
        assert int(lens[b]) == min(n, budget)
        for h, row in enumerate(want[b]):
            assert kept[b, h, :len(row)].tolist() == row, (b, h)
            assert torch.all(kept[b, h, len(row):] == -1)
            new_w[b, h, :n] = 0
            for i, p in enumerate(row):
                s, t = int(batch.block_tables[b, p // bs]), int(dst[b, i // bs])
                k[t, h, i % bs] = batch.k_cache[s, h, p % bs]
                v[t, h, i % bs] = batch.v_cache[s, h, p % bs]
                new_w[b, h, i] = w[b, h, p]
    assert torch.equal(bits(d.k_cache.cpu()), bits(k))
    assert torch.equal(bits(d.v_cache.cpu()), bits(v))
    assert torch.equal(bits(w_out.cpu()), bits(new_w))


EVICT = [  # ctxs, kv heads, D, block, dtype, budget, first, last
    ([5, 17, 33, 40, 0, 1], 4, 64, 16, F32, 16, 1, 2),
    ([5, 17, 33, 40, 0, 1], 4, 64, 16, F32, 1, 0, 0),
    ([100, 63, 64, 65], 2, 128, 16, BF16, 64, 4, 16),
    ([100, 63, 64, 65], 2, 128, 16, BF16, 63, 0, 63),
    ([100, 63, 64, 65], 2, 128, 16, BF16, 33, 33, 0),
    ([300, 31, 32, 33], 3, 64, 32, BF16, 31, 0, 0),
    ([500, 700], 1, 128, 64, F32, 300, 10, 100),
    ([1500, 900, 1200], 2, 128, 64, BF16, 1000, 4, 200),
    ([40], 2, 64, 16, BF16, 100, 0, 0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", EVICT, ids=str)
def test_eviction(pa, case, in_place):
    ctxs, hkv, D, bs, dtype, budget, first, last = case
    batch, w, dst = evict_case(ctxs, hkv, D, bs, dtype, budget, 406, max(ctxs) + 5)
    if in_place:
        dst = batch.block_tables
    d = batch.to(DEV)
    w_in = w.to(DEV)
    w_out = w_in if in_place else torch.full_like(w_in, 5.0)
    before = w if in_place else torch.full_like(w, 5.0)
    kept, lens = run_evict(pa, d, w_out, w_in, dst.to(DEV), budget, first, last)
    check_evict(batch, w, dst, budget, first, last, d, w_out, before, kept, lens)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("rows", [1, 2, 30])
def test_eviction_of_long_rows_in_place(pa, rows):
    """Thousands of kept tokens, at the column widths and cluster sizes that
    the number of rows leads to; in place, where order matters."""
    ctxs = [9000 - 411 * (i % 5) for i in range(rows)]
    hkv = 2 if rows < 30 else 1
    for dtype, D in ((BF16, 128), (F32, 64)):
        batch, w, _ = evict_case(ctxs, hkv, D, 16, dtype, 16, 407)
        d = batch.to(DEV)
        w_in = w.to(DEV)
        dst = batch.block_tables
        kept, lens = run_evict(pa, d, w_in, w_in, dst.to(DEV), 5001, 3, 777)
        check_evict_fast(batch, w, 5001, 3, 777, d, w_in, kept, lens)
    assert pa.pa_device_error() == 0


def check_evict_fast(batch, w, budget, first, last, d, w_out, kept, lens):
    """check_evict for in-place calls with every row longer than the budget."""
    assert torch.all(lens == budget)
    bs = batch.block_size
    k, v = d.k_cache.cpu(), d.v_cache.cpu()
    for b, n in enumerate(batch.context_lens.tolist()):
        for h in range(w.shape[1]):
            mid = w[b, h, first:n - last].double()
            cut = mid.sort(descending=True).values[budget - first - last - 1]
            take = mid > cut
            tie = mid == cut
            take |= tie & (tie.cumsum(0) <= budget - first - last - int(take.sum()))
            at = torch.cat((torch.arange(first), first + take.nonzero()[:, 0],
                            torch.arange(n - last, n)))
            assert torch.equal(kept[b, h].long(), at)
            t = batch.block_tables[b].long()
            src = (t[at // bs], at % bs)
            to = torch.arange(budget)
            to = (t[to // bs], to % bs)
            assert torch.equal(bits(k[to[0], h, to[1]]), bits(batch.k_cache[src[0], h, src[1]]))
            assert torch.equal(bits(v[to[0], h, to[1]]), bits(batch.v_cache[src[0], h, src[1]]))
            new = torch.zeros(n)
            new[:budget] = w[b, h, at]
            assert torch.equal(w_out[b, h, :n].cpu(), new)
            rest = torch.arange(budget, n)  # freed positions keep their bytes
            assert torch.equal(bits(k[t[rest // bs], h, rest % bs]),
                               bits(batch.k_cache[t[rest // bs], h, rest % bs]))


def test_shared_prefix_into_fresh_blocks(pa):
    """Rows that share their first blocks move them into blocks of their own and
    compact the rest in place: the shared blocks keep their bytes."""
    nb = 40
    batch = W.decode_batch([100, 90, 120], 2, 2, 64, 16, nb, BF16, seed=408, groups=[0, 0, 0],
                           prefix=48)
    batch.k_cache, batch.v_cache = oracle_after_append(batch)
    t = batch.block_tables
    assert torch.equal(t[0, :3], t[1, :3])
    free = [i for i in range(nb) if i not in set(t.flatten().tolist())]
    dst = t.clone()
    dst[:, :3] = torch.tensor(free[:9], dtype=torch.int32).reshape(3, 3)
    g = torch.Generator().manual_seed(409)
    w = torch.rand(3, 2, 120, generator=g)
    d = batch.to(DEV)
    w_in = w.to(DEV)
    kept, lens = run_evict(pa, d, w_in, w_in, dst.to(DEV), 70, 2, 10)
    check_evict(batch, w, dst, 70, 2, 10, d, w_in, w, kept, lens)
    assert pa.pa_device_error() == 0


def test_special_weights(pa):
    """NaN, infinities and signed zeros: NaN first, equal values by position."""
    batch, w, dst = evict_case([64], 1, 64, 16, BF16, 10, 410)
    w[:] = 0.0
    w[0, 0, ::3] = -0.0
    w[0, 0, 50] = float("nan")
    w[0, 0, 20] = float("inf")
    w[0, 0, 30] = float("-inf")
    w[0, 0, 31:40] = -1.0
    d = batch.to(DEV)
    out = torch.full_like(w, 5.0).to(DEV)
    kept, lens = run_evict(pa, d, out, w.to(DEV), dst.to(DEV), 10, 0, 1)
    assert kept[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 20, 50, 63]
    kept, lens = run_evict(pa, batch.to(DEV), out, w.to(DEV),
                           batch.block_tables.to(DEV), 63, 0, 0)
    assert kept[0, 0].tolist() == [i for i in range(64) if i != 30]


@pytest.mark.parametrize("n", [2400, 9000])  # one CTA, a cluster
@pytest.mark.parametrize("close", [127, 128, 129, 2047, 2049])
def test_close_weights_around_the_cut(pa, n, close):
    """As many weights within 2^-10 of each other as a selecting CTA ranks
    directly, or sets aside, and one more or less; many of them equal, and the
    cut at the first, in the middle and at the last of them."""
    batch, _, _ = evict_case([n], 3, 64, 16, BF16, 16, 413)
    g = torch.Generator().manual_seed(414 + close)
    w = torch.full((1, 3, n), 2.0 ** -7)
    at = torch.randperm(n, generator=g)
    w[0, :, at[:close]] = 1 + torch.randint(0, 600, (3, close), generator=g) * 2.0 ** -20
    w[0, :, at[close:close + 100]] = 64.0
    for need in (1, close // 2, close - 1):
        d = batch.to(DEV)
        w_in = w.to(DEV)
        dst = batch.block_tables
        kept, lens = run_evict(pa, d, w_in, w_in, dst.to(DEV), 100 + need, 0, 0)
        check_evict(batch, w, dst, 100 + need, 0, 0, d, w_in, w, kept, lens)
    assert pa.pa_device_error() == 0


def test_bad_ids_and_lengths_are_recorded(pa):
    batch, w, dst = evict_case([64, 40], 2, 64, 16, BF16, 32, 411)
    want = R.evict(w, batch.context_lens, 32, 0, 0)
    d = batch.to(DEV)
    dst[0, 1] = batch.num_blocks
    out = torch.full_like(w, 5.0).to(DEV)
    kept, _ = run_evict(pa, d, out, w.to(DEV), dst.to(DEV), 32, 0, 0)
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE
    assert kept[0, 0].tolist() == want[0][0]
    got = d.k_cache.cpu()[dst[1].long(), 1].reshape(-1, 64)[:32]
    src = torch.tensor(want[1][1])
    t = batch.block_tables[1].long()
    assert torch.equal(bits(got), bits(batch.k_cache[t[src // 16], 1, src % 16]))
    # a length above the host's bound is clamped to it
    d = batch.to(DEV)
    d.context_lens[0] = 1000
    kept, lens = run_evict(pa, d, out, w.to(DEV), batch.block_tables.to(DEV), 32, 0, 0, max_ctx=64)
    assert pa.pa_device_error(clear=True) == pa.PA_ERR_BAD_TABLE
    assert kept[0, 0].tolist() == want[0][0] and lens.tolist() == [32, 32]


def test_a_decode_loop_with_eviction(pa):
    """Decode steps that collect weights, an eviction in place, and more steps
    on the compacted cache, each step against the 64-bit form on the tokens the
    cache then holds."""
    bs, H, G, D, steps = 16, 2, 4, 64, 3
    g = torch.Generator().manual_seed(412)
    ctx = [90, 50, 33]
    nb = 40
    batch = W.decode_batch([c + steps * 2 for c in ctx], H * G, H, D, bs, nb, BF16, seed=413)
    d = batch.to(DEV)
    table = batch.block_tables
    d.k_cache.copy_(torch.randn(d.k_cache.shape, generator=g).to(BF16))
    d.v_cache.copy_(torch.randn(d.v_cache.shape, generator=g).to(BF16))
    weights = torch.zeros(3, H, 128, device=DEV)
    ref_w = torch.zeros(3, H, 128, dtype=torch.float64)
    lens = torch.tensor(ctx, dtype=torch.int32)
    n = pa.pa_decode_accumulate_weights_workspace_size(3, H * G, D, 128)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def step():
        lens.add_(1)
        key, value, q = (torch.randn(s, generator=g).to(BF16)
                         for s in ((3, H, D), (3, H, D), (3, H * G, D)))
        slots = torch.stack([table[b, (int(lens[b]) - 1) // bs].long() * bs +
                             (int(lens[b]) - 1) % bs for b in range(3)])
        dl = lens.to(DEV)
        pa.pa_reshape_and_cache(key.to(DEV), value.to(DEV), d.k_cache, d.v_cache, slots.to(DEV))
        out = torch.empty(3, H * G, D, dtype=BF16, device=DEV)
        pa.pa_decode_accumulate_weights(out, weights, weights, q.to(DEV), d.k_cache, d.v_cache,
                                        d.block_tables, dl, int(lens.max()), 0.125, 0, ws)
        ref, new = R.decode_weights(q, d.k_cache.cpu(), d.v_cache.cpu(), table, lens, 0.125,
                                    ref_w, 128)
        assert_close(out, ref, "step")
        for b in range(3):
            ref_w[b, :, :int(lens[b])] = new[b, :, :int(lens[b])]
        assert torch.allclose(weights.cpu().double(), ref_w, rtol=1e-4, atol=1e-4)

    for _ in range(steps):
        step()
    kept = torch.empty(3, H, 40, dtype=torch.int32, device=DEV)
    new_lens = torch.empty(3, dtype=torch.int32, device=DEV)
    pa.pa_evict_tokens(d.k_cache, d.v_cache, weights, weights, kept, new_lens, d.block_tables,
                       d.block_tables, lens.to(DEV), int(lens.max()), 40, 2, 8)
    for b in range(3):
        m = min(int(lens[b]), 40)
        for h in range(H):
            at = kept[b, h, :m].long().cpu()
            moved = ref_w[b, h, at].clone()
            ref_w[b, h] = 0
            ref_w[b, h, :m] = moved
    lens.copy_(new_lens.cpu())
    assert lens.tolist() == [40, 40, 36]
    for _ in range(steps):
        step()
    assert pa.pa_device_error() == 0


def test_both_in_a_graph_on_another_stream(pa):
    batch, w, dst = evict_case([500, 77, 300], 2, 128, 16, BF16, 100, 414)
    d = batch.to(DEV)
    s = torch.cuda.Stream()
    n = pa.pa_decode_accumulate_weights_workspace_size(3, 2, 128, 500, 64)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(d.q)
    old = torch.where(torch.isnan(w), torch.zeros(()), w).to(DEV)
    new, new2 = torch.zeros_like(old), torch.zeros_like(old)
    kept = torch.empty(3, 2, 100, dtype=torch.int32, device=DEV)
    lens = torch.empty(3, dtype=torch.int32, device=DEV)
    calls = [pa.prepare_decode_accumulate_weights(out, new, old, d.q, d.k_cache, d.v_cache,
                                                  d.block_tables, d.context_lens, 500,
                                                  batch.scale, 64, ws),
             pa.prepare_evict_tokens(d.k_cache, d.v_cache, new2, new, kept, lens, d.block_tables,
                                     dst.to(DEV), d.context_lens, 500, 100, 4, 20)]
    for c in calls:
        c()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, new, new2, kept, lens, d.k_cache)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for c in calls:
            c(stream=s)
    for t in (out, new, new2):
        t.zero_()
    kept.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip((out, new, new2, kept, lens, d.k_cache), want):
        if a.is_floating_point():
            a, b = bits(a), bits(b)
        assert torch.equal(a, b)
    assert pa.pa_device_error() == 0


def test_binding_refuses_mismatched_tensors(pa):
    batch, w, dst = evict_case([64, 40], 2, 64, 16, BF16, 32, 415)
    d = batch.to(DEV)
    z = dict(k=d.k_cache, v=d.v_cache, wo=torch.zeros_like(w).to(DEV), wi=w.to(DEV),
             kept=torch.zeros(2, 2, 32, dtype=torch.int32, device=DEV),
             nl=torch.zeros(2, dtype=torch.int32, device=DEV), t=d.block_tables, dt=dst.to(DEV),
             n=d.context_lens, m=64, budget=32, first=0, last=0)
    call = lambda **k: pa.pa_evict_tokens(*{**z, **k}.values())
    call()
    for bad, err in ((dict(wi=None), ValueError), (dict(wi=w.to(DEV).half()), TypeError),
                     (dict(kept=z["kept"][:, :, :31].contiguous()), ValueError),
                     (dict(dt=z["dt"][:1]), ValueError), (dict(n=z["n"].long()), TypeError),
                     (dict(first=30, last=3), pa.PAError), (dict(nl=z["n"]), pa.PAError),
                     (dict(m=65), pa.PAError), (dict(dt=z["dt"][:, :1].contiguous()), pa.PAError)):
        with pytest.raises(err):
            call(**bad)
    n = pa.pa_decode_accumulate_weights_workspace_size(2, 2, 64, 64)
    y = dict(o=torch.empty_like(d.q), wo=z["wo"], wi=z["wi"], q=d.q, k=d.k_cache, v=d.v_cache,
             t=d.block_tables, n=d.context_lens, m=64, scale=0.1, part=0,
             ws=torch.empty(n, dtype=torch.uint8, device=DEV))
    call = lambda **k: pa.pa_decode_accumulate_weights(*{**y, **k}.values())
    call()
    flat = torch.zeros(w.numel() + 8, device=DEV)
    a, b = flat[:w.numel()].view(w.shape), flat[4:4 + w.numel()].view(w.shape)
    for bad, err in ((dict(wo=w.to(DEV).double()), TypeError), (dict(wo=a, wi=b), pa.PAError),
                     (dict(ws=None), pa.PAError), (dict(ws=y["ws"][:n - 1]), pa.PAError),
                     (dict(m=65), pa.PAError), (dict(wi=z["wi"][:, :1]), ValueError)):
        with pytest.raises(err):
            call(**bad)
    torch.cuda.synchronize()
