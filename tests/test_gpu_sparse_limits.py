"""The operators that decode over part of a cache at their limits: pools whose
offsets pass 32 bits, rows whose scores or weights outgrow shared memory, weights
that no histogram tells apart, and a whole step captured in a graph and replayed
with changed inputs."""
import pytest
import torch

import sparse_reference as R
from helpers import assert_close, bits
from pagedattention_paged_kv_02_b200 import workloads as W

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


def test_offsets_past_32_bits(pa):
    """Blocks at the far end of a pool of 4.6e9 elements per cache."""
    NB, H, bs, D, G = 70000, 8, 64, 128, 2
    assert NB * H * bs * D > 1 << 32
    k = torch.empty(NB, H, bs, D, dtype=BF16, device=DEV)
    v = torch.empty(NB, H, bs, D, dtype=BF16, device=DEV)
    ctx = [150, 64, 300]
    far = torch.arange(NB - 1, NB - 16, -1, dtype=torch.int32)
    tables = torch.stack([far[0:5], far[5:10], far[10:15]])
    g = torch.Generator().manual_seed(501)
    hk = torch.randn(15, H, bs, D, generator=g).to(BF16)
    hv = torch.randn(15, H, bs, D, generator=g).to(BF16)
    k[far.long().to(DEV)] = hk.to(DEV)
    v[far.long().to(DEV)] = hv.to(DEV)
    near = tables - (NB - 15)          # the same rows in a pool of 15 blocks
    hk, hv = hk.flip(0), hv.flip(0)
    q = torch.randn(3, H * G, D, generator=g).to(BF16)
    lens = torch.tensor(ctx, dtype=torch.int32)
    dt, dl, dq = tables.to(DEV), lens.to(DEV), q.to(DEV)

    kb = torch.empty(NB, H, 2, D, dtype=BF16, device=DEV)
    pa.pa_update_key_bounds(kb, k, dt, dl, dl, 300)
    want_kb = R.update_key_bounds(torch.zeros(15, H, 2, D, dtype=BF16), hk, near, lens, lens)
    used = torch.cat([near[b, :-(-n // bs)] for b, n in enumerate(ctx)]).long()
    assert torch.equal(bits(kb[(used + NB - 15).to(DEV)].cpu()), bits(want_kb[used]))

    sel = torch.empty(3, H, 2, dtype=torch.int32, device=DEV)
    pa.pa_select_blocks(sel, dq, kb, dt, dl, 300, bs, 0, 1)
    want_sel = R.select_blocks(q, want_kb, near, lens, bs, 2, 0, 1)
    assert torch.equal(sel.cpu(), want_sel)

    out = torch.empty_like(dq)
    n = pa.pa_decode_selected_blocks_workspace_size(3, H * G, H, D, bs, 2)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    pa.pa_decode_selected_blocks(out, dq, k, v, dt, dl, sel, 0.1, 0, ws)
    assert_close(out, R.decode_selected(q, hk, hv, near, lens, want_sel, 0.1), "selected")

    w = torch.zeros(3, H, 300, device=DEV)
    n = pa.pa_decode_accumulate_weights_workspace_size(3, H * G, D, 300)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    pa.pa_decode_accumulate_weights(out, w, w, dq, k, v, dt, dl, 300, 0.1, 0, ws)
    ref, ref_w = R.decode_weights(q, hk, hv, near, lens, 0.1, None, 300)
    assert_close(out, ref, "weights")
    for b, c in enumerate(ctx):
        assert torch.allclose(w[b, :, :c].cpu().double(), ref_w[b, :, :c], rtol=1e-4, atol=1e-6)

    kept = torch.empty(3, H, 70, dtype=torch.int32, device=DEV)
    nl = torch.empty(3, dtype=torch.int32, device=DEV)
    host_w = w.cpu()
    pa.pa_evict_tokens(k, v, w, w, kept, nl, dt, dt, dl, 300, 70, 2, 8)
    want = R.evict(host_w, lens, 70, 2, 8)
    for b, c in enumerate(ctx):
        for h in range(H):
            assert kept[b, h, :min(c, 70)].tolist() == want[b][h]
            at = torch.tensor(want[b][h])
            got = k[dt[b, :2].long(), h].reshape(-1, D)[:len(at)].cpu()
            src = hk[near[b].long(), h].reshape(-1, D)[at]
            assert torch.equal(bits(got), bits(src))
    assert pa.pa_device_error() == 0


def test_selection_over_more_blocks_than_shared_memory_holds(pa):
    g = torch.Generator().manual_seed(502)
    n, H, D = 30000, 2, 64
    kb = torch.randn(n, H, 2, D, generator=g).sort(dim=2).values.to(BF16)
    table = torch.randperm(n, generator=g).int()[None]
    lens = torch.tensor([n * 16], dtype=torch.int32)
    q = torch.randn(1, 2 * H, D, generator=g).to(BF16)
    for equal in (False, True):
        if equal:      # three kinds of blocks: the exact path, on global memory
            kb[1:] = kb[torch.randint(0, 3, (n - 1,), generator=g)]
        want = R.select_blocks(q, kb, table, lens, 16, 700, 3, 4)
        got = torch.empty(1, H, 700, dtype=torch.int32, device=DEV)
        pa.pa_select_blocks(got, q.to(DEV), kb.to(DEV), table.to(DEV), lens.to(DEV), n * 16, 16,
                            3, 4)
        assert torch.equal(got.cpu(), want)
    assert pa.pa_device_error() == 0


def kept_of(pa, w, budget, first, last, lens=None):
    """Kept positions for weights alone: every block of the rows is block 0, the
    destinations are blocks of their own. The moved weights are checked here, in
    another buffer and in place."""
    B, H, n = w.shape
    bs = 64
    need = -(-budget // bs)
    k = torch.zeros(1 + B * need, H, bs, 64, dtype=BF16, device=DEV)
    src = torch.zeros(B, -(-n // bs), dtype=torch.int32, device=DEV)
    dst = torch.arange(1, 1 + B * need, dtype=torch.int32, device=DEV).reshape(B, need)
    kept = torch.full((B, H, budget), -9, dtype=torch.int32, device=DEV)
    nl = torch.empty(B, dtype=torch.int32, device=DEV)
    lens = torch.full((B,), n, dtype=torch.int32) if lens is None else lens
    out = torch.full_like(w, 5.0)
    same = w.clone()
    for w_out, w_in in ((out, w), (same, same)):
        pa.pa_evict_tokens(k, k.clone(), w_out, w_in, kept, nl, src, dst, lens.to(DEV), n, budget,
                           first, last)
    torch.cuda.synchronize()
    want = torch.zeros_like(w)
    want[:, :, :budget] = w.gather(2, kept.long())
    assert torch.equal(out, want) and torch.equal(same, want)
    return kept.cpu()


def best_of(w, budget, first, last):
    """The same by a stable sort, in 64 bits."""
    n = w.shape[-1]
    mid = w[..., first:n - last].double()
    top = mid.sort(dim=-1, descending=True, stable=True).indices[..., :budget - first - last]
    top = top.sort(dim=-1).values + first
    lead = w.shape[:-1]
    a = torch.arange(first).expand(*lead, first)
    z = torch.arange(n - last, n).expand(*lead, last)
    return torch.cat((a, top, z), -1).int()


@pytest.mark.parametrize("rows,n", [((1, 1), 400000), ((1, 150), 41500), ((2, 3), 30000),
                                    ((30, 5), 5000), ((1, 1), 65)])
def test_weights_that_outgrow_shared_memory_or_not(pa, rows, n):
    g = torch.Generator().manual_seed(503)
    w = torch.exp(3 * torch.randn(*rows, n, generator=g))
    budget = min(n - 1, 3000)
    got = kept_of(pa, w.to(DEV), budget, min(4, budget // 3), budget // 4)
    assert torch.equal(got, best_of(w, budget, min(4, budget // 3), budget // 4))


@pytest.mark.parametrize("rows", [(1, 2), (40, 5)])
@pytest.mark.parametrize("kind", ["zero", "close", "two", "spread", "negative", "subnormal"])
def test_weights_that_a_histogram_does_not_tell_apart(pa, rows, kind):
    """All equal; thousands within a few units in the last place; two values;
    ninety orders of magnitude; both signs; subnormals."""
    g = torch.Generator().manual_seed(504)
    n = 20000 if rows[0] == 1 else 9000
    u = torch.rand(*rows, n, generator=g)
    w = {"zero": torch.zeros_like(u),
         "close": 1.0 + (u * 64).floor() * 2.0 ** -23,
         "two": (u < 0.7).float() * 3.0,
         "spread": torch.exp((u - 0.5) * 170.0),
         "negative": (u - 0.9) * torch.exp(10 * u),
         "subnormal": (u * 500).floor() * 2.0 ** -149}[kind]
    w[..., :4] = w[..., :4].abs() + 1000.0
    for budget in (1, 777, n - 3):
        assert torch.equal(kept_of(pa, w.to(DEV), budget, 0, 0), best_of(w, budget, 0, 0)), budget


def test_a_step_in_a_graph(pa):
    """Append, bounds, selection and decode captured once; replays with new
    keys, queries and a later position follow them."""
    batch = W.decode_batch([700, 60, 1300], 16, 2, 128, 16, 200, BF16, seed=505)
    d = batch.to(DEV)
    NB, H, bs, D = d.k_cache.shape
    kb = torch.zeros(NB, H, 2, D, dtype=BF16, device=DEV)
    pa.pa_update_key_bounds(kb, d.k_cache, d.block_tables, d.context_lens - 1,
                            d.context_lens - 1, 1300)
    lens = d.context_lens.clone()
    ones = torch.ones_like(lens)
    sel = torch.empty(3, H, 20, dtype=torch.int32, device=DEV)
    out = torch.empty_like(d.q)
    n = pa.pa_decode_selected_blocks_workspace_size(3, 16, H, D, bs, 20)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    calls = [pa.prepare_reshape_and_cache(d.key, d.value, d.k_cache, d.v_cache, d.slot_mapping),
             pa.prepare_update_key_bounds(kb, d.k_cache, d.block_tables, lens, ones, 1),
             pa.prepare_select_blocks(sel, d.q, kb, d.block_tables, lens, 1310, bs, 1, 1),
             pa.prepare_decode_selected_blocks(out, d.q, d.k_cache, d.v_cache, d.block_tables,
                                               lens, sel, batch.scale, workspace=ws)]
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        for c in calls:
            c(stream=s)
    gen = torch.Generator().manual_seed(506)
    for step in range(3):
        if step:     # the next position of each row, still inside its last block
            lens.add_(1)
            d.slot_mapping.add_(1)
            for t in (d.key, d.value, d.q):
                t.copy_(torch.randn(t.shape, generator=gen).to(BF16))
        g.replay()
        torch.cuda.synchronize()
        k, v = d.k_cache.cpu(), d.v_cache.cpu()
        cl = lens.cpu()
        ref_kb = R.update_key_bounds(torch.zeros(NB, H, 2, D, dtype=BF16), k, batch.block_tables,
                                     cl, cl)
        want = R.select_blocks(d.q.cpu(), ref_kb, batch.block_tables, cl, bs, 20, 1, 1)
        assert torch.equal(sel.cpu(), want), step
        ref = R.decode_selected(d.q.cpu(), k, v, batch.block_tables, cl, want, batch.scale)
        assert_close(out, ref, f"step {step}")
    assert pa.pa_device_error() == 0


def test_selection_on_two_streams(pa):
    """Two selections in flight at once, a workspace each."""
    g = torch.Generator().manual_seed(507)
    n, H, D = 4000, 4, 128
    runs = []
    for i in range(2):
        kb = torch.randn(n, H, 2, D, generator=g).sort(dim=2).values.to(BF16)
        table = torch.randperm(n, generator=g).int()[None]
        q = torch.randn(1, 4 * H, D, generator=g).to(BF16)
        lens = torch.tensor([n * 16], dtype=torch.int32)
        want = R.select_blocks(q, kb, table, lens, 16, 64, 1, 1)
        sel = torch.empty(1, H, 64, dtype=torch.int32, device=DEV)
        call = pa.prepare_select_blocks(sel, q.to(DEV), kb.to(DEV), table.to(DEV), lens.to(DEV),
                                        n * 16, 16, 1, 1)
        runs.append((call, torch.cuda.Stream(), sel, want))
    torch.cuda.synchronize()
    for _ in range(10):
        for call, s, sel, _ in runs:
            with torch.cuda.stream(s):
                sel.zero_()
            call(stream=s)
        torch.cuda.synchronize()
        for _, _, sel, want in runs:
            assert torch.equal(sel.cpu(), want)
