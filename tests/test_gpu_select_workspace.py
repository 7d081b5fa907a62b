"""pa_select_blocks that brings its own workspace, on a stream that is not the
current one: memory that another stream still uses is left alone, and what the
call gives back is not handed out while its kernels run. Each stream that must
be behind spins for tens of milliseconds first."""
import pytest
import torch

import sparse_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16
SPIN = 100_000_000        # cycles: some 50 ms


@pytest.fixture(scope="module")
def pa():
    from pagedattention_paged_kv_02_b200 import build, pa as _pa
    build.build()
    torch.cuda.init()
    return _pa


@pytest.fixture(autouse=True)
def clean(pa):
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    pa.pa_device_error(clear=True)
    yield
    torch.cuda.synchronize()
    pa.pa_device_error(clear=True)


class Case:
    """One selection over 3000 blocks, and its workspace's size."""

    def __init__(self, pa, seed):
        g = torch.Generator().manual_seed(seed)
        n, H, D = 3000, 4, 64
        kb = torch.randn(n, H, 2, D, generator=g).sort(dim=2).values.to(BF16)
        table = torch.randperm(n, generator=g).int()[None]
        q = torch.randn(1, 2 * H, D, generator=g).to(BF16)
        lens = torch.tensor([n * 16], dtype=torch.int32)
        self.want = R.select_blocks(q, kb, table, lens, 16, 50, 1, 1)
        self.sel = torch.zeros(1, H, 50, dtype=torch.int32, device=DEV)
        self.args = (self.sel, q.to(DEV), kb.to(DEV), table.to(DEV), lens.to(DEV), n * 16, 16, 1, 1)
        self.bytes = pa.pa_select_blocks_workspace_size(1, H, 16, n * 16)
        torch.cuda.synchronize()

    def check(self):
        torch.cuda.synchronize()
        assert torch.equal(self.sel.cpu(), self.want)


@pytest.mark.parametrize("prepared", [False, True])
def test_memory_freed_on_the_current_stream_is_still_its_own(pa, prepared):
    case, s = Case(pa, 631), torch.cuda.Stream()
    freed = torch.full((case.bytes,), 7, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    copy = freed.clone()                     # runs after the spin
    del freed
    if prepared:
        call = pa.prepare_select_blocks(*case.args)
        call(stream=s)
    else:
        pa.pa_select_blocks(*case.args, stream=s)
    s.synchronize()
    case.check()
    assert bool((copy == 7).all())


@pytest.mark.parametrize("prepared", [False, True])
def test_a_workspace_given_back_is_not_handed_out_under_its_kernels(pa, prepared):
    case, s = Case(pa, 632), torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    if prepared:
        call = pa.prepare_select_blocks(*case.args)
        call(stream=s)
        del call
    else:
        pa.pa_select_blocks(*case.args, stream=s)
    others = [torch.full((case.bytes,), 9, dtype=torch.uint8, device=DEV) for _ in range(4)]
    case.check()
    for t in others:
        assert bool((t == 9).all())


def test_one_prepared_call_on_several_streams(pa):
    """Each stream's launches have a workspace of their own: the current stream,
    two others, and the first one again behind a spin."""
    case = Case(pa, 633)
    call = pa.prepare_select_blocks(*case.args)
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s in streams:
            case.sel.zero_()
            torch.cuda.synchronize()
            call(stream=s)
            case.check()
    case.sel.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    call()                                   # still to come when the next one runs
    call(stream=streams[1])
    case.check()


def test_a_graph_outlives_the_prepared_call(pa):
    """The captured launch's workspace belongs to the graph: dropping the call
    and using the memory it might have left changes nothing."""
    case, s = Case(pa, 634), torch.cuda.Stream()
    call = pa.prepare_select_blocks(*case.args)
    call(stream=s)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g, stream=s):
            call(stream=s)
    del call
    with torch.cuda.stream(s):
        on_s = [torch.full((case.bytes,), 3, dtype=torch.uint8, device=DEV) for _ in range(4)]
    here = [torch.full((case.bytes,), 4, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    for g in graphs:
        case.sel.zero_()
        g.replay()
        case.check()
    assert all(bool((t == 3).all()) for t in on_s) and all(bool((t == 4).all()) for t in here)


def test_the_call_refuses_a_stream_of_another_device(pa):
    case = Case(pa, 635)

    class Elsewhere:
        device_index = 1
        cuda_stream = 0

    with pytest.raises(ValueError):
        pa.prepare_select_blocks(*case.args)(stream=Elsewhere())
