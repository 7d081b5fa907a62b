"""Sizes that a C int does not hold are refused by the prepared calls, not cut
to their low 32 bits. (Only pointers are taken of the tensors, and the check
comes before any of them would be used: stand-ins for device tensors do.)"""
import ctypes

import pytest
import torch

from pagedattention_paged_kv_02_b200 import build as pa_build


@pytest.fixture()
def pa(monkeypatch):
    pa_build.build()
    from pagedattention_paged_kv_02_b200 import pa as _pa
    monkeypatch.setattr(_pa, "_p", lambda t: None if t is None else ctypes.c_void_p(t.data_ptr()))
    return _pa


B, H, NB, BS, D = 2, 2, 8, 16, 64
HUGE = (1 << 32) + 16          # its low 32 bits are a valid size


def tensors():
    int32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return dict(q=torch.zeros(B, H, D), cache=torch.zeros(NB, H, BS, D),
                bounds=torch.zeros(NB, H, 2, D), tables=int32(B, 4), lens=int32(B),
                sel=int32(B, H, 3), w=torch.zeros(B, H, 64), kept=int32(B, H, 8), new=int32(B))


def test_sizes_past_32_bits_are_refused(pa):
    t = tensors()
    ws = torch.zeros(4096, dtype=torch.uint8)
    rows = (t["tables"], t["lens"])
    calls = {
        "bounds": lambda n: pa.prepare_update_key_bounds(t["bounds"], t["cache"], *rows,
                                                         t["lens"], n),
        "select": lambda n: pa.prepare_select_blocks(t["sel"], t["q"], t["bounds"], *rows, n, BS,
                                                     workspace=ws),
        "first": lambda n: pa.prepare_select_blocks(t["sel"], t["q"], t["bounds"], *rows, 64, BS,
                                                    n, workspace=ws),
        "selected": lambda n: pa.prepare_decode_selected_blocks(
            t["q"].clone(), t["q"], t["cache"], t["cache"], *rows, t["sel"], 0.1, n, ws),
        "weights": lambda n: pa.prepare_decode_accumulate_weights(
            t["q"].clone(), t["w"], None, t["q"], t["cache"], t["cache"], *rows, n, 0.1,
            workspace=ws),
        "evict": lambda n: pa.prepare_evict_tokens(
            t["cache"], t["cache"].clone(), t["w"], t["w"], t["kept"], t["new"], t["tables"],
            t["tables"], t["lens"], n, 8),
    }
    for name, call in calls.items():
        call(16)
        for n in (HUGE, 1 << 31, -(1 << 31) - 1):
            with pytest.raises(ValueError, match="32-bit"):
                call(n)
