"""The attention binding's own arithmetic and checks on the CPU: slots of positions, windows."""
from types import SimpleNamespace

import pytest
import torch

import linear_exl3_input_amd as ex
from linear_exl3_input_amd import attention as at


def slots(pages, page_size, table, seq, positions):
    """KvCache.slots, which needs the cache's sizes alone."""
    return ex.KvCache.slots(SimpleNamespace(pages=pages, page_size=page_size), table, seq, positions)


TABLE = torch.tensor([[4, 2, -1, 5], [7, 9, 0, 10]], dtype=torch.int32)  # of a cache of 10 pages: 10 is a hole too


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_slots_are_those_of_the_page_table(dtype):
    seq, pos = torch.meshgrid(torch.arange(2), torch.arange(64), indexing="ij")
    got = slots(10, 16, TABLE, seq.flatten().to(dtype), pos.flatten().to(dtype))
    want = [TABLE[s, p // 16].item() * 16 + p % 16 if 0 <= TABLE[s, p // 16] < 10 else -1 for s in range(2) for p in range(64)]
    assert got.tolist() == want and got.dtype == torch.int32


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_positions_and_sequences_out_of_range_have_no_slot(dtype):
    pos = torch.tensor([-1, -16, -17, -2 ** 31, 64, 65, 2 ** 31 - 1, 3, 3, 3], dtype=dtype)
    seq = torch.tensor([1, 1, 0, 1, 1, 0, 1, -1, 2, 2 ** 31 - 1], dtype=dtype)
    assert slots(10, 16, TABLE, seq, pos).tolist() == [-1] * 10
    assert slots(10, 16, TABLE, seq[:1], torch.tensor([63], dtype=dtype)).tolist() == [-1]  # page 10


def test_page_numbers_that_wrap_have_no_slot():
    table = torch.tensor([[2 ** 28, 2 ** 28 + 3, -2 ** 28, 2 ** 31 - 1]], dtype=torch.int32)  # times 16: 0, 48, 0, -16
    got = slots(10, 16, table, torch.zeros(4, dtype=torch.int32), torch.arange(4, dtype=torch.int32) * 16 + 5)
    assert got.tolist() == [-1] * 4


def test_a_table_without_pages_has_no_slots():
    for shape in ((3, 0), (0, 4), (0, 0)):
        got = slots(10, 16, torch.zeros(shape, dtype=torch.int32), torch.tensor([0, 1]), torch.tensor([0, 17]))
        assert got.tolist() == [-1, -1] and got.dtype == torch.int32
    assert slots(10, 16, TABLE, torch.zeros(0, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)).shape == (0,)


def test_the_last_slot_of_the_largest_cache():
    pages = (2 ** 31 - 1) // 1024
    table = torch.tensor([[pages - 1]], dtype=torch.int32)
    assert slots(pages, 1024, table, torch.tensor([0]), torch.tensor([1023])).item() == pages * 1024 - 1


@pytest.mark.parametrize("window", [-1, 2 ** 30 + 1, 2 ** 32, 2 ** 32 + 1, 2 ** 63 - 1])
def test_windows_that_do_not_fit_are_refused(window):
    """2^32 + 1 would be a window of 1 in 32 bits, 2^32 none at all."""
    with pytest.raises(ValueError, match=f"window={window}, must be 0"):
        at._window(window)


def test_windows_that_fit_pass():
    assert [at._window(w) for w in (0, 1, 4096, 2 ** 30)] == [0, 1, 4096, 2 ** 30]


@pytest.mark.gpu
def test_calls_refuse_windows_that_do_not_fit():
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    cache = ex.KvCache.empty(1, 16, 4, 64)
    for window in (2 ** 32, 2 ** 32 + 1):
        with pytest.raises(ValueError, match="window="):
            ex.prompt_attention(q, q, q, cu, window=window)
        with pytest.raises(ValueError, match="window="):
            ex.paged_attention(cache, q, cu, cu[1:], cu[:1].view(1, 1), window=window)
