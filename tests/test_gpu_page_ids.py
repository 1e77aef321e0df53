"""Page ids that tg_page_tables meets in the caller's tables and free list, and the slots they give."""
import pytest
import torch

from learned_token_pruning_b200 import tokengate as tg
from test_gpu_kv4 import DEV, I32, _i32

pytestmark = pytest.mark.gpu


def test_page_ids_whose_slots_pass_32_bits_give_no_slot_and_are_reported():
    page = 1 << 20
    ids = [5, 2047, 2048, 4096, 2 ** 31 - 1]
    n = len(ids)
    lens, new, tables = _i32([0] * n), _i32([3] + [1] * (n - 1)), torch.full((n, 1), -1, dtype=I32, device=DEV)
    free, n_free = _i32(ids[::-1]), _i32([n])
    slots, start = torch.full((n + 4,), 7, dtype=I32, device=DEV), torch.empty(n + 1, dtype=I32, device=DEV)
    tg.tg_page_tables(lens, new, None, page, tables, free, n_free, lens, n_free, slots, start)
    with pytest.raises(tg.TokenGateError) as e:
        tg.tg_check_device_error()
    assert e.value.status == 8
    assert slots.tolist() == [5 * page, 5 * page + 1, 5 * page + 2, 2047 * page, -1, -1, -1, -1, -1]
    # the ids are looked at once the tables are made
    assert tables.flatten().tolist() == ids and lens.tolist() == [3, 1, 1, 1, 1] and int(n_free) == 0
    # a held page with such an id
    lens, new, tables = _i32([7, 1]), _i32([1, 1]), _i32([[4095], [3]])
    slots, start = torch.full((2,), 7, dtype=I32, device=DEV), torch.empty(3, dtype=I32, device=DEV)
    tg.tg_page_tables(lens, new, None, page, tables, free, n_free, lens, n_free, slots, start)
    with pytest.raises(tg.TokenGateError):
        tg.tg_check_device_error()
    assert slots.tolist() == [-1, 3 * page + 1]
