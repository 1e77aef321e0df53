"""What tg_page_tables_by_request refuses on the host (CPU)."""
import ctypes

import pytest
import torch

from learned_token_pruning_b200 import build, tokengate as tg

P = ctypes.c_void_p(256)  # a non-null dummy: validation fails before it is ever dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return tg.lib()


def test_validation(L):
    f = L.tg_page_tables_by_request

    def call(lens=P, new=P, rel=None, nreq=4, page=16, tab=P, mp=8, free=P, cap=32, nf=P, lo=P, nfo=P, slots=P, rs=None):
        return f(lens, new, rel, nreq, page, tab, mp, free, cap, nf, lo, nfo, slots, rs, None)

    assert call(lens=None) == 1 and call(new=None) == 1 and call(tab=None) == 1 and call(lo=None) == 1
    assert call(nf=None) == 1 and call(nfo=None) == 1 and call(slots=None) == 1 and call(free=None) == 1
    assert call(nreq=-1) == 1 and call(page=0) == 1 and call(mp=0) == 1 and call(cap=-1) == 1
    assert call(nreq=4097) == 4 and call(page=1 << 20, mp=1 << 11) == 4


def test_binding_wants_one_slot_a_request(L):
    z, i32 = torch.zeros, torch.int32
    for slots in (2, 4):
        with pytest.raises(tg.TokenGateError):
            tg.tg_page_tables_by_request(z(3, dtype=i32), z(3, dtype=i32), None, 16, z(3, 4, dtype=i32), z(9, dtype=i32),
                                         z(1, dtype=i32), z(3, dtype=i32), z(1, dtype=i32), z(slots, dtype=i32))
