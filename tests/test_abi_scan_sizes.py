"""Sizes that deltanet_scan_* and deltanet_step refuse before a GPU is touched: what the kernels'
32-bit counters of tokens and channels do not hold, tokens without a sequence, slots of more
requests than the search for repeated ones is made for."""
import pytest

from deltanet_chunkwise_delta_b200 import _lib as L
from deltanet_chunkwise_delta_b200 import build as B
from tests.test_abi_block_ops import desc, ref

MOST = 2 ** 31 - 16385


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


@pytest.mark.parametrize("T,D", [(1, MOST + 1), (1, 2 ** 31 - 1), (17, MOST + 1), (MOST + 1, 1), (1, 2 ** 31)])
def test_rows_past_the_counters(lib, T, D):
    # made-up addresses far enough apart for the sizes: what refuses is the size
    at = lambda i, *s, t=L.DN_BF16: desc(list(s), t, 1 + i * 2 ** 10)
    x, g, out = at(0, 1, T, D), at(1, 1, T, D), at(2, 1, T, D)
    state, fin = at(3, 1, D, t=L.DN_F32), at(4, 1, D, t=L.DN_F32)
    more = [at(5, 1, T, D), at(6, 1, T, D)]
    args = lambda *a: [None if x is None else ref(x) for x in a] + [None]
    assert lib.deltanet_scan_fwd(*args(x, g, None, None, out, fin)) == L.DN_ERR_INVALID_ARG
    assert lib.deltanet_scan_bwd(*args(g, out, None, None, x, None, *more, None)) == L.DN_ERR_INVALID_ARG
    assert lib.deltanet_scan_step(*args(x, g, state, None, out)) == L.DN_ERR_INVALID_ARG


def test_tokens_of_no_sequence(lib):
    """cu_seqlens of one entry: nothing would be written, and no kernel run to report it."""
    x, g, out, dx, dg = (desc([1, 5, 8], L.DN_F32, i) for i in (1, 2, 3, 4, 5))
    cu = desc([1], L.DN_I32, 6)
    a = [None if t is None else ref(t) for t in (x, g, None, cu, out, None)] + [None]
    assert lib.deltanet_scan_fwd(*a) == L.DN_ERR_INVALID_ARG
    a = [None if t is None else ref(t) for t in (g, out, None, cu, x, None, dx, dg, None)] + [None]
    assert lib.deltanet_scan_bwd(*a) == L.DN_ERR_INVALID_ARG


def test_slots_of_too_many_requests(lib):
    N = 2 ** 20 + 1
    at = lambda i, *s, t=L.DN_F32: desc(list(s), t, 1 + i * 2 ** 8)
    a = [at(0, N, 1, 8), at(1, N, 1, 8), at(2, N, 8), at(3, N, t=L.DN_I32), at(4, N, 1, 8)]
    assert lib.deltanet_scan_step(*map(ref, a), None) == L.DN_ERR_INVALID_ARG
    q, k, v, out = (at(i, N, 1, 1, 64, t=L.DN_BF16) for i in range(4))
    beta, state, slots = at(4, N, 1, 1), at(5, 4, 1, 64, 64), at(6, N, t=L.DN_I32)
    assert lib.deltanet_step(ref(q), ref(k), ref(v), ref(beta), None, 1, ref(state), ref(slots), ref(out),
                             None) == L.DN_ERR_INVALID_ARG
