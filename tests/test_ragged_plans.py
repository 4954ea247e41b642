"""Workspace queries of paged calls over the whole range of sizes and hints (no GPU needed)."""
import ctypes
import itertools

import pytest

import factorized_sparse_self_b200 as st
from factorized_sparse_self_b200 import _CacheDesc, _Desc, _PackedDesc

BIG = 2 ** 31 - 1
PARTS = 32  # most key ranges


def query(kind, mode, T, l, seqs, total, H, Hkv, max_q):
    n = ctypes.c_size_t()
    x = _PackedDesc(seqs, total, H, Hkv, 64, 0, 0, 0, 0, 0, 0)
    c = _CacheDesc(8, 16, 1, 16 * Hkv * 64, Hkv * 64, 64)
    p = _Desc(kind, mode, T, l, 1)
    code = st.lib().st_paged_attn_workspace(ctypes.byref(p), st.ST_BF16, ctypes.byref(x), ctypes.byref(c), max_q, ctypes.byref(n))
    assert code == st.ST_OK or (seqs == 2 ** 30 and code == st.ST_ERR_UNSUPPORTED)  # units may be too many to number
    return n.value


@pytest.mark.parametrize("kind,mode", [(0, 0), (0, 1), (1, 0), (1, 1), (2, 0)])
def test_any_hints_give_a_bounded_plan(kind, mode):
    """Parts hold fp32 rows and their LSE, at most 32 ranges in each of two orders, and few where rows are many."""
    for T, l, max_q, (seqs, total) in itertools.product(
            (1, 300, 65536, BIG), (1, 4, 300, BIG), (1, 17, 600, BIG),
            ((1, 0), (1, 1), (64, 64), (3, 700), (2 ** 30, 5), (2 ** 30, 0), (1, 2 ** 20))):
        for H, Hkv in ((1, 1), (32, 8), (15, 3)):
            size = query(kind, mode, T, l, seqs, total, H, Hkv, max_q)
            rows = total * H
            assert size <= 2 * PARTS * (rows * 65 * 4 + 256) + 512
            assert size <= 2 * ((256 << 20) + rows * 64 * 4) * 65 // 64 + 2 * PARTS * 256 + 1024
            assert size == query(kind, mode, T, l, seqs, total, H, Hkv, max_q)


def test_more_units_than_can_be_numbered():
    """Refused before any launch: 2^25 sequences of 64 heads, each with a unit of its own."""
    L, ptr, n = st.lib(), ctypes.c_void_p(4096), ctypes.c_size_t()
    for kind, seqs in ((2, 2 ** 25), (1, 2 ** 25), (0, 2 ** 26)):
        p = _Desc(kind, 0, 100, 16, 1)
        x = _PackedDesc(seqs, 100, 64, 64, 64, 0, 0, 0, 0, 0, 0)
        c = _CacheDesc(8, 16, 1, 16 * 64 * 64, 64 * 64, 64)
        a, b, e = ctypes.byref(p), ctypes.byref(x), ctypes.byref(c)
        codes = [L.st_packed_attn_fwd_workspace(a, st.ST_BF16, b, ctypes.byref(n)),
                 L.st_packed_attn_bwd_workspace(a, st.ST_BF16, b, ctypes.byref(n)),
                 L.st_packed_attn_fwd(a, st.ST_BF16, b, 0.0, *[ptr] * 7, 1 << 60, None),
                 L.st_packed_attn_bwd(a, st.ST_BF16, b, 0.0, *[ptr] * 11, 1 << 60, None)]
        if kind != 0:  # strided chunks may go to a kernel that numbers them otherwise
            codes += [L.st_paged_attn_workspace(a, st.ST_BF16, b, e, 100, ctypes.byref(n)),
                      L.st_paged_attn(a, st.ST_BF16, b, e, 100, 0.0, *[ptr] * 9, 1 << 60, None)]
        assert codes == [st.ST_ERR_UNSUPPORTED] * len(codes), (kind, codes)
