"""Refusals of the ragged and paged calls: bad arguments are turned away before any CUDA call (no GPU needed)."""
import ctypes

import pytest

import factorized_sparse_self_b200 as st
from factorized_sparse_self_b200 import _CacheDesc, _Desc, _PackedDesc

PTR = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)
NULL = ctypes.c_void_p(0)
DENSE = dict(kind=2, head_mode=0, T=100, l=1, c=1)
OK = dict(n_seqs=2, total=100, H=4, Hkv=2, d=64)
CACHE = dict(num_pages=8, page_size=16, max_pages=4, page_stride=16 * 128, slot_stride=128, head_stride=64)


def by(x):
    return ctypes.byref(x)


def desc(**kw):
    return _PackedDesc(**{**OK, **kw})


def cache(**kw):
    return _CacheDesc(**{**CACHE, **kw})


def pattern(**kw):
    return _Desc(**{**DENSE, **kw})


def every_call(p, dt, x, c, ptr=PTR, ws=PTR, wn=1 << 40, max_q=1):
    """Status of every entry point for these arguments."""
    L = st.lib()
    n = ctypes.c_size_t()
    pa, xa, ca = (by(p) if p is not None else None), (by(x) if x is not None else None), (by(c) if c is not None else None)
    return {
        "fwd_ws": L.st_packed_attn_fwd_workspace(pa, dt, xa, by(n)),
        "bwd_ws": L.st_packed_attn_bwd_workspace(pa, dt, xa, by(n)),
        "paged_ws": L.st_paged_attn_workspace(pa, dt, xa, ca, max_q, by(n)),
        "fwd": L.st_packed_attn_fwd(pa, dt, xa, 0.0, ptr, ptr, ptr, ptr, ptr, ptr, ws, wn, None),
        "bwd": L.st_packed_attn_bwd(pa, dt, xa, 0.0, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ws, wn, None),
        "paged": L.st_paged_attn(pa, dt, xa, ca, max_q, 0.0, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ws, wn, None),
    }


@pytest.mark.parametrize("bad", [dict(kind=3), dict(kind=-1), dict(T=0), dict(kind=0, l=0), dict(kind=0, l=4, head_mode=2),
                                 dict(kind=1, l=4, c=0), dict(kind=1, l=4, c=5)], ids=str)
def test_bad_patterns(bad):
    for name, code in every_call(pattern(**bad), st.ST_BF16, desc(), cache()).items():
        assert code == st.ST_ERR_INVALID, name


@pytest.mark.parametrize("bad", [dict(n_seqs=0), dict(total=-1), dict(H=0), dict(Hkv=0), dict(H=5), dict(d=0),
                                 dict(q_stride=128), dict(q_stride=300), dict(q_stride=-256)], ids=str)
def test_bad_sizes(bad):
    for name, code in every_call(pattern(), st.ST_BF16, desc(**bad), cache()).items():
        assert code == st.ST_ERR_INVALID, name


def test_bad_key_strides():
    for bad in (dict(k_stride=64), dict(v_stride=200)):
        got = every_call(pattern(), st.ST_BF16, desc(**bad), cache())
        assert got["fwd"] == got["bwd"] == got["fwd_ws"] == got["bwd_ws"] == st.ST_ERR_INVALID
    for bad in (dict(dq_stride=64), dict(dk_stride=200), dict(dv_stride=-128)):
        assert every_call(pattern(), st.ST_BF16, desc(**bad), cache())["bwd"] == st.ST_ERR_INVALID


@pytest.mark.parametrize("dt,d", [(st.ST_BF16, 32), (st.ST_F16, 96), (st.ST_BF16, 256), (st.ST_F32, 16), (st.ST_F32, 256)])
def test_head_sizes_without_kernels(dt, d):
    c = cache(page_stride=16 * 2 * d, slot_stride=2 * d, head_stride=d)
    for name, code in every_call(pattern(), dt, desc(d=d), c).items():
        assert code == st.ST_ERR_UNSUPPORTED, name


def test_row_numbers_past_31_bits():
    for name, code in every_call(pattern(), st.ST_BF16, desc(total=1 << 30, H=4, Hkv=4), cache()).items():
        assert code == st.ST_ERR_UNSUPPORTED, name
    got = every_call(pattern(), st.ST_BF16, desc(), cache(num_pages=1 << 30, page_size=64, page_stride=64 * 128))
    assert got["paged"] == got["paged_ws"] == st.ST_ERR_UNSUPPORTED
    got = every_call(pattern(), st.ST_BF16, desc(), cache(max_pages=1 << 30, page_size=64))
    assert got["paged"] == got["paged_ws"] == st.ST_ERR_UNSUPPORTED


@pytest.mark.parametrize("keys", [0x7fff0001, 0x7fffffff])
def test_key_and_row_numbers_leave_room_for_a_tile(keys):
    """Tile ends are rounded up in 32 bits."""
    c = cache(num_pages=1, page_size=keys, max_pages=1, page_stride=0, slot_stride=0)
    codes = every_call(pattern(), st.ST_BF16, desc(n_seqs=1), c)
    assert codes["paged"] == codes["paged_ws"] == st.ST_ERR_UNSUPPORTED
    codes = every_call(pattern(), st.ST_BF16, desc(n_seqs=1, total=keys, H=1, Hkv=1), cache())
    assert set(codes.values()) == {st.ST_ERR_UNSUPPORTED}


@pytest.mark.parametrize("big", [1 << 62, 1 << 61, (1 << 63) - 64], ids=hex)
@pytest.mark.parametrize("which", ["page_stride", "slot_stride", "head_stride"])
def test_cache_strides_past_64_bits(which, big):
    """Sums of such strides would wrap around to small numbers."""
    codes = every_call(pattern(), st.ST_BF16, desc(Hkv=4), cache(page_size=129, num_pages=129, **{which: big}))
    assert codes["paged"] == codes["paged_ws"] == st.ST_ERR_UNSUPPORTED


def test_cache_extent_past_64_bits():
    n = 0x7fff0000
    codes = every_call(pattern(), st.ST_BF16, desc(Hkv=4, n_seqs=1),
                       cache(num_pages=n, page_size=n, max_pages=1, page_stride=64 * n, slot_stride=64 * n, head_stride=64 * n))
    assert codes["paged"] == codes["paged_ws"] == st.ST_ERR_UNSUPPORTED


def test_null_and_unknown():
    for name, code in every_call(None, st.ST_BF16, desc(), cache()).items():
        assert code == st.ST_ERR_INVALID, name
    for name, code in every_call(pattern(), st.ST_BF16, None, cache()).items():
        assert code == st.ST_ERR_INVALID, name
    for name, code in every_call(pattern(), 7, desc(), cache()).items():
        assert code == st.ST_ERR_INVALID, name
    assert every_call(pattern(), st.ST_BF16, desc(), None)["paged"] == st.ST_ERR_INVALID
    assert every_call(pattern(), st.ST_BF16, desc(), cache(), max_q=0)["paged"] == st.ST_ERR_INVALID
    L = st.lib()
    assert L.st_packed_attn_fwd_workspace(by(pattern()), st.ST_BF16, by(desc()), None) == st.ST_ERR_INVALID
    assert L.st_packed_attn_bwd_workspace(by(pattern()), st.ST_BF16, by(desc()), None) == st.ST_ERR_INVALID


def test_pointers_and_workspace():
    for ptr in (NULL, ODD):
        got = every_call(pattern(), st.ST_BF16, desc(), cache(), ptr=ptr)
        assert got["fwd"] == got["bwd"] == got["paged"] == st.ST_ERR_INVALID
    two = pattern(kind=0, l=8, head_mode=1)  # joined from two orders: needs a workspace
    n = ctypes.c_size_t()
    L = st.lib()
    for query in (L.st_packed_attn_fwd_workspace, L.st_packed_attn_bwd_workspace):
        assert query(by(two), st.ST_BF16, by(desc()), by(n)) == st.ST_OK and n.value > 0
    for ws, wn in ((NULL, 1 << 40), (PTR, 16), (ctypes.c_void_p(4096 + 16), 1 << 40)):
        got = every_call(two, st.ST_BF16, desc(), cache(), ws=ws, wn=wn)
        assert got["fwd"] == got["bwd"] == got["paged"] == st.ST_ERR_WORKSPACE


def test_no_tokens_is_no_work():
    got = every_call(pattern(), st.ST_BF16, desc(total=0), cache(), ptr=NULL, ws=NULL, wn=0)
    assert set(got.values()) == {st.ST_OK}
    L = st.lib()
    assert L.st_cache_append(st.ST_BF16, by(desc(total=0)), by(cache()), NULL, NULL, NULL, NULL, NULL, NULL, NULL, None) == st.ST_OK


@pytest.mark.parametrize("bad", [dict(num_pages=0), dict(page_size=0), dict(max_pages=0), dict(slot_stride=100), dict(page_stride=-2048)], ids=str)
def test_bad_caches(bad):
    got = every_call(pattern(), st.ST_BF16, desc(), cache(**bad))
    assert got["paged"] == got["paged_ws"] == st.ST_ERR_INVALID
    L = st.lib()
    args = [PTR] * 7
    assert L.st_cache_append(st.ST_BF16, by(desc()), by(cache(**bad)), *args, None) == st.ST_ERR_INVALID


def test_append_refusals():
    L = st.lib()
    args = [PTR] * 7
    assert L.st_cache_append(9, by(desc()), by(cache()), *args, None) == st.ST_ERR_INVALID
    assert L.st_cache_append(st.ST_BF16, None, by(cache()), *args, None) == st.ST_ERR_INVALID
    assert L.st_cache_append(st.ST_BF16, by(desc()), None, *args, None) == st.ST_ERR_INVALID
    assert L.st_cache_append(st.ST_BF16, by(desc(k_stride=100)), by(cache()), *args, None) == st.ST_ERR_INVALID
    c = cache(page_stride=16 * 24, slot_stride=24, head_stride=12)
    assert L.st_cache_append(st.ST_BF16, by(desc(d=12)), by(c), *args, None) == st.ST_ERR_UNSUPPORTED
    for at in range(7):
        bad = list(args)
        bad[at] = NULL
        assert L.st_cache_append(st.ST_BF16, by(desc()), by(cache()), *bad, None) == st.ST_ERR_INVALID


def test_binding_refuses_host_tensors():
    import torch
    P = st.st_pattern("dense")
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        st.st_packed_attn_fwd(P, q, k, k, cu, 4)
    with pytest.raises(KeyError):
        st.st_pattern("sideways")
