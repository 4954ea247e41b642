"""Packed and paged attention on the GPU where callers' data lie at the edges: rows before the first sequence, rows that
are not finite, lengths past the cache, first calls inside a capture. Reference and bounds: tests/ragged_ref.py."""
import subprocess
import sys

import pytest
import torch

import factorized_sparse_self_b200 as st
from conftest import ROOT
from ragged_ref import One, check
from test_gpu_ragged import DT, make_cache, packed, paged, randn, starts

pytestmark = pytest.mark.gpu

THREE = [("bf16", 64), ("f16", 128), ("f32", 64)]
KINDS = [("dense", "merged", 1, 1), ("strided", "merged", 16, 1), ("strided", "split", 9, 1), ("fixed", "merged", 32, 4),
         ("fixed", "split", 20, 6)]


# ---- rows before the first sequence: whole units of them ----------------------------------------


@pytest.mark.parametrize("lead", [64, 300, 1000])
@pytest.mark.parametrize("ty", THREE, ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("pat", KINDS, ids=lambda p: "-".join(map(str, p)))
def test_packed_rows_before_the_first_sequence(pat, ty, lead):
    """A batch that is a view into a longer one (cu[2:6], say): the rows in front are not touched."""
    for x, (H, Hkv) in enumerate([(1, 1), (4, 1), (15, 3)]):
        packed(pat, H, Hkv, ty[1], ty[0], [[100, 100], [0, 1, 300], [257]][x], seed=x, backward=True, lead=lead)


@pytest.mark.parametrize("lead", [64, 300, 1000])
@pytest.mark.parametrize("ty", THREE, ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("pat", KINDS, ids=lambda p: "-".join(map(str, p)))
def test_paged_rows_before_the_first_sequence(pat, ty, lead):
    dtype, d = ty
    dt = DT[dtype]
    for x, (H, Hkv) in enumerate([(1, 1), (4, 1), (15, 3)]):
        for lens, new, hint in (([1, 90, 700], [1, 1, 1], 1), ([300, 20, 40], [200, 20, 1], 200), ([300, 20], [200, 20], 1)):
            g = torch.Generator(device="cuda").manual_seed(x)
            kc, vc, table = make_cache(g, lens, 16, Hkv, d, dt)
            ks, vs = ([randn(g, n, Hkv, d, dtype=dt) for n in lens] for _ in range(2))
            kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
            front = torch.full((lead, Hkv, d), float("nan"), dtype=dt, device="cuda")
            st.st_cache_append(torch.cat([front, *ks]), torch.cat([front, *vs]), kc, vc, table, starts(lens) + lead, kv)
            for s, n in enumerate(lens):
                for p in range(n):
                    if p % 61 == 0 or p == n - 1:
                        at = int(table[s, p // 16]), p % 16
                        assert torch.equal(kc[at], ks[s][p]) and torch.equal(vc[at], vs[s][p])
            q = randn(g, lead + sum(new), H, d, dtype=dt)
            q[:lead] = float("nan")
            o = torch.full_like(q, 7.0)
            lse = torch.full((q.shape[0], H), 7.0, device="cuda")
            st.st_paged_attn(st.st_pattern(*pat), q, kc, vc, table, starts(new) + lead, kv, hint, max(lens), o=o, lse=lse)
            assert st.st_last_device_status() == st.ST_OK
            assert bool((o[:lead] == 7.0).all()) and bool((lse[:lead] == 7.0).all())
            a = lead
            for s, n in enumerate(new):
                ro, to, rl, tl = One(pat, q[a:a + n], ks[s], vs[s], dt).outputs()
                check("o", o[a:a + n], ro, to)
                check("lse", lse[a:a + n], rl, tl)
                a += n


# ---- query rows that are not finite ---------------------------------------------------------------


def spoil(q, rows):
    """q with NaN in one entry of the first of `rows`, infinities in the second, overflowing scores in the third (float16
    cannot reach them: infinities of both signs)."""
    bad = q.clone()
    bad[rows[0], :, 5] = float("nan")
    bad[rows[1]] = float("inf")
    if q.dtype == torch.float16:
        bad[rows[2]] = float("-inf")
    else:
        bad[rows[2]] = 3e38
    return bad


def only_those(rows, good, bad):
    """Rows of NaN among `rows`, the others bit by bit as without them."""
    keep = torch.ones(good.shape[0], dtype=torch.bool, device=good.device)
    keep[rows] = False
    assert torch.equal(good[keep], bad[keep])
    assert bool(torch.isnan(bad[rows]).all())
    assert not bool(torch.isnan(good).any())


# one part a row; key ranges; two orders, the second joining the first, and with key ranges
SPLITS = [(("dense", "merged", 1, 1), [300, 140], 24, 6), (("dense", "merged", 1, 1), [2100, 90], 2, 1),
          (("strided", "merged", 16, 1), [300, 900], 72, 24), (("strided", "merged", 3, 1), [2100, 90], 2, 1),
          (("fixed", "merged", 40, 30), [2100, 90], 2, 1)]


@pytest.mark.parametrize("ty", THREE, ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("pat,lens,H,Hkv", SPLITS, ids=str)
def test_packed_query_rows_that_are_not_finite(pat, lens, H, Hkv, ty):
    dtype, d = ty
    g = torch.Generator(device="cuda").manual_seed(1)
    n = sum(lens)
    q, k, v, dout = (randn(g, n, h, d, dtype=DT[dtype]) for h in (H, Hkv, Hkv, H))
    P, cu = st.st_pattern(*pat), starts(lens)
    rows = [lens[0] - 1, lens[0] - 40, 200]
    bad = spoil(q, rows)
    good_out = st.st_packed_attn_fwd(P, q, k, v, cu, max(lens))
    bad_out = st.st_packed_attn_fwd(P, bad, k, v, cu, max(lens))
    for a, b in zip(good_out, bad_out):
        only_those(rows, a, b)
    # the gradients of the other sequence, and dQ of the other rows
    a = st.st_packed_attn_bwd(P, q, k, v, *good_out, dout, cu, max(lens))
    b = st.st_packed_attn_bwd(P, bad, k, v, *bad_out, dout, cu, max(lens))
    only_those(rows, a[0], b[0])
    for x, y in zip(a[1:], b[1:]):
        assert torch.equal(x[lens[0]:], y[lens[0]:])
    assert st.st_last_device_status() == st.ST_OK


@pytest.mark.parametrize("ty", THREE, ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("pat", [("dense", "merged", 1, 1), ("strided", "merged", 16, 1), ("fixed", "merged", 40, 30)], ids=str)
def test_paged_query_rows_that_are_not_finite(pat, ty):
    """Decoding and chunks, with one key range and several (max_kv steers the split only)."""
    dtype, d = ty
    H, Hkv = 4, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    for lens, new, rows in (([3000, 2500, 2000, 40], [1, 1, 1, 1], [0, 1, 2]), ([3000, 40], [300, 9], [299, 0, 100])):
        kc, vc, table = make_cache(g, lens, 16, Hkv, d, DT[dtype])
        kc.normal_(generator=g)
        vc.normal_(generator=g)
        q = randn(g, sum(new), H, d, dtype=DT[dtype])
        bad = spoil(q, rows)
        kv, cu = torch.tensor(lens, dtype=torch.int32, device="cuda"), starts(new)
        for max_kv in (1, 3000):
            for max_q in (1, max(new), 100000):
                out = [st.st_paged_attn(st.st_pattern(*pat), x, kc, vc, table, cu, kv, max_q, max_kv) for x in (q, bad)]
                for a, b in zip(*out):
                    only_those(rows, a, b)
    assert st.st_last_device_status() == st.ST_OK


# ---- a process whose first call is captured ---------------------------------------------------------

FIRST = r"""
import torch
import factorized_sparse_self_b200 as st

calls = {calls!r}
g = torch.Generator(device="cuda").manual_seed(0)
n, H, Hkv, d = 200, 4, 2, 64
q, k, v, dout = (torch.randn(n, h, d, generator=g, device="cuda").to(torch.{dtype}) for h in (H, Hkv, Hkv, H))
P = st.st_pattern("strided", "merged", 16)
cu = torch.tensor([0, 150, n], dtype=torch.int32, device="cuda")
kc, vc = (torch.zeros(14, 16, Hkv, d, dtype=q.dtype, device="cuda") for _ in range(2))
table = torch.arange(20, dtype=torch.int32, device="cuda").remainder(14).view(2, 10).contiguous()
table[1] = torch.tensor([10, 11, 12, 13, 0, 0, 0, 0, 0, 0], dtype=torch.int32)
kv = torch.tensor([150, 50], dtype=torch.int32, device="cuda")

def run():
    out = []
    if "packed" in calls:
        o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, 150)
        out += [o, lse, *st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, 150)]
    if "append" in calls:
        st.st_cache_append(k, v, kc, vc, table, cu, kv)
        out += [kc, vc]
    if "paged" in calls:
        out += st.st_paged_attn(P, q, kc, vc, table, cu, kv, 150, 150)
    return out

torch.cuda.synchronize()
if {query}:
    st.st_packed_attn_fwd_workspace(P, q, k, v, cu, 150)
    st.st_paged_attn_workspace(P, q, kc, vc, table, cu, kv, 150, 150)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
for x in got:
    x.zero_()
graph.replay()
torch.cuda.synchronize()
assert st.st_last_device_status() == st.ST_OK
got = [x.clone() for x in got]
assert any(bool((x != 0).any()) for x in got)
for a, b in zip(got, run()):
    assert torch.equal(a, b)
print("FIRST CALL OK")
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("query,calls", [(True, ("packed",)), (False, ("packed",)), (False, ("append", "paged"))], ids=str)
def test_first_call_of_a_process_under_capture(query, calls, dtype):
    """Nothing ran before, at most a workspace query: the status word is made while the stream is captured."""
    got = subprocess.run([sys.executable, "-c", FIRST.format(query=query, calls=calls, dtype=dtype)], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "FIRST CALL OK" in got.stdout, got.stderr[-2000:]


# ---- lengths outside the page table -----------------------------------------------------------------


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 32)])
def test_append_reports_lengths_outside_the_page_table(dtype, d):
    """Two pages of 16 slots a sequence. Tokens that the length puts past the last slot, or before the first, are
    dropped; the others are written; the length is reported either way."""
    Hkv, page = 2, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32, device="cuda")
    k, v = (randn(g, 7, Hkv, d, dtype=DT[dtype]) for _ in range(2))
    new = [3, 4]
    for bad in (33, 34, 60, 2 ** 31 - 1, -1, -30, -2 ** 31):
        for which in (0, 1):
            lens = [20, 20]
            lens[which] = bad
            kc, vc = (torch.full((4, page, Hkv, d), x, dtype=DT[dtype], device="cuda") for x in (3.0, 4.0))
            want_k, want_v = kc.clone(), vc.clone()
            a = 0
            for s, (n, m) in enumerate(zip(lens, new)):
                for t in range(m):
                    p = n - m + t
                    if 0 <= p < 2 * page:
                        want_k[int(table[s, p // page]), p % page] = k[a + t]
                        want_v[int(table[s, p // page]), p % page] = v[a + t]
                a += m
            st.st_cache_append(k, v, kc, vc, table, starts(new), torch.tensor(lens, dtype=torch.int32, device="cuda"))
            assert st.st_last_device_status() == st.ST_ERR_INVALID, bad
            assert st.st_last_device_status() == st.ST_OK
            assert torch.equal(kc, want_k) and torch.equal(vc, want_v), bad
    # the largest length, and rows at negative positions, are no error
    st.st_cache_append(k, v, kc, vc, table, starts(new), torch.tensor([32, 2], dtype=torch.int32, device="cuda"))
    assert st.st_last_device_status() == st.ST_OK


# ---- waits that run out -----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128)])
def test_a_launch_that_times_out_ends_at_once(dtype, d):
    """32 k units, more than 200 for every SM. Each CTA that runs meets a tile that never comes and gives up after the
    limit of 20 ms (and as long again for the copies that it waits for); units that have not started are dropped. One
    CTA after the other would take more than 4 s. The next call is right."""
    n, H, Hkv = 4000, 16, 8
    g = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (randn(g, n, h, d, dtype=DT[dtype]) for h in (H, Hkv, Hkv))
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    P = st.st_pattern("dense")
    want = st.st_packed_attn_fwd(P, q, k, v, cu, 1)
    assert st.st_last_device_status() == st.ST_OK
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    st.st_set_wait_limit(20_000_000, force_timeout=True)
    try:
        begin.record()
        st.st_packed_attn_fwd(P, q, k, v, cu, 1)
        end.record()
        assert st.st_last_device_status() == st.ST_ERR_DEVICE_TIMEOUT
        assert begin.elapsed_time(end) < 1000
    finally:
        st.st_set_wait_limit(0, force_timeout=False)
    assert st.st_last_device_status() == st.ST_OK
    for a, b in zip(want, st.st_packed_attn_fwd(P, q, k, v, cu, 1)):
        assert torch.equal(a, b)
    assert st.st_last_device_status() == st.ST_OK


def test_a_forced_time_out_waits_for_a_kernel_with_waits():
    """Calls whose kernels have none (a decoding step, float32) pass it by; a chunk takes it, once."""
    g = torch.Generator(device="cuda").manual_seed(7)
    kc, vc, table = make_cache(g, [400, 300], 16, 2, 64, torch.bfloat16)
    kc.normal_(generator=g)
    vc.normal_(generator=g)
    q = randn(g, 200, 8, 64, dtype=torch.bfloat16)
    kv, P = torch.tensor([400, 300], dtype=torch.int32, device="cuda"), st.st_pattern("dense")

    def step(m):
        return st.st_paged_attn(P, q[:2 * m], kc, vc, table, starts([m, m]), kv, m, 400)

    want = step(1), step(100)
    x = randn(g, 50, 2, 64, dtype=torch.float32)
    st.st_set_wait_limit(20_000_000, force_timeout=True)
    try:
        got = step(1)
        st.st_packed_attn_fwd(P, x, x, x, starts([50]), 50)
        assert st.st_last_device_status() == st.ST_OK
        step(100)
        assert st.st_last_device_status() == st.ST_ERR_DEVICE_TIMEOUT
        for a, b in zip(want[0] + want[1], got + step(100)):
            assert torch.equal(a, b)
        assert st.st_last_device_status() == st.ST_OK
    finally:
        st.st_set_wait_limit(0, force_timeout=False)


def test_shortest_wait_limit_leaves_time_for_copies_under_way():
    """A limit of a nanosecond counts as a millisecond: no wait of these calls is that long."""
    g = torch.Generator(device="cuda").manual_seed(8)
    lens = [700, 300, 1]
    q, k, v, dout = (randn(g, 1001, h, 64, dtype=torch.bfloat16) for h in (8, 4, 4, 8))
    cu, P = starts(lens), st.st_pattern("strided", "merged", 20)

    def run():
        o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, 700)
        return (o, lse, *st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, 700))

    want = run()
    torch.cuda.synchronize()
    st.st_set_wait_limit(1, force_timeout=False)
    try:
        got = run()
        assert st.st_last_device_status() == st.ST_OK
    finally:
        st.st_set_wait_limit(0, force_timeout=False)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


# ---- batches without tokens ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [0, 5])
def test_batches_of_empty_sequences(rows, dtype):
    """The longest sequence is 0 long; rows of no sequence stay as they were."""
    H, Hkv, d, dt = 4, 2, 64, DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(9)
    P, cu = st.st_pattern("strided", "merged", 8), starts([0, 0, 0])
    q, k, v, dout = (randn(g, rows, h, d, dtype=dt) for h in (H, Hkv, Hkv, H))
    o, lse, dq, dk, dv = (torch.full((rows, *s), 7.0, dtype=t, device="cuda") for s, t in (
        ((H, d), dt), ((H,), torch.float32), ((H, d), dt), ((Hkv, d), dt), ((Hkv, d), dt)))
    st.st_packed_attn_fwd_workspace(P, q, k, v, cu, 0)
    st.st_packed_attn_bwd_workspace(P, q, k, v, cu, 0)
    st.st_packed_attn_fwd(P, q, k, v, cu, 0, o=o, lse=lse)
    st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, 0, dq=dq, dk=dk, dv=dv)
    kc, vc, table = make_cache(g, [0, 0, 0], 16, Hkv, d, dt)
    kv = torch.zeros(3, dtype=torch.int32, device="cuda")
    st.st_cache_append(k, v, kc, vc, table, cu, kv)
    st.st_paged_attn_workspace(P, q, kc, vc, table, cu, kv, 0, 0)
    st.st_paged_attn(P, q, kc, vc, table, cu, kv, 0, 0, o=o, lse=lse)
    assert st.st_last_device_status() == st.ST_OK
    assert all(bool((x == 7.0).all()) for x in (o, lse, dq, dk, dv)) and bool(torch.isnan(kc).all())
    for bad in (-1, -5):
        with pytest.raises(st.StatusError):
            st.st_packed_attn_fwd(P, q, k, v, cu, bad)
        with pytest.raises(st.StatusError):
            st.st_paged_attn(P, q, kc, vc, table, cu, kv, bad, 0)


# ---- alignment, groups and starts at their limits -----------------------------------------------------


def sixteen_bytes_on(shape, dtype, fill=7.0):
    """A contiguous tensor whose first element lies 16 bytes past a 256-byte boundary."""
    n, skip = 1, 16 // torch.empty((), dtype=dtype).element_size()
    for x in shape:
        n *= x
    return torch.full((n + skip,), fill, dtype=dtype, device="cuda")[skip:].view(shape)


@pytest.mark.parametrize("ty", THREE, ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("pat,lens,H,Hkv", SPLITS, ids=str)
def test_tensors_on_16_byte_boundaries_only(pat, lens, H, Hkv, ty):
    """Rows are stored 32 bytes at a time where they can be: the results are the same where they cannot."""
    dtype, d = ty
    dt, n = DT[dtype], sum(lens)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = [randn(g, n, h, d, dtype=dt) for h in (H, Hkv, Hkv, H)]
    P, cu = st.st_pattern(*pat), starts(lens)
    o, lse = st.st_packed_attn_fwd(P, *x[:3], cu, max(lens))
    grads = st.st_packed_attn_bwd(P, *x[:3], o, lse, x[3], cu, max(lens))
    y = [sixteen_bytes_on(t.shape, dt).copy_(t) for t in x]
    assert all(t.data_ptr() % 32 == 16 for t in y)
    o2, lse2, *grads2 = (sixteen_bytes_on(t.shape, t.dtype) for t in (o, lse, *grads))
    st.st_packed_attn_fwd(P, *y[:3], cu, max(lens), o=o2, lse=lse2)
    st.st_packed_attn_bwd(P, *y[:3], o2, lse2, y[3], cu, max(lens), dq=grads2[0], dk=grads2[1], dv=grads2[2])
    assert st.st_last_device_status() == st.ST_OK
    for a, b in zip((o, lse, *grads), (o2, lse2, *grads2)):
        assert torch.equal(a, b)
    # the same rows as a chunk and as single tokens over a cache that starts there
    page = 16
    kc, vc = (sixteen_bytes_on((-(-n // page), page, Hkv, d), dt, float("nan")) for _ in range(2))
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None].contiguous()
    kv = torch.tensor([n], dtype=torch.int32, device="cuda")
    st.st_cache_append(y[1], y[2], kc, vc, table, starts([n]), kv)
    for m in (1, 90):
        out = [st.st_paged_attn(P, q, kc, vc, table, starts([m]), kv, m, n, o=o3, lse=lse3) for q, o3, lse3 in (
            (x[0][-m:].contiguous(), None, None),
            (sixteen_bytes_on((m, H, d), dt).copy_(x[0][-m:]), sixteen_bytes_on((m, H, d), dt), sixteen_bytes_on((m, H), torch.float32)))]
        for a, b in zip(*out):
            assert torch.equal(a, b)
        ro, to, rl, tl = One(pat, x[0][-m:], x[1], x[2], dt).outputs()
        check("o", out[1][0], ro, to)
    assert st.st_last_device_status() == st.ST_OK


@pytest.mark.parametrize("ty", THREE, ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("G", [64, 128, 129, 300])
def test_groups_of_a_tile_of_heads_and_more(G, ty):
    """One query's heads fill a tile, or several."""
    dtype, d = ty
    for pat in (("dense", "merged", 1, 1), ("strided", "merged", 5, 1), ("fixed", "split", 6, 2)):
        packed(pat, G, 1, d, dtype, [19, 1, 40], backward=True, lead=2)
        paged(pat, G, 1, d, dtype, [70, 33, 2], [1, 5, 1], 16)
        paged(pat, G, 1, d, dtype, [70, 33, 2], [1, 1, 1], 16, max_q=1)


@pytest.mark.parametrize("ty", THREE, ids=lambda t: f"{t[0]}-d{t[1]}")
def test_starts_outside_the_rows_are_clamped(ty):
    dtype, d = ty
    g = torch.Generator(device="cuda").manual_seed(5)
    n, H, Hkv = 310, 4, 2
    q, k, v, dout = (randn(g, n, h, d, dtype=DT[dtype]) for h in (H, Hkv, Hkv, H))
    P = st.st_pattern("strided", "merged", 12)

    def run(cu):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, n)
        return (o, lse, *st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, n))

    for wild, tame in (([-5, 100, 10 ** 9], [0, 100, n]), ([-2 ** 31, -7, 2 ** 31 - 1, 2 ** 31 - 1], [0, 0, n, n])):
        for a, b in zip(run(wild), run(tame)):
            assert torch.equal(a, b)
    assert st.st_last_device_status() == st.ST_OK


def test_packed_offsets_past_32_bits():
    """Tensors of more than 2^32 elements, and parts of them in fp32: the last sequence's rows and gradients."""
    long, short, H, d = 1_060_000, 300, 32, 128
    g = torch.Generator(device="cuda").manual_seed(6)
    n = long + short
    assert n * H * d > 2 ** 32
    q, k, v, dout = (torch.randn(n, h, d, generator=g, device="cuda", dtype=torch.bfloat16) for h in (H, 1, 1, H))
    P, cu = st.st_pattern("strided", "merged", 512), starts([long, short])
    o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, long)
    grads = st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, long)
    assert st.st_last_device_status() == st.ST_OK
    a = long
    one = One(("strided", "merged", 512, 1), q[a:], k[a:], v[a:], torch.bfloat16)
    ro, to, rl, tl = one.outputs()
    check("o", o[a:], ro, to)
    check("lse", lse[a:], rl, tl)
    for name, got, (want, tol) in zip(("dq", "dk", "dv"), grads, one.backward(dout[a:])):
        check(name, got[a:], want, tol)
    # causal: the first rows of the long sequence have what they would have alone
    m = 200
    one = One(("strided", "merged", 512, 1), q[:m], k[:m], v[:m], torch.bfloat16)
    ro, to, rl, tl = one.outputs()
    check("o", o[:m], ro, to)
    check("lse", lse[:m], rl, tl)
    del q, dout, o, grads
    torch.cuda.empty_cache()


@pytest.mark.parametrize("ty", THREE, ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("pat,lens,H,Hkv", SPLITS, ids=str)
def test_results_repeat_bit_by_bit(pat, lens, H, Hkv, ty):
    """One part a row, key ranges, two orders; units go to whichever SM is free, sums do not."""
    dtype, d = ty
    dt, n = DT[dtype], sum(lens)
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v, dout = (randn(g, n, h, d, dtype=dt) for h in (H, Hkv, Hkv, H))
    P, cu = st.st_pattern(*pat), starts(lens)
    kc, vc, table = make_cache(g, lens, 16, Hkv, d, dt)
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st.st_cache_append(k, v, kc, vc, table, cu, kv)

    def run():
        o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, max(lens))
        out = [o, lse, *st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, max(lens))]
        for m in (1, 64):
            out += st.st_paged_attn(P, q[:2 * m], kc, vc, table, starts([m, m]), kv, m, max(lens))
        return out

    first = run()
    for _ in range(8):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)
