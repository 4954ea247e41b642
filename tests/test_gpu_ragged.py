"""Attention over packed sequences and paged caches on the GPU, against plain 64-bit attention
(tests/ragged_ref.py derives the tolerances entry by entry)."""
import pytest
import torch

import factorized_sparse_self_b200 as st
from ragged_ref import One, check

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def randn(gen, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def packed(pat, H, Hkv, d, dtype, lens, seed=0, tail=3, backward=False, fused=False, std=1.0, scale=None, lead=0):
    """Runs the packed calls and checks everything against the reference. `lead`, `tail`: rows of no sequence before
    the first and behind the last, filled with NaN on input and with a sentinel on output."""
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(lens)
    total = lead + n + tail
    if fused:
        qkv = randn(g, total, H + 2 * Hkv, d, dtype=dt, std=std)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:
        q, k, v = (randn(g, total, h, d, dtype=dt, std=std) for h in (H, Hkv, Hkv))
    dout = randn(g, total, H, d, dtype=dt)
    for x in (q, k, v, dout):
        x[:lead] = float("nan")
        x[lead + n:] = float("nan")
    at = [lead]
    for m in lens:
        at.append(at[-1] + m)
    cu = torch.tensor(at, dtype=torch.int32, device="cuda")
    P = st.st_pattern(*pat)
    mark = 7.0
    o = torch.full((total, H, d), mark, dtype=dt, device="cuda")
    lse = torch.full((total, H), mark, device="cuda")
    st.st_packed_attn_fwd(P, q, k, v, cu, max(max(lens), 1), scale=scale, o=o, lse=lse)
    grads = None
    if backward:
        if fused:
            dqkv = torch.full_like(qkv, mark)
            grads = dqkv[:, :H], dqkv[:, H:H + Hkv], dqkv[:, H + Hkv:]
        else:
            grads = tuple(torch.full_like(x, mark) for x in (q, k, v))
        st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, max(max(lens), 1), scale=scale, dq=grads[0], dk=grads[1],
                              dv=grads[2])
    torch.cuda.synchronize()
    assert st.st_last_device_status() == st.ST_OK
    for x in (o, lse, *(grads or ())):
        assert bool((x[:lead] == mark).all()) and bool((x[lead + n:] == mark).all()), "rows of no sequence were written"
    for a, b in zip(at[:-1], at[1:]):
        if a == b:
            continue
        one = One(pat, q[a:b], k[a:b], v[a:b], dt, scale)
        ro, to, rl, tl = one.outputs()
        check("o", o[a:b], ro, to)
        check("lse", lse[a:b], rl, tl)
        if backward:
            for name, got, (want, tol) in zip(("dq", "dk", "dv"), grads, one.backward(dout[a:b])):
                check(name, got[a:b], want, tol)
    return o, lse, grads


PATTERNS = [("dense", "merged", 1, 1), ("strided", "split", 16, 1), ("strided", "merged", 16, 1), ("strided", "split", 1, 1),
            ("strided", "merged", 1, 1), ("strided", "merged", 7, 1), ("strided", "split", 300, 1), ("strided", "merged", 5000, 1),
            ("fixed", "split", 16, 4), ("fixed", "merged", 16, 4), ("fixed", "merged", 128, 8), ("fixed", "split", 40, 40),
            ("fixed", "merged", 40, 40), ("fixed", "split", 5000, 3), ("fixed", "merged", 1, 1), ("fixed", "split", 7, 2)]
LENS = [[1], [0, 5, 0], [130, 1, 64, 257], [700], [128, 256], [129, 0, 0, 3, 383]]
HEADS = [(1, 1), (4, 1), (6, 3), (5, 1), (15, 3), (2, 2)]
TYPES = [("bf16", 64), ("f16", 64), ("bf16", 128), ("f16", 128), ("f32", 32), ("f32", 64), ("f32", 128)]


@pytest.mark.parametrize("ty", TYPES, ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("pat", PATTERNS, ids=lambda p: "-".join(map(str, p)))
def test_packed_forward_and_backward(pat, ty):
    dtype, d = ty
    # every pattern meets every list of lengths and every grouping, in a rotation of its own
    for x in range(6):
        lens, (H, Hkv) = LENS[x], HEADS[(x + PATTERNS.index(pat) + TYPES.index(ty)) % 6]
        packed(pat, H, Hkv, d, dtype, lens, seed=x, backward=True, lead=x % 2)


@pytest.mark.parametrize("ty", [("bf16", 64), ("f16", 128), ("f32", 64)], ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("heads", [(8, 2), (7, 7), (6, 2)], ids=str)
def test_packed_slices_of_fused_tensors(ty, heads):
    packed(("fixed", "merged", 32, 4), *heads, ty[1], ty[0], [200, 61], fused=True, backward=True)
    packed(("strided", "split", 9, 1), *heads, ty[1], ty[0], [33, 300], fused=True, backward=True, tail=0)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f16", 64), ("f32", 64)])
def test_packed_longer_sequences(dtype, d):
    packed(("dense", "merged", 1, 1), 4, 2, d, dtype, [2049, 1000], backward=True)
    packed(("strided", "merged", 45, 1), 4, 1, d, dtype, [2500, 77], backward=True)
    packed(("fixed", "merged", 128, 8), 2, 2, d, dtype, [2200, 2047], backward=True)
    packed(("fixed", "split", 64, 8), 4, 2, d, dtype, [2300], backward=True)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("pat", [("dense", "merged", 1, 1), ("fixed", "split", 20, 9), ("strided", "merged", 10, 1), ("strided", "split", 200, 1)], ids=str)
def test_many_units_of_different_lengths(pat, dtype, d):
    """Several units for every CTA, of no, few and many key tiles, one behind the other."""
    packed(pat, 24, 6, d, dtype, [1500, 3, 0, 700, 129, 1, 260], backward=True)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128), ("f32", 64)])
@pytest.mark.parametrize("pat", [(kind, mode, l, c) for kind in ("strided", "fixed") for mode in ("split", "merged")
                                 for l, c in ((2 ** 31 - 1, 5), (2 ** 31 - 1, 2 ** 31 - 1))], ids=str)
def test_largest_strides(pat, dtype, d):
    """One class, window or block holds the whole sequence."""
    packed(pat, 4, 2, d, dtype, [300, 1, 129], backward=True)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128), ("f32", 64)])
@pytest.mark.parametrize("pat", [("strided", "merged", 16, 1), ("strided", "split", 7, 1), ("fixed", "merged", 16, 4), ("fixed", "split", 40, 40),
                                 ("fixed", "split", 20, 3)], ids=str)
def test_many_key_units(pat, dtype, d):
    """Key tiles enough for each key order to go by itself, the last one adding what the first one left."""
    packed(pat, 72, 24, d, dtype, [900, 0, 1, 250, 129, 19, 385], backward=True)
    packed(pat, 64, 32, d, dtype, [200] * 7, backward=True, fused=True, lead=3)


@pytest.mark.parametrize("pat,H,Hkv,d,dtype,lens", [
    (("dense", "merged", 1, 1), 20, 4, 128, "bf16", [2518, 78, 177]), (("dense", "merged", 1, 1), 4, 2, 64, "bf16", [2000]),
    (("strided", "split", 100, 1), 16, 8, 128, "f16", [79, 1159, 19, 52, 10]), (("fixed", "split", 20, 9), 10, 2, 128, "bf16", [3, 2276, 57]),
    (("strided", "merged", 10, 1), 10, 2, 128, "bf16", [7, 48, 16, 3, 1668, 459]), (("strided", "merged", 174, 1), 32, 8, 128, "bf16", [80, 86]),
    (("strided", "merged", 130, 1), 8, 2, 64, "f16", [1000, 300, 20])], ids=str)
def test_gradients_lose_no_more_than_their_roundings(pat, H, Hkv, d, dtype, lens):
    """dQ and dK are sums of products with dS rounded to 16 bits, then rounded themselves: two independent errors of one
    size, the square root of 2 together. What D loses to the rounding of o would come on top; 6 % is left for it."""
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(12)
    n, at = sum(lens), [0]
    q, k, v, dout = (randn(g, n, h, d, dtype=dt) for h in (H, Hkv, Hkv, H))
    P, cu = st.st_pattern(*pat), starts(lens)
    o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, max(lens))
    got = st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, max(lens))
    want = [[], [], []]
    for m in lens:
        a, b = at[-1], at[-1] + m
        at.append(b)
        for x, (ref, _) in zip(want, One(pat, q[a:b], k[a:b], v[a:b], dt).backward(dout[a:b])):
            x.append(ref)
    for name, x, ref in zip(("dq", "dk", "dv"), got, want):
        ref = torch.cat(ref)
        lost, rounding = (float((y.double() - ref).norm()) for y in (x, ref.to(dt)))
        assert lost <= 1.5 * rounding, (name, lost / rounding)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128), ("f32", 32)])
@pytest.mark.parametrize("pat", [("dense", "merged", 1, 1), ("strided", "merged", 3, 1), ("fixed", "merged", 4, 2)], ids=str)
def test_thousands_of_sequences_of_one_token(pat, dtype, d):
    """One key each: O is its value row, dV the sum of dO over the group, dQ and dK are zero but for roundings."""
    dt, H, Hkv, n = DT[dtype], 6, 2, 3001
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v, dout = (randn(g, n, h, d, dtype=dt) for h in (H, Hkv, Hkv, H))
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda").repeat_interleave(2)  # an empty one behind each
    P = st.st_pattern(*pat)
    o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, 1)
    dq, dk, dv = st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, 1)
    assert st.st_last_device_status() == st.ST_OK
    rep = lambda x: x.double().repeat_interleave(H // Hkv, 1)
    e, eps = torch.finfo(dt).eps / 2, 2.0 ** -24
    s = (q.double() * rep(k)).sum(2) * d ** -0.5
    size = (q.double() * rep(k)).abs().sum(2) * d ** -0.5
    # P = exp(s - LSE): the sums of d products and the logarithm's fp32 roundings, and the approximate exp2's
    off = (d + 16) * eps * (size + 1) + 2.0 ** -20
    assert bool(((lse.double() - s).abs() <= off).all())
    assert bool(((o.double() - rep(v)).abs() <= (2 * e + off[..., None]) * rep(v).abs()).all())
    gd = dout.double().view(n, Hkv, H // Hkv, d)
    tol = (2 * e + off.view(n, Hkv, -1).amax(2)[..., None]) * gd.abs().sum(2) + e * gd.abs().sum(2)
    assert bool(((dv.double() - gd.sum(2)).abs() <= tol).all())
    # dS = P (dP - D): what o lost to its rounding, at most, where D is not mended
    ds = (2 * e + 2 * off) * (dout.double() * rep(v)).abs().sum(2) + (d + 16) * eps * (dout.double() * rep(v)).abs().sum(2)
    assert bool((dq.double().abs() <= (ds * d ** -0.5)[..., None] * rep(k).abs() * (1 + 4 * e) + 2.0 ** -24).all())
    lim = ((ds * d ** -0.5)[..., None] * q.double().abs()).view(n, Hkv, -1, d).sum(2) * (1 + 4 * e) + 2.0 ** -24
    assert bool((dk.double().abs() <= lim).all())


def test_two_calls_at_once():
    """Two streams, a workspace each, started together and repeated: each keeps its results."""
    P = st.st_pattern("strided", "merged", 24)
    g = torch.Generator(device="cuda").manual_seed(9)
    data, want = [], []
    for n in (1500, 1100):
        q, k, v, dout = (randn(g, n, h, 64, dtype=torch.bfloat16) for h in (8, 4, 4, 8))
        data.append((q, k, v, dout, starts([n - 300, 300]), n))

    def run(x, stream=None):
        q, k, v, dout, cu, n = x
        o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, n, stream=stream)
        return (o, lse, *st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, n, stream=stream))

    want = [run(x) for x in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[] for _ in data]
    for _ in range(5):
        for i, x in enumerate(data):
            got[i].append(run(x, streams[i]))
    torch.cuda.synchronize()
    assert st.st_last_device_status() == st.ST_OK
    for w, all_of in zip(want, got):
        for out in all_of:
            for a, b in zip(w, out):
                assert torch.equal(a, b)


def test_large_scores_and_given_scale():
    # scores up to about +-60: the running maximum moves by far more than a rounding
    packed(("dense", "merged", 1, 1), 2, 1, 64, "bf16", [700, 300], std=3.0, backward=True)
    packed(("strided", "merged", 20, 1), 2, 1, 128, "f16", [600], std=2.5, backward=True)
    packed(("dense", "merged", 1, 1), 4, 2, 64, "f16", [500], scale=0.31, backward=True)


def test_maximum_that_jumps_late():
    # the largest score of a row is its last key's, far above all before it
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (randn(g, 900, 1, 64, dtype=torch.bfloat16, std=0.2) for _ in range(3))
    k[600:] = k[600:] + 4 * q[600:]
    k[899] = 30 * q[899]
    cu = torch.tensor([0, 900], dtype=torch.int32, device="cuda")
    o, lse = st.st_packed_attn_fwd(st.st_pattern("dense"), q, k, v, cu, 900)
    ro, to, rl, tl = One(("dense", "merged", 1, 1), q, k, v, torch.bfloat16).outputs()
    check("o", o, ro, to)
    check("lse", lse, rl, tl)


def test_neighbours_do_not_mix():
    """A sequence's results do not depend on what is packed around it, infinities and NaN included."""
    P = st.st_pattern("strided", "merged", 24)
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [100, 333, 77]
    q, k, v = (randn(g, 510, h, 64, dtype=torch.bfloat16) for h in (4, 2, 2))
    dout = randn(g, 510, 4, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 100, 433, 510], dtype=torch.int32, device="cuda")

    def run():
        o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, max(lens))
        return [x[100:433].clone() for x in (o, lse, *st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, max(lens)))]

    first = run()
    for x in (q, k, v, dout):
        x[:100] = float("inf")
        x[433:] = float("nan")
    for a, b in zip(first, run()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("pat", [("dense", "merged", 1, 1), ("strided", "merged", 16, 1), ("fixed", "split", 32, 4)], ids=str)
def test_gradient_against_differences(pat):
    """<grad, u> against the central difference of the 64-bit loss along u."""
    g = torch.Generator(device="cuda").manual_seed(11)
    n, H, Hkv, d = 150, 4, 2, 32
    q, k, v = (randn(g, n, h, d, dtype=torch.float32) for h in (H, Hkv, Hkv))
    dout = randn(g, n, H, d, dtype=torch.float32)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    P = st.st_pattern(*pat)
    o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, n)
    grads = st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, n)

    def loss(x):
        return float((One(pat, *x, torch.float32).outputs()[0] * dout.double()).sum())

    for which in range(3):
        u = torch.randn(grads[which].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        x = [t.double() for t in (q, k, v)]
        up = loss([t + h * u if y == which else t for y, t in enumerate(x)])
        dn = loss([t - h * u if y == which else t for y, t in enumerate(x)])
        want = (up - dn) / (2 * h)
        got = float((grads[which].double() * u).sum())
        # truncation: the third derivative along u times h^2 / 6 (h^2 = 1e-8, derivatives of order |u|^3 per row);
        # gradient: fp32 rounding of n * H * d terms
        size = float((grads[which].double() * u).abs().sum())
        assert abs(got - want) <= 1e-5 * size, (which, got, want, size)


def test_reproducible_streams_and_capture():
    P = st.st_pattern("fixed", "merged", 32, 4)
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k, v, dout = (randn(g, 1200, h, 64, dtype=torch.bfloat16) for h in (4, 2, 2, 4))
    cu = torch.tensor([0, 500, 900, 1200], dtype=torch.int32, device="cuda")

    def run(stream=None):
        o, lse = st.st_packed_attn_fwd(P, q, k, v, cu, 700, stream=stream)
        return (o, lse, *st.st_packed_attn_bwd(P, q, k, v, o, lse, dout, cu, 700, stream=stream))

    first = run()
    for a, b in zip(first, run()):
        assert torch.equal(a, b), "not reproducible"
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [run(s) for s in (s1, s2, s1, s2)]
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(first, out):
            assert torch.equal(a, b), "differs on another stream"
    # captured once, replayed with other sequence lengths: they are read on the device
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for lens in ([0, 500, 900, 1200], [0, 1, 700, 1000], [0, 0, 0, 1200]):
        cu.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[lens[0]:lens[-1]], b[lens[0]:lens[-1]])
    assert st.st_last_device_status() == st.ST_OK


# ---- paged cache ---------------------------------------------------------------------------


def make_cache(g, lens, page, Hkv, d, dt, layout="nhd", extra=2):
    """Caches filled with NaN, a page table with unused entries of -1, and the keys and values to write: per sequence."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    if layout == "nhd":
        kc, vc = (torch.full((pages, page, Hkv, d), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    elif layout == "hnd":
        kc, vc = (torch.full((pages, Hkv, page, d), float("nan"), dtype=dt, device="cuda").transpose(1, 2) for _ in range(2))
    else:  # keys and values of a page next to each other
        both = torch.full((pages, 2, page, Hkv, d), float("nan"), dtype=dt, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    return kc, vc, table


def starts(ns):
    at = [0]
    for n in ns:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def paged(pat, H, Hkv, d, dtype, lens, new, page, layout="nhd", seed=0, max_q=None, max_kv=None, tail=2):
    """Fills a cache by st_cache_append, then attends the new tokens. lens may be below new (rows at negative positions)."""
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    kc, vc, table = make_cache(g, lens, page, Hkv, d, dt, layout)
    ks = [randn(g, n, Hkv, d, dtype=dt) for n in lens]
    vs = [randn(g, n, Hkv, d, dtype=dt) for n in lens]
    if sum(lens):
        st.st_cache_append(torch.cat(ks), torch.cat(vs), kc, vc, table, starts(lens),
                           torch.tensor(lens, dtype=torch.int32, device="cuda"))
    total = sum(new) + tail
    q = randn(g, total, H, d, dtype=dt)
    q[sum(new):] = float("nan")
    o = torch.full((total, H, d), 7.0, dtype=dt, device="cuda")
    lse = torch.full((total, H), 7.0, device="cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = starts(new)
    st.st_paged_attn(st.st_pattern(*pat), q, kc, vc, table, cu, kv, max_q or max(new), max_kv or max(max(lens), 1), o=o, lse=lse)
    torch.cuda.synchronize()
    assert st.st_last_device_status() == st.ST_OK
    assert bool((o[sum(new):] == 7.0).all()) and bool((lse[sum(new):] == 7.0).all())
    a = 0
    for s, n in enumerate(new):
        skip = max(0, n - lens[s])
        if skip:
            assert bool((o[a:a + skip] == 0).all()) and bool(torch.isneginf(lse[a:a + skip]).all())
        if n > skip:
            ro, to, rl, tl = One(pat, q[a + skip:a + n], ks[s], vs[s], dt).outputs()
            check("o", o[a + skip:a + n], ro, to)
            check("lse", lse[a + skip:a + n], rl, tl)
        a += n
    return o, lse


@pytest.mark.parametrize("ty", TYPES, ids=lambda t: f"{t[0]}-d{t[1]}")
@pytest.mark.parametrize("pat", PATTERNS, ids=lambda p: "-".join(map(str, p)))
def test_paged_decode_and_chunks(pat, ty):
    dtype, d = ty
    x = PATTERNS.index(pat) + TYPES.index(ty)
    H, Hkv = HEADS[x % 6]
    page = (1, 16, 20, 64, 128, 7)[x % 6]
    layout = ("nhd", "hnd", "both")[x % 3]
    paged(pat, H, Hkv, d, dtype, [1, 700, 65, 129, 0], [1, 1, 1, 1, 1], page, layout, seed=x)
    paged(pat, H, Hkv, d, dtype, [400, 33, 900], [200, 33, 1], page, layout, seed=x + 1)
    paged(pat, H, Hkv, d, dtype, [1000, 3, 0, 130], [3, 5, 2, 0], page, layout, seed=x + 2)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f16", 128), ("f32", 64)])
def test_paged_long_contexts(dtype, d):
    """Few rows over long caches: the keys are split and joined."""
    paged(("dense", "merged", 1, 1), 8, 2, d, dtype, [5000], [1], 16)
    paged(("dense", "merged", 1, 1), 32, 1, d, dtype, [3001, 17], [1, 1], 48)
    paged(("strided", "merged", 64, 1), 4, 4, d, dtype, [6000, 4000], [1, 40], 64)
    paged(("strided", "split", 100, 1), 8, 2, d, dtype, [5000, 10], [130, 1], 16)
    paged(("fixed", "merged", 128, 8), 8, 8, d, dtype, [6100], [4], 32)
    paged(("fixed", "split", 64, 8), 2, 1, d, dtype, [4097, 4096], [1, 300], 20)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("pat", [("dense", "merged", 1, 1), ("fixed", "merged", 700, 600), ("strided", "split", 4000, 1)], ids=str)
def test_paged_chunks_in_ranges_of_different_lengths(pat, dtype, d):
    """More key ranges than SMs: long ones first, a short sequence in fewer of them, one with a single row."""
    paged(pat, 32, 8, d, dtype, [5100, 1300, 4000, 40], [300, 70, 1, 33], 16, layout="hnd")


def test_paged_lengths_are_hints():
    """max_q and max_kv steer the split only."""
    for mq, mk in ((1, 1), (5000, 100000), (1, 100000)):
        paged(("dense", "merged", 1, 1), 8, 2, 64, "bf16", [900, 300], [150, 1], 16, max_q=mq, max_kv=mk)
        paged(("strided", "merged", 16, 1), 8, 2, 64, "f16", [900, 300], [1, 1], 16, max_q=mq, max_kv=mk)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128), ("f32", 64)])
@pytest.mark.parametrize("pat", [p for p in PATTERNS if p[0] == "strided"], ids=lambda p: "-".join(map(str, p)))
def test_paged_strided_chunks_of_few_and_many_rows(pat, dtype, d):
    """The expected chunk chooses the kernel: rows of a few queries, or tiles of 256 rows."""
    for mq in (1, 100000):
        paged(pat, 6, 3, d, dtype, [1300, 90, 0, 700], [300, 100, 2, 129], 24, seed=mq, max_q=mq)
        paged(pat, 5, 1, d, dtype, [650], [600], 64, layout="hnd", seed=mq + 1, max_q=mq)


@pytest.mark.parametrize("pat", [("dense", "merged", 1, 1), ("strided", "merged", 12, 1), ("fixed", "split", 16, 3)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_decode_agrees_with_the_whole_prompt(pat, dtype):
    """Used together: append a prompt in chunks, decode token by token; every row is the packed call's row."""
    dt, H, Hkv, d, n = DT[dtype], 4, 2, 64, 170
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (randn(g, n, h, d, dtype=dt) for h in (H, Hkv, Hkv))
    one = One(pat, q, k, v, dt)
    ro, to, rl, tl = one.outputs()
    P = st.st_pattern(*pat)
    o, lse = st.st_packed_attn_fwd(P, q, k, v, starts([n]), n)
    check("o", o, ro, to)
    kc, vc, table = make_cache(g, [n], 16, Hkv, d, dt)
    a = 0
    for m in (90, 60, 1, 1, 1, 1, 16):
        kv = torch.tensor([a + m], dtype=torch.int32, device="cuda")
        st.st_cache_append(k[a:a + m], v[a:a + m], kc, vc, table, starts([m]), kv)
        o, lse = st.st_paged_attn(P, q[a:a + m], kc, vc, table, starts([m]), kv, m, n)
        check("o", o, ro[a:a + m], to[a:a + m])
        check("lse", lse, rl[a:a + m], tl[a:a + m])
        a += m
    assert a == n and st.st_last_device_status() == st.ST_OK


def test_captured_decoding_step():
    """Append and attend in one graph, replayed while the lengths grow."""
    P, H, Hkv, d = st.st_pattern("fixed", "merged", 16, 4), 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    lens = [40, 7]
    kc, vc, table = make_cache(g, [64, 64], 16, Hkv, d, torch.bfloat16)
    ks, vs, qs = ([randn(g, 64, h, d, dtype=torch.bfloat16) for _ in lens] for h in (Hkv, Hkv, H))
    st.st_cache_append(torch.cat([x[:n] for x, n in zip(ks, lens)]), torch.cat([x[:n] for x, n in zip(vs, lens)]), kc, vc,
                       table, starts(lens), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(2, h, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    cu = starts([1, 1])
    st.st_paged_attn(P, q, kc, vc, table, cu, kv, 1, 64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.add_(1)
        st.st_cache_append(k, v, kc, vc, table, cu, kv)
        o, lse = st.st_paged_attn(P, q, kc, vc, table, cu, kv, 1, 64)
    for step in range(20):
        for s, n in enumerate(lens):
            q[s], k[s], v[s] = qs[s][n + step], ks[s][n + step], vs[s][n + step]
        graph.replay()
        torch.cuda.synchronize()
        for s, n in enumerate(lens):
            m = n + step + 1
            ro, to, rl, tl = One(("fixed", "merged", 16, 4), q[s:s + 1], ks[s][:m], vs[s][:m], torch.bfloat16).outputs()
            check("o", o[s:s + 1], ro, to)
    assert st.st_last_device_status() == st.ST_OK


def test_bad_pages_and_lengths_are_reported():
    """Every table entry and length is checked by the kernels: bad ones set the status, nothing outside is touched."""
    P = st.st_pattern("dense")
    for dtype, d in (("bf16", 64), ("f32", 64)):
        dt = DT[dtype]
        kc = torch.zeros(4, 16, 2, d, dtype=dt, device="cuda")
        vc = torch.zeros_like(kc)
        q, k = torch.zeros(2, 4, d, dtype=dt, device="cuda"), torch.ones(2, 2, d, dtype=dt, device="cuda")
        cu = starts([1, 1])
        for bad, kv in (([[0, 4], [1, 2]], [20, 20]), ([[0, -1], [1, 2]], [20, 20]), ([[0, 3], [1, 2]], [20, 33]),
                        ([[0, 3], [1, 2]], [-1, 3])):
            table = torch.tensor(bad, dtype=torch.int32, device="cuda")
            lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
            for max_q in (1, 200):
                st.st_paged_attn(P, q, kc, vc, table, cu, lens, max_q, 32)
                assert st.st_last_device_status() == st.ST_ERR_INVALID, (bad, kv)
                assert st.st_last_device_status() == st.ST_OK
        before = kc.clone()
        table = torch.tensor([[0, 4], [-1, 2]], dtype=torch.int32, device="cuda")
        st.st_cache_append(k, k, kc, vc, table, cu, torch.tensor([20, 4], dtype=torch.int32, device="cuda"))
        assert st.st_last_device_status() == st.ST_ERR_INVALID
        assert torch.equal(kc, before)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "f16"), (40, "bf16"), (64, "f32"), (4, "f32")])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "both"])
def test_append_writes_the_new_slots_and_no_others(d, dtype, layout):
    dt, Hkv, page = DT[dtype], 3, 12
    g = torch.Generator(device="cuda").manual_seed(1)
    lens, new = [50, 1, 13, 0, 30], [17, 1, 0, 2, 30]
    kc, vc, table = make_cache(g, lens, page, Hkv, d, dt, layout)
    kc.fill_(3.0)
    vc.fill_(4.0)
    want_k, want_v = kc.clone(), vc.clone()
    kv_fused = randn(g, sum(new) + 2, 2 * Hkv, d, dtype=dt)
    k, v = kv_fused[:, :Hkv], kv_fused[:, Hkv:]
    a = 0
    for s, (n, m) in enumerate(zip(lens, new)):
        for t in range(m):
            p = n - m + t
            if p >= 0:
                want_k[int(table[s, p // page]), p % page] = k[a + t]
                want_v[int(table[s, p // page]), p % page] = v[a + t]
        a += m
    st.st_cache_append(k, v, kc, vc, table, starts(new), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert st.st_last_device_status() == st.ST_OK
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: the last pages are read and written."""
    page, Hkv, d = 1024, 8, 128
    pages = (1 << 32) // (page * Hkv * d) + 2  # 4.3e9 elements, 8.6 GB each
    kc = torch.zeros(pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator(device="cuda").manual_seed(6)
    n = 1500
    k, v = (randn(g, n, Hkv, d, dtype=torch.bfloat16) for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    kv = torch.tensor([n], dtype=torch.int32, device="cuda")
    st.st_cache_append(k, v, kc, vc, table, starts([n]), kv)
    for m in (1, 200):
        q = randn(g, m, 16, d, dtype=torch.bfloat16)
        o, lse = st.st_paged_attn(st.st_pattern("dense"), q, kc, vc, table, starts([m]), kv, m, n)
        ro, to, rl, tl = One(("dense", "merged", 1, 1), q, k, v, torch.bfloat16).outputs()
        check("o", o, ro, to)
        check("lse", lse, rl, tl)
    assert st.st_last_device_status() == st.ST_OK
