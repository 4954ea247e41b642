"""Packed and paged attention on the GPU where callers' data lie at the edges: rows before the first sequence, rows that
are not finite, lengths past the cache, first calls inside a capture. Reference and bounds: tests/ragged_ref.py."""
import pytest
import torch

import factorized_sparse_self_b200 as st
from ragged_ref import One, check
from test_gpu_ragged import DT, make_cache, packed, randn, starts

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
