"""Plain 64-bit attention over ragged sequences, with bounds on what the kernels' roundings may
move each result by.

One sequence at a time: dense scores, a table of truth values for the sets, softmax, gradients
by formula. The bounds follow the arithmetic: e is half a step of the 16-bit type (0 for float32
tensors: `torch.finfo(t).eps / 2` is then the fp32 step, counted in w):
  weights  P is rounded to 16 bits before P V (and P^T dO), so entry by entry
           |dP| <= (e + w) P, where w bounds the fp32 arithmetic behind a weight: a score is a sum
           of d products (relative error (d + 4) u of the sum of their magnitudes, u = 2^-24), its
           exponential errs by as much absolutely, and n weights are summed in fp32
  dS       = P (dP - D), rounded to 16 bits; D = dO . O is formed from the rounded O
  results  rounded once more to the tensor's type.
Below the type's smallest normal number the step no longer shrinks with the value: half a step is
a = smallest_normal * eps / 2 there (fp16: 2^-25; fp16's smallest normal number is 2^-14, so small
weights and gradients do meet it). Every rounding to the type therefore counts a beside its
relative term: a itself for a result, a |v| for each weight of a row (weights are rounded before
the division by their sum, which is at least 1), a |q|, a |k|, a |dO| for each entry of dS and P.
"""
import torch

U = 2.0 ** -24


def keeps(kind, mode, l, c, i, j, parity):
    """Truth table [len(i), len(j)] of the set of a head of the given parity."""
    i, j = i[:, None], j[None, :]
    past = (j <= i) & (i >= 0)
    if kind == "dense":
        return past
    if kind == "strided":
        sets = [past & (j >= i - l), past & (torch.remainder(i - j, l) == 0)]
    else:
        sets = [past & (torch.div(i, l, rounding_mode="floor") == torch.div(j, l, rounding_mode="floor")),
                past & (torch.remainder(j, l) >= l - c)]
    return sets[0] | sets[1] if mode == "merged" else sets[parity]


class One:
    """One sequence in float64: q [nq, H, d] at positions nk - nq .., k, v [nk, Hkv, d]."""

    def __init__(self, pat, q, k, v, dtype, scale=None):
        kind, mode, l, c = pat
        nq, H, d = q.shape
        nk, Hkv, _ = k.shape
        G = H // Hkv
        self.scale = scale or d ** -0.5
        self.q = q.double().permute(1, 0, 2)
        self.k = k.double().permute(1, 0, 2).repeat_interleave(G, 0)
        self.v = v.double().permute(1, 0, 2).repeat_interleave(G, 0)
        self.G, self.Hkv = G, Hkv
        i = torch.arange(nk - nq, nk, device=q.device)
        j = torch.arange(nk, device=q.device)
        live = torch.stack([keeps(kind, mode, l, c, i, j, h % 2) for h in range(H)])
        s = (self.q @ self.k.transpose(1, 2)) * self.scale
        s = s.masked_fill(~live, float("-inf"))
        self.lse = torch.logsumexp(s, 2) if nk else torch.full((H, nq), float("-inf"), dtype=torch.float64, device=q.device)
        base = torch.where(torch.isinf(self.lse), torch.zeros_like(self.lse), self.lse)
        self.p = torch.exp(s - base[:, :, None])
        self.o = self.p @ self.v
        top = ((self.q.abs() @ self.k.abs().transpose(1, 2)) * self.scale * live).amax() if nq * nk else torch.zeros(())
        self.w = float(U * (2 * (d + 4) * float(top) + nk + 64))
        self.eps = torch.finfo(dtype).eps / 2
        self.e = 0.0 if dtype == torch.float32 else self.eps
        self.a = torch.finfo(dtype).smallest_normal * self.eps
        self.a_in = 0.0 if dtype == torch.float32 else self.a
        self.live = live.double()
        self.o_tol = self.eps * self.o.abs() + self.a + (self.e + 2 * self.w) * (self.p @ self.v.abs()) + \
            self.a_in * (self.live @ self.v.abs())
        self.lse_tol = (self.w + 4 * U * base.abs()) * torch.ones_like(base)

    def outputs(self):
        """o, its bound [nq, H, d]; lse, its bound [nq, H]."""
        f = lambda x: x.permute(1, 0, 2)  # noqa: E731
        return f(self.o), f(self.o_tol), self.lse.T, self.lse_tol.T

    def backward(self, dout):
        """(dq, bound), (dk, bound), (dv, bound)."""
        do = dout.double().permute(1, 0, 2)
        p, e, w = self.p, self.e, self.w
        d = self.q.shape[-1]
        D = (do * self.o).sum(-1, keepdim=True)
        dp = do @ self.v.transpose(1, 2)
        ds = p * (dp - D)
        # D from the rounded O, dP from d products, P from the rounded LSE
        d_err = (do.abs() * (self.o_tol + U * d * self.o.abs())).sum(-1, keepdim=True)
        dp_err = U * (d + 4) * (do.abs() @ self.v.abs().transpose(1, 2))
        ds_err = (e + 4 * w) * ds.abs() + p * (d_err + dp_err) * (1 + e) + self.a_in * self.live
        n = self.p.shape[1] * self.G + self.p.shape[2]
        acc = U * (n + 8)  # a sum of n products in fp32

        def group(x):
            return x.view(self.Hkv, self.G, *x.shape[1:]).sum(1)

        def out(x, tol):
            return x.permute(1, 0, 2), (tol + self.eps * x.abs() + self.a).permute(1, 0, 2)

        s = self.scale
        dq, dk, dv = ds @ self.k * s, group(ds.transpose(1, 2) @ self.q) * s, group(p.transpose(1, 2) @ do)
        dq_tol = s * (ds_err + acc * ds.abs()) @ self.k.abs()
        dk_tol = s * group((ds_err + acc * ds.abs()).transpose(1, 2) @ self.q.abs())
        dv_tol = group(((e + 4 * w + acc) * p + self.a_in * self.live).transpose(1, 2) @ do.abs())
        return out(dq, dq_tol * (1 + self.eps)), out(dk, dk_tol * (1 + self.eps)), out(dv, dv_tol * (1 + self.eps))


def check(name, got, want, tol):
    got = got.double()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf), f"{name}: infinities differ"
    bad = (~inf) & ~((got - want).abs() <= tol)
    if bad.any():
        off = torch.where(inf | torch.isnan(got), torch.zeros_like(got), (got - want).abs() / tol.clamp(min=1e-300))
        at = [int(x) for x in torch.nonzero(bad)[0]]
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values off, the first at {at}: got "
                             f"{float(got[tuple(at)]):.6g}, want {float(want[tuple(at)]):.6g} +- {float(tol[tuple(at)]):.3g}; "
                             f"worst {float(off.max()):.3g} times its bound")
