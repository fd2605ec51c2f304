"""Inputs, references in 64 bits and error bounds for the adapter operators.

The references are plain torch in float64, adapter by adapter over its own
tokens. The bounds are derived, not tuned:

* every output is rounded once to bf16: half a step, 2^-8 of the value;
* an fp32 sum of n terms is off by at most n * 2^-23 * sum |terms| (2^-24 per
  rounded addition, a whole step where the tensor cores truncate);
* u and v are held as fp32 or as a bf16 leading and trailing part, which
  leaves at most 2^-16 of each.
"""
import numpy as np
import torch

import oracle
import synth
from gpu_util import to_dev

F64 = torch.float64
HALF_STEP = 2.0 ** -8
SUM = 2.0 ** -23
PAIR = 2.0 ** -16


def ids_of(kind: str, m: int, adapters: int, gen) -> torch.Tensor | None:
    if kind == "null":
        return None
    if kind == "nobody":
        return torch.full((m,), -1, dtype=torch.int32)
    ids = torch.randint(0, adapters, (m,), generator=gen)
    if kind == "runs":
        ids = torch.sort(ids).values
    elif kind == "holes":   # every kind of "no adapter"
        bad = torch.tensor([-1, adapters, -2 ** 31, 2 ** 31 - 1, adapters + 7])
        take = torch.rand(m, generator=gen) < 0.4
        ids = torch.where(take, bad[torch.randint(0, 5, (m,), generator=gen)], ids)
    elif kind == "last":    # only the last adapter has tokens
        ids = torch.full((m,), adapters - 1)
    else:
        assert kind == "mixed", kind
    return ids.to(torch.int32)


class Case:
    """Inputs of one layer with adapters, on the GPU, from a seed."""

    def __init__(self, m, n, k, g, bits, adapters, rank, kind, seed=0, dev="cuda:0"):
        self.m, self.n, self.k, self.g, self.bits = m, n, k, g, bits
        self.adapters, self.rank, self.dev = adapters, rank, dev
        gen = torch.Generator().manual_seed(seed * 1009 + m * 31 + n + k + rank)

        def normal(*shape):
            return torch.randn(*shape, generator=gen)

        idx, lut, al, be = synth.random_any4(n, k, g, seed, layer=f"lora{n}x{k}")
        if bits < 4:
            idx = idx & (0x77 if bits == 3 else 0x33)
        self.q = oracle.Any4Tensors(idx, lut, al, be, g)
        bf = torch.bfloat16
        self.x = (normal(m, k) * torch.exp(0.5 * normal(k))).to(bf).to(dev)
        self.dy = (0.1 * normal(m, n)).to(bf).to(dev)
        self.a = (normal(adapters, rank, k) / k ** 0.5).to(bf).to(dev)
        self.b = (0.05 * normal(adapters, n, rank)).to(bf).to(dev)
        self.scale = (16.0 / rank * torch.exp(0.3 * normal(adapters))).to(dev)
        ids = ids_of(kind, m, adapters, gen)
        self.ids = None if ids is None else ids.to(dev)
        self.tokens = [torch.nonzero((ids if ids is not None else torch.zeros(m)) == l).flatten().to(dev)
                       for l in range(adapters)]
        self._w = None

    def packed(self):
        import learned_bit_lut_b200 as a4
        q = self.q
        return a4.any4_pack_bits(self.bits, *(to_dev(t, self.dev) for t in (q.idx_nib, q.lut, q.alpha, q.beta)), self.g)

    def weight(self):
        """W_hat as the format defines it, in float64 (rounded by the oracle)."""
        if self._w is None:
            bits = oracle.dequant(self.q)
            self._w = to_dev(bits, self.dev).view(torch.bfloat16).to(F64)
        return self._w

    def shape(self):
        return self.n, self.k, self.g

    # ---- references: value and bound of the error before the output's rounding

    def u_ref(self):
        x = self.x.to(F64)
        u, bound = torch.zeros(self.m, self.rank, dtype=F64, device=self.dev), None
        bound = torch.zeros_like(u)
        for l, t in enumerate(self.tokens):
            a, s = self.a[l].to(F64), self.scale[l].to(F64)
            u[t] = s * (x[t] @ a.T)
            bound[t] = (self.k + 2) * SUM * s * (x[t].abs() @ a.abs().T)
        return u, bound

    def y_ref(self):
        x, w = self.x.to(F64), self.weight()
        u, ub = self.u_ref()
        y = x @ w.T
        bound = (self.k + 2 * self.rank + 8) * SUM * (x.abs() @ w.abs().T)
        for l, t in enumerate(self.tokens):
            b = self.b[l].to(F64)
            y[t] += u[t] @ b.T
            bound[t] += (ub[t] + PAIR * u[t].abs()) @ b.abs().T
            bound[t] += (self.k + 2 * self.rank + 8) * SUM * (u[t].abs() @ b.abs().T)
        return y, bound

    def v_ref(self):
        dy = self.dy.to(F64)
        v = torch.zeros(self.m, self.rank, dtype=F64, device=self.dev)
        bound = torch.zeros_like(v)
        for l, t in enumerate(self.tokens):
            b, s = self.b[l].to(F64), self.scale[l].to(F64)
            v[t] = s * (dy[t] @ b)
            bound[t] = (self.n + 2) * SUM * s * (dy[t].abs() @ b.abs())
        return v, bound

    def grad_ref(self, x, u):
        """(dx, da, db) with bounds for a kept input x and inner activation u."""
        dy, w = self.dy.to(F64), self.weight()
        x, u = x.to(F64), u.to(F64)
        v, vb = self.v_ref()
        dx = dy @ w
        terms = self.n + 2 * self.rank + 8
        dxb = terms * SUM * (dy.abs() @ w.abs())
        da = torch.zeros(self.adapters, self.rank, self.k, dtype=F64, device=self.dev)
        db = torch.zeros(self.adapters, self.n, self.rank, dtype=F64, device=self.dev)
        dab, dbb = torch.zeros_like(da), torch.zeros_like(db)
        for l, t in enumerate(self.tokens):
            a = self.a[l].to(F64)
            dx[t] += v[t] @ a
            dxb[t] += (vb[t] + PAIR * v[t].abs()) @ a.abs() + terms * SUM * (v[t].abs() @ a.abs())
            da[l] = v[t].T @ x[t]
            dab[l] = (vb[t] + PAIR * v[t].abs()).T @ x[t].abs() + (2 * len(t) + 8) * SUM * (v[t].abs().T @ x[t].abs())
            db[l] = dy[t].T @ u[t]
            dbb[l] = (2 * len(t) + 8) * SUM * (dy[t].abs().T @ u[t].abs())
        return (dx, dxb), (da, dab), (db, dbb)


def check(got: torch.Tensor, ref: torch.Tensor, bound: torch.Tensor, what: str):
    """Every element within its bound plus half a bf16 step; the same NaN and
    infinite places."""
    got = got.to(F64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN places differ"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    err = (got - ref).abs()[fin]
    # the computed value is rounded, so half a step of |ref| + bound; 1e-37: outputs near zero
    limit = (bound + HALF_STEP * (ref.abs() + bound) + 1e-37)[fin]
    bad = err > limit
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float((err / limit).max()):.2f} of the bound")
    if err.numel() > 4096:   # the rounding errors as a whole: no element's sum can hide a lost term
        # a rounding to bf16 is off by 2^-8 / sqrt(3) of the value on its binade's mean square at most
        off, size, room = float(err.norm()), float(ref[fin].norm()), float(bound[fin].norm())
        assert off <= 2.0 ** -8 / 3 ** 0.5 * size + room, f"{what}: off by {off} of {size}"


def guarded(shape, dtype=torch.bfloat16, dev="cuda:0", tail=64):
    """A contiguous tensor in the middle of a larger buffer of a known pattern,
    and a check that the buffer around it is untouched."""
    count = int(np.prod(shape))
    size = torch.empty((), dtype=dtype).element_size()
    pad = tail * 16 // size
    buf = torch.full(((count + 2 * pad) * size,), 0x5A, dtype=torch.uint8, device=dev).view(dtype)
    inner = buf[pad:pad + count].view(*shape)

    def untouched():
        edge = torch.cat((buf[:pad], buf[pad + count:])).view(torch.uint8)
        return bool((edge == 0x5A).all())

    return inner, untouched
