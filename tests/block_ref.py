"""64-bit forms of the operators around the layer, on CPU tensors, with the
magnitudes that the tolerances are counted in (U: half a step of fp32)."""
from __future__ import annotations

import torch

U = 2.0 ** -24
D = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def d(t):
    return None if t is None else t.detach().cpu().to(D)


def plan(ids, E):
    """Counts, offsets, positions and slots of ids [T][K], slot by slot."""
    T, K = ids.shape
    flat = ids.reshape(-1).tolist()
    by = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            by[e].append(i)
    counts = [len(b) for b in by]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    slot = [i for b in by for i in b]
    pos = [-1] * len(flat)
    for q, i in enumerate(slot):
        pos[i] = q
    slot += [-1] * (len(flat) - len(slot))
    i32 = torch.int32
    return (torch.tensor(counts, dtype=i32), torch.tensor(offsets, dtype=i32),
            torch.tensor(pos, dtype=i32).reshape(T, K), torch.tensor(slot, dtype=i32))


def gather_sum(pos, w, rows, base, H):
    """(sum, sum of magnitudes) of base + w rows[pos]; positions outside the rows add nothing."""
    T, K = pos.shape
    y = torch.zeros((T, H), dtype=D) if base is None else d(base).clone()
    a = y.abs()
    for t in range(T):
        for k in range(K):
            q = int(pos[t, k])
            if 0 <= q < rows.shape[0]:
                r = d(rows[q]) * (1.0 if w is None else float(w[t, k]))
                y[t] += r
                a[t] += r.abs()
    return y, a


def norm_scale(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


class Norm:
    """block_norm and its gradient in 64 bits; None parameters as in the library."""

    def __init__(self, prev, next, token=None):
        # prev: dict(post_norm, post_gain, gate, x_scale, y_scale, eps) or None; next: dict(pre_gain, eps) or None
        self.prev, self.next = prev, next
        self.u = torch.ones((), dtype=D) if token is None else d(token).unsqueeze(1)

    def _p(self):
        one = torch.ones((), dtype=D)
        p = self.prev
        f = lambda t: one if t is None else d(t)  # noqa: E731
        # the scales and eps are fp32 in the library
        g = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
        return f(p.get("post_gain")), f(p.get("gate")), g(p.get("x_scale", 1.0)), g(p.get("y_scale", 1.0)), \
            g(p.get("eps", 1e-6)), p.get("post_norm", False)

    def _n(self):
        q = self.next.get("pre_gain")
        return (torch.ones((), dtype=D) if q is None else d(q)), float(torch.tensor(self.next.get("eps", 1e-6),
                                                                                    dtype=torch.float32))

    def x_out(self, x, y):
        """(x_out unrounded, magnitude of its two terms)."""
        p, g, xs, ys, eps, post = self._p()
        b = ys * self.u * g * p * y * (norm_scale(y, eps) if post else 1.0)
        return xs * x + b, (xs * x).abs() + b.abs()

    def n(self, s):
        q, eps = self._n()
        return s * norm_scale(s, eps) * q

    def backward(self, s, y, dxo, dn):
        """dict of (gradient, magnitude): the magnitudes add the absolute values of every product of the formula."""
        H = s.shape[1]
        dxo = torch.zeros_like(s) if dxo is None else dxo
        ds, Ds, out = dxo, dxo.abs(), {}
        if self.next is not None:
            q, eps = self._n()
            r = norm_scale(s, eps)
            sh = s * r
            m1, M1 = (sh * q * dn).mean(1, keepdim=True), (sh * q * dn).abs().mean(1, keepdim=True)
            ds = ds + r * (q * dn - sh * m1)
            Ds = Ds + r * ((q * dn).abs() + sh.abs() * M1)
            out["dpre"] = ((sh * dn).sum(0), (sh * dn).abs().sum(0))
        if self.prev is None:
            out["dx"] = (ds, Ds)
            return out
        p, g, xs, ys, eps, post = self._p()
        out["dx"] = (xs * ds, abs(xs) * Ds)
        rho = norm_scale(y, eps) if post else torch.ones((), dtype=D)
        yh = y * rho
        dz, Dz = ys * self.u * g * ds, (ys * self.u * g).abs() * Ds
        z = yh * p
        dg, Dg = ys * self.u * z * ds, (ys * self.u * z).abs() * Ds
        du, Du = ys * g * z * ds, (ys * g * z).abs() * Ds
        out["dgate"] = (dg.sum(0), Dg.sum(0))
        out["dtoken"] = (du.sum(1), Du.sum(1))
        out["dpost"] = ((yh * dz).sum(0), (yh.abs() * Dz).sum(0))
        if post:
            m2, M2 = (yh * p * dz).mean(1, keepdim=True), ((yh * p).abs() * Dz).mean(1, keepdim=True)
            out["dy"] = (rho * (p * dz - yh * m2), rho * (p.abs() * Dz + yh.abs() * M2))
        else:
            out["dy"] = (dz, Dz)
        return out


def assert_near(got, ref, mag, coeff, name, dtype=None):
    """|got - ref| <= coeff * U * mag + half a step of the output's type (relative to the value)."""
    got = d(got)
    dtype = dtype or torch.float32
    tol = 1.01 * (coeff * U * mag + half_step(dtype) * ref.abs()) + torch.finfo(dtype).tiny
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(((got - ref).abs() / tol).nan_to_num(float("inf")).reshape(-1).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values off, worst at {i}: "
                             f"{float(got.reshape(-1)[i])} against {float(ref.reshape(-1)[i])}, "
                             f"tolerance {float(tol.expand_as(ref).reshape(-1)[i])}")
