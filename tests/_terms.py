"""Plain 64-bit forms of the attentions with learned score terms, and element-wise error bounds.

The forms follow the definitions over a dense [S, S] mask of allowed keys, one lane at a time, with
gradients by the chain rule.  The bounds add up what the kernels' arithmetic can lose, r being the
unit roundoff of the inputs' type (2^-8 bf16, 2^-11 f16) and eta half its subnormal spacing:

* a score is a binary32 sum of exact products: D 2^-24 scale |q|.|k|, the terms added to it and its
  scaling lose 4 2^-24 of the magnitudes, and exp2 (2 ulp) 2^-22: together the relative error `es` of
  an unnormalised weight (doubled for the weight itself, whose denominator has it too);
* the forward rounds each weight to the inputs' type (r, and eta of the row's largest) before the
  product with V; its denominator adds the rounded weights (r at most) or the exact ones; the
  result is rounded once more;
* the backward's weights come from the log-sum-exp (r at most off when the denominator added
  rounded weights, checked by the tests), Delta from the stored, rounded outputs; P and dS are
  rounded before their products; binary32 sums of n terms lose n 2^-24 of the magnitudes.
"""
import numpy as np
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
ETA = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
ACC = 2.0 ** -24


def allowed(rp, ci, S, block):
    """[S, S]: the keys each query may see (its CSR row's blocks, keys up to the query)."""
    M = torch.zeros((S, S), dtype=torch.bool)
    rp, ci = np.asarray(rp), np.asarray(ci)
    for i in range(len(rp) - 1):
        for j in ci[rp[i]:rp[i + 1]]:
            M[i * block:(i + 1) * block, j * block:(j + 1) * block] = True
    return M & torch.ones((S, S), dtype=torch.bool).tril()


def bucket_of(S, starts):
    """[S, S]: the bucket of q - k (0 where it is negative)."""
    d = (torch.arange(S)[:, None] - torch.arange(S)[None]).clamp(min=0)
    b = torch.zeros_like(d)
    for i, s in enumerate(starts):
        b = torch.where(d >= s, i, b)
    return b


def softmax(z, M):
    """Weights and log-sum-exp over M; rows without keys have no weight and -inf."""
    z = z.masked_fill(~M, -np.inf)
    m = z.max(-1, keepdim=True).values
    m = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(z - m)
    t = e.sum(-1, keepdim=True)
    return e / torch.where(t > 0, t, 1.0), (m + torch.log(t)).squeeze(-1)


def lanes(x):
    return x.detach().cpu().double().reshape((-1,) + tuple(x.shape[-2:]))


def _weights(q, k, M, scale, z_extra, D):
    z = scale * (q @ k.T)
    mag = scale * (q.abs() @ k.abs().T) * D
    if z_extra is not None:
        z = z + z_extra
        mag = mag + 4 * z_extra.abs().nan_to_num(0.0, 0.0, 0.0)
    P, lse = softmax(z, M)
    es = (mag + 4 * z.abs().nan_to_num(0.0, 0.0, 0.0).masked_fill(~M, 0)) * ACC
    # the row's log-sum-exp carries the same kind of error, relative to its own weights
    es = es + (P * es).sum(-1, keepdim=True) + 4 * ACC * lse.abs().nan_to_num(0.0, 0.0, 0.0)[:, None] + 2.0 ** -21
    return P, lse, es


class Grads:
    """The softmax gradient of one map of one lane, with its bound: dS and its error."""

    def __init__(self, P, es, dP, edP, delta_err, r, eta, lse_err, M):
        delta = (P * dP).sum(-1, keepdim=True)
        self.P, self.eP = P, P * (es + lse_err)
        self.dS = P * (dP - delta)
        self.exact_err = self.eP * (dP - delta).abs() + P * (delta_err[:, None] + edP)  # before its rounding
        self.eS = self.exact_err + r * self.dS.abs() + eta * M
        self.ePr = self.eP + r * P + eta * M  # P rounded before its product


def _close(got, ref, err, what):
    got = got.detach().cpu().double().reshape(ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - err
    worst = over.argmax()
    assert (over <= 0).all(), (f"{what}: {int((over > 0).sum())} of {over.numel()} elements over the bound; worst "
                               f"{got.reshape(-1)[worst]:.6g} for {ref.reshape(-1)[worst]:.6g}, allowed "
                               f"{err.reshape(-1)[worst]:.3g}")


def biased(Q, K, V, rp, ci, block, scale, bias, starts, dO=None):
    """{name: (value, bound)} of O and, with dO, dQ, dK, dV, dbias; "lse" with its value only."""
    dt = Q.dtype
    r, eta = U[dt], ETA[dt]
    q, k, v = lanes(Q), lanes(K), lanes(V)
    L, S, D = q.shape
    H = bias.shape[0]
    b = bias.detach().cpu().double()
    b = torch.where(b <= -1e30, -np.inf, b)
    M, at = allowed(rp, ci, S, block), bucket_of(S, starts)
    out = {"O": (torch.zeros_like(q), torch.zeros_like(q)), "lse": torch.zeros(L, S, dtype=torch.float64)}
    if dO is not None:
        g = lanes(dO)
        for n in ("dQ", "dK", "dV"):
            out[n] = (torch.zeros_like(q), torch.zeros_like(q))
        out["dbias"] = (torch.zeros_like(b), torch.zeros_like(b))
    n = S * ACC
    for l in range(L):
        P, lse, es = _weights(q[l], k[l], M, scale, b[l % H][at], D)
        O = P @ v[l]
        raw = (P * (2 * r + 2 * es + n) + eta * M) @ v[l].abs()
        out["O"][0][l], out["O"][1][l] = O, raw + r * O.abs() + eta
        out["lse"][l] = lse
        if dO is None:
            continue
        dP = g[l] @ v[l].T
        edP = D * ACC * (g[l].abs() @ v[l].abs().T)
        delta_err = (g[l].abs() * (out["O"][1][l] + D * ACC * O.abs())).sum(-1)
        m = Grads(P, es, dP, edP, delta_err, r, eta, r, M)
        for name, val, err in (("dQ", scale * (m.dS @ k[l]), scale * ((m.eS + n * m.dS.abs()) @ k[l].abs())),
                               ("dK", scale * (m.dS.T @ q[l]), scale * ((m.eS + n * m.dS.abs()).T @ q[l].abs())),
                               ("dV", m.P.T @ g[l], (m.ePr + n * m.P).T @ g[l].abs())):
            out[name][0][l], out[name][1][l] = val, err + r * val.abs() + eta
        # the bucket sums: dS as it is before its rounding.  The open last bucket's row sums are minus
        # the sum of the row's others, so they carry the others' errors and not their own
        last = at == len(starts) - 1
        for bucket in range(len(starts) - 1):
            here = at == bucket
            out["dbias"][0][l % H, bucket] += m.dS[here].sum()
            out["dbias"][1][l % H, bucket] += (m.exact_err + 8 * n * m.dS.abs())[here].sum()
        rows = (last & M).any(-1)
        out["dbias"][0][l % H, -1] += m.dS[last].sum()
        out["dbias"][1][l % H, -1] += (m.exact_err + 8 * n * m.dS.abs()).masked_fill(last, 0)[rows].sum()
    if dO is not None:
        out["dbias"] = (out["dbias"][0], out["dbias"][1] + r * out["dbias"][0].abs() + eta)
    return out


def differential(Q, K, V, rp, ci, block, scale, lambdas, init, dO=None):
    """{name: (value, bound)} of O, O2 and, with dO, dQ, dK, dV, dlq1, dlk1, dlq2, dlk2; "lse" [2, L, S]."""
    dt = Q.dtype
    r, eta = U[dt], ETA[dt]
    q, k, v = lanes(Q), lanes(K), lanes(V)
    L, S, D = q.shape
    w = D // 2
    lam4 = [x.detach().cpu().double().reshape(-1, w) for x in lambdas]
    heads = lam4[0].shape[0]
    H = Q.shape[1] if Q.dim() == 4 else L
    e1, e2 = torch.exp((lam4[0] * lam4[1]).sum(-1)), torch.exp((lam4[2] * lam4[3]).sum(-1))
    # its two products are binary32 sums of w terms; exp is 2 ulp off at most
    e_lam = sum(e * ((a.abs() * b.abs()).sum(-1) * w * ACC + 2.0 ** -22)
                for e, a, b in ((e1, *lam4[:2]), (e2, *lam4[2:]))) + 4 * ACC * (e1 + e2 + abs(init))
    M = allowed(rp, ci, S, block)
    new = lambda: (torch.zeros_like(q), torch.zeros_like(q))  # noqa: E731
    out = {"O": new(), "O2": new(), "lse": torch.zeros(2, L, S, dtype=torch.float64)}
    if dO is not None:
        g = lanes(dO)
        out.update(dQ=new(), dK=new(), dV=new())
        dlam, edlam = torch.zeros(heads, dtype=torch.float64), torch.zeros(heads, dtype=torch.float64)
    n = S * ACC
    for l in range(L):
        h = (l % H) if heads > 1 else 0
        lam, el = (e1 - e2 + init)[h].item(), e_lam[h].item()
        maps, O, raw = [], [], []
        for m in range(2):
            P, lse, es = _weights(q[l][:, m * w:m * w + w], k[l][:, m * w:m * w + w], M, scale, None, D)
            out["lse"][m, l] = lse
            maps.append((P, es))
            O.append(P @ v[l])
            raw.append((P * (2 * r + 2 * es + n) + eta * M) @ v[l].abs())
        val = O[0] - lam * O[1]
        out["O"][0][l] = val
        out["O"][1][l] = raw[0] + abs(lam) * raw[1] + el * O[1].abs() + r * val.abs() + eta + \
            4 * ACC * (O[0].abs() + abs(lam) * O[1].abs())
        out["O2"][0][l], out["O2"][1][l] = O[1], raw[1] + r * O[1].abs() + eta
        if dO is None:
            continue
        dP = g[l] @ v[l].T
        edP = D * ACC * (g[l].abs() @ v[l].abs().T)
        d2 = (g[l].abs() * (out["O2"][1][l] + D * ACC * O[1].abs())).sum(-1)
        d1 = (g[l].abs() * (out["O"][1][l] + D * ACC * val.abs())).sum(-1) + abs(lam) * d2 + el * (g[l] * O[1]).sum(-1).abs()
        m1 = Grads(maps[0][0], maps[0][1], dP, edP, d1, r, eta, 0.0, M)
        m2 = Grads(maps[1][0], maps[1][1], dP, edP, d2, r, eta, 0.0, M)  # -lambda is applied below
        dQ, eQ = [], []
        dK, eK = [], []
        for m, f, ef, part in ((m1, 1.0, 0.0, slice(0, w)), (m2, -lam, el, slice(w, D))):
            dS, eS = f * m.dS, abs(f) * (m.exact_err + r * m.dS.abs()) + ef * m.dS.abs() + eta * M + n * abs(f) * m.dS.abs()
            dQ.append(scale * (dS @ k[l][:, part])), eQ.append(scale * (eS @ k[l][:, part].abs()))
            dK.append(scale * (dS.T @ q[l][:, part])), eK.append(scale * (eS.T @ q[l][:, part].abs()))
        for name, val, err in (("dQ", torch.cat(dQ, 1), torch.cat(eQ, 1)), ("dK", torch.cat(dK, 1), torch.cat(eK, 1))):
            out[name][0][l], out[name][1][l] = val, err + r * val.abs() + eta
        val = (m1.P - lam * m2.P).T @ g[l]
        err = (m1.ePr + abs(lam) * m2.ePr + el * m2.P + n * (m1.P + abs(lam) * m2.P)).T @ g[l].abs()
        out["dV"][0][l], out["dV"][1][l] = val, err + r * val.abs() + eta
        dlam[h] -= (m2.P * dP).sum()
        edlam[h] += (m2.eP * dP.abs() + m2.P * edP + 8 * n * m2.P * dP.abs()).sum()
    if dO is not None:
        for i, (name, e, f) in enumerate((("dlq1", e1, 1), ("dlk1", e1, 1), ("dlq2", e2, -1), ("dlk2", e2, -1))):
            other = lam4[i ^ 1]
            val = (f * dlam * e)[:, None] * other
            rel = (lam4[i].abs() * other.abs()).sum(-1) * w * ACC + 2.0 ** -20
            err = ((edlam + dlam.abs() * rel) * e)[:, None] * other.abs()
            out[name] = (val, err + r * val.abs() + eta)
    return out
