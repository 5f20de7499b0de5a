"""The 64-bit forms that the GPU tests compare with: their gradients against differences of their own
outputs, and their outputs against formulations of another kind."""
import numpy as np
import pytest
import torch

from _terms import allowed, biased, bucket_of, differential

S, D, BLOCK = 70, 64, 32
RP, CI = np.array([0, 1, 2, 5], np.int32), np.array([0, 1, 0, 1, 2], np.int32)  # row 1 without block 0
STARTS = [0, 2, 2, 9, 40]


def _inputs(seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((1, 2, S, D), generator=g).half() for _ in range(4)]


def _difference(f, x, at, h):
    """Central difference of the scalar f(x) in direction `at`; x in 64 bits, beyond the 16-bit grid."""
    return (f(x + h * at) - f(x - h * at)) / (2 * h)


@pytest.mark.parametrize("which", ["Q", "K", "V", "bias"])
def test_biased_gradients_are_differences(which):
    q, k, v, do = _inputs()
    bias = torch.randn((2, len(STARTS)), generator=torch.Generator().manual_seed(1)).half()
    x = dict(Q=q, K=k, V=v, bias=bias)
    grads = biased(q, k, v, RP, CI, BLOCK, 0.125, bias, STARTS, do)

    def f(t):
        y = {n: t if n == which else u for n, u in x.items()}
        y["Q"] = _Half(y["Q"])
        O = biased(y["Q"], y["K"], y["V"], RP, CI, BLOCK, 0.125, y["bias"], STARTS)["O"][0]
        return float((O * do.double().reshape(O.shape)).sum())

    at = torch.randn(x[which].shape, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    want = float((grads["d" + which][0].reshape(at.shape) * at).sum())
    got = _difference(f, x[which].double(), at, 1e-4)
    assert abs(got - want) <= 1e-6 * (1 + abs(want))


class _Half(torch.Tensor):
    """A 64-bit tensor that says float16: the forms take the rounding unit of their bounds from it."""

    @staticmethod
    def __new__(cls, x):
        return torch.Tensor._make_subclass(cls, x)

    dtype = torch.float16

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        with torch._C.DisableTorchFunctionSubclass():
            return func(*[a.as_subclass(torch.Tensor) if isinstance(a, cls) else a for a in args], **(kwargs or {}))


@pytest.mark.parametrize("which", ["Q", "K", "V", "lq1", "lk1", "lq2", "lk2"])
def test_differential_gradients_are_differences(which):
    q, k, v, do = _inputs(3)
    g = torch.Generator().manual_seed(4)
    x = dict(Q=q, K=k, V=v, **{n: (0.3 * torch.randn((2, D // 2), generator=g)).half() for n in ("lq1", "lk1", "lq2", "lk2")})
    args = lambda y: (y["Q"], y["K"], y["V"], RP, CI, BLOCK, 0.2, [y[n] for n in ("lq1", "lk1", "lq2", "lk2")], 0.4)  # noqa: E731
    grads = differential(*args(x), do)

    def f(t):
        y = {n: t if n == which else u for n, u in x.items()}
        y["Q"] = _Half(y["Q"])
        O = differential(*args(y))["O"][0]
        return float((O * do.double().reshape(O.shape)).sum())

    at = torch.randn(x[which].shape, generator=torch.Generator().manual_seed(5), dtype=torch.float64)
    want = float((grads["d" + which][0].reshape(at.shape) * at).sum())
    got = _difference(f, x[which].double(), at, 1e-4)
    assert abs(got - want) <= 1e-6 * (1 + abs(want))


def test_outputs_by_another_formulation():
    """Row by row over explicit key lists, with scipy's softmax."""
    from scipy.special import softmax
    q, k, v, _ = _inputs(6)
    bias = torch.randn((2, len(STARTS)), generator=torch.Generator().manual_seed(7)).half()
    O = biased(q, k, v, RP, CI, BLOCK, 0.125, bias, STARTS)["O"][0].numpy()
    Q, K, V, b = (x.double().numpy() for x in (q[0], k[0], v[0], bias))
    for h in range(2):
        for t in (0, 33, 64, 69):
            keys = [j * BLOCK + c for j in CI[RP[t // BLOCK]:RP[t // BLOCK + 1]] for c in range(BLOCK) if j * BLOCK + c <= t]
            z = [0.125 * Q[h, t] @ K[h, x] + b[h, np.searchsorted(STARTS, t - x, side="right") - 1] for x in keys]
            assert np.allclose(O[h, t], softmax(z) @ V[h, keys], atol=1e-12)


def test_masks():
    M = allowed(RP, CI, S, BLOCK)
    assert M[0, 0] and not M[0, 1] and not M[40, 3] and M[40, 33] and M[69, 3] and M[69, 69]
    at = bucket_of(S, STARTS)
    assert at[5, 5] == 0 and at[5, 3] == 2 and at[5, 4] == 0 and at[60, 51] == 3 and at[60, 20] == 4
