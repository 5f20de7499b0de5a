"""The differential forward at D = 64 and more than 1024 tiles, on both sides of an average row of 16 blocks
(three thread blocks per SM for shorter rows, two for longer ones)."""
import numpy as np
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _terms import _close, differential
from test_gpu_biased import DEV, _dev

pytestmark = pytest.mark.gpu


def _csr(S, block, per):
    """Rows of the `per` blocks up to their own."""
    nb = -(-S // block)
    rows = [list(range(max(0, i + 1 - per), i + 1)) for i in range(nb)]
    return np.cumsum([0] + [len(r) for r in rows]).astype(np.int32), np.array([j for r in rows for j in r], np.int32)


@pytest.mark.parametrize("per", [15, 16, 17, 30])
@pytest.mark.parametrize("block,dtype", [(64, torch.float16), (128, torch.bfloat16), (32, torch.float16)])
def test_forward(per, block, dtype):
    per = per * 64 // block  # the same tokens a row
    S, D = 2630, 64
    H = 1024 // 42 + 1
    g = torch.Generator().manual_seed(per)
    q, k, v = (torch.randn((1, H, S, D), generator=g).to(dtype) for _ in range(3))
    lam = [(0.2 * torch.randn((H, D // 2), generator=g)).to(dtype) for _ in range(4)]
    rp, ci = _csr(S, block, per)
    out, out2, _ = tsa.tsa_differential_attention_fwd(*(x.to(DEV) for x in (q, k, v)), *_dev(rp, ci),
                                                      *(x.to(DEV) for x in lam), 0.5, block=block)
    assert tsa.tsa_last_device_status() == 0
    for h in (0, H - 1):
        ref = differential(q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], rp, ci, block, 32 ** -0.5, [x[h:h + 1] for x in lam], 0.5)
        _close(out[:, h], *ref["O"], f"O of head {h}")
        _close(out2[:, h], *ref["O2"], f"O2 of head {h}")
