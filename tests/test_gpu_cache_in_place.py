"""What the rotary and paged cache calls write in place is a new version to autograd, and has no gradient."""
import pytest
import torch

import topology_scheduled_gb300 as tsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _new(*shape):
    return torch.randn(shape, device=DEV, dtype=torch.float16)


def _calls(x, y):
    """Calls that write to x, and (the second output) to y, each [2, 1, 16, 64]."""
    f = tsa.rotary_frequencies(64)
    table, lens, t = _ints([[0], [1]]), _ints([16, 3]), _new(2, 1, 16, 64)
    q = _new(2, 1024, 64)
    return {"rotary": lambda: tsa.tsa_rotary(_new(2, 1, 16, 64), _new(2, 1, 16, 64), f, out=x, out_k=y),
            "in place": lambda: tsa.tsa_rotary(x, y, f, out=x, out_k=y),
            "append": lambda: tsa.tsa_paged_append(None, t, t, x, y, table, lens),
            "query": lambda: tsa.tsa_paged_append(x, t, t, y, _new(2, 1, 16, 64), table, lens, None, f, out=x),
            "decode": lambda: tsa.tsa_paged_attention_decode(q[:, :16].contiguous(), t, t, table, lens, out=x.view(2, 16, 64))}


WAYS = ["rotary", "in place", "append", "query", "decode"]


@pytest.mark.parametrize("way", WAYS)
def test_a_saved_tensor_that_is_written_is_noticed(way):
    x, y = _new(2, 1, 16, 64), _new(2, 1, 16, 64)
    w = _new(2, 1, 16, 64).requires_grad_()
    for written in (x,) if way == "decode" else (x, y):
        loss = (w * written).sum()
        _calls(x, y)[way]()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    # a tensor that is only read is not
    q = _new(2, 1, 16, 64)
    loss = (w * q).sum()
    tsa.tsa_rotary(q, None, tsa.rotary_frequencies(64))
    loss.backward()


@pytest.mark.parametrize("way", WAYS)
def test_an_output_that_requires_a_gradient_is_refused(way):
    for which in (0,) if way == "decode" else (0, 1):
        xy = [_new(2, 1, 16, 64), _new(2, 1, 16, 64)]
        xy[which].requires_grad_()
        before = [t.detach().clone() for t in xy]
        with pytest.raises(ValueError, match="gradient"):
            _calls(*xy)[way]()
        assert all(torch.equal(a.detach(), b) for a, b in zip(xy, before))
        with torch.no_grad():
            _calls(*xy)[way]()


def test_inference_tensors():
    with torch.inference_mode():
        x, y = _new(2, 1, 16, 64), _new(2, 1, 16, 64)
        for way in WAYS:
            _calls(x, y)[way]()
    for way in WAYS:  # written outside too, as caches made in that mode are
        with torch.no_grad():
            if way != "decode":
                _calls(x, y)[way]()
    assert tsa.tsa_last_device_status() == 0
