"""The operators on the rows' contents record no gradient: tensors that require one are refused, not
dropped from the graph. Refusals run without a GPU: they come before every other check."""

import pytest
import torch

from serving_pb_lru_amd import Engine, head_rows, latent_rows, pack_rows, rotate


def calls(device, grad):
    t = lambda *s: torch.zeros(s, device=device)
    with_grad = lambda *s: t(*s).requires_grad_(grad)
    pos = torch.zeros(1, dtype=torch.int32, device=device)
    keys = t(1, 1, 1, 1, 64)
    return {
        "latent channels": lambda: pack_rows(latent_rows(), with_grad(1, 1, 512), t(1, 1, 64)),
        "rotary channels": lambda: pack_rows(latent_rows(), t(1, 1, 512), with_grad(1, 1, 64)),
        "keys": lambda: pack_rows(head_rows(1, 64), with_grad(1, 1, 1, 1, 64), keys),
        "values": lambda: pack_rows(head_rows(1, 64), keys, with_grad(1, 1, 1, 1, 64)),
        "x": lambda: rotate(with_grad(1, 1, 64), pos),
        "out": lambda: rotate(t(1, 1, 64), pos, out=with_grad(1, 1, 64)),
        "in place": lambda: (lambda x: rotate(x, pos, out=x))(with_grad(1, 1, 64)),
    }


@pytest.mark.parametrize("what", list(calls("cpu", False)))
def test_refused(what):
    with pytest.raises(ValueError, match="gradient"):
        calls("cpu", True)[what]()
    with pytest.raises(ValueError, match="CUDA"):          # no gradient: the next check
        calls("cpu", False)[what]()
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        calls("cpu", True)[what]()


def test_attend_refuses():
    sel = torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="gradient"):
        Engine.attend(None, 0, 0, sel, torch.zeros((1, 1, 576)).requires_grad_(), latent_rows())
    for kw in (dict(out=torch.zeros((1, 1, 512)).requires_grad_()), dict(lse=torch.zeros((1, 1)).requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            Engine.attend(None, 0, 0, sel, torch.zeros((1, 1, 576)), latent_rows(), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("what", list(calls("cpu", False)))
def test_without_gradients_they_run(what):
    """Under no_grad, as a model's decode step runs, parameters and views of them may go in."""
    plain = calls("cuda", False)[what]()
    with torch.no_grad():
        got = calls("cuda", True)[what]()
    assert torch.equal(got, plain) and got.grad_fn is None
