"""clip_grad_norm's lists read by the C reader, and by attributes where it does not serve: the same results."""
import pytest
import torch

pytestmark = pytest.mark.gpu


class Other(torch.Tensor):
    pass


def lists(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    grads = [torch.randn(1 + 37 * k % 1000, generator=g, device="cuda").to(torch.bfloat16 if k % 3 else torch.float32)
             for k in range(200)] + [torch.zeros((0, 3), device="cuda")]
    return grads, [torch.full_like(t, 7.0) for t in grads]


@pytest.mark.parametrize("how", ["no interface", "a class of its own", "tuples", "parameters"])
@pytest.mark.parametrize("place", ["in place", "out"])
def test_same_results(cuda_lib, how, place, monkeypatch):
    fq = cuda_lib
    grads, outs = lists(1)
    g2, o2 = lists(1)
    norm = fq.clip_grad_norm(grads, 0.5, out=None if place == "in place" else outs)
    if how == "no interface":
        monkeypatch.setattr(fq, "_LISTS", (None,))
    elif how == "a class of its own":
        g2, o2 = [t.as_subclass(Other) for t in g2], [t.as_subclass(Other) for t in o2]
    elif how == "tuples":
        g2, o2 = tuple(g2), tuple(o2)
    else:
        g2 = [torch.nn.Parameter(t) for t in g2]
    norm2 = fq.clip_grad_norm(g2, 0.5, out=None if place == "in place" else o2)
    assert torch.equal(norm, norm2)
    for a, b, c, d in zip(grads, g2, outs, o2):
        assert torch.equal(a, b.detach().as_subclass(torch.Tensor)) and torch.equal(c, d.as_subclass(torch.Tensor))


def test_refusals(cuda_lib):
    fq = cuda_lib
    a = torch.ones(8, device="cuda")
    for bad in (a.half(), a.double(), a[::2], torch.ones(8)):
        with pytest.raises(ValueError, match="gradients"):
            fq.clip_grad_norm([a, bad], 1.0)
    for bad in ([a.bfloat16()], [a[:4]], [torch.ones(16, device="cuda")[::2]], [torch.ones(8)]):
        with pytest.raises(ValueError, match="out tensors"):
            fq.clip_grad_norm([a], 1.0, out=bad)
    with pytest.raises(ValueError, match="one tensor per gradient"):
        fq.clip_grad_norm([a], 1.0, out=[])
    assert bool((a == 1).all())
