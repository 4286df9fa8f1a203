"""CPU tests of the float64 references that the GPU tests of include/cbk_nn.h compare with: their
gradients against central differences and autograd."""
import pytest

import nn_reference as ref

torch = pytest.importorskip("torch")


def _tensors(T, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: (torch.randn(*s, generator=g, dtype=torch.float64) * 0.5)  # noqa: E731
    return mk(T, K), mk(N, K), mk(N, K), mk(T, N)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_ffn_gradient_against_differences(act):
    x, wg, wu, dh = _tensors(3, 7, 5, 1)
    (dx, _), (dg, _), (du, _) = ref.ffn_bwd(act, x, wg, wu, dh)
    f = lambda x: (ref.ffn(act, x, wg, wu)[0] * dh).sum()  # noqa: E731
    e = 1e-5
    for i in range(3):
        for k in range(5):
            p, m = x.clone(), x.clone()
            p[i, k] += e
            m[i, k] -= e
            assert abs((f(p) - f(m)) / (2 * e) - dx[i, k]) < 1e-8
    named = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
             "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[act]
    g, u = (x @ wg.T).requires_grad_(), (x @ wu.T).requires_grad_()
    (named(g) * u * dh).sum().backward()
    assert torch.allclose(g.grad, dg, atol=1e-12) and torch.allclose(u.grad, du, atol=1e-12)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_slopes_stay_within_the_bounds_used(act):
    z = torch.linspace(-30, 30, 60001, dtype=torch.float64)
    _, d, b1, b2 = ref.act(act, z)
    assert float(d.abs().max()) <= b1
    assert float(((d[1:] - d[:-1]) / (z[1:] - z[:-1])).abs().max()) <= b2


def test_xent_gradient_against_differences():
    x, w, _, _ = _tensors(4, 9, 5, 2)
    labels = torch.tensor([3, -100, 0, 8])
    dloss = torch.tensor([0.5, 2.0, 1.5, -1.0], dtype=torch.float64)
    dx, _ = ref.xent_bwd(x, w, labels, dloss, -100)
    f = lambda x: (ref.xent(x, w, labels, -100)[0][0] * dloss).sum()  # noqa: E731
    e = 1e-5
    for i in range(4):
        for k in range(5):
            p, m = x.clone(), x.clone()
            p[i, k] += e
            m[i, k] -= e
            assert abs((f(p) - f(m)) / (2 * e) - dx[i, k]) < 1e-8
    assert bool((dx[1] == 0).all())
    loss = ref.xent(x, w, labels, -100)[0][0]
    assert torch.allclose(loss, torch.nn.functional.cross_entropy(x @ w.T, labels, reduction="none", ignore_index=-100))
