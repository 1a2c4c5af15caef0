"""The operators together: a feed-forward network under emulated ZeRO-3.

A rank's gradients against float64 autograd of the same network on the same 16-bit parameters.
Activations and gradients are rounded to bf16 (2^-8) at each of about ten places on the way through
a layer; the errors are independent, so that their norm stays within 2^-8 sqrt(10 layers) of the
gradient's, doubled for the roundings' spread: 0.03 at two layers.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def norm64(a, w, eps):
    return a / torch.sqrt((a * a).mean(1, keepdim=True) + eps) * w


@pytest.mark.parametrize("dim,inner,rows", [(128, 320, 96), (72, 136, 33)])
def test_gradients(dim, inner, rows):
    from zero_sharded_mixed_03_gb300.feed_forward import ShardedFeedForward
    model = ShardedFeedForward(2, dim, inner, 3, rows, residual_scale=0.5, seed=3)
    try:
        gen = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randn(rows, dim, generator=gen, device="cuda").to(torch.bfloat16)
        dy = torch.randn(rows, dim, generator=gen, device="cuda").to(torch.bfloat16)
        got = model.forward(x)
        model.backward(1, dy)
        units = []
        for u in range(2):
            units.append(model.unit16(u).double().clone().requires_grad_(True))
            model.group.release(u)
        vectors = model.vectors16.double().requires_grad_(True)
        y = x.double()
        for l in range(2):
            w1, b1, w2, b2 = (units[l][a:b] for a, b in zip(model.at, model.at[1:] + [model.at[3] + dim]))
            z = norm64(y, vectors[l, 0], model.eps) @ w1.view(dim, inner) + b1
            h = z * 0.5 * torch.erfc(-z * 0.5 ** 0.5) @ w2.view(inner, dim) + b2
            y = y + 0.5 * vectors[l, 2] * norm64(h, vectors[l, 1], model.eps)
        grads = torch.autograd.grad(y, units + [vectors], dy.double())
        assert float((got.double() - y).norm() / y.norm()) < 0.03
        used = model.at[3] + dim
        for u in range(2):
            want = grads[u][:used]
            off = float((model.contribs[u][1][:used].double() - want).norm() / want.norm())
            assert off < 0.03, (u, off)
            assert not bool(model.contribs[u][0].any()), "another rank's contribution was written"
        off = float((model.rank_vector_grads[1].double() - grads[2]).norm() / grads[2].norm())
        assert off < 0.03, off
    finally:
        torch.cuda.synchronize()
        model.close()


def test_it_learns():
    from zero_sharded_mixed_03_gb300.feed_forward import train
    losses = train(steps=60)
    assert losses[-1] < 0.35 * losses[0], losses[::10]
