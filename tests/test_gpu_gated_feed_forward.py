"""The operators together: gated feed-forward blocks whose matrices take orthogonalised updates, in one step with a plan of
the vectors.

A rank's gradients against float64 autograd of the same network on the same 16-bit parameters.  Activations and gradients
are rounded to bf16 (2^-8) at each of about twelve places on the way through a layer; the errors are independent, so that
their norm stays within 2^-8 sqrt(12 layers) of the gradient's, doubled for the roundings' spread: 0.04 at two layers.
"""
import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    Z.zero_operators_check()


def norm64(a, w, eps):
    return a / torch.sqrt((a * a).mean(1, keepdim=True) + eps) * w


@pytest.mark.parametrize("dim,inner,rows", [(128, 320, 96), (72, 136, 33), (50, 77, 20)])
def test_gradients(dim, inner, rows):
    from zero_sharded_mixed_03_gb300.feed_forward import GatedFeedForward
    model = GatedFeedForward(2, dim, inner, 3, rows, residual_scale=0.5, seed=3)
    try:
        gen = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randn(rows, dim, generator=gen, device="cuda").to(torch.bfloat16)
        dy = torch.randn(rows, dim, generator=gen, device="cuda").to(torch.bfloat16)
        got = model.forward(x)
        model.backward(1, dy)
        w = [p.double().requires_grad_(True) for p in model.params16]
        flat = model.group.full16.view(torch.bfloat16).double().requires_grad_(True)
        sizes = [dim, dim, dim, inner, inner, dim]
        y = x.double()
        for l in range(2):
            pre, post, gate, bg, bu, bd = (flat[a:a + n] for a, n in zip(model.at[6 * l:6 * l + 6], sizes))
            z = norm64(y, pre, model.eps)
            g = z @ w[3 * l] + bg
            h = (g * torch.sigmoid(g) * (z @ w[3 * l + 1] + bu)) @ w[3 * l + 2] + bd
            y = y + 0.5 * gate * norm64(h, post, model.eps)
        grads = torch.autograd.grad(y, w + [flat], dy.double())
        assert float((got.double() - y).norm() / y.norm()) < 0.04
        for have, want in zip(model.grads[1] + [model.contribs[1]], grads):
            off = float((have.double() - want).norm() / want.norm())
            assert off < 0.04, (tuple(want.shape), off)
        assert not any(bool(g.any()) for g in model.grads[0] + [model.contribs[0]]), "another rank's was written"
    finally:
        torch.cuda.synchronize()
        model.close()


def test_training_runs_and_a_bad_step_is_left_out():
    from zero_sharded_mixed_03_gb300.feed_forward import GatedFeedForward, train
    losses = train(steps=5, rows=64, gated=True)
    assert len(losses) == 5 and all(torch.isfinite(torch.tensor(losses)))
    model = GatedFeedForward(1, 64, 96, 2, 32)
    try:
        x = torch.ones(32, 64, dtype=torch.bfloat16, device="cuda")
        h, muon = Z.hyper(max_grad_norm=1.0), Z.muon_hyper()
        for k in range(3):
            for r in range(2):
                model.forward(x)
                model.backward(r, x)
            if k == 1:
                model.grads[1][2][5, 5] = float("nan")
            kept = [p.clone() for p in model.params] + [model.group.full16.clone()]
            model.step(h, muon)
            now = model.params + [model.group.full16]
            same = all(torch.equal(a, b) for a, b in zip(kept, now))
            assert same == (k == 1)
        assert model.group.t() == 2 and Z.zero_muon_read(model.muon, model._stream()).t == 2
    finally:
        torch.cuda.synchronize()
        model.close()
