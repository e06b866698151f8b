"""examples/delta_block.py: layer norm, causal convolution, delta rule, layer norm
of each head and AdamW together.  It runs, its gradients are those of the same
model in float64, and answering token by token gives the logits of the
whole-sequence pass."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("delta_block", os.path.join(ROOT, "examples", "delta_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(model, ids, w):
    """The model's logits in the type of the weights w, by elementary torch operations, token by token."""
    f, H, D = torch.nn.functional, model.heads, model.dim
    lin = lambda x, p: x @ p.reshape(p.shape[0], -1).T
    x = f.one_hot(ids, model.symbols).to(w["w_in"].dtype)
    h = lin(x, w["w_in"])
    n = f.layer_norm(h, (model.width,), w["norm1"], w["shift1"])
    u = lin(n, w["w_qkv"])
    K = model.taps
    pad = torch.cat([torch.zeros_like(u[:, :K - 1]), u], 1)
    c = f.silu(sum(pad[:, j:j + u.shape[1]] * w["w_conv"][:, j] for j in range(K)) + w["bias"])
    q, k, v = (t.unflatten(-1, (H, D)) for t in c.split(model.width, -1))
    q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    a = lin(n, w["w_gates"])
    g, beta = -f.softplus(a[..., :H] - 2), torch.sigmoid(a[..., H:])
    S, out = torch.zeros(ids.shape[0], H, D, D, dtype=x.dtype, device=x.device), []
    for t in range(ids.shape[1]):
        S = S * g[:, t].exp()[..., None, None]
        e = v[:, t] - (S * k[:, t][..., None]).sum(2)
        S = S + k[:, t][..., None] * (beta[:, t][..., None] * e)[:, :, None]
        out.append(D ** -0.5 * (S * q[:, t][..., None]).sum(2))
    z = f.layer_norm(torch.stack(out, 1), (D,), w["norm2"], w["shift2"])
    return lin(h + lin(z.flatten(-2), w["w_o"]), w["w_out"])


def test_gradients_are_those_of_the_model_in_64_bits(example):
    """About ten roundings to bf16 lie on the way to a logit and as many on the way back, 2**-9 of a value each in the mean;
    independent, they make sqrt(20) 2**-9 = 0.9% of a gradient's norm.  Layer norms and unit lengths of short vectors amplify
    some; eight times that, 7%, is allowed."""
    model = example.DeltaBlock(seed=3)
    ids, targets, weight = example.batch(torch.Generator(device="cuda").manual_seed(4), 5, 70, model.symbols)
    logits, saved = model.forward(ids)
    loss, dlogits = model.loss(logits, targets, weight)
    grads = model.backward(dlogits, saved)
    w = {n: p.double().requires_grad_() for n, p in model.w.items()}
    ref = _plain(model, ids, w)
    assert float((logits - ref.detach()).norm()) <= 0.07 * float(ref.detach().norm())
    model.loss(ref, targets, weight)[0].backward()
    for n, p in w.items():
        assert float((grads[n].double() - p.grad).norm()) <= 0.07 * float(p.grad.norm()), n


def test_it_trains_and_runs(example):
    model, losses = example.train(steps=8)
    assert all(torch.isfinite(torch.tensor(losses)))
    assert all(bool(torch.isfinite(p).all()) for p in model.master.values())
    for n, c in model.copies.items():
        assert torch.equal(c, model.master[n].to(torch.bfloat16)), n


def test_token_by_token_equals_whole_sequence(example):
    """The two forms of the recurrence round differently, by less than 2**-16; each value then passes four roundings to bf16 that may
    fall to the other side, two of them behind layer norms of heads."""
    model, _ = example.train(steps=5)
    ids, _, _ = example.batch(torch.Generator(device="cuda").manual_seed(7), 3, 80, model.symbols)
    whole, _ = model.forward(ids)
    state = model.start(3)
    steps = torch.stack([model.answer(ids[:, t], state) for t in range(80)], 1)
    assert float((steps - whole).abs().amax()) <= 8 * 2.0 ** -8 * float(whole.abs().amax())
