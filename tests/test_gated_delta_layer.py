"""The example that runs the operators together, as its users would run it."""
import importlib.util
import os

import pytest

from conftest import ROOT


def example():
    path = os.path.join(ROOT, "examples", "gated_delta_layer.py")
    spec = importlib.util.spec_from_file_location("gated_delta_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_example_loads_without_a_gpu():
    pytest.importorskip("torch")
    model = example().Model()
    assert model.qkv.out_features == (2 * model.Hk + model.Hv) * 128


@pytest.mark.gpu
def test_training_lowers_the_loss_and_matches_plain_gradients():
    torch = pytest.importorskip("torch")
    ex = example()
    torch.manual_seed(0)
    model = ex.Model().cuda()
    tokens = torch.randint(0, 384, (2, 71), device="cuda")
    model.loss(tokens).backward()
    got = {n: p.grad.double() for n, p in model.named_parameters()}
    # the same loss with the mixing written out, in 64 bits from the same (bf16) heads
    for p in model.parameters():
        p.grad = None
    x = model.embed[tokens[:, :-1]]
    q, k, v, g, beta = (t.double() for t in model.heads(x))
    q, k = (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    q, k = (t.repeat_interleave(model.Hv // model.Hk, 2) for t in (q, k))
    S, outs = 0.0, []
    for i in range(q.shape[1]):
        S = S * g[:, i, :, None, None].exp() if i else torch.zeros(2, model.Hv, 128, 128, device="cuda", dtype=torch.double)
        d = beta[:, i, :, None] * (v[:, i] - (S * k[:, i, :, :, None]).sum(-2))
        S = S + k[:, i, :, :, None] * d[:, :, None]
        outs.append(model.scale * (S * q[:, i, :, :, None]).sum(-2))
    logits = model.logits(x, torch.stack(outs, 1))
    torch.nn.functional.cross_entropy(logits.flatten(0, 1), tokens[:, 1:].flatten()).backward()
    for n, p in model.named_parameters():
        want = p.grad.double()
        # bf16 results at each of the few operators in a row: a few times 2^-8 of the gradient
        assert (got[n] - want).norm() <= 0.03 * want.norm(), n
    losses = ex.train(model)
    assert losses[-1] < 0.9 * losses[0]


@pytest.mark.gpu
def test_decoding_keeps_the_states_of_the_kept_tokens():
    torch = pytest.importorskip("torch")
    import gated_delta_rule_39_gb300 as kda
    ex = example()
    torch.manual_seed(0)
    model = ex.Model().cuda()
    ex.train(model, steps=5)
    seen, last, states, kept = ex.serve(model)
    assert kda.kda_fwd_get_error() == 0
    assert 0 < kept <= 4
    assert ((0 <= last) & (last < 384)).all()
    for n, s in enumerate(seen):
        t = torch.tensor(s, dtype=torch.int32, device="cuda")
        want = model.prompt(t[None], torch.tensor([0, len(s)], dtype=torch.int32, device="cuda"))[1][0]
        # fp32 steps after an fp16-operand prompt against one of the whole: 2^-11 per operand,
        # and bf16 projections whose sums depend on the batch's shape
        assert (states[n] - want).norm() <= 0.02 * want.norm()
