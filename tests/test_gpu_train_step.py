"""The operators together, as a training step uses them (examples/train_step.py): the
gradients of the first step against automatic differentiation of the same model in
32 bits, and a short run that has to learn."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _gpu(require_gpu):
    yield


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_first_step_gradients(example):
    """bfloat16 logits and logit gradients are the only roundings between the two: 2^-9
    each of what flows through them, and the logits' (up to ~5 here, so 2^-7 absolute)
    again in the probabilities; 3 % of each gradient's norm covers their sum."""
    model = example.Model(vocab=512, hidden=128)
    ids, following = example.batch(4096, 512, 0)
    loss, _ = example.loss_and_gradient(model, ids, following)
    w = {n: getattr(model, n).float().requires_grad_() for n in ("table", "mats", "out")}
    h = torch.nn.functional.embedding(ids, w["table"])
    for b in range(0, len(w["mats"]), 2):
        h = h + torch.relu(h @ w["mats"][b].t()) @ w["mats"][b + 1].t()
    logp = torch.log_softmax(h @ w["out"].t(), 1)
    asked = following >= 0
    entropy = -(logp.exp() * logp).sum(1)
    lp = logp.gather(1, following.clamp(min=0)[:, None])[:, 0]
    want = -((lp + 0.01 * entropy) * asked).sum() / asked.sum()
    want.backward()
    assert abs(float(loss) - float(want.detach())) < 0.01 * abs(float(want.detach()))
    for n, t in w.items():
        off = float((model.grads[n] - t.grad).norm() / t.grad.norm())
        assert off < 0.03, (n, off)


def test_it_learns(example):
    history = example.train(steps=60)
    assert history[-1][0] < 0.5 * history[0][0] and history[-1][1] > 0.8, (history[0], history[-1])
