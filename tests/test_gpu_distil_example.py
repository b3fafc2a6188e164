"""The example of distilling and serving runs, and its gradient is the formula's (needs a GB300)."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from decode_step_token_gb300 import build
    build.build_library()
    spec = importlib.util.spec_from_file_location("distil_and_serve", os.path.join(ROOT, "examples", "distil_and_serve.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("rows,vocab,width,top,block", [(64, 4096, 256, 32, 16), (33, 5003, 100, 128, 32), (150, 777, 65, 5, 16)])
def test_runs(example, rows, vocab, width, top, block):
    got = example.run(rows=rows, vocab=vocab, width=width, top=top, rounds=2, tokens=5, block=block)
    assert len(got["divergence"]) == 2 and np.isfinite(got["divergence"]).all() and min(got["divergence"]) >= 0
    assert got["tokens"].shape == (5, rows) and ((got["tokens"] >= 0) & (got["tokens"] < vocab)).all()
    assert np.isfinite(got["logprob"].numpy()).all() and (got["logprob"] <= 0).all()


@pytest.mark.parametrize("rows,vocab,width,top", [(24, 1000, 64, 20), (7, 9001, 33, 128)])
def test_gradient(example, rows, vocab, width, top):
    """The weight's gradient against 64-bit automatic differentiation of the loss on the same lists.

    A logit is a sum of `width` products in fp32 and so is off by e = width 2^-24 sum |h w| at most, a probability
    by 2 e of itself; the kernel's own error is 16 roundings of p + q (the exponential's 2^-22 among them); the
    weight's gradient is a sum of `rows` products in fp32.
    """
    import torch

    import decode_step_token_gb300 as d

    gen = torch.Generator(device="cuda:0").manual_seed(vocab)
    hidden = torch.randn((rows, width), generator=gen, device="cuda:0")
    teacher = 2.0 * torch.randn((vocab, width), generator=gen, device="cuda:0") / width ** 0.5
    student = torch.randn((vocab, width), generator=gen, device="cuda:0") / width ** 0.5
    with d.Sampler(max_rows=rows, max_vocab=vocab) as sampler:
        lesson = example.Lesson(sampler, rows, vocab, top, torch.device("cuda:0"))
        lesson.hear(hidden @ teacher.t())
        got = lesson.step(hidden, student, token_coef=0.25).double()
    w = student.double().requires_grad_(True)
    logp = torch.log_softmax(hidden.double() @ w.t(), 1)
    ids, lq = lesson.ids.long(), lesson.logprobs.double()
    inside = torch.zeros_like(logp, dtype=torch.bool).scatter_(1, ids, True)
    rest = torch.logsumexp(logp.masked_fill(inside, -float("inf")), 1)
    lr = lesson.rest.double()
    kl = (lq.exp() * (lq - logp.gather(1, ids))).sum(1) + lr.exp() * (lr - rest)
    loss = (kl - 0.25 * logp.gather(1, ids[:, :1])[:, 0]).mean()
    loss.backward()
    p = logp.detach().exp()
    q = p.clone().scatter_(1, ids, lq.exp())
    e = width * 2.0 ** -24 * (hidden.double().abs() @ student.double().abs().t()).amax()
    off = (2 * e + 16 * 2.0 ** -24) * (p + q) * 1.25 / rows
    off.scatter_add_(1, ids[:, :1], torch.full((rows, 1), 0.25 * 2.0 ** -23 / rows, dtype=torch.float64, device="cuda:0"))
    g = (1.25 * p + q) / rows
    bound = (off + rows * 2.0 ** -24 * g).t() @ hidden.double().abs()
    bad = (got - w.grad).abs() > bound + 1e-12
    assert not bad.any(), ((got - w.grad).abs() / bound).max().item()
    assert abs(lesson.loss.item() - loss.item()) <= 4 * e.item() * (1 + 0.25) + 1e-6 * abs(loss.item())
