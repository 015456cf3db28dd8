"""The training step's operators together (examples/policy_training.py): one update against a plain
torch one in 64 bits, and a short run that has to learn."""
import os
import sys

import pytest
import torch

from _training_util import F64, act64

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_reduced_gradient_against_autograd(symar):
    """The sum over ranks of every tensor's gradient against autograd in 64 bits on the same bfloat16
    weights.  The kernels round activations, logits and their gradients to bfloat16 (2^-8 each, six of
    them on the longest path): 6 x 2^-8 of the gradient's size, by 2-norm."""
    from policy_training import Policy

    p = Policy(ranks=3, batch=200, seed=3)
    try:
        g = torch.Generator("cuda")
        g.manual_seed(5)
        n = p.batch
        batches = []
        w = [v.to(F64).requires_grad_() for v in p.views(p.weights)]
        loss = 0.0
        for _ in range(p.ranks):
            x = torch.randn(n, p.shapes[0][1], generator=g, device="cuda").to(torch.bfloat16)
            a = torch.randint(0, p.shapes[4][0], (n,), generator=g, device="cuda")
            adv, weight = torch.randn(n, generator=g, device="cuda"), torch.full((n,), 1.0 / (n * p.ranks), device="cuda")
            h1 = act64(x.to(F64) @ w[0].t() + w[1], "gelu")
            h2 = act64(h1 @ w[2].t() + w[3], "gelu") + h1
            logp = (h2 @ w[4].t() + w[5]).log_softmax(1).gather(1, a[:, None])[:, 0]
            old = (logp.detach() + 0.05 * torch.randn(n, generator=g, device="cuda")).float()
            ref = (logp.detach() + 0.2 * torch.randn(n, generator=g, device="cuda")).float()
            ratio, k = (logp - old.to(F64)).exp(), ref.to(F64) - logp
            loss = loss + (weight.to(F64) * (-torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv) +
                                             0.01 * (k.exp() - k - 1))).sum()
            batches.append((x, a, old, ref, adv, weight))
        loss.backward()
        stats = p.update(batches, lr=0.0)
        assert symar.sym_stream_status() == symar.SYM_OK
        assert abs(stats[0] - loss.detach()) < 6 * 2.0 ** -8 * abs(adv).mean()
        norm = torch.sqrt(sum(v.grad.square().sum() for v in w))
        got = p.views(p.recv.tensor(torch.float32)[1])
        for a, b in zip(got, w):
            assert (a.to(F64) - b.grad).norm() <= 6 * 2.0 ** -8 * b.grad.norm() + 2.0 ** -8 * norm
        assert abs(p.norm[0] - norm) <= 6 * 2.0 ** -8 * norm
    finally:
        p.free()


@pytest.mark.parametrize("states", ["f32", "mx8"])
def test_short_run_learns(symar, states):
    from policy_training import train

    rewards = train(steps=60, ranks=4, states=states)
    assert sum(rewards[:5]) / 5 < 0.12 < 0.3 < sum(rewards[-5:]) / 5
