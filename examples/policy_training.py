"""Data-parallel training of a small policy over R rank windows of one GPU.

Every rank draws its own contexts, samples an action from the shared policy and is rewarded when it is
the teacher's.  One update:

    forward     sym_linear x 3 (gelu with its pre-activation kept, a residual block, the action head)
    loss        sym_policy_loss: clipped ratio and KL to a frozen reference, with its gradient in one pass
    backward    sym_linear_backward x 3, each dw and dbias written straight into the rank's send window
    reduction   sym_allreduce over the R windows (float32 sum)
    optimizer   sym_grad_norm and sym_adamw_step on the sum: float32 master weights, bfloat16 copies for
                the next forward pass, 8-bit or 32-bit states

    python examples/policy_training.py [--steps 120] [--ranks 4] [--states mx8|f32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import symmetric_memory_allreduce_gb300 as sm  # noqa: E402


class Policy:
    """logits = W3 h2 + b3, h2 = gelu(W2 h1 + b2) + h1, h1 = gelu(W1 x + b1); R ranks share the weights."""

    def __init__(self, inputs=48, hidden=256, actions=16, ranks=4, batch=512, states="mx8", seed=0):
        self.shapes = [(hidden, inputs), (hidden,), (hidden, hidden), (hidden,), (actions, hidden), (actions,)]
        sizes = [torch.Size(s).numel() for s in self.shapes]
        starts = [0]
        for n in sizes[:-1]:
            starts.append(starts[-1] + -(-n // 32) * 32)     # each tensor at a multiple of 32 elements
        self.total = starts[-1] + -(-sizes[-1] // 32) * 32
        self.spans, self.ranks, self.batch = list(zip(starts, sizes)), ranks, batch
        g = torch.Generator("cuda")
        g.manual_seed(seed)
        z = dict(device="cuda")
        self.master, self.weights = torch.zeros(self.total, **z), torch.zeros(self.total, dtype=torch.bfloat16, **z)
        for s, v in zip(self.shapes, self.views(self.master)):
            if len(s) == 2:
                v.copy_(torch.randn(s, generator=g, **z) * s[1] ** -0.5)
        self.weights.copy_(self.master)
        self.reference = self.weights.clone()
        self.send, self.recv = sm.Window(ranks, self.total * 4), sm.Window(ranks, self.total * 4)
        self.grads = self.send.tensor(torch.float32)[:, :self.total]
        self.grads.zero_()                                   # the gaps between tensors stay 0
        if states == "mx8":
            m, v = (torch.zeros(self.total, dtype=torch.uint8, **z) for _ in "mv")
            ms, vs = (torch.zeros(self.total // 32, dtype=torch.uint8, **z) for _ in "mv")
            scales = dict(m_scales=[ms[a // 32:a // 32 + -(-n // 32)] for a, n in self.spans],
                          v_scales=[vs[a // 32:a // 32 + -(-n // 32)] for a, n in self.spans])
        else:
            (m, v), scales = (torch.zeros(self.total, **z) for _ in "mv"), {}
        flat = lambda t: [t[a:a + n] for a, n in self.spans]  # noqa: E731
        self.adamw = sm.AdamW(flat(self.master), flat(self.recv.tensor(torch.float32)[0]), flat(m), flat(v),
                              copies=flat(self.weights), **scales)
        self.norm, self.step = torch.zeros(2, **z), 0
        half = lambda *s: torch.empty(*s, dtype=torch.bfloat16, **z)  # noqa: E731
        self.h1, self.z1, self.h2, self.z2 = (half(batch, hidden) for _ in range(4))
        self.dh1, self.dh2 = half(batch, hidden), half(batch, hidden)
        self.logits, self.dlogits = half(batch, actions), half(batch, actions)

    def views(self, flat):
        return [flat[a:a + n].view(s) for (a, n), s in zip(self.spans, self.shapes)]

    def forward(self, x, weights=None):
        w1, b1, w2, b2, w3, b3 = self.views(self.weights if weights is None else weights)
        sm.sym_linear(x, w1, self.h1, bias=b1, pre=self.z1, act="gelu")
        sm.sym_linear(self.h1, w2, self.h2, bias=b2, residual=self.h1, pre=self.z2, act="gelu")
        sm.sym_linear(self.h2, w3, self.logits, bias=b3)
        return self.logits

    def backward(self, x, rank):
        """From self.dlogits, into the rank's part of the send window."""
        _, _, w2, _, w3, _ = self.views(self.weights)
        d1, e1, d2, e2, d3, e3 = self.views(self.grads[rank])
        sm.sym_linear_backward(self.dlogits, self.h2, w3, dx=self.dh2, dw=d3, dbias=e3)
        sm.sym_linear_backward(self.dh2, self.h1, w2, pre=self.z2, dx=self.dh1, dw=d2, dbias=e2, act="gelu")
        self.dh1 += self.dh2                                 # the residual's gradient
        sm.sym_linear_backward(self.dh1, x, self.views(self.weights)[0], pre=self.z1, dw=d1, dbias=e1, act="gelu")

    def update(self, batches, lr):
        """One optimizer step from every rank's (x, actions, old_logp, ref_logp, advantages, weights)."""
        losses = torch.empty(self.ranks, 4, device="cuda")
        logp, lse = torch.empty(self.batch, device="cuda"), torch.empty(self.batch, device="cuda")
        for r, (x, actions, old, ref, adv, w) in enumerate(batches):
            sm.sym_policy_loss(self.forward(x), actions, old, adv, w, losses[r], logp, lse, ref_logp=ref,
                               dlogits=self.dlogits, kl_coef=0.01)
            self.backward(x, r)
        sm.sym_allreduce(self.send, self.recv, self.total)
        sm.sym_grad_norm(self.adamw, self.norm, max_norm=1.0)
        self.step += 1
        sm.sym_adamw_step(self.adamw, lr=lr, weight_decay=0.01, step=self.step, grad_scale=self.norm[1:], seed=self.step)
        return losses.sum(0)

    def free(self):
        self.adamw.free()
        self.send.free()
        self.recv.free()


def train(steps=120, ranks=4, states="mx8", seed=0, lr=2e-3, say=None):
    """Mean reward of every step."""
    p = Policy(ranks=ranks, states=states, seed=seed)
    g = torch.Generator("cuda")
    g.manual_seed(seed + 1)
    inputs, actions, n = p.shapes[0][1], p.shapes[4][0], p.batch
    teacher = torch.randn(actions, inputs, generator=g, device="cuda")
    stats, logp, ref, lse = (torch.empty(k, device="cuda") for k in (4, n, n, n))
    zero, ones = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    rewards = []
    try:
        for step in range(steps):
            batches, reward = [], 0.0
            for _ in range(ranks):
                x = torch.randn(n, inputs, generator=g, device="cuda").to(torch.bfloat16)
                logits = p.forward(x)
                a = torch.multinomial(logits.float().softmax(1), 1, generator=g)[:, 0]
                sm.sym_policy_loss(logits, a, zero, zero, ones, stats, logp, lse)            # the sampler's log-probabilities
                old = logp.clone()
                sm.sym_policy_loss(p.forward(x, p.reference), a, zero, zero, ones, stats, ref, lse)
                hit = (a == (x.float() @ teacher.t()).argmax(1)).float()
                reward += hit.mean()
                batches.append((x, a, old, ref.clone(), (hit - hit.mean()) / (hit.std() + 1e-3), ones / (n * ranks)))
            for _ in range(2):                               # the second one is off the sampling policy: ratios and clipping
                loss = p.update(batches, lr)
            rewards.append(float(reward / ranks))
            if say and step % 10 == 0:
                say(f"step {step:4d}  reward {rewards[-1]:.3f}  loss {loss[0]:+.4f}  kl {loss[2]:.4f}  "
                    f"clipped {loss[3]:.3f}  gradient norm {p.norm[0]:.3f}")
        status = sm.sym_stream_status()
        assert status == sm.SYM_OK, sm.sym_last_error()
        return rewards
    finally:
        p.free()


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=120)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--states", choices=("mx8", "f32"), default="mx8")
    o = ap.parse_args()
    train(o.steps, o.ranks, o.states, say=print)
