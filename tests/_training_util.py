"""Plain 64-bit forms of the training operators and the roundoffs that tolerances are derived from."""
import math

import torch

F64 = torch.float64
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}     # half a step at 1
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}  # smallest step
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: 0.5 * z * torch.erfc(-z / math.sqrt(2))}[act]()


def slope64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(F64)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def linear64(x, w, bias=None, residual=None, act="none"):
    """(y, z, sum of |terms|) of the linear layer in 64 bits."""
    z, size = x.to(F64) @ w.to(F64).t(), x.to(F64).abs() @ w.to(F64).abs().t()
    if bias is not None:
        z, size = z + bias.to(F64), size + bias.to(F64).abs()
    y = act64(z, act)
    return (y if residual is None else y + residual.to(F64)), z, size


def close(got, want, tol, what=""):
    """Every element within its own tolerance; NaN and infinities in the same places."""
    got = got.to(F64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: finite in other places"
    assert torch.equal(torch.isnan(want), torch.isnan(got)), f"{what}: NaN in other places"
    bad = ((got - want).abs() > tol) & fine
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: "
                             f"{got[tuple(i)].item()} for {want[tuple(i)].item()}")


def policy64(logits, targets, old, adv, weights, ref=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
             temperature=1.0, grad_out=1.0):
    """stats, logp, lse, dlogits in 64 bits, row by row from the definition."""
    T, V = logits.shape
    stats = torch.zeros(4, dtype=F64)
    logp, lse = torch.zeros(T, dtype=F64), torch.zeros(T, dtype=F64)
    grad = torch.zeros(T, V, dtype=F64)
    for t in range(T):
        w = 1.0 if weights is None else float(weights[t])
        y = int(targets[t])
        if w == 0 or not 0 <= y < V:
            continue
        z = logits[t].detach().cpu().to(F64) / temperature
        lse[t] = torch.logsumexp(z, 0)
        logp[t] = z[y] - lse[t]
        A, d = float(adv[t]), float(logp[t]) - float(old[t])
        rho = math.exp(min(max(d, -20.0), 20.0))
        cut = min(max(rho, 1 - clip_low), 1 + clip_high)
        clipped = cut * A < rho * A
        policy, slope = -min(rho * A, cut * A), 0.0 if clipped or abs(d) > 20 else -A * rho
        kl = 0.0
        if ref is not None:
            k = float(ref[t]) - float(logp[t])
            kr = math.exp(min(max(k, -20.0), 20.0))
            kl = kr - min(max(k, -20.0), 20.0) - 1
            slope += 0.0 if abs(k) > 20 else kl_coef * (1 - kr)
        stats += torch.tensor([w * (policy + kl_coef * kl), w * policy, w * kl, w * clipped], dtype=F64)
        p = torch.exp(z - lse[t])
        p[y] -= 1
        grad[t] = -grad_out * w * slope / temperature * p
    return stats, logp, lse, grad
