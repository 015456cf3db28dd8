"""Training-step operators around the AllReduce, as cases to be measured.

Three operators: the linear layer (forward and backward), the clipped policy
loss with its KL term (loss, loss with gradient in one call, or forward and
backward apart), and the AdamW step over many tensors.  ``own`` chooses the
side: False computes the plain form in elementary 32-bit torch operations,
True calls this package's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 32                    # elements per scale of an 8-bit state
CLIP = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.05, temperature=0.9)
ADAM = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
STEP, SEED, MAX_NORM = 1000, 77, 1.0


# ------------------------------------------------------------------ the cases

def _linear(name, rows, inp, out, dtype, act, bias=True, residual=False, pre=False):
    return dict(name=name, op="linear", rows=rows, inp=inp, out=out, dtype=dtype, act=act, bias=bias,
                residual=residual, pre=pre)


def _linear_grad(name, rows, inp, out, dtype, act, grads):
    return dict(name=name, op="linear_grad", rows=rows, inp=inp, out=out, dtype=dtype, act=act, grads=grads)


def _loss(name, rows, vocab, dtype, mode):
    return dict(name=name, op="loss", rows=rows, vocab=vocab, dtype=dtype, mode=mode)


def _adamw(name, tensors, width, params, grads, states, copy=False, clip=False, packed=False):
    return dict(name=name, op="adamw", tensors=tensors, width=width, params=params, grads=grads, states=states,
                copy=copy, clip=clip, packed=packed)


def listed():
    return [
        # one token being generated: the weights are read once, latency counts
        _linear("linear one token", 1, 4096, 16384, "bf16", "gelu"),
        # a ragged batch through an odd-sized projection back into the residual stream
        _linear("linear odd", 333, 1001, 777, "f16", "silu", residual=True),
        # a value head or a probe kept in 32 bits
        _linear("linear f32", 512, 2048, 2048, "f32", "relu", residual=True),
        # the widening layer of a training batch, its pre-activation kept for the backward pass
        _linear("linear large", 8192, 4096, 16384, "bf16", "gelu", pre=True),
        # backward of a layer in the middle of a network
        _linear_grad("linear grad", 4096, 4096, 4096, "bf16", "gelu", "same"),
        # gradients in 32 bits for the AllReduce, from a batch of ragged length
        _linear_grad("linear grad f32 sums", 1000, 2048, 1544, "f16", "none", "f32"),
        # a micro-batch's last few answer tokens: few rows, a wide vocabulary
        _loss("loss few tokens", 8, 131072, "bf16", "grad"),
        # an odd vocabulary in 32 bits, forward and backward apart (as an autograd engine calls them)
        _loss("loss odd", 509, 50003, "f32", "split"),
        # a training batch's answers, loss and gradient in one call
        _loss("loss large", 8192, 131072, "bf16", "grad"),
        # a small network's step: latency counts
        _adamw("adamw small", 12, 96, "f32", "f32", "f32", packed=True),
        # a network trained in 16 bits with its states in 8
        _adamw("adamw 8 bit", 30, 2048, "bf16", "bf16", "mx8"),
        # 32-bit master weights with a 16-bit copy for the next forward pass, gradients clipped by their norm
        _adamw("adamw large", 24, 4096, "f32", "f32", "f32", copy=True, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear_grad", "loss", "loss", "adamw", "adamw"])
    half = rng.choice(["bf16", "f16"])
    act = rng.choice(["none", "relu", "gelu", "silu"])
    if kind in ("linear", "linear_grad"):
        dtype = rng.choice([half, half, half, "f32"])
        rows = _log(rng, 1, 8192 if dtype != "f32" else 1024)
        inp, out = _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.6:                       # widths are multiples of 8 more often than not
            inp, out = -(-inp // 8) * 8, -(-out // 8) * 8
        if kind == "linear":
            c = _linear("", rows, inp, out, dtype, act, rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.4)
        else:
            c = _linear_grad("", rows, inp, out, dtype, act, "f32" if act == "none" and rng.random() < 0.5 else "same")
    elif kind == "loss":
        dtype = rng.choice([half, half, "f32"])
        c = _loss("", _log(rng, 1, 4096), _log(rng, 2000, 131072), dtype, rng.choice(["loss", "grad", "split"]))
    else:
        states = rng.choice(["f32", "mx8"])
        params = rng.choice(["f32", half])
        c = _adamw("", rng.randint(1, 48), _log(rng, 33, 2048), params, rng.choice(["f32", half]), states,
                   params == "f32" and rng.random() < 0.4, states == "f32" and rng.random() < 0.5,
                   states == "f32" and rng.random() < 0.3)
    del c["name"]
    return c


def sizes(case):
    """Elements of each tensor: the matrices and vectors of a stack of two-layer blocks of this width."""
    w, n = case["width"], case["tensors"]
    block = [w * w, w, 4 * w * w, 4 * w, 4 * w * w, w]
    return (block * (n // 6 + 1))[:n]


def _spans(case):
    """(start, size) of each tensor in the flat buffers: packed, or each at the next multiple of a block."""
    at, got = 0, []
    for n in sizes(case):
        got.append((at, n))
        at += n if case["packed"] else -(-n // BLOCK) * BLOCK
    return got, at


def work(case):
    if case["op"] in ("linear", "linear_grad"):
        M, K, N, e = case["rows"], case["inp"], case["out"], SIZE[case["dtype"]]
        if case["op"] == "linear":
            b = M * K + N * K + M * N * (1 + case["residual"] + case["pre"]) + N * case["bias"]
            return {"bytes": e * b, "flops": 2 * M * N * K}
        ge = 4 if case["grads"] == "f32" else e
        b = e * (M * N * (1 + (case["act"] != "none")) + 2 * M * K + N * K) + ge * (N * K + N)
        return {"bytes": b, "flops": 4 * M * N * K}
    if case["op"] == "loss":
        passes = 1 if case["mode"] == "loss" else 2
        live = case["rows"] * case["vocab"] * SIZE[case["dtype"]]
        return {"bytes": passes * live + 32 * case["rows"], "flops": passes * 4 * case["rows"] * case["vocab"]}
    n = sum(sizes(case))
    state = 16 if case["states"] == "f32" else 4 + 4 / BLOCK
    b = n * (2 * SIZE[case["params"]] + SIZE[case["grads"]] + state + 2 * case["copy"])
    return {"bytes": b, "flops": 16 * n}


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] in ("linear", "linear_grad"):
        M, K, N, t = case["rows"], case["inp"], case["out"], DTYPES[case["dtype"]]
        s["x"], s["w"] = _normal(g, (M, K), t), _normal(g, (N, K), t, K ** -0.5)
        if case["op"] == "linear":
            s["bias"] = _normal(g, (N,), t, 0.5) if case["bias"] else None
            s["residual"] = _normal(g, (M, N), t) if case["residual"] else None
            s["y"] = torch.empty(M, N, device="cuda", dtype=t)
            s["pre"] = torch.empty(M, N, device="cuda", dtype=t) if case["pre"] else None
        else:
            gt = torch.float32 if case["grads"] == "f32" else t
            s["dy"] = _normal(g, (M, N), t)
            s["pre"] = _normal(g, (M, N), t) if case["act"] != "none" else None
            s["dx"] = torch.empty(M, K, device="cuda", dtype=t)
            s["dw"], s["dbias"] = torch.empty(N, K, device="cuda", dtype=gt), torch.empty(N, device="cuda", dtype=gt)
    elif case["op"] == "loss":
        T, V, t = case["rows"], case["vocab"], DTYPES[case["dtype"]]
        s["logits"] = torch.empty(T, V, device="cuda", dtype=t)
        s["targets"] = torch.empty(T, device="cuda", dtype=torch.int64)
        logp = torch.empty(T, device="cuda")
        for i in range(0, T, 512):                   # in pieces: the draws are larger than the logits
            z = _normal(g, (min(512, T - i), V), t, 2.0)
            s["logits"][i:i + 512] = z
            z = z.float() / CLIP["temperature"]
            noise = torch.rand(z.shape, generator=g, device="cuda").clamp_(1e-12, 1 - 1e-7).log_().neg_().log_()
            y = (z - noise).argmax(1)                # a sample of softmax(z)
            s["targets"][i:i + 512] = y
            logp[i:i + 512] = z.gather(1, y[:, None])[:, 0] - z.logsumexp(1)
        s["old_logp"] = logp + _normal(g, (T,), scale=0.15)      # the policy that sampled: a few steps older
        s["ref_logp"] = logp + _normal(g, (T,), scale=0.4)
        s["advantages"] = _normal(g, (T,))
        live = torch.rand(T, generator=g, device="cuda") >= 0.1  # the others are padding
        live[T // 2] = True
        s["weights"] = live.float() / live.sum()
        s["stats"] = torch.empty(4, device="cuda")
        s["logp"], s["lse"] = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        s["dlogits"] = torch.empty_like(s["logits"]) if case["mode"] != "loss" else None
    else:
        spans, total = _spans(case)
        inside = torch.zeros(total, device="cuda", dtype=torch.bool)
        for at, n in spans:
            inside[at:at + n] = True
        grads = _normal(g, (total,), scale=1e-2) * torch.exp(_normal(g, (total,)))   # heavy-tailed, as gradients are
        s["params"] = (_normal(g, (total,), scale=0.05) * inside).to(DTYPES[case["params"]])
        s["grads"] = (grads * inside).to(DTYPES[case["grads"]])
        m = _normal(g, (total,), scale=3e-3) * inside
        v = (1e-2 * torch.exp(_normal(g, (total,)))).square() * inside
        del grads
        if case["states"] == "f32":
            s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
        else:
            mx, me = _to_blocks(m)
            rx, re = _to_blocks(v.sqrt())
            s["m"], s["m_scale"] = mx.to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1), me
            s["v"], s["v_scale"] = rx.to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1), re
        s["copy"] = torch.empty(total, device="cuda", dtype=torch.bfloat16) if case["copy"] else None
        # the clip factor of a step whose norm was taken before, where this step does not take it itself
        s["grad_scale"] = torch.rand(1, generator=g, device="cuda") * 0.5 + 0.5
        s["norm"] = torch.empty(2, device="cuda")
        if own:
            import symmetric_memory_allreduce_gb300 as sm

            def cut(t, per=1):
                return [t[at // per:at // per + -(-n // per)] for at, n in spans] if t is not None else None

            s["plan"] = sm.AdamW(cut(s["params"]), cut(s["grads"]), cut(s["m"]), cut(s["v"]),
                                 m_scales=cut(s["m_scale"], BLOCK), v_scales=cut(s["v_scale"], BLOCK),
                                 copies=cut(s["copy"]))
    return s


# ------------------------------------------------------------------ the plain forms

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _plain_linear(s):
    act = s["case"]["act"]
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, act)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(s["y"].dtype)}
    if s["pre"] is not None:
        out["pre"] = z.to(s["y"].dtype)
    return out


def _plain_linear_grad(s):
    dz = s["dy"].float()
    if s["pre"] is not None:
        dz = dz * _act_grad(s["pre"].float(), s["case"]["act"])
    return {"dx": (dz @ s["w"].float()).to(s["dx"].dtype), "dw": (dz.t() @ s["x"].float()).to(s["dw"].dtype),
            "dbias": dz.sum(0).to(s["dbias"].dtype)}


def _plain_loss(s):
    w, a = s["weights"], s["advantages"]
    z = s["logits"].float() * (1 / CLIP["temperature"])
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + torch.exp(z - top).sum(1).log()
    logp = z.gather(1, s["targets"][:, None])[:, 0] - lse
    live = w != 0
    lse, logp = torch.where(live, lse, 0.0), torch.where(live, logp, 0.0)
    d, k = logp - s["old_logp"], s["ref_logp"] - logp
    ratio, kr = torch.exp(d.clamp(-20, 20)), torch.exp(k.clamp(-20, 20))
    bounded = ratio.clamp(1 - CLIP["clip_low"], 1 + CLIP["clip_high"])
    clipped = bounded * a < ratio * a
    policy = -torch.minimum(ratio * a, bounded * a)
    kl = kr - k.clamp(-20, 20) - 1
    each = torch.where(live, policy + CLIP["kl_coef"] * kl, 0.0)
    stats = torch.stack([(w * each).sum(), (w * torch.where(live, policy, 0.0)).sum(),
                         (w * torch.where(live, kl, 0.0)).sum(), (w * clipped).sum()])
    out = {"stats": stats, "logp": logp, "lse": lse}
    if s["dlogits"] is not None:
        dlogp = torch.where(clipped | (d.abs() > 20), 0.0, -a * ratio)
        dlogp = dlogp + CLIP["kl_coef"] * torch.where(k.abs() > 20, 0.0, 1 - kr)
        c = torch.where(live, w * dlogp, 0.0) * (1 / CLIP["temperature"])
        grad = torch.exp(z - lse[:, None]) * -c[:, None]
        grad.scatter_add_(1, s["targets"][:, None], c[:, None])
        out["dlogits"] = torch.where(live[:, None], grad, 0.0).to(s["logits"].dtype)
    return out


def _to_blocks(x):
    """Blocks of 32 scaled by the power of two that brings the largest into (224, 448], and that power + 127."""
    x = torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)
    bits = x.abs().amax(1).view(torch.int32)
    e = ((bits + 0x1FFFFF) >> 23).sub(135).clamp(-127, 127)
    return torch.ldexp(x, -e[:, None]), e.add(127).to(torch.uint8)


def _from_blocks(codes, scale, n):
    x = codes.view(torch.float8_e4m3fn).to(torch.float32).view(-1, BLOCK)
    return torch.ldexp(x, (scale.to(torch.int32) - 127)[:, None]).reshape(-1)[:n]


def _mix(x):
    """32-bit integer mixing in 64-bit arithmetic: xor-shifts and two odd multipliers."""
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _round_up_or_down(y):
    """y in [0, 448] to e4m3 codes: the step above with the probability of its nearness, never 0 from above 0."""
    at = torch.arange(y.numel(), device=y.device)
    h = _mix((at * 0x9E3779B1 + SEED) & 0xFFFFFFFF) >> 12
    e = ((y.reshape(-1).to(torch.float32).view(torch.int32) >> 23) - 127).clamp(min=-6)
    k = torch.floor(torch.ldexp(y.reshape(-1), 3 - e) + h.to(y.dtype) * 2.0 ** -20)
    k = torch.where((k == 0) & (y.reshape(-1) > 0), 1.0, k).to(torch.int32)
    return ((e + 6) * 8 + k).to(torch.uint8)


def _plain_adamw(s):
    case, n = s["case"], s["params"].numel()
    g = s["grads"].float()
    out = {}
    scale = s["grad_scale"]
    if case["clip"]:
        norm = (g * g).sum().sqrt()
        scale = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
        out["norm"] = torch.stack([norm, scale])
    g = g * scale
    if case["states"] == "f32":
        m, v = s["m"], s["v"]
    else:
        m = _from_blocks(s["m"], s["m_scale"], n)
        v = _from_blocks(s["v"], s["v_scale"], n)
        v = v * v
    a = ADAM
    m = m * a["beta1"] + g * (1 - a["beta1"])
    v = v * a["beta2"] + (g * g) * (1 - a["beta2"])
    root = v.sqrt()
    denom = root * (1 / math.sqrt(1 - a["beta2"] ** STEP)) + a["eps"]
    p = s["params"].float() * (1 - a["lr"] * a["weight_decay"])
    p = p - (m / denom) * (a["lr"] / (1 - a["beta1"] ** STEP))
    s["params"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if case["states"] == "f32":
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        mx, me = _to_blocks(m)
        rx, re = _to_blocks(root)
        s["m"].copy_(mx.to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1)[:s["m"].numel()])
        s["v"].copy_(_round_up_or_down(rx)[:s["v"].numel()])
        s["m_scale"].copy_(me)
        s["v_scale"].copy_(re)
    return out


def _adamw_out(s, out):
    """What a step leaves: parameters, states (8-bit ones as float8 values and exponents), the copy."""
    out["params"], out["copy"] = s["params"], s["copy"]
    if s["case"]["states"] == "f32":
        out["m"], out["v"] = s["m"], s["v"]
    else:
        out["m"], out["v"] = s["m"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
        out["m_scale"], out["v_scale"] = s["m_scale"], s["v_scale"]
    return out


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "linear":
            return _plain_linear(s)
        if case["op"] == "linear_grad":
            return _plain_linear_grad(s)
        if case["op"] == "loss":
            return _plain_loss(s)
        return _adamw_out(s, _plain_adamw(s))
    import symmetric_memory_allreduce_gb300 as sm

    if case["op"] == "linear":
        sm.sym_linear(s["x"], s["w"], s["y"], bias=s["bias"], residual=s["residual"], pre=s["pre"], act=case["act"])
        return {"y": s["y"], "pre": s["pre"]}
    if case["op"] == "linear_grad":
        sm.sym_linear_backward(s["dy"], s["x"], s["w"], pre=s["pre"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"],
                               act=case["act"])
        return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"]}
    if case["op"] == "loss":
        sm.sym_policy_loss(s["logits"], s["targets"], s["old_logp"], s["advantages"], s["weights"], s["stats"],
                           s["logp"], s["lse"], ref_logp=s["ref_logp"],
                           dlogits=s["dlogits"] if case["mode"] == "grad" else None, **CLIP)
        if case["mode"] == "split":
            sm.sym_policy_loss_backward(s["logits"], s["targets"], s["old_logp"], s["advantages"], s["weights"],
                                        s["logp"], s["lse"], s["dlogits"], ref_logp=s["ref_logp"], **CLIP)
        return {"stats": s["stats"], "logp": s["logp"], "lse": s["lse"], "dlogits": s["dlogits"]}
    out, scale = {}, s["grad_scale"]
    if case["clip"]:
        sm.sym_grad_norm(s["plan"], s["norm"], max_norm=MAX_NORM)
        out["norm"], scale = s["norm"], s["norm"][1:]
    sm.sym_adamw_step(s["plan"], step=STEP, grad_scale=scale, seed=SEED, **ADAM)
    return _adamw_out(s, out)


# ------------------------------------------------------------------ 64 bits

def _exact_linear(s):
    act = s["case"]["act"]
    z = torch.mm(s["x"].double(), s["w"].double().transpose(0, 1))
    if s["bias"] is not None:
        z += s["bias"].double()
    y = {"none": lambda t: t, "relu": lambda t: torch.where(t > 0, t, torch.zeros_like(t)),
         "gelu": lambda t: t * torch.erfc(t * -(0.5 ** 0.5)) / 2, "silu": lambda t: t * torch.sigmoid(t)}[act](z)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": y, "pre": z if s["pre"] is not None else None}


def _exact_linear_grad(s):
    dz = s["dy"].double()
    if s["pre"] is not None:
        z, act = s["pre"].double(), s["case"]["act"]
        if act == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        elif act == "gelu":
            dz = dz * (torch.erfc(z * -(0.5 ** 0.5)) / 2 + z * torch.exp(z.square() / -2) / (2 * math.pi) ** 0.5)
        elif act == "silu":
            dz = dz * torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    return {"dx": torch.mm(dz, s["w"].double()), "dw": torch.mm(dz.transpose(0, 1), s["x"].double()),
            "dbias": dz.sum(0)}


def _exact_loss(s):
    T, temp = s["case"]["rows"], CLIP["temperature"]
    w, a = s["weights"].double(), s["advantages"].double()
    logp, lse = torch.zeros(T, device="cuda", dtype=torch.float64), torch.zeros(T, device="cuda", dtype=torch.float64)
    rows = w.nonzero()[:, 0]
    for part in rows.split(512):
        z = s["logits"][part].double() / temp
        lse[part] = torch.logsumexp(z, 1)
        logp[part] = z[torch.arange(len(part), device="cuda"), s["targets"][part]] - lse[part]
    d = (logp - s["old_logp"].double())
    k = (s["ref_logp"].double() - logp)
    rho, kr = d.clamp(-20, 20).exp(), k.clamp(-20, 20).exp()
    lo, hi = 1 - CLIP["clip_low"], 1 + CLIP["clip_high"]
    stopped = ((a > 0) & (rho > hi)) | ((a < 0) & (rho < lo))
    policy = torch.where(stopped, -a * rho.clamp(lo, hi), -a * rho)
    kl = kr - 1 - k.clamp(-20, 20)
    stats = torch.stack([(w * (policy + CLIP["kl_coef"] * kl)).sum(), (w * policy).sum(), (w * kl).sum(),
                         (w * stopped).sum()])
    out = {"stats": stats, "logp": logp, "lse": lse}
    if s["dlogits"] is not None:
        slope = torch.where(stopped | (d.abs() > 20), 0.0, -a * rho)
        slope = slope + torch.where(k.abs() > 20, 0.0, CLIP["kl_coef"] * (1 - kr))
        c = w * slope / temp
        grad = torch.zeros(s["logits"].shape, device="cuda", dtype=torch.float64)
        for part in rows.split(512):
            p = torch.softmax(s["logits"][part].double() / temp, 1)
            p[torch.arange(len(part), device="cuda"), s["targets"][part]] -= 1
            grad[part] = p * -c[part, None]
        out["dlogits"] = grad
    return out


def _exact_adamw(s):
    a, case, n = ADAM, s["case"], s["params"].numel()
    g = s["grads"].double()
    out = {"norm": None} if case["clip"] else {}
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        out["norm"] = torch.stack([norm, torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)])
        g = g * out["norm"][1]
    else:
        g = g * s["grad_scale"].double()
    if case["states"] == "f32":
        m, v = s["m"].double(), s["v"].double()
    else:
        def value(codes, e):
            x = codes.view(torch.float8_e4m3fn).to(torch.float64).view(-1, BLOCK)
            return (x * torch.exp2(e.double() - 127)[:, None]).view(-1)[:n]
        m, v = value(s["m"], s["m_scale"]), value(s["v"], s["v_scale"]).square()
    m = a["beta1"] * m + (1 - a["beta1"]) * g
    v = a["beta2"] * v + (1 - a["beta2"]) * g.square()
    mh, vh = m / (1 - a["beta1"] ** STEP), v / (1 - a["beta2"] ** STEP)
    p = s["params"].double()
    p = p - a["lr"] * (mh / (vh.sqrt() + a["eps"]) + a["weight_decay"] * p)
    out["params"], out["copy"] = p, p if s["copy"] is not None else None
    if case["states"] == "f32":
        out["m"], out["v"] = m, v
    else:                                            # what 8 bits hold has no value in 64
        out["m"] = out["v"] = out["m_scale"] = out["v_scale"] = None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "linear_grad": _exact_linear_grad, "loss": _exact_loss,
            "adamw": _exact_adamw}[case["op"]](s)
