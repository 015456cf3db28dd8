"""The clipped policy loss with its KL term against its definition in 64 bits.

Tolerances: lse is a log of a sum of at most V terms held in 32 bits, off by at most
E = (V/256 + 64) 2^-23 (a thread adds at most V/256 of them, then a tree) + 2^-21 max|z| (scaling,
exponents); logp by 2E.  rho, exp(k) and p are off by 2E + 2^-20 of themselves, products add a few
roundings, the gradient is rounded once to its type."""
import pytest
import torch

from _training_util import DTYPES, F64, TINY, UNIT, close, policy64

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1), (1, 2), (3, 31), (2, 1000), (5, 4097), (7, 8193), (33, 2056), (2, 50003), (1, 131072), (2, 300_001), (300, 96)]
HYPER = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.1, temperature=0.8)


def _inputs(T, V, dtype, seed, spread=0.5):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    logits = (n(T, V) * 3).to(DTYPES[dtype])
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    z = logits.double() / HYPER["temperature"]
    logp = (z.gather(1, targets[:, None])[:, 0] - z.logsumexp(1)).float()
    weights = torch.rand(T, generator=g, device="cuda") / T
    weights[::3] = 0 if T > 1 else 0.7
    return dict(logits=logits, targets=targets, old_logp=logp + n(T) * spread, advantages=n(T), weights=weights,
                ref_logp=logp + n(T) * spread)


def _outputs(T):
    return dict(stats=torch.full((4,), 7.0, device="cuda"), logp=torch.full((T,), 7.0, device="cuda"),
                lse=torch.full((T,), 7.0, device="cuda"))


def _compare(inp, hyper, out, dlogits, grad_out=1.0):
    T, V = inp["logits"].shape
    dtype = inp["logits"].dtype
    host = {k: None if v is None else v.cpu() for k, v in inp.items()}
    stats, logp, lse, grad = policy64(host["logits"], host["targets"], host["old_logp"], host["advantages"],
                                      host["weights"], host["ref_logp"], grad_out=grad_out, **hyper)
    z = host["logits"].double() / hyper["temperature"]
    top = torch.where(torch.isfinite(z), z.abs(), 0.0).amax(1)
    E = (V / 256 + 64) * 2.0 ** -23 + 2.0 ** -21 * top
    live = host["weights"] != 0 if host["weights"] is not None else torch.ones(T, dtype=torch.bool)
    close(out["lse"].cpu(), lse, E, "lse")
    close(out["logp"].cpu(), logp, 2 * E, "logp")
    w = (host["weights"].double() if host["weights"] is not None else torch.ones(T, dtype=F64)) * live
    d = (logp - host["old_logp"].double()).clamp(-20, 20)
    k = (host["ref_logp"].double() - logp).clamp(-20, 20) if host["ref_logp"] is not None else torch.full((T,), -60.0).double()
    rel = 2 * E + 2.0 ** -19
    pol = host["advantages"].double().abs() * d.exp()
    kl = k.exp() + 1 + k.abs().clamp(max=20)
    err = torch.stack([(w * (pol + hyper["kl_coef"] * kl) * rel).sum(), (w * pol * rel).sum(), (w * kl * rel).sum(),
                       w.sum() * 2.0 ** -22]) + (T + 4) * 2.0 ** -23 * stats.abs()
    close(out["stats"].cpu(), stats, err, "stats")
    if dlogits is None:
        return
    p = torch.where(live[:, None], torch.exp(z - lse[:, None]), 0.0)
    onehot = torch.zeros(T, V, dtype=F64).scatter_(1, host["targets"][:, None].clamp(0, V - 1), 1.0)
    c = abs(grad_out) * w / hyper["temperature"] * (pol + hyper["kl_coef"] * (k.exp() + 1))
    tol = UNIT[dtype] * 1.01 * grad.abs() + TINY[dtype] + (c * rel)[:, None] * 2 * (p + onehot)
    close(dlogits.cpu(), grad, tol, "dlogits")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_loss_and_gradient(symar, shape, dtype):
    T, V = shape
    for kl, weighted in [(True, True), (False, False)]:
        inp = _inputs(T, V, dtype, 10 * T + V + kl)
        if not kl:
            inp["ref_logp"] = None
        if not weighted:
            inp["weights"] = None
        out, d = _outputs(T), torch.full((T, V), 7.0, device="cuda", dtype=DTYPES[dtype])
        symar.sym_policy_loss(**inp, **out, dlogits=d, **HYPER)
        assert symar.sym_stream_status() == symar.SYM_OK, symar.sym_last_error()
        _compare(inp, HYPER, out, d)
        # the loss alone, then the gradient alone with an upstream factor, then in place
        out2, d2, go = _outputs(T), torch.full_like(d, 7.0), torch.full((1,), -2.5, device="cuda")
        symar.sym_policy_loss(**inp, **out2, **HYPER)
        _compare(inp, HYPER, out2, None)
        symar.sym_policy_loss_backward(**inp, logp=out2["logp"], lse=out2["lse"], dlogits=d2, grad_out=go, **HYPER)
        _compare(inp, HYPER, out2, d2, -2.5)
        x = inp["logits"].clone()
        symar.sym_policy_loss(**{**inp, "logits": x}, **out2, dlogits=x, **HYPER)
        assert torch.equal(x, d)


@pytest.mark.parametrize("dtype,T,V", [("bf16", 2500, 2056), ("f16", 2500, 96), ("f32", 400, 9001), ("bf16", 90, 70001)])
def test_many_rows_with_runs_of_masked_ones(symar, dtype, T, V):
    """More rows than the GPU takes at once, masked in runs of every length."""
    inp = _inputs(T, V, dtype, T + V)
    live = torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.4
    live[T // 3:T // 2], live[-T // 5:] = False, True
    inp["weights"] = (live.float() / T).cuda()
    for d in (torch.full_like(inp["logits"], 7.0), None):
        out = _outputs(T)
        symar.sym_policy_loss(**inp, **out, dlogits=d, **HYPER)
        assert symar.sym_stream_status() == symar.SYM_OK, symar.sym_last_error()
        _compare(inp, HYPER, out, d)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_strided_and_misaligned_rows(symar, dtype):
    T = 5
    for V in (130, 8200):
        for off, pad in [(1, 0), (3, 6), (8, 24)]:
            inp = _inputs(T, V, dtype, V + off)
            buf = torch.full((T, V + off + pad), float("nan"), device="cuda", dtype=DTYPES[dtype])
            buf[:, off:off + V] = inp["logits"]
            g = torch.full((T, V + pad + 1), 7.0, device="cuda", dtype=DTYPES[dtype])
            inp["logits"], d = buf[:, off:off + V], g[:, 1:1 + V]
            out = _outputs(T)
            symar.sym_policy_loss(**inp, **out, dlogits=d, **HYPER)
            _compare(inp, HYPER, out, d)
            assert (g[:, 0] == 7).all() and (g[:, 1 + V:] == 7).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [40, 5000])
def test_masked_vocabulary_and_rows(symar, V, dtype):
    """Columns at -inf and at the type's lowest value; weight-0 rows full of NaN and infinities; all rows off."""
    T = 6
    inp = _inputs(T, V, dtype, 5)
    x = inp["logits"]
    inp["weights"] = torch.full((T,), 0.25, device="cuda")
    x[0, V // 2:] = float("-inf")
    x[1, : V - 3] = float("-inf")
    x[2, ::2] = torch.finfo(x.dtype).min
    inp["targets"][:3] = torch.tensor([1, V - 1, 1])
    inp["weights"][3:5] = 0
    x[3], x[4, ::2] = float("nan"), float("inf")
    x[5] = 0.5                                              # a flat row
    z = x.double() / HYPER["temperature"]
    lp = (z.gather(1, inp["targets"][:, None])[:, 0] - z.logsumexp(1)).float()
    inp["old_logp"] = torch.where(torch.isfinite(lp), lp + 0.05, 0.0)
    inp["ref_logp"] = inp["old_logp"] + 0.3
    hyper = HYPER
    out, d = _outputs(T), torch.full_like(x, 7.0)
    symar.sym_policy_loss(**inp, **out, dlogits=d, **hyper)
    assert symar.sym_stream_status() == symar.SYM_OK
    _compare(inp, hyper, out, d)
    assert (d[3:5] == 0).all() and (d[0, V // 2:] == 0).all() and (out["logp"][3:5] == 0).all()
    inp["weights"] = torch.zeros(T, device="cuda")
    symar.sym_policy_loss(**inp, **out, dlogits=d, **hyper)
    assert (d == 0).all() and (out["stats"] == 0).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_a_live_row_without_a_distribution_is_nan(symar, dtype):
    inp = _inputs(3, 5000, dtype, 6)
    inp["weights"] = torch.ones(3, device="cuda")
    inp["logits"][1] = float("-inf")
    inp["logits"][2, 7] = float("nan")
    out, d = _outputs(3), torch.empty_like(inp["logits"])
    symar.sym_policy_loss(**inp, **out, dlogits=d, **HYPER)
    assert torch.isnan(out["logp"][1:]).all() and torch.isfinite(out["logp"][0])
    assert torch.isnan(out["stats"][0]) and torch.isfinite(d[0].float()).all()
    assert torch.isnan(d[1:].float()).all()


def test_extreme_ratios_are_clamped(symar):
    """logp 50 away from old and ref on either side: finite loss, no gradient through the clamped terms."""
    inp = _inputs(4, 64, "f32", 7)
    inp["weights"] = torch.ones(4, device="cuda")
    z = inp["logits"].double() / HYPER["temperature"]
    lp = (z.gather(1, inp["targets"][:, None])[:, 0] - z.logsumexp(1)).float()
    inp["old_logp"] = lp + torch.tensor([50.0, -50.0, 50.0, -50.0], device="cuda")
    inp["ref_logp"] = lp + torch.tensor([50.0, 50.0, -50.0, -50.0], device="cuda")
    inp["advantages"] = torch.tensor([1.0, 1.0, -1.0, -1.0], device="cuda")
    out, d = _outputs(4), torch.empty_like(inp["logits"])
    symar.sym_policy_loss(**inp, **out, dlogits=d, **HYPER)
    _compare(inp, HYPER, out, d)
    assert (d == 0).all()


def test_bad_target_is_reported(symar):
    inp = _inputs(4, 100, "bf16", 8)
    inp["weights"] = torch.tensor([0.5, 0.5, 0.0, 0.5], device="cuda")
    inp["targets"][1], inp["targets"][2], inp["targets"][3] = 100, -100, -1      # row 2's is not looked at
    out, d = _outputs(4), torch.full_like(inp["logits"], 7.0)
    symar.sym_policy_loss(**inp, **out, dlogits=d, **HYPER)
    assert symar.sym_stream_status() == 6 and "policy loss target" in symar.sym_last_error()
    assert symar.sym_stream_status() == symar.SYM_OK                             # reported once
    _compare(inp, HYPER, out, None)
    assert (d[1:] == 0).all() and d[0].abs().sum() > 0
    symar.sym_policy_loss_backward(**inp, logp=out["logp"], lse=out["lse"], dlogits=d, **HYPER)
    assert symar.sym_stream_status() == 6


def test_gradient_against_differences(symar):
    """dlogits along a direction against central differences of the loss in 64 bits (step 1e-5)."""
    T, V = 6, 50
    inp = _inputs(T, V, "f32", 9, spread=0.05)               # far from the clip's corners
    out, d = _outputs(T), torch.empty_like(inp["logits"])
    symar.sym_policy_loss(**inp, **out, dlogits=d, **HYPER)
    u = torch.randn(T, V, dtype=F64, generator=torch.Generator().manual_seed(3))
    host = {k: v.cpu() for k, v in inp.items()}

    def f(h):
        return policy64(host["logits"].double() + h * u, host["targets"], host["old_logp"], host["advantages"],
                        host["weights"], host["ref_logp"], **HYPER)[0][0]

    want, got = (f(1e-5) - f(-1e-5)) / 2e-5, (d.cpu().double() * u).sum()
    assert abs(want - got) < 1e-4 * (d.cpu().double() * u).abs().sum()


def test_stream_graph_and_no_rows(symar):
    T, V = 9, 6000
    inp, out = _inputs(T, V, "bf16", 11), _outputs(T)
    d = torch.empty_like(inp["logits"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    symar.sym_policy_loss(**inp, **out, dlogits=d, stream=st, **HYPER)
    st.synchronize()
    _compare(inp, HYPER, out, d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        symar.sym_policy_loss(**inp, **out, dlogits=d, **HYPER)
    other = _inputs(T, V, "bf16", 12)
    for k, v in other.items():
        inp[k].copy_(v)
    g.replay()
    _compare(other, HYPER, out, d)
    e = torch.empty(0, 10, device="cuda")
    z = torch.empty(0, device="cuda")
    stats = torch.full((4,), 7.0, device="cuda")
    symar.sym_policy_loss(e, torch.empty(0, device="cuda", dtype=torch.int64), z, z, z, stats, z, z, dlogits=e)
    assert (stats == 0).all()


def test_refusals(symar):
    inp, out = _inputs(4, 16, "bf16", 13), _outputs(4)
    n = symar.sym_launch_count()
    for b in [dict(targets=inp["targets"].int()), dict(old_logp=inp["old_logp"][:3]), dict(advantages=inp["advantages"].double()),
              dict(logits=inp["logits"].t()), dict(logits=inp["logits"].cpu()), dict(dlogits=inp["logits"].float()),
              dict(stats=torch.empty(3, device="cuda")), dict(temperature=0.0), dict(temperature=float("nan")),
              dict(clip_low=-0.1), dict(kl_coef=float("inf")), dict(dlogits=inp["logits"].view(-1)[:32].view(4, 8))]:
        with pytest.raises((ValueError, symar.SymError)):
            symar.sym_policy_loss(**{**inp, **out, **HYPER, **b})
    buf = torch.zeros(5, 16, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(symar.SymError):                      # the gradient shifted over the logits
        symar.sym_policy_loss(**{**inp, "logits": buf[:4]}, **out, dlogits=buf[1:], **HYPER)
    assert symar.sym_launch_count() == n
