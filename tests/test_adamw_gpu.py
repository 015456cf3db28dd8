"""AdamW over many tensors: bit for bit against the same operations in numpy float32 (each rounded
once, in the documented order), and against the formula in 64 bits.

In 64 bits: m and v are sums of two products, off by at most 4 roundings of the terms' magnitudes; the
update carries those through a root and a quotient, 16 roundings of itself and of m's terms' share."""
import math

import numpy as np
import pytest
import torch

from _training_util import DTYPES, F64, TINY, UNIT, close

pytestmark = pytest.mark.gpu
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
LISTS = {"one": [1], "scalars": [1, 1, 1], "edges": [31, 32, 33, 2047, 2048, 2049], "empty among": [0, 5, 0, 70, 0],
         "odd": [7, 4099, 1, 12345, 64, 3], "large": [300_001, 65_536]}


def _mix(x):
    x = x.astype(np.uint32)
    x ^= x >> np.uint32(16)
    x *= np.uint32(0x7FEB352D)
    x ^= x >> np.uint32(15)
    x *= np.uint32(0x846CA68B)
    return x ^ (x >> np.uint32(16))


def _exponent(amax):
    e = ((amax.view(np.int32).astype(np.int64) + 0x1FFFFF) >> 23) - 135
    return np.clip(e, -127, 127)


def _blocks(x):
    return np.pad(x, (0, -len(x) % 32)).reshape(-1, 32)


def _value(codes, scale):
    n = len(codes)
    c = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    return (_blocks(c) * np.ldexp(np.float32(1), scale.astype(np.int64) - 127).astype(np.float32)[:, None]).reshape(-1)[:n]


def _nearest(m):
    e = _exponent(np.abs(_blocks(m)).max(1))
    y = np.ldexp(_blocks(m), -e[:, None]).astype(np.float32).reshape(-1)[:len(m)]
    return torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), (e + 127).astype(np.uint8)


def _stochastic(r, base, seed):
    e = _exponent(_blocks(r).max(1))
    y = np.ldexp(_blocks(r), -e[:, None]).astype(np.float32).reshape(-1)[:len(r)]
    with np.errstate(over="ignore"):
        h = _mix((np.arange(len(r), dtype=np.uint32) + np.uint32(base)) * np.uint32(0x9E3779B1) + np.uint32(seed))
    u = (h >> np.uint32(12)).astype(np.float32) * np.float32(2.0 ** -20)
    k = np.maximum((y.view(np.int32) >> 23) - 127, -6)
    q = np.floor(np.ldexp(y, 3 - k).astype(np.float32) + u)
    q = np.where((q == 0) & (y > 0), 1, q).astype(np.int64)
    return ((k + 6) * 8 + q).astype(np.uint8), (e + 127).astype(np.uint8)


def _step32(p, g, m, v, gs, t, h):
    """The documented operations in float32; p, g, m, v, gs float32 arrays."""
    f = np.float32
    g = g * gs
    m = m * f(h["beta1"]) + g * f(1 - h["beta1"])
    v = v * f(h["beta2"]) + (g * g) * f(1 - h["beta2"])
    r = np.sqrt(v)
    d = r * f(1 / math.sqrt(1 - h["beta2"] ** t)) + f(h["eps"])
    p = p * f(1 - h["lr"] * h["weight_decay"]) - (m / d) * f(h["lr"] / (1 - h["beta1"] ** t))
    return p, m, v, r


def _tensors(counts, dtype, seed, offset=0, scale=1.0):
    """Views at `offset` elements into buffers of their own, with guards around."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in counts:
        b = torch.full((n + offset + 9,), 7.0, dtype=torch.float32)
        b[offset:offset + n] = torch.randn(n, generator=g) * scale
        out.append(b.to(dtype).cuda()[offset:offset + n])
    return out


def _np(t):
    return t.detach().cpu().float().numpy()


def _u8(counts, per, seed):
    return [torch.zeros(-(-n // per), dtype=torch.uint8, device="cuda") for n in counts]


@pytest.mark.parametrize("offset", [0, 1, 3, 8])
@pytest.mark.parametrize("grads", list(DTYPES))
@pytest.mark.parametrize("params", list(DTYPES))
@pytest.mark.parametrize("name", list(LISTS))
def test_f32_states_bit_exact(symar, name, params, grads, offset):
    counts = LISTS[name]
    if name == "large" and (params, grads) not in [("f32", "f32"), ("bf16", "bf16"), ("f32", "f16")]:
        pytest.skip("the large list runs on three type pairs")
    p, g = _tensors(counts, DTYPES[params], 1, offset), _tensors(counts, DTYPES[grads], 2, offset)
    # offset 1: v stands elsewhere than the others, so they share no vector boundary; 3: all share one
    m, v = _tensors(counts, torch.float32, 3, offset, 0.1), _tensors(counts, torch.float32, 4, 0 if offset == 1 else offset)
    for x in v:
        x.square_()
    copies = _tensors(counts, torch.bfloat16, 5, offset) if params == "f32" else None
    state = [[_np(t) for t in ts] for ts in (p, g, m, v)]
    gs = torch.tensor([0.37], device="cuda")
    with symar.AdamW(p, g, m, v, copies=copies) as plan:
        for t in (1, 2):
            symar.sym_adamw_step(plan, step=t, grad_scale=gs if t == 1 else None, **HYPER)
            for i, n in enumerate(counts):
                s = [x[i] for x in state]
                a, b, c, _ = _step32(*s, np.float32(0.37 if t == 1 else 1.0), t, HYPER)
                if t == 1:
                    p64, m64, v64 = (x.astype(np.float64) for x in (s[0], s[2], s[3]))
                    g64 = s[1].astype(np.float64) * float(np.float32(0.37))
                    m1, v1 = 0.9 * m64 + 0.1 * g64, 0.99 * v64 + 0.01 * g64 ** 2
                    q = (HYPER["lr"] / 0.1) / (np.sqrt(v1 / 0.01) + 1e-8)
                    want = p64 * (1 - 1e-3) - q * m1
                    tol = 16 * 2.0 ** -24 * (np.abs(want) + np.abs(p64) + q * (np.abs(0.9 * m64) + np.abs(0.1 * g64)))
                    u = UNIT[p[i].dtype]
                    close(p[i].cpu(), torch.from_numpy(want), torch.from_numpy(tol + u * 1.01 * np.abs(want) + TINY[p[i].dtype]), "p")
                    close(m[i].cpu(), torch.from_numpy(m1), torch.from_numpy(4 * 2.0 ** -24 * (np.abs(0.9 * m64) + np.abs(0.1 * g64))), "m")
                    close(v[i].cpu(), torch.from_numpy(v1), torch.from_numpy(4 * 2.0 ** -24 * np.abs(v1)), "v")
                a_t = torch.from_numpy(a).to(p[i].dtype)
                assert torch.equal(p[i].cpu(), a_t), (i, n, t)
                assert np.array_equal(_np(m[i]), b) and np.array_equal(_np(v[i]), c), (i, n, t)
                if copies:
                    assert torch.equal(copies[i].cpu(), torch.from_numpy(a).to(torch.bfloat16))
                state[0][i], state[2][i], state[3][i] = a_t.float().numpy(), b, c
        for ts in (p, g, m, v):                                 # the guards after each tensor
            for x in ts:
                base = x._base if x._base is not None else x
                assert (base[x.storage_offset() + x.numel():] == 7).all()
    assert symar.sym_stream_status() == symar.SYM_OK


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("grads", list(DTYPES))
@pytest.mark.parametrize("params", list(DTYPES))
@pytest.mark.parametrize("name", list(LISTS))
def test_8_bit_states_bit_exact(symar, name, params, grads, offset):
    counts = LISTS[name]
    if name == "large" and (params, grads) not in [("f32", "f32"), ("bf16", "bf16"), ("f32", "f16")]:
        pytest.skip("the large list runs on three type pairs")
    p, g = _tensors(counts, DTYPES[params], 1, offset), _tensors(counts, DTYPES[grads], 2, offset)
    for x in g[:1]:
        x[: len(x) // 2] *= 1e-3                            # blocks of unlike sizes
    m, v = ([torch.zeros(n + 8, dtype=torch.uint8, device="cuda")[offset:offset + n] for n in counts] for _ in "mv")
    ms, vs = _u8(counts, 32, 0), _u8(counts, 32, 0)
    state = [_np(t) for t in p], [_np(t) for t in g], [_np(t).astype(np.uint8) for t in m], [_np(t).astype(np.uint8) for t in v], \
            [x.cpu().numpy() for x in ms], [x.cpu().numpy() for x in vs]
    with symar.AdamW(p, g, m, v, m_scales=ms, v_scales=vs) as plan:
        for t in (1, 2, 3):
            symar.sym_adamw_step(plan, step=t, seed=100 + t, **HYPER)
            base = 0
            for i, n in enumerate(counts):
                pi, gi, mi, vi, msi, vsi = (x[i] for x in state)
                m32, r32 = _value(mi, msi), _value(vi, vsi)
                a, b, c, r = _step32(pi, gi, m32, r32 * r32, np.float32(1), t, HYPER)
                a_t = torch.from_numpy(a).to(p[i].dtype)
                if n:
                    mc, me = _nearest(b)
                    vc, ve = _stochastic(r, base, 100 + t)
                    assert torch.equal(p[i].cpu(), a_t), (i, n, t)
                    assert np.array_equal(m[i].cpu().numpy(), mc) and np.array_equal(ms[i].cpu().numpy(), me), (i, n, t)
                    assert np.array_equal(v[i].cpu().numpy(), vc) and np.array_equal(vs[i].cpu().numpy(), ve), (i, n, t)
                    for k, val in enumerate((a_t.float().numpy(), gi, mc, vc, me, ve)):
                        state[k][i] = val
                base += -(-n // 32) * 32
    assert symar.sym_stream_status() == symar.SYM_OK


def test_8_bit_values_are_near_and_unbiased(symar):
    """A block's values are within half a step of e4m3 (m) or one (the root), and the root's mean over
    seeds is within 5 standard errors; a root above zero never becomes zero."""
    n, reps = 4096, 64
    g = torch.cat([torch.randn(n // 2), torch.randn(n // 2) * torch.logspace(-6, 0, n // 2)]).cuda()
    total = torch.zeros(n, dtype=F64, device="cuda")
    for seed in range(reps):
        p, m, v = torch.zeros(n, device="cuda"), *(torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in "mv")
        ms, vs = (torch.zeros(n // 32, dtype=torch.uint8, device="cuda") for _ in "mv")
        with symar.AdamW([p], [g], [m], [v], m_scales=[ms], v_scales=[vs]) as plan:
            symar.sym_adamw_step(plan, step=1, seed=seed, **HYPER)
            torch.cuda.synchronize()
        r = torch.from_numpy(_value(v.cpu().numpy(), vs.cpu().numpy())).cuda().double()
        mm = torch.from_numpy(_value(m.cpu().numpy(), ms.cpu().numpy())).cuda().double()
        r0, m0 = g.double().abs() * 0.1, g.double() * 0.1
        scale = torch.exp2(vs.double() - 127).repeat_interleave(32)
        step = torch.exp2(torch.floor(torch.log2((r0 / scale).clamp(min=2.0 ** -6))) - 3) * scale
        mscale = torch.exp2(ms.double() - 127).repeat_interleave(32)
        mstep = torch.exp2(torch.floor(torch.log2((m0.abs() / mscale).clamp(min=2.0 ** -6))) - 3) * mscale
        assert ((r - r0).abs() <= step * 1.0001).all() and ((mm - m0).abs() <= mstep * 0.5001).all()
        assert ((r > 0) == (r0 > 0)).all()
        total += (r - r0) / step
    fine = r0 > 8 * scale * 2.0 ** -9                        # where zero is out of reach
    mean = total[fine].sum() / (reps * fine.sum())
    assert abs(mean) < 5 * 0.5 / math.sqrt(reps * int(fine.sum()))


def test_8_bit_second_moment_follows_a_change(symar):
    """400 steps of gradients 4 times as large move the stored root there (to nearest it would stay put);
    v's distance falls by 0.99^400 = 0.018, and single roots scatter by an e4m3 step or so."""
    n = 8192
    g = torch.full((n,), 1.0, device="cuda")
    p, m, v = torch.zeros(n, device="cuda"), *(torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in "mv")
    ms, vs = (torch.zeros(n // 32, dtype=torch.uint8, device="cuda") for _ in "mv")
    with symar.AdamW([p], [g], [m], [v], m_scales=[ms], v_scales=[vs]) as plan:
        for t in range(1, 801):
            if t == 401:
                g.fill_(4.0)
            symar.sym_adamw_step(plan, step=t, seed=t, **HYPER)
        torch.cuda.synchronize()
    r = _value(v.cpu().numpy(), vs.cpu().numpy())
    assert abs(r.mean() - 4.0) < 0.25


@pytest.mark.parametrize("grads", list(DTYPES))
@pytest.mark.parametrize("name", list(LISTS))
def test_grad_norm(symar, name, grads):
    """Squares added in 32 bits by threads of at most 256 + 32 terms each: 300 roundings at most."""
    counts = LISTS[name]
    for offset in (0, 1):
        g = _tensors(counts, DTYPES[grads], 3, offset)
        p = [t.float().clone() for t in g]
        m, v = ([torch.zeros_like(x) for x in p] for _ in "mv")
        out, again = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
        with symar.AdamW(p, g, m, v) as plan:
            want = math.sqrt(sum(float(x.double().square().sum()) for x in g))
            symar.sym_grad_norm(plan, out, max_norm=0.5)
            symar.sym_grad_norm(plan, again, max_norm=0.5)
            assert torch.equal(out, again)
            assert abs(out[0].item() - want) <= 300 * 2.0 ** -24 * want
            assert abs(out[1].item() - min(1.0, 0.5 / (want + 1e-6))) <= 310 * 2.0 ** -24
            symar.sym_grad_norm(plan, out, max_norm=1e9)
            assert out[1].item() == 1.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_step_without_a_finite_norm_is_skipped(symar, bad):
    g = _tensors([5000, 33], torch.float16, 1)
    p, m, v = _tensors([5000, 33], torch.float32, 2), _tensors([5000, 33], torch.float32, 3), _tensors([5000, 33], torch.float32, 4)
    before = [x.clone() for ts in (p, m, v) for x in ts]
    g[1][7] = bad
    out = torch.empty(2, device="cuda")
    with symar.AdamW(p, g, m, v) as plan:
        symar.sym_grad_norm(plan, out, max_norm=1.0)
        assert torch.isnan(out[1]) and not torch.isfinite(out[0])
        symar.sym_adamw_step(plan, step=1, grad_scale=out[1:], **HYPER)
        assert all(torch.equal(a, b) for a, b in zip(before, [x for ts in (p, m, v) for x in ts]))
        g[1][7] = 0
        symar.sym_grad_norm(plan, out, max_norm=1.0)
        symar.sym_adamw_step(plan, step=1, grad_scale=out[1:], **HYPER)
        assert not torch.equal(before[0], p[0])


def test_window_gradients_stream_and_graph(symar):
    """Gradients as views of a rank's window (odd offsets), the step on its own stream and replayed."""
    R, counts = 2, [100, 33, 4097]
    w = symar.Window(R, 4 * sum(counts))
    try:
        flat = w.tensor(torch.float32)[1, :sum(counts)]
        flat.copy_(torch.randn(sum(counts), generator=torch.Generator().manual_seed(1)))
        g = list(flat.split(counts))
        p, m, v = _tensors(counts, torch.float32, 2), _tensors(counts, torch.float32, 3), [torch.ones(n, device="cuda") for n in counts]
        ref = [[_np(t) for t in ts] for ts in (p, g, m, v)]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with symar.AdamW(p, g, m, v) as plan:
            symar.sym_adamw_step(plan, step=3, stream=st, **HYPER)
            st.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                symar.sym_adamw_step(plan, step=3, **HYPER)
            graph.replay()
            torch.cuda.synchronize()
        for i in range(3):
            a = [x[i] for x in ref]
            for _ in range(2):
                a[0], a[2], a[3], _ = _step32(*a, np.float32(1), 3, HYPER)
            assert np.array_equal(_np(p[i]), a[0]) and np.array_equal(_np(m[i]), a[2])
    finally:
        w.free()


def test_no_tensors(symar):
    out = torch.empty(2, device="cuda")
    with symar.AdamW([], [], [], []) as plan:
        symar.sym_adamw_step(plan, step=1, lr=1e-3)
        symar.sym_grad_norm(plan, out, max_norm=1.0)
    assert out.tolist() == [0.0, 1.0]


def test_refusals(symar):
    f = lambda n, d=torch.float32: torch.zeros(n, device="cuda", dtype=d)  # noqa: E731
    for args, kw in [(([f(4)], [f(5)], [f(4)], [f(4)]), {}), (([f(4)], [], [f(4)], [f(4)]), {}),
                     (([f(4).cpu()], [f(4)], [f(4)], [f(4)]), {}), (([f(4)], [f(4)], [f(4).half()], [f(4)]), {}),
                     (([f(4), f(4).half()], [f(4), f(4)], [f(4), f(4)], [f(4), f(4)]), {}),
                     (([f(8)[::2]], [f(4)], [f(4)], [f(4)]), {}), (([f(4).double()], [f(4)], [f(4)], [f(4)]), {}),
                     (([f(40)], [f(40)], [f(40, torch.uint8)], [f(40, torch.uint8)]),
                      dict(m_scales=[f(1, torch.uint8)], v_scales=[f(2, torch.uint8)])),
                     (([f(4)], [f(4)], [f(4)], [f(4)]), dict(m_scales=[f(1, torch.uint8)]))]:
        with pytest.raises((ValueError, symar.SymError)):
            symar.AdamW(*args, **kw)
    with symar.AdamW([f(4)], [f(4)], [f(4)], [f(4)]) as plan:
        n = symar.sym_launch_count()
        for kw in [dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=float("nan")),
                   dict(weight_decay=float("inf"))]:
            with pytest.raises(symar.SymError):
                symar.sym_adamw_step(plan, **{**dict(lr=1e-3, step=1), **kw})
        with pytest.raises(ValueError):
            symar.sym_adamw_step(plan, lr=1e-3, step=1, grad_scale=f(2))
        with pytest.raises(symar.SymError):
            symar.sym_grad_norm(plan, f(2), max_norm=0.0)
        assert symar.sym_launch_count() == n
