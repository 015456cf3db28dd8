"""The linear layer (sym_linear, sym_linear_backward) against its definition in 64 bits.

Tolerances: a sum of K terms held in 32 bits is off by at most (K+4) 2^-23 times the sum of the
terms' magnitudes (2^-23 a step: the tensor cores may truncate); activations have slopes below 1.13
and are evaluated to 2^-20; each output is rounded once to its type.  The backward products also
carry dz's own rounding."""
import ctypes

import pytest
import torch

from _training_util import DTYPES, F64, TINY, UNIT, act64, close, linear64, slope64

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "silu"]
# one row to several tiles; sizes around the tiles' edges (8, 16, 64, 128, 256), odd ones
SIZES = [(1, 1, 1), (1, 64, 128), (1, 257, 640), (2, 1000, 96), (3, 65, 4100), (4, 2050, 260), (7, 130, 24), (8, 33, 1001), (9, 33, 1001), (13, 300, 1003), (16, 512, 2048), (17, 128, 4096), (32, 131, 260),
         (33, 264, 136), (64, 640, 328), (100, 72, 1000), (127, 129, 65), (128, 256, 64), (129, 257, 63),
         (200, 136, 200), (256, 512, 512), (333, 777, 1001), (1030, 304, 520)]


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _forward_tol(ref, z_size, K, dtype, residual=None):
    size = z_size + (0 if residual is None else residual.to(F64).abs())
    return UNIT[dtype] * ref.abs() * 1.01 + TINY[dtype] + 1.13 * ((K + 4) * 2.0 ** -23 + 2.0 ** -20) * size


def _check_forward(sm, x, w, y, bias, residual, pre, act):
    r0 = residual.clone() if residual is not None else None
    sm.sym_linear(x, w, y, bias=bias, residual=residual, pre=pre, act=act)
    assert sm.sym_stream_status() == sm.SYM_OK, sm.sym_last_error()
    want, z, size = linear64(x, w, bias, r0, act)
    K = x.shape[1]
    close(y, want, _forward_tol(want, size, K, x.dtype, r0), "y")
    if pre is not None:
        close(pre, z, _forward_tol(z, size, K, x.dtype), "pre")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(symar, size, dtype):
    M, N, K = size
    t = DTYPES[dtype]
    x, w = _rand((M, K), t, 1), _rand((N, K), t, 2, K ** -0.5)
    bias, residual = _rand((N,), t, 3), _rand((M, N), t, 4)
    for i, act in enumerate(ACTS):
        y = torch.full((M, N), 7.0, device="cuda", dtype=t)
        pre = torch.full((M, N), 7.0, device="cuda", dtype=t) if i % 2 else None
        _check_forward(symar, x, w, y, bias if i != 1 else None, residual if i != 2 else None, pre, act)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_forward_strided_and_misaligned(symar, M, dtype):
    """Rows inside wider buffers, starting at odd elements; bytes outside the outputs stay as they are."""
    t, N, K = DTYPES[dtype], 150, 203
    for off, pad in [(0, 5), (8, 13), (1, 0), (3, 21), (8, 32)]:
        bx, bw = _rand((M, K + off + pad), t, 5), _rand((N, K + off + pad), t, 6, 0.1)
        by = torch.full((M, N + off + pad), 7.0, device="cuda", dtype=t)
        bp, br = by.clone(), _rand((M, N + off + pad), t, 7)
        x, w, y, p, r = (b[:, off:off + n] for b, n in [(bx, K), (bw, K), (by, N), (bp, N), (br, N)])
        _check_forward(symar, x, w, y, _rand((N + 1,), t, 8)[1:], r, p, "gelu")
        for b in (by, bp):
            assert (b[:, :off] == 7).all() and (b[:, off + N:] == 7).all()


def test_residual_in_place(symar):
    for M, N, K in [(1, 256, 128), (70, 300, 64), (260, 520, 72)]:
        x, w, y = _rand((M, K), torch.bfloat16, 1), _rand((N, K), torch.bfloat16, 2, 0.1), _rand((M, N), torch.bfloat16, 3)
        _check_forward(symar, x, w, y, None, y, None, "silu")


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_special_values_stay_in_their_rows_and_columns(symar, dtype):
    t, (M, N, K) = DTYPES[dtype], (130, 140, 96)
    x, w = _rand((M, K), t, 1), _rand((N, K), t, 2, 0.1)
    x[3, 5], x[129, 0], w[7, 9] = float("nan"), float("inf"), float("-inf")
    y = torch.empty(M, N, device="cuda", dtype=t)
    symar.sym_linear(x, w, y)
    want = x.to(F64) @ w.to(F64).t()
    assert torch.isnan(y[3]).all() and torch.equal(torch.isnan(y), torch.isnan(want))
    wild = torch.isinf(want)
    assert torch.equal(torch.isinf(y), wild) and torch.equal(y[wild].to(F64), want[wild])


def test_empty(symar):
    e = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    n = symar.sym_launch_count()
    symar.sym_linear(e(0, 8), e(5, 8), e(0, 5))
    symar.sym_linear(e(3, 8), e(0, 8), e(3, 0))
    assert symar.sym_launch_count() == n
    y, b, r = e(3, 5), _rand((5,), torch.bfloat16, 1), _rand((3, 5), torch.bfloat16, 2)
    symar.sym_linear(e(3, 0), e(5, 0), y, bias=b, residual=r, act="relu")
    assert torch.equal(y, (b.float().clamp(min=0) + r.float()).to(torch.bfloat16))
    dw, db = torch.full((5, 8), 3.0, device="cuda"), torch.full((5,), 3.0, device="cuda")
    symar.sym_linear_backward(e(0, 5), e(0, 8), e(5, 8), dw=dw, dbias=db, accumulate=True)
    assert (dw == 3).all() and (db == 3).all()
    symar.sym_linear_backward(e(0, 5), e(0, 8), e(5, 8), dx=e(0, 8), dw=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()
    dx = _rand((3, 8), torch.bfloat16, 4)
    symar.sym_linear_backward(e(3, 0), e(3, 8), e(0, 8), dx=dx, dw=e(0, 8), dbias=e(0))
    assert (dx == 0).all()                                   # a layer without outputs
    assert symar.sym_stream_status() == symar.SYM_OK


def _check_backward(sm, dy, x, w, pre, dx, dw, db, act, accumulate):
    M, K = x.shape
    N, t = w.shape[0], x.dtype
    dw0, db0 = (None if g is None else g.to(F64).clone() for g in (dw, db))
    sm.sym_linear_backward(dy, x, w, pre=pre, dx=dx, dw=dw, dbias=db, act=act, accumulate=accumulate)
    assert sm.sym_stream_status() == sm.SYM_OK, sm.sym_last_error()
    dz = dy.to(F64) * (slope64(pre.to(F64), act) if pre is not None else 1.0)
    slack = 2.0 ** -20 + (UNIT[t] if act != "none" else 0)   # dz's evaluation, and its rounding to the operand type
    size = dz.abs() + (dy.to(F64).abs() * 2.0 ** -20 + TINY[t] if act != "none" else 0)

    def tol(ref, sums, n, dtype, more=0):
        return UNIT[dtype] * 1.01 * ref.abs() + TINY[dtype] + (slack + (n + 4) * 2.0 ** -23) * sums * 1.01 + more

    if dx is not None:
        want = dz @ w.to(F64)
        close(dx, want, tol(want, size @ w.to(F64).abs(), N, t), "dx")
    evaluated = 2.0 ** -20 * (dy.to(F64).abs().t() @ x.to(F64).abs()) if dw is not None else 0
    if dw is not None:
        want = dz.t() @ x.to(F64) + (dw0 if accumulate else 0)
        close(dw, want, tol(want, size.t() @ x.to(F64).abs() + (dw0.abs() if accumulate else 0), M, dw.dtype, evaluated),
              "dw")
    if db is not None:
        want = dz.sum(0) + (db0 if accumulate else 0)
        sums = size.sum(0) + (db0.abs() if accumulate else 0)
        close(db, want, UNIT[db.dtype] * 1.01 * want.abs() + TINY[db.dtype] + ((M + 4) * 2.0 ** -23 + 2.0 ** -20) *
              (sums + dy.to(F64).abs().sum(0)), "dbias")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(symar, size, dtype):
    M, N, K = size
    t = DTYPES[dtype]
    dy, x, w = _rand((M, N), t, 1), _rand((M, K), t, 2), _rand((N, K), t, 3, K ** -0.5)
    pre = _rand((M, N), t, 4, 2.0)
    for i, act in enumerate(ACTS):
        gt = torch.float32 if i in (0, 3) else t
        dx = torch.full((M, K), 7.0, device="cuda", dtype=t)
        dw, db = _rand((N, K), gt, 5), _rand((N,), gt, 6)
        _check_backward(symar, dy, x, w, pre if act != "none" else None, dx, dw, db, act, accumulate=i >= 2)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_backward_strided_misaligned_and_partial(symar, dtype):
    t, M, N, K = DTYPES[dtype], 70, 150, 203
    for off, pad in [(1, 0), (3, 21), (8, 32)]:
        bufs = [_rand((r, c + off + pad), t, 10 + i) for i, (r, c) in
                enumerate([(M, N), (M, K), (N, K), (M, N), (M, K), (N, K)])]
        dy, x, w, pre, dx, dw = (b[:, off:b.shape[1] - pad] for b in bufs)
        edge = [b.clone() for b in bufs]
        _check_backward(symar, dy, x, w, pre, dx, dw, None, "silu", True)
        for b, e in zip(bufs, edge):
            assert torch.equal(b[:, :off], e[:, :off]) and torch.equal(b[:, b.shape[1] - pad:], e[:, e.shape[1] - pad:])
        db = torch.empty(N, device="cuda")
        _check_backward(symar, dy, x, w, pre, dx, None, None, "gelu", False)
        _check_backward(symar, dy, x, w, None, None, dw, None, "none", False)
        _check_backward(symar, dy, x, w, pre, None, None, db, "relu", False)


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(symar, act):
    """<dx, u> + <dw, v> + <db, s> against central differences of sum(c * y) in 64 bits, step 1e-5: their
    own error is below 1e-7 here, the kernel's 32-bit one below 1e-4 of the sums' size."""
    M, N, K, t = 9, 21, 34, torch.float32
    x, w, b = _rand((M, K), t, 1), _rand((N, K), t, 2, 0.2), _rand((N,), t, 3)
    c = _rand((M, N), t, 4)
    y, pre = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    symar.sym_linear(x, w, y, bias=b, pre=pre, act=act)
    dx, dw, db = (torch.empty_like(v) for v in (x, w, b))
    symar.sym_linear_backward(c, x, w, pre=pre, dx=dx, dw=dw, dbias=db, act=act)
    u, v, s = _rand((M, K), F64, 5), _rand((N, K), F64, 6), _rand((N,), F64, 7)

    def f(h):
        z = (x.to(F64) + h * u) @ (w.to(F64) + h * v).t() + b.to(F64) + h * s
        return (c.to(F64) * act64(z, act)).sum()

    want = (f(1e-5) - f(-1e-5)) / 2e-5
    got = (dx.to(F64) * u).sum() + (dw.to(F64) * v).sum() + (db.to(F64) * s).sum()
    size = (dx.to(F64) * u).abs().sum() + (dw.to(F64) * v).abs().sum() + (db.to(F64) * s).abs().sum()
    assert abs(want - got) < 1e-4 * size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_calls_give_equal_bits(symar, dtype):
    t, (M, N, K) = DTYPES[dtype], (48, 520, 4096)
    x, w, dy = _rand((M, K), t, 1), _rand((N, K), t, 2, 0.02), _rand((M, N), t, 3)
    seen = []
    for _ in range(5):
        y, dx, dw, db = (torch.empty(s, device="cuda", dtype=t) for s in [(M, N), (M, K), (N, K), (N,)])
        symar.sym_linear(x, w, y, act="gelu")
        symar.sym_linear_backward(dy, x, w, pre=y, dx=dx, dw=dw, dbias=db, act="gelu")
        seen.append((y, dx, dw, db))
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))


def test_other_stream_and_graph(symar):
    """Calls on a stream of their own, and captured: replays see the inputs of the moment."""
    M, N, K, t = 60, 300, 203, torch.bfloat16                # odd K: the call needs a workspace
    x, w = _rand((M, K), t, 1), _rand((N, K), t, 2, 0.1)
    y, dx, dw, db = (torch.empty(s, device="cuda", dtype=t) for s in [(M, N), (M, K), (N, K), (N,)])
    pre, dy = torch.empty(M, N, device="cuda", dtype=t), _rand((M, N), t, 3)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def step(**kw):
        symar.sym_linear(x, w, y, pre=pre, act="gelu", **kw)
        symar.sym_linear_backward(dy, x, w, pre=pre, dx=dx, dw=dw, dbias=db, act="gelu", **kw)

    step(stream=st)
    st.synchronize()
    first = [v.clone() for v in (y, dx, dw, db)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for v in (y, dx, dw, db):
        v.zero_()
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw, db)))
    x.copy_(_rand((M, K), t, 9))
    g.replay()
    want, _, size = linear64(x, w, act="gelu")
    close(y, want, _forward_tol(want, size, K, t), "replayed y")


def test_gradient_into_a_window_and_allreduce(symar):
    """dw written straight into each rank's send window, summed by the AllReduce in 32 bits."""
    R, M, N, K, t = 4, 50, 96, 72, torch.bfloat16
    w = _rand((N, K), t, 1)
    send, recv = symar.Window(R, N * K * 4), symar.Window(R, N * K * 4)
    try:
        want, size = 0, 0
        for r in range(R):
            x, dy = _rand((M, K), t, 10 + r), _rand((M, N), t, 20 + r)
            dw = send.tensor(torch.float32)[r, :N * K].view(N, K)
            symar.sym_linear_backward(dy, x, w, dw=dw)
            want, size = want + dy.to(F64).t() @ x.to(F64), size + dy.to(F64).abs().t() @ x.to(F64).abs()
        symar.sym_allreduce(send, recv, N * K)
        assert symar.sym_stream_status() == symar.SYM_OK
        for r in range(R):
            close(recv.tensor(torch.float32)[r, :N * K].view(N, K), want, (M + R + 4) * 2.0 ** -23 * size, "sum")
    finally:
        send.free()
        recv.free()


def test_refusals(symar):
    t = torch.bfloat16
    x, w, y = _rand((4, 8), t, 1), _rand((6, 8), t, 2), torch.empty(4, 6, device="cuda", dtype=t)
    bad = [dict(w=w.float()), dict(w=w[:, :7]), dict(y=y[:, :5]), dict(y=y.float()), dict(x=x.cpu()),
           dict(x=_rand((8, 4), t, 3).t()), dict(x=x.double()), dict(bias=x[0]), dict(residual=y[:3])]
    n = symar.sym_launch_count()
    for b in bad:
        with pytest.raises((ValueError, symar.SymError)):
            symar.sym_linear(**{**dict(x=x, w=w, y=y), **b})
    big = torch.empty(64, device="cuda", dtype=t)
    with pytest.raises(symar.SymError):                      # y over x
        symar.sym_linear(big[:32].view(4, 8), w, big[16:40].view(4, 6))
    with pytest.raises(symar.SymError):                      # y shifted over the residual
        symar.sym_linear(x, w, big[:24].view(4, 6), residual=big[6:30].view(4, 6))
    with pytest.raises(ctypes.ArgumentError):
        symar.sym_linear(x, w, y, act="tanh")
    dw = torch.empty(6, 8, device="cuda", dtype=t)
    with pytest.raises(symar.SymError):                      # the activation's gradient needs pre
        symar.sym_linear_backward(y, x, w, dw=dw, act="relu")
    with pytest.raises(ValueError):
        symar.sym_linear_backward(y, x, w, dw=dw, dbias=torch.empty(6, device="cuda"))
    with pytest.raises(symar.SymError):                      # too small a workspace
        symar.sym_linear_backward(y, x, w, pre=y.clone(), dw=dw, act="relu",
                                  workspace=torch.empty(16, device="cuda", dtype=torch.uint8))
    assert symar.sym_launch_count() == n
