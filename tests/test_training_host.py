"""Host-side argument checks of the training operators' C entries: no GPU, nothing is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from symmetric_memory_allreduce_gb300 import build

    build.build()
    from symmetric_memory_allreduce_gb300 import _binding

    return _binding.load()


A = 1 << 20            # addresses that are only looked at


def _linear(lib, **kw):
    a = dict(x=A, ldx=64, w=2 * A, ldw=64, bias=None, residual=None, ldr=64, y=3 * A, ldy=64, pre=None, ldp=64, M=8,
             N=64, K=64, dtype=1, act=0, ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.sym_linear(*a.values())


def test_linear_refusals(lib):
    for kw in [dict(x=None), dict(w=None), dict(y=None), dict(dtype=3), dict(act=4), dict(act=-1), dict(ldx=63), dict(ldw=1),
               dict(ldy=63), dict(residual=4 * A, ldr=63), dict(pre=4 * A, ldp=3), dict(x=A + 1), dict(y=3 * A + 1),
               dict(y=A + 16), dict(y=2 * A), dict(pre=3 * A + 64), dict(residual=3 * A + 2), dict(bias=3 * A + 128),
               dict(wsb=16)]:
        assert _linear(lib, **kw) == 1, kw
    for kw in [dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31)]:
        assert _linear(lib, **kw) == 5, kw
    assert _linear(lib, M=0) == 0 and _linear(lib, N=0) == 0
    assert lib.sym_launch_count() == 0


def test_linear_workspace_covers_unaligned_rows(lib):
    f = lib.sym_linear_workspace
    assert f(A, 64, 2 * A, 64, 100, 100, 64, 1) == 0
    assert f(A, 64, 2 * A, 64, 100, 100, 64, 0) == 0
    assert f(A, 64, 2 * A, 64, 0, 100, 64, 1) == 0
    assert f(A + 2, 64, 2 * A, 64, 100, 50, 64, 1) >= 100 * 64 * 2      # x at an odd element
    assert f(A, 65, 2 * A, 65, 100, 50, 65, 2) >= (100 + 50) * 72 * 2   # odd rows, both padded to 72
    assert f(A + 4, 65, 2 * A, 65, 100, 50, 65, 0) == 0
    assert _linear(lib, ldx=65, ws=None) == 1
    assert _linear(lib, ldx=65, ws=9 * A + 8, wsb=1 << 20) == 1
    assert _linear(lib, ldx=65, ws=A + 256, wsb=1 << 20) == 1           # over x


def _backward(lib, **kw):
    a = dict(dy=A, lddy=64, x=2 * A, ldx=64, w=3 * A, ldw=64, pre=None, ldp=64, dx=4 * A, lddx=64, dw=5 * A, lddw=64,
             dbias=6 * A, M=8, N=64, K=64, dtype=1, gdtype=1, act=0, acc=0, ws=8 * A, wsb=1 << 22, stream=None)
    a.update(kw)
    return lib.sym_linear_backward(*a.values())


def test_linear_backward_refusals(lib):
    for kw in [dict(dy=None), dict(x=None), dict(w=None), dict(act=1), dict(dtype=7), dict(gdtype=2), dict(gdtype=5),
               dict(lddy=63), dict(lddx=63), dict(lddw=63), dict(dx=4 * A + 1), dict(gdtype=0, dw=5 * A + 2),
               dict(ws=None), dict(ws=8 * A + 8), dict(dx=A), dict(dw=4 * A + 64), dict(dbias=5 * A),
               dict(act=1, pre=7 * A, wsb=0), dict(act=1, pre=7 * A, ws=4 * A)]:
        assert _backward(lib, **kw) == 1, kw
    assert _backward(lib, M=1 << 31) == 5
    assert _backward(lib, dx=None, dw=None, dbias=None) == 0
    need = lambda act, ld=64: lib.sym_linear_backward_workspace(A, ld, 2 * A, 64, 3 * A, 64, 8, 64, 64, 1, act)  # noqa: E731
    assert need(1) >= 8 * 64 * 2 and need(0) == 0
    assert need(0, 65) >= need(0) + 8 * 64 * 2 and need(1, 65) == need(1)
    assert lib.sym_launch_count() == 0


def _policy(lib, **kw):
    a = dict(logits=A, ld=100, T=4, V=100, dtype=1, targets=2 * A, old=3 * A, ref=None, adv=4 * A, weights=None, lo=0.2,
             hi=0.2, kl=0.0, temp=1.0, stats=5 * A, logp=6 * A, lse=7 * A, d=None, ldd=100, go=None, stream=None)
    a.update(kw)
    return lib.sym_policy_loss(*a.values())


def test_policy_refusals(lib):
    for kw in [dict(logits=None), dict(targets=None), dict(old=None), dict(adv=None), dict(stats=None), dict(logp=None),
               dict(lse=None), dict(ld=99), dict(V=0), dict(dtype=3), dict(lo=-1.0), dict(hi=float("nan")), dict(temp=0.0),
               dict(temp=-1.0), dict(kl=float("nan")), dict(logits=A + 1), dict(targets=2 * A + 4), dict(old=3 * A + 2),
               dict(d=8 * A, ldd=99), dict(d=A + 200), dict(d=A, ldd=104)]:
        assert _policy(lib, **kw) == 1, kw
    assert _policy(lib, T=1 << 31) == 5
    assert lib.sym_policy_loss_backward(A, 100, 4, 100, 1, 2 * A, 3 * A, None, 4 * A, None, 0.2, 0.2, 0.0, 1.0, 6 * A, 7 * A,
                                        None, 100, None, None) == 1
    assert lib.sym_launch_count() == 0


def test_adamw_refusals(lib):
    h = ctypes.c_void_p(5)
    one = (ctypes.c_size_t * 1)(16)
    ok = (ctypes.c_void_p * 1)(A)
    odd = (ctypes.c_void_p * 1)(A + 2)
    nul = (ctypes.c_void_p * 1)(None)

    def create(counts=one, p=ok, g=ok, m=ok, v=ok, ms=None, vs=None, c=None, pt=0, gt=0, ct=0):
        return lib.sym_adamw_create(1, counts, p, g, m, v, ms, vs, c, pt, gt, ct, ctypes.byref(h))

    assert create(counts=None) == 1 and h.value is None
    for kw in [dict(p=nul), dict(g=nul), dict(m=nul), dict(v=nul), dict(c=nul), dict(ms=ok), dict(vs=ok), dict(pt=3), dict(gt=9),
               dict(ct=-1), dict(p=odd), dict(m=odd), dict(ms=nul, vs=ok), dict(c=odd)]:
        assert create(**kw) == 1, kw
    assert create(counts=(ctypes.c_size_t * 1)((1 << 42) + 1)) == 5
    assert lib.sym_adamw_create(1, one, ok, ok, ok, ok, None, None, None, 0, 0, 0, None) == 1
    assert lib.sym_adamw_step(None, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, None, 0, None) == 1
    assert lib.sym_grad_norm(None, 1.0, A, None) == 1
    assert lib.sym_adamw_free(None) == 0
    assert lib.sym_launch_count() == 0
