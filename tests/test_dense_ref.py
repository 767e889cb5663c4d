"""CPU checks behind the dense operators' tests: the plain 64-bit gradients
against central differences of the plain forwards, the optimiser's rounding
rules against their definitions, and the C ABI's refusals (host checks: no
kernel runs)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import dense_ref as R


def _differences(fn, x, dout, h=1e-5):
    """d <fn(x), dout> / dx by central differences."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = ((fn(a) - fn(b)) * dout).sum() / (2 * h)
    return g


# central differences of O(1) smooth functions at h = 1e-5: the third
# derivative's term is h^2 / 6 = 2e-11, the rounding of fn about 1e-15 / h =
# 1e-10 times the sum's size; 1e-7 leaves two orders
FD = dict(rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("T,d", [(1, 1), (3, 5), (2, 8)])
def test_rmsnorm_backward_is_the_derivative(T, d):
    rng = np.random.default_rng(T * 10 + d)
    s, w, dy = rng.standard_normal((T, d)), rng.standard_normal(d), rng.standard_normal((T, d))
    eps = 1e-2
    _, rstd = R.rmsnorm(s, w, eps)
    ds, dw = R.rmsnorm_backward(dy, s, w, rstd)
    np.testing.assert_allclose(ds, _differences(lambda a: R.rmsnorm(a, w, eps)[0], s, dy), **FD)
    np.testing.assert_allclose(dw, _differences(lambda a: R.rmsnorm(s, a, eps)[0], w, dy), **FD)


@pytest.mark.parametrize("T,d,f", [(1, 4, 3), (3, 2, 5)])
def test_ffn_backward_is_the_derivative(T, d, f):
    rng = np.random.default_rng(T + d)
    x, w1, w2, dy = (rng.standard_normal(k) for k in ((T, d), (2 * f, d), (d, f), (T, d)))
    _, h, gu = R.ffn(x, w1, w2)
    dx, dw1, dw2, _ = R.ffn_backward(dy, x, gu, h, w1, w2)
    np.testing.assert_allclose(dx, _differences(lambda a: R.ffn(a, w1, w2)[0], x, dy), **FD)
    np.testing.assert_allclose(dw1, _differences(lambda a: R.ffn(x, a, w2)[0], w1, dy), **FD)
    np.testing.assert_allclose(dw2, _differences(lambda a: R.ffn(x, w1, a)[0], w2, dy), **FD)


def test_state_exponent_is_the_smallest_that_holds_the_block():
    a = np.concatenate([np.exp2(np.random.default_rng(1).uniform(-100, 100, 2000)), [448.0, 448.0 * (1 + 2e-16), 1.75,
                                                                                     np.nextafter(1.75, 2), 2.0]])
    e = R.state_exponent(a)
    assert np.all(a <= 448 * np.exp2(e)) and np.all(a > 448 * np.exp2(e - 1))
    assert R.state_exponent(np.array([0.0]))[0] == -127


def test_random_rounding_lands_on_the_neighbouring_codes_in_proportion():
    grid = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    grid = np.unique(grid[np.isfinite(grid)])
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.uniform(-448, 448, 500), rng.uniform(-0.05, 0.05, 500), [0.0, 448.0, 2.0 ** -6, 2.0 ** -9]])
    x = x.astype(np.float32).astype(np.float64)
    every = np.arange(65536, dtype=np.uint64)
    for v in x:
        got = R.e4m3_random(np.full(65536, v), every)
        lo, hi = grid[grid <= v].max(), grid[grid >= v].min()
        assert set(np.unique(got)) <= {lo, hi}, v
        # over all 2^16 values of the bits the mean is v, but for the value's own bits below them (one part in 2^16)
        assert abs(got.mean() - v) <= (hi - lo) * 2.0 ** -15
    b = R.bf16_random(np.full(65536, np.float32(0.3)), every)
    assert abs(b.mean() - np.float32(0.3)) <= 2.0 ** -9 * 2.0 ** -15 and len(np.unique(b)) == 2


def test_random_bits_are_spread():
    r = R.random_bits(7, 12, 3, 1 << 16)
    # 2^16 draws: each of the 32 bits is set 2^15 times within 5 standard deviations (128 each)
    for k in range(32):
        assert abs(int(((r >> np.uint64(k)) & np.uint64(1)).sum()) - (1 << 15)) <= 5 * 128, k
    assert not np.array_equal(r, R.random_bits(7, 13, 3, 1 << 16))
    assert not np.array_equal(r, R.random_bits(7, 12, 4, 1 << 16))
    assert not np.array_equal(r, R.random_bits(8, 12, 3, 1 << 16))


# ------------------------------------------------------------------ refusals

OK, INVALID, UNSUPPORTED, ALIGN, WS = 0, 1, 2, 3, 4
FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    from dropless_moe_expert_amd import build, ops
    if not os.path.exists(ops.LIB_PATH):
        build.build()
    return ops.load_library(require_gpu=False)


def _norm(L, **k):
    a = dict(x=FAKE, ldx=64, w=FAKE, wt=0, r=None, rt=0, ldr=0, s=None, lds=0, T=4, d=64, eps=1e-6, y=FAKE, q=None,
             qs=None, rstd=None)
    a.update(k)
    return L.moe_add_rmsnorm(*a.values(), None)


def test_norm_refusals(L):
    assert _norm(L, T=0) == OK
    assert _norm(L, T=-1) == INVALID
    assert _norm(L, d=0) == INVALID
    assert _norm(L, eps=-1.0) == INVALID and _norm(L, eps=float("nan")) == INVALID
    assert _norm(L, d=32769, ldx=32769) == UNSUPPORTED
    assert _norm(L, T=1 << 31) == UNSUPPORTED
    assert _norm(L, x=None) == INVALID and _norm(L, w=None) == INVALID
    assert _norm(L, y=None) == INVALID                               # no output
    assert _norm(L, q=FAKE) == INVALID and _norm(L, qs=FAKE) == INVALID   # codes without scales
    assert _norm(L, q=FAKE, qs=FAKE, d=48) == UNSUPPORTED
    assert _norm(L, r=FAKE, ldr=64) == INVALID                        # a residual needs s
    assert _norm(L, s=FAKE, lds=64) == INVALID                        # and s a residual
    assert _norm(L, r=FAKE, ldr=64, s=FAKE, lds=32) == INVALID
    assert _norm(L, ldx=63) == INVALID
    assert _norm(L, wt=2) == UNSUPPORTED and _norm(L, r=FAKE, rt=5, ldr=64, s=FAKE, lds=64) == UNSUPPORTED
    assert _norm(L, x=FAKE + 1) == ALIGN and _norm(L, rstd=FAKE + 2) == ALIGN
    assert _norm(L, r=FAKE + 2, rt=1, ldr=64, s=FAKE, lds=64) == ALIGN
    # codes are written by the 16-byte path alone
    assert _norm(L, q=FAKE, qs=FAKE, x=FAKE + 2) == ALIGN
    assert _norm(L, q=FAKE, qs=FAKE, ldx=65) == ALIGN
    assert _norm(L, q=FAKE + 4, qs=FAKE) == ALIGN


def _norm_bwd(L, **k):
    a = dict(dy=FAKE, lddy=64, s=FAKE, st=0, lds=64, w=FAKE, wt=0, rstd=FAKE, dres=None, lddres=0, T=4, d=64, dx=FAKE,
             ds=None, dw=FAKE, ws=FAKE, n=1 << 30)
    a.update(k)
    return L.moe_add_rmsnorm_backward(*a.values(), None)


def test_norm_backward_refusals(L):
    for name in ("dy", "s", "w", "rstd", "dx", "dw"):
        assert _norm_bwd(L, **{name: None}) == INVALID, name
    assert _norm_bwd(L, T=-1) == INVALID and _norm_bwd(L, d=0) == INVALID
    assert _norm_bwd(L, st=1) == INVALID and _norm_bwd(L, ds=FAKE) == INVALID    # ds with fp32 s, and only then
    assert _norm_bwd(L, lddy=63) == INVALID and _norm_bwd(L, dres=FAKE, lddres=1) == INVALID
    assert _norm_bwd(L, d=40000, lddy=40000, lds=40000) == UNSUPPORTED
    assert _norm_bwd(L, st=3) == UNSUPPORTED
    assert _norm_bwd(L, dx=FAKE + 1) == ALIGN
    need = L.moe_add_rmsnorm_backward_workspace_bytes(4, 64)
    assert need >= 4 * 64 * 4
    assert _norm_bwd(L, n=need - 1) == WS and _norm_bwd(L, ws=None) == WS and _norm_bwd(L, ws=FAKE + 64) == ALIGN
    assert L.moe_add_rmsnorm_backward_workspace_bytes(-1, 64) == 0
    assert L.moe_add_rmsnorm_backward_workspace_bytes(1 << 30, 32768) == 512 * 32768 * 4


def _ffn(L, **k):
    a = dict(x=FAKE, ldx=64, w1=FAKE, w2=FAKE, res=None, ldr=0, T=4, d=64, f=32, h=None, gu=None, y=2 * FAKE, ws=FAKE,
             n=1 << 40)
    a.update(k)
    return L.moe_gated_ffn(*a.values(), None)


def test_ffn_refusals(L):
    assert _ffn(L, T=0) == OK
    for name in ("x", "w1", "w2", "y"):
        assert _ffn(L, **{name: None}) == INVALID, name
    assert _ffn(L, T=-1) == INVALID and _ffn(L, d=0) == INVALID and _ffn(L, f=0) == INVALID
    assert _ffn(L, d=60, ldx=60) == UNSUPPORTED and _ffn(L, f=12) == UNSUPPORTED
    assert _ffn(L, d=1 << 15, ldx=1 << 15, f=1 << 15) == UNSUPPORTED     # the weight's offsets pass 32 bits
    assert _ffn(L, gu=FAKE) == INVALID                                    # pre-activations without h
    assert _ffn(L, y=FAKE) == INVALID                                     # onto x
    assert _ffn(L, ldx=56) == INVALID and _ffn(L, res=FAKE, ldr=8) == INVALID
    assert _ffn(L, res=2 * FAKE, ldr=72) == INVALID                       # in place at another pitch
    assert _ffn(L, ldx=(1 << 23) + 8) == UNSUPPORTED and _ffn(L, res=FAKE, ldr=1 << 24) == UNSUPPORTED
    assert _ffn(L, ldx=65) == ALIGN and _ffn(L, res=FAKE, ldr=68) == ALIGN
    for name in ("x", "w1", "w2", "res", "y"):
        assert _ffn(L, **{"ldr": 64, name: 2 * FAKE + 8}) == ALIGN, name
    need = L.moe_gated_ffn_workspace_bytes(4, 64, 32, 0, 0)
    assert need >= 256 + 4 * 32 * 2
    assert _ffn(L, n=need - 1) == WS and _ffn(L, ws=None) == WS and _ffn(L, ws=FAKE + 16) == ALIGN
    assert L.moe_gated_ffn_workspace_bytes(4, 60, 32, 0, 0) == 0


def _ffn_bwd(L, **k):
    a = dict(dy=FAKE, x=FAKE, gu=FAKE, h=FAKE, w1=FAKE, w2=FAKE, T=4, d=64, f=32, dt=0, dgu=FAKE, dx=FAKE, dw1=FAKE,
             dw2=FAKE, ws=FAKE, n=1 << 40)
    a.update(k)
    return L.moe_gated_ffn_backward(*a.values(), None)


def test_ffn_backward_refusals(L):
    for name in ("dy", "x", "gu", "h", "w1", "w2", "dgu", "dx", "dw1", "dw2"):
        assert _ffn_bwd(L, **{name: None}) == INVALID, name
        assert _ffn_bwd(L, **{name: FAKE + 8}) == ALIGN, name
    assert _ffn_bwd(L, d=60) == UNSUPPORTED and _ffn_bwd(L, f=12) == UNSUPPORTED and _ffn_bwd(L, dt=4) == UNSUPPORTED
    assert _ffn_bwd(L, T=-1) == INVALID and _ffn_bwd(L, T=1 << 31) == UNSUPPORTED
    need = L.moe_gated_ffn_backward_workspace_bytes(4, 64, 32)
    assert need >= 256 and L.moe_gated_ffn_backward_workspace_bytes(4, 60, 32) == 0
    assert _ffn_bwd(L, n=need - 1) == WS and _ffn_bwd(L, ws=FAKE + 16) == ALIGN


def _adamw(L, step=FAKE, gs=None, count=None, **k):
    from dropless_moe_expert_amd import ops
    t = dict(p=FAKE, master=0, g=FAKE, m=FAKE, v=FAKE, ms=0, vs=0, n=100)
    c = dict(lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, bits=32, pt=0, gt=0, seed=0)
    for key, val in k.items():
        (t if key in t else c)[key] = val
    cfg = ops.AdamwConfig(*c.values())
    table = (ctypes.c_int64 * 8)(*[x or 0 for x in t.values()])
    return L.moe_adamw_step(table, 1 if count is None else count, ctypes.byref(cfg), step, gs, None)


def test_adamw_refusals(L):
    for name in ("p", "g", "m", "v"):
        assert _adamw(L, **{name: 0}) == INVALID, name
    assert _adamw(L, step=None) == INVALID and _adamw(L, count=-1) == INVALID
    assert _adamw(L, n=-1) == INVALID and _adamw(L, n=1 << 40) == UNSUPPORTED
    for bad in (dict(b1=1.0), dict(b2=1.0), dict(b1=-0.1), dict(eps=-1.0), dict(lr=float("nan")), dict(b2=float("nan")),
                dict(wd=float("inf")), dict(eps=float("inf"))):
        assert _adamw(L, **bad) == INVALID, bad
    assert _adamw(L, bits=16) == UNSUPPORTED and _adamw(L, pt=2) == UNSUPPORTED and _adamw(L, gt=-1) == UNSUPPORTED
    assert _adamw(L, bits=8) == INVALID                       # 8-bit states without scales
    assert _adamw(L, pt=1, master=FAKE) == INVALID            # a master of an fp32 weight
    assert _adamw(L, p=FAKE + 1) == ALIGN and _adamw(L, gt=1, g=FAKE + 2) == ALIGN and _adamw(L, m=FAKE + 2) == ALIGN
    assert _adamw(L, step=FAKE + 2) == ALIGN and _adamw(L, gs=FAKE + 1) == ALIGN
    # one of two entries with a master copy
    from dropless_moe_expert_amd import ops
    cfg = ops.AdamwConfig(1e-3, 0.9, 0.99, 1e-8, 0.1, 32, 0, 0, 0)
    two = (ctypes.c_int64 * 16)(FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, 8, FAKE, 0, FAKE, FAKE, FAKE, 0, 0, 8)
    assert L.moe_adamw_step(two, 2, ctypes.byref(cfg), FAKE, None, None) == INVALID
