"""The dense operators around the layer on the GPU (norm, gated feed-forward
block, optimiser step) against plain 64-bit forms, element by element.

Bounds: a rounding to a type is off by at most half a step (dense_ref.ULP*,
relative); an fp32 sum of n terms by n * 2^-24 of the sum of their magnitudes;
hardware exp, reciprocal and their kin by a few fp32 steps, counted as 16."""
import numpy as np
import pytest
import torch

import dense_ref as R
from dense_ref import ULP16, ULP32, f64
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from dropless_moe_expert_amd import ops as _ops
    _ops.load_library()
    return _ops


def _t(rng, shape, dtype=torch.bfloat16, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype).cuda()


def _pitched(t, ld, shift=0):
    """t's values as rows of pitch ld that start `shift` elements into a buffer."""
    T, d = t.shape
    buf = torch.zeros(T * ld + shift, dtype=t.dtype, device=t.device)
    v = buf[shift:shift + T * ld].view(T, ld)[:, :d]
    v.copy_(t)
    return v


def _within(got, ref, bound, what):
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - ref)[bad].max()), np.argwhere(bad)[:3].tolist())


def _bits_equal(a, b, what):
    n = a.element_size()
    it = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[n]
    assert a.shape == b.shape and torch.equal(a.contiguous().view(it), b.contiguous().view(it)), what


# ------------------------------------------------------------------ norm

def _check_norm(ops, x, w, r, eps, mxfp8=False, **kw):
    o = ops.add_rmsnorm(x, w, r, eps=eps, mxfp8=mxfp8, keep_rstd=True, **kw)
    torch.cuda.synchronize()
    if r is None:
        assert o["s"] is x
    else:
        s = f64(x) + f64(r)
        # the fp32 sum, then (bf16) the stored rounding
        _within(o["s"], s, (ULP32 + (ULP16 if r.dtype == torch.bfloat16 else 0)) * np.abs(s) * (1 + ULP16), "s")
    d = x.shape[1]
    y, rstd = R.rmsnorm(f64(o["s"]), f64(w), eps)
    # a thread sums at most 32 squares, then 6 + 16 partial sums: 54 steps,
    # halved by the square root; its division, root and product a step each
    n = (54 / 2 + 4) * ULP32
    _within(o["rstd"], rstd, n * rstd, "rstd")
    _within(o["y"], y, (ULP16 + (n + 2 * ULP32) * (1 + ULP16)) * np.abs(y) + 2.0 ** -133, "y")
    if mxfp8:
        q, sc = ops.mxfp8_quantize(o["y"], 0)
        _bits_equal(o["q"], q, "codes")
        _bits_equal(o["scale"], sc, "scales")
        only = ops.add_rmsnorm(x, w, r, eps=eps, bf16=False, mxfp8=True)
        assert only["y"] is None and only["rstd"] is None
        _bits_equal(only["q"], q, "codes alone")
        _bits_equal(only["scale"], sc, "scales alone")
    return o


@pytest.mark.parametrize("T,d", [(1, 1), (1, 7168), (3, 7), (5, 32), (2, 511), (1025, 40), (7, 1023), (1500, 96),
                                 (3, 2048), (1100, 2048), (1030, 4096), (2, 4104), (1029, 7168), (1, 8200), (2, 8191),
                                 (1, 32768), (1, 32767), (1027, 8448), (64, 65), (1026, 1000)])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
def test_add_rmsnorm(ops, T, d, res):
    say("add_rmsnorm", T, d, res)
    rng = np.random.default_rng(T * 7 + d)
    x = _t(rng, (T, d), scale=3.0)
    r = None if res is None else _t(rng, (T, d), res, 2.0)
    w = _t(rng, (d,), torch.float32 if T % 2 else torch.bfloat16)
    _check_norm(ops, x, w, r, 1e-5, mxfp8=d % 32 == 0)


def test_add_rmsnorm_pitch_alignment_and_place(ops):
    rng = np.random.default_rng(5)
    x, w = _t(rng, (9, 256)), _t(rng, (256,))
    for res in (torch.bfloat16, torch.float32):
        r = _t(rng, (9, 256), res)
        want = _check_norm(ops, x, w, r, 1e-6, mxfp8=True)
        for ld, shift in ((264, 0), (256 + 32, 8), (259, 0), (256, 1), (300, 3)):
            say("add_rmsnorm pitch", res, ld, shift)
            xs, rs = _pitched(x, ld, shift), _pitched(r, ld, shift)
            got = _check_norm(ops, xs, w, rs, 1e-6)
            _bits_equal(got["s"], want["s"], "s")
            # in place: the residual's rows, nothing beside them
            whole = rs.clone()
            pad_before = torch.as_strided(rs, (9, ld), (ld, 1), rs.storage_offset())[:8, 256:].clone()
            o = ops.add_rmsnorm(xs, w, rs, eps=1e-6, out_s=rs)
            assert o["s"] is rs
            _bits_equal(rs, want["s"], "in place")
            _bits_equal(o["y"], got["y"], "y, in place")
            assert torch.equal(torch.as_strided(rs, (9, ld), (ld, 1), rs.storage_offset())[:8, 256:], pad_before)
            rs.copy_(whole)
    say("add_rmsnorm codes refuse odd pitches")
    with pytest.raises(ops.MoeError):
        ops.add_rmsnorm(_pitched(x, 259), w, mxfp8=True)


def test_add_rmsnorm_special_values(ops):
    rng = np.random.default_rng(6)
    x, w = _t(rng, (6, 64)), _t(rng, (64,))
    x[1] = 0                     # an empty row: y = 0, whatever eps is
    x[2, 5] = float("nan")
    x[3, 40] = float("inf")
    x[4] = 1e-30                 # squares below fp32's range: eps decides
    o = ops.add_rmsnorm(x, w, eps=1e-6, mxfp8=True, keep_rstd=True)
    q, sc = ops.mxfp8_quantize(o["y"], 0)
    _bits_equal(o["scale"], sc, "scales")
    assert torch.isnan(o["y"][2]).all() and (o["scale"][2] == 255).all()
    assert torch.isnan(o["y"][3, 40]) and (o["y"][3, :40] == 0).all()
    assert (o["y"][1] == 0).all() and (o["scale"][1] == 0).all()
    assert abs(float(o["rstd"][4]) - 1e3) < 1e-3
    for i in (0, 1, 4, 5):
        _bits_equal(o["q"][i], q[i], "codes")
    # eps 0 and an empty row: 0 * inf
    assert torch.isnan(ops.add_rmsnorm(x, w, eps=0.0)["y"][1]).all()
    # no rows
    e = ops.add_rmsnorm(x[:0], w, mxfp8=True, keep_rstd=True)
    assert e["y"].shape == (0, 64) and e["scale"].shape == (0, 2) and e["rstd"].shape == (0,)


def _check_norm_bwd(ops, dy, s, w, rstd, dres):
    o = ops.add_rmsnorm_backward(dy, s, w, rstd, dresidual=dres)
    torch.cuda.synchronize()
    T, d = dy.shape
    D, S, W, K = f64(dy), f64(s), f64(w), f64(rstd)
    DR = None if dres is None else f64(dres)
    ds, dw = R.rmsnorm_backward(D, S, W, K, DR)
    xh = S * K[:, None]
    mag = np.abs(W * D)
    # the row's mean of w dy xh: 3 roundings a term, 32 + 6 + 16 additions
    c = (np.abs(W * D * xh)).mean(-1, keepdims=True)
    b = ULP32 * (K[:, None] * (6 * mag + (54 + 10) * np.abs(xh) * c) + (0 if DR is None else 2 * np.abs(ds)))
    if s.dtype == torch.float32:
        _within(o["ds"], ds, b, "ds")
    else:
        assert o["ds"] is o["dx"]
    _within(o["dx"], ds, b * (1 + ULP16) + ULP16 * np.abs(ds) + 2.0 ** -133, "dx")
    # columns: the rows of one of at least min(T, 512) workgroups in turn, then up to 32 + 64 + 32 partial sums
    n = -(-T // min(T, 512)) + 130 if T else 0
    _within(o["dweight"], dw, n * ULP32 * np.abs(D * xh).sum(0), "dweight")
    return o


@pytest.mark.parametrize("T,d", [(1, 1), (1, 7168), (3, 7), (515, 64), (2, 511), (1025, 40), (2049, 512), (7, 1023),
                                 (1500, 96), (600, 2048), (513, 4096), (2, 4104), (520, 7168), (1, 8200), (2, 8191),
                                 (1, 32768), (2, 32767), (700, 65), (0, 128)])
@pytest.mark.parametrize("st", [torch.bfloat16, torch.float32])
def test_add_rmsnorm_backward(ops, T, d, st):
    say("add_rmsnorm_backward", T, d, st)
    rng = np.random.default_rng(T * 5 + d)
    s, dy = _t(rng, (T, d), st, 2.0), _t(rng, (T, d))
    w = _t(rng, (d,), torch.float32 if T % 2 else torch.bfloat16)
    rstd = torch.rsqrt(s.float().square().mean(-1) + 1e-6)
    for dres in (None, _t(rng, (T, d), st)):
        o = _check_norm_bwd(ops, dy, s, w, rstd, dres)
        again = ops.add_rmsnorm_backward(dy, s, w, rstd, dresidual=dres)
        for k in ("dx", "ds", "dweight"):
            _bits_equal(o[k], again[k], k)


def test_add_rmsnorm_backward_pitch(ops):
    rng = np.random.default_rng(8)
    for st in (torch.bfloat16, torch.float32):
        s, dy, dr, w = _t(rng, (33, 136), st), _t(rng, (33, 136)), _t(rng, (33, 136), st), _t(rng, (136,))
        rstd = torch.rsqrt(s.float().square().mean(-1) + 1e-6)
        for ld, shift in ((144, 0), (136, 8), (141, 0), (136, 3)):
            say("add_rmsnorm_backward pitch", st, ld, shift)
            _check_norm_bwd(ops, _pitched(dy, ld, shift), _pitched(s, ld, shift), w, rstd, _pitched(dr, ld, shift))


# ------------------------------------------------------------------ gated block

def _ffn_inputs(T, d, f, seed):
    rng = np.random.default_rng(seed)
    return _t(rng, (T, d)), _t(rng, (2 * f, d), scale=d ** -0.5), _t(rng, (d, f), scale=f ** -0.5), _t(rng, (T, d))


def _check_ffn(ops, x, w1, w2, res):
    y, saved = ops.gated_ffn(x, w1, w2, res, keep=True)
    torch.cuda.synchronize()
    d, f = w2.shape
    X, W1, W2 = f64(x), f64(w1), f64(w2)
    _, h, gu = R.ffn(X, W1, W2)
    e = d * ULP32 * (np.abs(X) @ np.abs(W1).T) + 2.0 ** -126
    _within(saved["gu"], gu, ULP16 * np.abs(gu) + e * (1 + ULP16), "gu")
    # |silu'| <= 1.1; exp, reciprocal and two products
    eg, eu, g, u = e[:, :f], e[:, f:], gu[:, :f], gu[:, f:]
    eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(R.silu(g)) * eu + 16 * ULP32 * np.abs(h)
    _within(saved["h"], h, ULP16 * np.abs(h) + eh * (1 + ULP16) + 2.0 ** -126, "h")
    H = f64(saved["h"])
    yr = H @ W2.T
    mag = np.abs(H) @ np.abs(W2).T
    if res is not None:
        yr = yr + f64(res)
        mag = mag + np.abs(f64(res))
    ey = (f + 2) * ULP32 * mag
    _within(y, yr, ULP16 * np.abs(yr) + ey * (1 + ULP16) + 2.0 ** -126, "y")
    # without the kept tensors: the same product of an h within its own bound
    alone = ops.gated_ffn(x, w1, w2, res)
    torch.cuda.synchronize()
    slack = (2 * (ULP16 * np.abs(h) + eh * (1 + ULP16) + 2.0 ** -126)) @ np.abs(W2).T
    _within(alone, yr, ULP16 * np.abs(yr) + (ey + slack) * (1 + ULP16) + 2.0 ** -126, "y alone")
    return y, saved, alone


FFN_SIZES = [(1, 8, 8), (1, 64, 8), (1, 512, 256), (2, 72, 40), (15, 264, 136), (16, 1024, 96), (17, 8, 8), (17, 72, 40),
             (33, 520, 264), (63, 200, 72), (64, 128, 64), (65, 1032, 200), (100, 2048, 768), (129, 136, 1032),
             (200, 264, 72), (255, 64, 64), (300, 4096, 64), (1000, 256, 520), (6200, 640, 1024), (4200, 3008, 64), (8, 2048, 8704),
             (5, 4104, 4096), (1500, 2056, 1032)]


@pytest.mark.parametrize("T,d,f", FFN_SIZES)
@pytest.mark.parametrize("with_res", [False, True])
def test_gated_ffn(ops, T, d, f, with_res):
    say("gated_ffn", T, d, f, with_res)
    x, w1, w2, r = _ffn_inputs(T, d, f, T + d + f)
    res = r if with_res else None
    y, saved, alone = _check_ffn(ops, x, w1, w2, res)
    y2, saved2 = ops.gated_ffn(x, w1, w2, res, keep=True)
    _bits_equal(y, y2, "the same call twice")
    _bits_equal(saved["h"], saved2["h"], "h twice")


@pytest.mark.parametrize("T", [1, 20, 90, 6200])
def test_gated_ffn_pitch_and_place(ops, T):
    d, f = 640, 1024
    x, w1, w2, r = _ffn_inputs(T, d, f, T)
    want, _, _ = _check_ffn(ops, x, w1, w2, r)
    say("gated_ffn pitch", T)
    xs, rs = _pitched(x, d + 8), _pitched(r, d + 24, 8)
    _check_ffn(ops, xs, w1, w2, rs)
    say("gated_ffn in place", T)
    out = r.clone()
    assert ops.gated_ffn(x, w1, w2, out, out=out) is out
    _bits_equal(out, ops.gated_ffn(x, w1, w2, r), "in place")


def test_gated_ffn_special_values(ops):
    """A NaN or infinity stays in its token's row, in every form."""
    for T, d, f in ((3, 64, 40), (40, 72, 40), (6200, 640, 1024)):
        say("gated_ffn special", T)
        x, w1, w2, _ = _ffn_inputs(T, d, f, 9)
        clean = ops.gated_ffn(x, w1, w2)
        x[1, 5] = float("nan")
        y = ops.gated_ffn(x, w1, w2)
        keep = [i for i in range(T) if i != 1]
        assert torch.isnan(y[1]).all()
        _bits_equal(y[keep], clean[keep], "the other rows")
    x, w1, w2, r = _ffn_inputs(5, 64, 40, 3)
    assert ops.gated_ffn(x[:0], w1, w2).shape == (0, 64)
    z = ops.gated_ffn(torch.zeros_like(x), w1, w2, r)
    _bits_equal(z, r, "zero tokens leave the residual")


def _check_ffn_bwd(ops, dy, x, saved, w1, w2, out_dtype):
    o = ops.gated_ffn_backward(dy, x, saved, w1, w2, out_dtype=out_dtype)
    torch.cuda.synchronize()
    T, d = dy.shape
    f = w2.shape[1]
    DY, X, GU, H, W1, W2 = (f64(t) for t in (dy, x, saved["gu"], saved["h"], w1, w2))
    dh = DY @ W2
    e = d * ULP32 * (np.abs(DY) @ np.abs(W2))      # dh is not rounded
    dgu = R.dswiglu(GU, dh)
    lin = np.abs(R.dswiglu(GU, np.ones_like(dh)))
    mag = np.concatenate([np.abs(GU[:, f:]) * (1 + np.abs(GU[:, :f])), np.abs(GU[:, :f])], 1) * np.tile(np.abs(dh), 2)
    b = lin * np.tile(e, 2) + 16 * ULP32 * mag
    _within(o["dgu"], dgu, ULP16 * np.abs(dgu) + b * (1 + ULP16) + 2.0 ** -126, "dgu")
    G = f64(o["dgu"])
    out = ULP16 if out_dtype == torch.bfloat16 else 0.0
    dx, dw1, dw2 = G @ W1, G.T @ X, DY.T @ H
    _within(o["dx"], dx, ULP16 * np.abs(dx) + 2 * f * ULP32 * 1.01 * (np.abs(G) @ np.abs(W1)) + 2.0 ** -126, "dx")
    _within(o["dw1p"], dw1, out * np.abs(dw1) + T * ULP32 * 1.01 * (np.abs(G).T @ np.abs(X)) + 2.0 ** -126, "dw1p")
    _within(o["dw2"], dw2, out * np.abs(dw2) + T * ULP32 * 1.01 * (np.abs(DY).T @ np.abs(H)) + 2.0 ** -126, "dw2")
    assert o["dw1p"].dtype == out_dtype and o["dw2"].dtype == out_dtype
    return o


@pytest.mark.parametrize("T,d,f", [(1, 64, 32), (1, 128, 64), (2, 64, 96), (33, 128, 160), (255, 320, 64), (257, 64, 288),
                                   (300, 1024, 256), (1000, 256, 768), (1100, 2112, 64),
                                   (1, 8, 8), (3, 72, 40), (65, 200, 136), (130, 1032, 24), (31, 8, 264), (6200, 2112, 64),
                                   (6200, 640, 2304), (1000, 7168, 2048)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_gated_ffn_backward(ops, T, d, f, out_dtype):
    say("gated_ffn_backward", T, d, f, out_dtype)
    x, w1, w2, dy = _ffn_inputs(T, d, f, T + f)
    _, saved = ops.gated_ffn(x, w1, w2, keep=True)
    o = _check_ffn_bwd(ops, dy, x, saved, w1, w2, out_dtype)
    p = ops.gated_ffn_backward(dy, x, saved, w1, w2, out_dtype=out_dtype)
    for k in ("dx", "dw1p", "dw2", "dgu"):
        _bits_equal(o[k], p[k], k)


def test_gated_ffn_backward_no_tokens(ops):
    x, w1, w2, dy = _ffn_inputs(4, 64, 32, 1)
    z = dict(gu=torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), h=torch.empty(0, 32, dtype=torch.bfloat16,
                                                                                      device="cuda"))
    o = ops.gated_ffn_backward(dy[:0], x[:0], z, w1, w2)
    assert (o["dw1p"] == 0).all() and (o["dw2"] == 0).all() and o["dx"].shape == (0, 64)


def test_gated_ffn_refuses(ops):
    x, w1, w2, r = _ffn_inputs(4, 64, 32, 2)
    for call in (lambda: ops.gated_ffn(x.float(), w1, w2), lambda: ops.gated_ffn(x, w1[:-8], w2),
                 lambda: ops.gated_ffn(x, w1, w2, r[:2]), lambda: ops.gated_ffn(x, w1, w2, out=x),
                 lambda: ops.gated_ffn(x.t(), w1, w2), lambda: ops.gated_ffn(x.cpu(), w1, w2),
                 lambda: ops.gated_ffn(_pitched(x, 65), w1, w2),
                 lambda: ops.add_rmsnorm(x, w1[0], bf16=False), lambda: ops.add_rmsnorm(x, w1[0], out_s=r),
                 lambda: ops.add_rmsnorm(x, w1[0], r.half()), lambda: ops.add_rmsnorm(x, w1[0][:32])):
        with pytest.raises(ops.MoeError):
            call()


# ------------------------------------------------------------------ optimiser

HYPER = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 31, 32, 33, 64, 100, 2048, 2049, 8191, 8192, 8193, 20000, 65536]


def _adam_case(rng, sizes, bits, params, grad, dev="cuda"):
    """params: 'master', 'bf16' or 'f32'."""
    pt = torch.float32 if params == "f32" else torch.bfloat16
    master = [_t(rng, (n,), torch.float32, 0.05) for n in sizes]
    st = dict(params=[m.to(pt) for m in master], masters=master if params == "master" else None,
              grads=[_t(rng, (n,), grad, 1e-2) for n in sizes],
              step=torch.full((1,), 4, dtype=torch.int32, device=dev))
    m = [_t(rng, (n,), torch.float32, 1e-2) for n in sizes]
    rv = [(_t(rng, (n,), torch.float32, 1e-2).abs() + 1e-4) for n in sizes]
    if bits == 32:
        st.update(exp_avg=m, exp_avg_sq=[v * v for v in rv], exp_avg_scale=None, exp_avg_sq_scale=None)
    else:
        for name, ts in (("exp_avg", m), ("exp_avg_sq", rv)):
            qs, es = [], []
            for t in ts:
                b = R.blocks(f64(t))
                e = R.state_exponent(np.abs(b).max(1))
                qs.append(torch.from_numpy((b / np.exp2(e)[:, None]).reshape(-1)[:t.numel()].astype(np.float32)).to(
                    torch.float8_e4m3fn).cuda())
                es.append(torch.from_numpy((e + 127).astype(np.uint8)).cuda().view(torch.float8_e8m0fnu))
            st[name], st[name + "_scale"] = qs, es
    return st


def _call(ops, st, gs=None, seed=11, **hyper):
    h = dict(HYPER)
    h.update(hyper)
    ops.adamw_step(st["params"], st["grads"], st["exp_avg"], st["exp_avg_sq"], st["step"], masters=st["masters"],
                   exp_avg_scale=st["exp_avg_scale"], exp_avg_sq_scale=st["exp_avg_sq_scale"], grad_scale=gs, seed=seed, **h)


def _copy(st):
    cp = lambda v: [t.clone() for t in v] if isinstance(v, list) else v.clone() if isinstance(v, torch.Tensor) else v  # noqa
    return {k: cp(v) for k, v in st.items()}


def _check_codes(codes, scale, want, err, r16, what):
    """codes, scale of values `want` known within err (absolute): the scale is
    the one that `want`'s interval allows, and each code lies between the
    roundings of the interval's two ends by the same random bits."""
    n = len(want)
    q = codes.detach().cpu().view(torch.float8_e4m3fn).float().double().numpy()
    e = scale.detach().cpu().view(torch.uint8).numpy().astype(int) - 127
    lo, hi = R.blocks(want - err), R.blocks(want + err)
    top = np.maximum(np.abs(lo), np.abs(hi)).max(1)
    low = np.where((lo <= 0) & (hi >= 0), 0, np.minimum(np.abs(lo), np.abs(hi))).max(1)
    assert np.all((e >= R.state_exponent(low)) & (e <= R.state_exponent(top))), what
    k = np.exp2(-e.astype(float))[:, None]
    a = np.clip((lo * k).reshape(-1)[:n], -448, 448)
    b = np.clip((hi * k).reshape(-1)[:n], -448, 448)
    # magnitudes are rounded, so the rounding is monotonic on each side of zero and through it
    ra, rb = R.e4m3_random(a.astype(np.float32).astype(np.float64), r16), R.e4m3_random(b.astype(np.float32).astype(np.float64), r16)
    bad = ~((np.minimum(ra, rb) <= q) & (q <= np.maximum(ra, rb)))
    assert not bad.any(), (what, np.argwhere(bad)[:3].tolist(), q[bad][:3], ra[bad][:3], rb[bad][:3])


def _check_adamw(before, after, t, gs=1.0, seed=11, **hyper):
    h = dict(HYPER)
    h.update(hyper)
    (b1, b2), lr, eps, wd = h["betas"], h["lr"], h["eps"], h["weight_decay"]
    assert int(after["step"].item()) == t
    for i, g in enumerate(before["grads"]):
        G, n = f64(g), g.numel()
        P = f64(before["params"][i] if before["masters"] is None else before["masters"][i])
        if before["exp_avg_scale"] is None:
            M, V = f64(before["exp_avg"][i]), f64(before["exp_avg_sq"][i])
        else:
            M = R.decode(before["exp_avg"][i], before["exp_avg_scale"][i])
            V = R.decode(before["exp_avg_sq"][i], before["exp_avg_sq_scale"][i]) ** 2
        p, m, v = R.adamw(P, G, M, V, t, lr, b1, b2, eps, wd, gs)
        # constants rounded to fp32, two products and a sum each
        em = 5 * ULP32 * (b1 * np.abs(M) + (1 - b1) * np.abs(G * gs)) + 2.0 ** -126
        ev = 7 * ULP32 * (b2 * np.abs(V) + (1 - b2) * (G * gs) ** 2) + 2.0 ** -126
        den = np.sqrt(v / (1 - b2 ** t)) + eps
        upd = np.abs(m / (1 - b1 ** t)) / den
        # v's error reaches its root halved
        eu = em / (1 - b1 ** t) / den + upd * (16 * ULP32 + 0.5 * ev / np.maximum(v, 1e-300))
        ep = 3 * ULP32 * np.abs(P) + lr * (eu + 4 * ULP32 * (wd * np.abs(P) + upd))
        if before["exp_avg_scale"] is None:
            _within(after["exp_avg"][i], m, em, ("m", i))
            _within(after["exp_avg_sq"][i], v, ev, ("v", i))
        r = R.random_bits(seed, t, i, n)
        if before["exp_avg_scale"] is not None:
            _check_codes(after["exp_avg"][i], after["exp_avg_scale"][i], m, em + 2 * ULP32 * np.abs(m), r & np.uint64(0xFFFF),
                         ("m codes", i))
            sv = np.sqrt(v)
            _check_codes(after["exp_avg_sq"][i], after["exp_avg_sq_scale"][i], sv,
                         sv * (0.5 * ev / np.maximum(v, 1e-300) + 4 * ULP32), r >> np.uint64(16), ("sqrt v codes", i))
        if before["masters"] is not None:
            _within(after["masters"][i], p, ep, ("master", i))
            _bits_equal(after["params"][i], after["masters"][i].to(torch.bfloat16), ("param of master", i))
        elif before["params"][i].dtype == torch.float32:
            _within(after["params"][i], p, ep, ("param", i))
        else:
            r16 = R.mix(r + np.uint64(0x9E3779B9)) & np.uint64(0xFFFF)
            a, b = R.bf16_random((p - ep).astype(np.float32), r16), R.bf16_random((p + ep).astype(np.float32), r16)
            got = f64(after["params"][i])
            bad = ~((np.minimum(a, b) <= got) & (got <= np.maximum(a, b)))
            assert not bad.any(), ("bf16 param", i, np.argwhere(bad)[:3].tolist())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("params", ["master", "bf16", "f32"])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_adamw_step(ops, bits, params, grad):
    say("adamw", bits, params, grad)
    rng = np.random.default_rng(bits + len(params))
    st = _adam_case(rng, SIZES, bits, params, grad)
    before = _copy(st)
    gs = torch.full((1,), 0.25, device="cuda")
    _call(ops, st, gs=gs)
    torch.cuda.synchronize()
    _check_adamw(before, st, 5, gs=0.25)
    for a, b in zip(before["grads"], st["grads"]):
        _bits_equal(a, b, "gradients are read only")
    again = _copy(before)
    _call(ops, again, gs=gs)
    for k in ("params", "exp_avg", "exp_avg_sq"):
        for a, b in zip(again[k], st[k]):
            _bits_equal(a, b, k)
    before = _copy(st)
    _call(ops, st)               # and a step on what the first one left
    torch.cuda.synchronize()
    _check_adamw(before, st, 6)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_many_tensors_from_the_start(ops, bits):
    """More tensors than one launch takes, empty ones among them, from adamw_state's zeros."""
    rng = np.random.default_rng(4)
    sizes = [(37 * i) % 300 for i in range(101)] + [9000]
    p = [_t(rng, (n,), torch.bfloat16, 0.05) for n in sizes]
    s = ops.adamw_state(p, bits)
    st = dict(params=p, masters=None, grads=[_t(rng, (n,), torch.float32, 1e-2) for n in sizes], **s)
    say("adamw many", bits)
    before = _copy(st)
    _call(ops, st)
    torch.cuda.synchronize()
    _check_adamw(before, st, 1)
    before = _copy(st)
    _call(ops, st, betas=(0.0, 0.0), eps=1e-3, weight_decay=0.0)
    torch.cuda.synchronize()
    _check_adamw(before, st, 2, betas=(0.0, 0.0), eps=1e-3, weight_decay=0.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_unaligned_views(ops, bits):
    """Tensors that start anywhere in a buffer; what lies beside them stays."""
    rng = np.random.default_rng(3)
    sizes = [100, 333]
    st = _adam_case(rng, sizes, bits, "bf16", torch.bfloat16)
    want = _copy(st)
    _call(ops, want)
    for k in ("params", "grads", "exp_avg", "exp_avg_sq"):
        bufs, views = [], []
        for t in st[k]:
            raw = torch.full((t.numel() + 6,), 7, dtype=torch.uint8, device="cuda").view(t.dtype) if t.element_size() == 1 \
                else torch.full((t.numel() + 6,), 7, dtype=t.dtype, device="cuda")
            v = raw[3:3 + t.numel()]
            v.copy_(t)
            bufs.append(raw)
            views.append(v)
        st[k], st[k + "_buf"] = views, bufs
    say("adamw unaligned", bits)
    fence = {k: [(b[:3].clone(), b[-3:].clone()) for b in st[k + "_buf"]] for k in ("params", "exp_avg", "exp_avg_sq")}
    _call(ops, st)
    torch.cuda.synchronize()
    for k in ("params", "exp_avg", "exp_avg_sq"):
        for a, b, buf, (lo, hi) in zip(st[k], want[k], st[k + "_buf"], fence[k]):
            _bits_equal(a, b, k)
            _bits_equal(buf[:3], lo, "before")
            _bits_equal(buf[-3:], hi, "behind")


def test_adamw_skips_a_step_of_infinite_scale(ops):
    rng = np.random.default_rng(2)
    for bits in (32, 8):
        st = _adam_case(rng, [100, 5000], bits, "master", torch.bfloat16)
        before = _copy(st)
        for bad in (float("inf"), float("nan")):
            _call(ops, st, gs=torch.full((1,), bad, device="cuda"))
        torch.cuda.synchronize()
        assert int(st["step"].item()) == 4
        for k in ("params", "masters", "exp_avg", "exp_avg_sq"):
            for a, b in zip(before[k], st[k]):
                _bits_equal(a, b, k)


def test_adamw_nan_and_zero_states(ops):
    """A NaN gradient marks its element (8 bits: its block) and no other; a block of zeros stays zero."""
    rng = np.random.default_rng(1)
    for bits in (32, 8):
        say("adamw nan", bits)
        st = _adam_case(rng, [256], bits, "master", torch.float32)
        st["grads"][0][40] = float("nan")
        st["grads"][0][64:96] = 0
        st["exp_avg"][0].view(torch.uint8 if bits == 8 else torch.float32)[64:96] = 0
        st["exp_avg_sq"][0].view(torch.uint8 if bits == 8 else torch.float32)[64:96] = 0
        _call(ops, st)
        torch.cuda.synchronize()
        bad = torch.isnan(st["masters"][0]).nonzero().flatten().tolist()
        assert bad == [40]
        if bits == 8:
            e = st["exp_avg_scale"][0].view(torch.uint8)
            assert e[1] == 255 and e[2] == 0 and e[0] not in (0, 255) and e[3] not in (0, 255)
            assert (st["exp_avg"][0].view(torch.uint8)[64:96] == 0).all()
            assert (st["exp_avg_sq_scale"][0].view(torch.uint8)[2] == 0)
        else:
            assert torch.isnan(st["exp_avg"][0]).nonzero().flatten().tolist() == [40]


def test_adamw_random_rounding_keeps_the_mean(ops):
    """With no gradient v decays by beta2 a step; each step moves it by far
    less than half a code, so only the random rounding lets it go, and on
    average exactly: sqrt(v)'s expectation is multiplied by sqrt(beta2).  200
    steps at 0.999 round with a relative variance of at most 200 * 0.0005 / 8
    an element: a standard deviation of 0.112 / sqrt(65536) = 4.4e-4 of the
    mean, and five of them are allowed."""
    n = 65536
    rng = np.random.default_rng(12)
    st = _adam_case(rng, [n], 8, "bf16", torch.bfloat16)
    st["grads"][0].zero_()
    sv = R.decode(st["exp_avg_sq"][0], st["exp_avg_sq_scale"][0]).sum()
    for _ in range(200):
        _call(ops, st, lr=0.0, betas=(0.9, 0.999))
    torch.cuda.synchronize()
    got = R.decode(st["exp_avg_sq"][0], st["exp_avg_sq_scale"][0]).sum() / sv
    assert abs(got / 0.999 ** 100 - 1) <= 5 * 4.4e-4, got


def test_adamw_refuses(ops):
    rng = np.random.default_rng(0)
    st = _adam_case(rng, [64, 64], 32, "master", torch.bfloat16)
    for k, v in (("params", [st["params"][0]] * 2), ("exp_avg", st["exp_avg"][:1]), ("step", st["step"].cpu()),
                 ("grads", [st["grads"][0], st["grads"][1].float()]), ("exp_avg", [t.half() for t in st["exp_avg"]]),
                 ("masters", [t[:32] for t in st["masters"]]), ("exp_avg_scale", st["exp_avg"]),
                 ("params", [t.view(8, 8).t() for t in st["params"]]), ("grads", [st["grads"][0], None]),
                 ("grads", st["grads"][:1]), ("exp_avg_sq", [None, None])):
        bad = dict(st)
        bad[k] = v
        with pytest.raises(ops.MoeError):
            _call(ops, bad)
    with pytest.raises(ops.MoeError):
        _call(ops, st, betas=(1.0, 0.9))


# ------------------------------------------------------------------ offsets past 32 bits

def test_norm_past_32_bit_offsets(ops):
    """More than 2^31 elements (and, in fp32, 2^33 bytes): the last rows are the small call's."""
    T, d = 330_000, 6560
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    r = torch.zeros((T, d), dtype=torch.float32, device="cuda")
    rng = np.random.default_rng(21)
    tail = 40
    x[-tail:], r[-tail:] = _t(rng, (tail, d)), _t(rng, (tail, d), torch.float32)
    w = _t(rng, (d,))
    say("norm past 32 bits")
    big = ops.add_rmsnorm(x, w, r, mxfp8=True, keep_rstd=True)
    small = ops.add_rmsnorm(x[-tail:].clone(), w, r[-tail:].clone(), mxfp8=True, keep_rstd=True)
    # a wavefront's and a workgroup's sums of one row differ in order: the same bound as against 64 bits
    _within(big["rstd"][-tail:], f64(small["rstd"]), 62 * ULP32 * f64(small["rstd"]), "rstd")
    for k in ("y", "s"):
        _within(big[k][-tail:], f64(small[k]), 2 * ULP16 * np.abs(f64(small[k])), k)
        assert not big[k][:-tail].any(), k
    q, sc = ops.mxfp8_quantize(big["y"][-tail:].clone(), 0)
    _bits_equal(big["q"][-tail:], q, "codes")
    _bits_equal(big["scale"][-tail:], sc, "scales")
    dy = torch.zeros_like(x)
    dy[-tail:] = _t(rng, (tail, d))
    b = ops.add_rmsnorm_backward(dy, big["s"], w, big["rstd"], dresidual=r)
    D, S, K = f64(dy[-tail:]), f64(big["s"][-tail:]), f64(big["rstd"][-tail:])
    ds, dw = R.rmsnorm_backward(D, S, f64(w), K, f64(r[-tail:]))
    _within(b["ds"][-tail:], ds, 80 * ULP32 * (np.abs(ds) + K[:, None] * np.abs(f64(w) * D) + np.abs(S * K[:, None])), "ds")
    _within(b["dweight"], dw, (T // 512 + 131) * ULP32 * np.abs(D * S * K[:, None]).sum(0), "dweight")


@pytest.mark.parametrize("pitch", [0, 8])
def test_ffn_past_32_bit_offsets(ops, pitch):
    T, d, f = 1_100_000, 64, 1024        # gu: 2.25e9 elements
    rng = np.random.default_rng(22)
    w1, w2 = _t(rng, (2 * f, d), scale=d ** -0.5), _t(rng, (d, f), scale=f ** -0.5)
    x = torch.zeros((T, d + pitch), dtype=torch.bfloat16, device="cuda")[:, :d]
    tail = 70
    x[-tail:] = _t(rng, (tail, d))
    say("ffn past 32 bits", pitch)
    y, saved = ops.gated_ffn(x, w1, w2, x, keep=True)
    _, h, gu = R.ffn(f64(x[-tail:]), f64(w1), f64(w2))
    e = d * ULP32 * (np.abs(f64(x[-tail:])) @ np.abs(f64(w1)).T)
    _within(saved["gu"][-tail:], gu, ULP16 * np.abs(gu) + e * (1 + ULP16), "gu")
    H = f64(saved["h"][-tail:])
    yr = H @ f64(w2).T + f64(x[-tail:])
    _within(y[-tail:], yr, ULP16 * np.abs(yr) + 1.01 * (f + 2) * ULP32 * (np.abs(H) @ np.abs(f64(w2)).T + np.abs(f64(x[-tail:]))),
            "y")
    assert not y[:-tail].any() and not saved["h"][:-tail].any()
    if pitch:
        return
    dy = torch.zeros_like(y)
    dy[-tail:] = _t(rng, (tail, d))
    o = ops.gated_ffn_backward(dy, x, saved, w1, w2)
    cut = {k: saved[k][-tail:].clone() for k in saved}
    p = ops.gated_ffn_backward(dy[-tail:].clone(), x[-tail:].clone(), cut, w1, w2)
    G = f64(p["dgu"])
    _within(o["dgu"][-tail:], G, 2 * ULP16 * np.abs(G) + 2.0 ** -126, "dgu")
    dw1 = f64(o["dgu"][-tail:]).T @ f64(x[-tail:])
    _within(o["dw1p"], dw1, ULP16 * np.abs(dw1) + 1.01 * tail * ULP32 * (np.abs(G).T @ np.abs(f64(x[-tail:]))) + 2.0 ** -126, "dw1p")


def test_adamw_past_32_bit_elements(ops):
    """An element's random bits and its block lie where its 64-bit index says."""
    n, tail = (1 << 32) + 3001, 5000
    rng = np.random.default_rng(23)
    dev = torch.device("cuda")
    p = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    p[-tail:], g[-tail:] = _t(rng, (tail,), scale=0.05), _t(rng, (tail,), scale=1e-2)
    st = ops.adamw_state([p], 8)
    before = p[-tail:].clone()
    say("adamw past 32 bits")
    ops.adamw_step([p], [g], st["exp_avg"], st["exp_avg_sq"], st["step"], exp_avg_scale=st["exp_avg_scale"],
                   exp_avg_sq_scale=st["exp_avg_sq_scale"], seed=11, **HYPER)
    torch.cuda.synchronize()
    i = np.arange(n - tail, n, dtype=np.uint64)
    key = R.mix(R.mix(R.mix(11) ^ np.uint64(1)) ^ np.uint64(0))
    r = R.mix((i & np.uint64(0xFFFFFFFF)) + R.mix(key ^ (i >> np.uint64(32))))
    want, m, v = R.adamw(f64(before), f64(g[-tail:]), 0.0, 0.0, 1, HYPER["lr"], *HYPER["betas"], HYPER["eps"],
                         HYPER["weight_decay"])
    ep = 4 * ULP32 * np.abs(f64(before)) + HYPER["lr"] * 40 * ULP32
    r16 = R.mix(r + np.uint64(0x9E3779B9)) & np.uint64(0xFFFF)
    a, b = R.bf16_random((want - ep).astype(np.float32), r16), R.bf16_random((want + ep).astype(np.float32), r16)
    got = f64(p[-tail:])
    assert ((np.minimum(a, b) <= got) & (got <= np.maximum(a, b))).all()
    assert not p[:-tail].any() and not st["exp_avg"][0].view(torch.uint8)[:-tail].any()
    # whole blocks of the tail: their codes from the same bits
    skip = -(n - tail) % 32
    at = (n - tail + skip) // 32
    _check_codes(st["exp_avg"][0][n - tail + skip:], st["exp_avg_scale"][0][at:], m[skip:], 8 * ULP32 * np.abs(m[skip:]),
                 r[skip:] & np.uint64(0xFFFF), "m codes")


def _some_rows(T, n=4096):
    """Rows at both ends and around the 2^20 workgroups that one launch dimension takes."""
    return torch.cat([torch.arange(0, n), torch.arange(T - n, T)]).cuda()


@pytest.mark.parametrize("d,rows", [(1, 32), (8, 32), (9000, 1)])
def test_norm_of_more_workgroups_than_one_dimension(ops, d, rows):
    """rows: of a workgroup."""
    T = (1 << 20) * rows + 4095
    if d == 9000:
        T = (1 << 20) + 130
    gen = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randint(-8, 9, (T, d), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    w = _t(np.random.default_rng(31), (d,))
    say("norm workgroups", T, d)
    o = ops.add_rmsnorm(x, w, keep_rstd=True)
    at = _some_rows(T, 4096 if d < 100 else 100)
    y, rstd = o["y"][at], o["rstd"][at]
    S = f64(x[at])
    k = 1 / np.sqrt((S * S).mean(1) + 1e-6)
    # the sum of squares of integers is exact; division, sum, root and reciprocal: four roundings and the hardware's
    _within(rstd, k, 16 * ULP32 * k, "rstd")
    ref = S * k[:, None] * f64(w)
    _within(y, ref, (ULP16 + 20 * ULP32) * np.abs(ref) * (1 + ULP16) + 2.0 ** -126, "y")


def test_ffn_of_more_workgroups_than_one_dimension(ops):
    T, d, f = (1 << 28) + 300, 8, 8      # 2^20 + 2 tiles of 256 rows
    rng = np.random.default_rng(32)
    w1, w2 = _t(rng, (2 * f, d), scale=d ** -0.5), _t(rng, (d, f), scale=f ** -0.5)
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    at = _some_rows(T)
    x[at] = _t(rng, (len(at), d))
    say("ffn workgroups", T)
    y = ops.gated_ffn(x, w1, w2)
    small, kept = ops.gated_ffn(x[at], w1, w2, keep=True)
    _, h, _ = R.ffn(f64(x[at]), f64(w1), f64(w2))
    # one stage of K in either call, in one order: the same sums
    _bits_equal(y[at], small, "y")
    H = f64(kept["h"])
    ref = H @ f64(w2).T
    _within(small, ref, ULP16 * np.abs(ref) + 1.01 * (f + 2) * ULP32 * (np.abs(H) @ np.abs(f64(w2)).T) + 2.0 ** -126, "y")
    assert not y[4096:-4096].any()


def test_ffn_backward_of_more_workgroups_than_one_dimension(ops):
    T, d, f = (1 << 27) + 300, 8, 8      # 2^20 + 3 tiles of 128 rows for dx alone
    rng = np.random.default_rng(33)
    w1, w2 = _t(rng, (2 * f, d), scale=d ** -0.5), _t(rng, (d, f), scale=f ** -0.5)
    zeros = lambda n: torch.zeros((T, n), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, dy, saved = zeros(d), zeros(d), dict(h=zeros(f), gu=zeros(2 * f))
    at = _some_rows(T)
    cut_x, cut_dy = _t(rng, (len(at), d)), _t(rng, (len(at), d))
    _, cut = ops.gated_ffn(cut_x, w1, w2, keep=True)
    x[at], dy[at], saved["h"][at], saved["gu"][at] = cut_x, cut_dy, cut["h"], cut["gu"]
    say("ffn backward workgroups", T)
    o = ops.gated_ffn_backward(dy, x, saved, w1, w2, out_dtype=torch.float32)
    p = ops.gated_ffn_backward(cut_dy, cut_x, cut, w1, w2, out_dtype=torch.float32)
    for k in ("dgu", "dx"):
        _bits_equal(o[k][at], p[k], k)
        assert not o[k][4096:-4096].any(), k
    # rows of zeros add nothing: 8192 terms, in whatever order
    G = f64(p["dgu"])
    for k, (a, b) in dict(dw1p=(G, f64(cut_x)), dw2=(f64(cut_dy), f64(cut["h"]))).items():
        _within(o[k], a.T @ b, len(at) * ULP32 * (np.abs(a).T @ np.abs(b)), k)


def test_in_place_norm_refuses_other_rows(ops):
    """In place, the rows read and written are the same ones."""
    buf = torch.zeros(4 * 80, dtype=torch.bfloat16, device="cuda")
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    r = buf.as_strided((4, 64), (80, 1))
    with pytest.raises(ops.MoeError):
        ops.add_rmsnorm(x, w, r, out_s=buf.as_strided((4, 64), (64, 1)))
    with pytest.raises(ops.MoeError):
        ops.add_rmsnorm(r, w, x, out_s=buf.as_strided((4, 64), (72, 1)))
    ops.add_rmsnorm(x, w, r, out_s=r)
    ops.add_rmsnorm(r, w, x, out_s=r)


# ------------------------------------------------------------------ as they are used

def _replayed(make, run, outputs, other):
    """run captured into a graph and replayed on new inputs, against eager calls."""
    state = make(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            run(state)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(state)
    for k in range(1, 4):
        fresh = make(k)
        want = [t.clone() for t in outputs(run(fresh))]
        other(state, make(k))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outputs(out), want):
            _bits_equal(a, b, ("replay", k))


def _refill(a, b):
    """a's tensors take b's values."""
    for k in a:
        if isinstance(a[k], torch.Tensor):
            a[k].copy_(b[k])
        elif isinstance(a[k], list):
            for s, t in zip(a[k], b[k]):
                s.view(torch.uint8 if s.element_size() == 1 else s.dtype).copy_(
                    t.view(torch.uint8 if t.element_size() == 1 else t.dtype))


@pytest.mark.parametrize("T", [1, 40, 300, 6200])
def test_graph_replay_of_a_block(ops, T):
    """Norm, shared expert with the residual, their backward and the step on
    its weights, captured together."""
    d, f = 640, 1024

    def make(k):
        rng = np.random.default_rng(100 + k)
        x, w1, w2, r = _ffn_inputs(T, d, f, 50 + k)
        c = _adam_case(rng, [2 * f * d, d * f, d], 8, "bf16", torch.bfloat16)
        c.pop("grads")
        return dict(x=x, r=r, dy=_t(rng, (T, d)), w=_t(rng, (d,)), **c)

    def run(s):
        w1, w2 = s["params"][0].view(2 * f, d), s["params"][1].view(d, f)
        n = ops.add_rmsnorm(s["x"], s["w"], s["r"], mxfp8=True, keep_rstd=True)
        y, saved = ops.gated_ffn(n["y"], w1, w2, n["s"], keep=True)
        b = ops.gated_ffn_backward(s["dy"], n["y"], saved, w1, w2)
        nb = ops.add_rmsnorm_backward(b["dx"], n["s"], s["w"], n["rstd"], dresidual=s["dy"])
        _call(ops, dict(s, grads=[b["dw1p"].view(-1), b["dw2"].view(-1), nb["dweight"].to(torch.bfloat16)]))
        return dict(y=y, q=n["q"], dx=nb["dx"], dw=nb["dweight"], s=s)

    def outputs(o):
        return [o["y"], o["q"], o["dx"], o["dw"]] + o["s"]["params"] + o["s"]["exp_avg"] + o["s"]["exp_avg_sq"] + [o["s"]["step"]]

    say("graph replay", T)
    _replayed(make, run, outputs, _refill)


@pytest.mark.parametrize("T", [1, 100, 6200])
def test_two_streams_at_once(ops, T):
    d, f = 640, 1024
    a, b = _ffn_inputs(T, d, f, 1), _ffn_inputs(T, d, f, 2)
    want = [ops.gated_ffn(*v[:3], v[3], keep=True) for v in (a, b)]
    grads = [ops.gated_ffn_backward(v[3], v[0], w[1], *v[1:3]) for v, w in zip((a, b), want)]
    torch.cuda.synchronize()
    say("two streams", T)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, v in enumerate((a, b)):
            with torch.cuda.stream(s[i]):
                y, saved = ops.gated_ffn(*v[:3], v[3], keep=True)
                got[i].append((y, ops.gated_ffn_backward(v[3], v[0], saved, *v[1:3])))
    torch.cuda.synchronize()
    for i in range(2):
        for y, g in got[i]:
            _bits_equal(y, want[i][0], "beside another stream's calls")
            for k in ("dx", "dw1p", "dw2"):
                _bits_equal(g[k], grads[i][k], k)


def test_the_block_around_the_layer(ops):
    """norm -> routed experts + shared expert -> backward -> step, each link on
    the other's outputs, and the MXFP8 output as the grouped GEMM's operand."""
    from dropless_moe_expert_amd import inputs
    L = inputs.workload("tiny")
    dev = lambda t: t.contiguous().cuda()  # noqa: E731
    x, logits, w1p, w2 = dev(L.x), dev(L.logits), dev(L.w1p), dev(L.w2)
    T, d = x.shape
    rng = np.random.default_rng(1)
    sw1, sw2 = _t(rng, (256, d), scale=d ** -0.5), _t(rng, (d, 128), scale=128 ** -0.5)
    w, r = _t(rng, (d,)), _t(rng, (T, d))
    n = ops.add_rmsnorm(x, w, r, mxfp8=True, keep_rstd=True)
    y, saved = ops.moe_forward(logits, n["y"], w1p, w2, L.K, keep=True)
    base = y.clone()
    y2, sh = ops.gated_ffn(n["y"], sw1, sw2, y, keep=True, out=y)
    assert y2 is y
    want, _, _ = R.ffn(f64(n["y"]), f64(sw1), f64(sw2), f64(base))
    H = f64(sh["h"])
    yr = H @ f64(sw2).T + f64(base)
    _within(y, yr, ULP16 * np.abs(yr) + 130 * ULP32 * (np.abs(H) @ np.abs(f64(sw2)).T + np.abs(f64(base))) * 1.01, "sum of both")
    # the norm's codes are the grouped GEMM's operand: the same product as from the quantiser's
    q, sc = ops.mxfp8_quantize(n["y"], 0)
    bq, bs = ops.quantize_weights(sw1.view(1, 256, d))
    rows = torch.tensor([T], dtype=torch.int32, device="cuda")
    _bits_equal(ops.grouped_gemm_mxfp8(n["q"], n["scale"], bq, bs, rows), ops.grouped_gemm_mxfp8(q, sc, bq, bs, rows), "MXFP8")
    dy = dev(L.dy)
    gb = ops.moe_backward(dy, saved, w1p, w2, L.K)
    sb = ops.gated_ffn_backward(dy, n["y"], sh, sw1, sw2)
    dn = gb["dx"] + sb["dx"]
    nb = ops.add_rmsnorm_backward(dn, n["s"], w, n["rstd"])
    weights = [w1p, w2, sw1, sw2, w]
    grads = [gb["dw1p"], gb["dw2"], sb["dw1p"], sb["dw2"], nb["dweight"].to(torch.bfloat16)]
    masters = [t.float() for t in weights]
    st = ops.adamw_state(weights)
    before = dict(params=[t.clone() for t in weights], masters=[t.clone() for t in masters], grads=grads,
                  **{k: ([t.clone() for t in v] if v is not None else None) for k, v in st.items() if k != "step"})
    ops.adamw_step(weights, grads, st["exp_avg"], st["exp_avg_sq"], st["step"], masters=masters, **HYPER)
    torch.cuda.synchronize()
    flat = lambda s: {k: [t.reshape(-1) for t in v] if isinstance(v, list) else v for k, v in s.items()}  # noqa: E731
    _check_adamw(flat(before), flat(dict(params=weights, masters=masters, **st)), 1)
    ops.pack_weights(w1p, ops.MOE_EPI_SWIGLU)        # the stepped weights go where weights go
