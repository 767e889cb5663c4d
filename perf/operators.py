"""The dense operators around the expert layer, as cases to be timed and compared.

Each case is one pass of one operator on inputs of a stated size:

  norm      add_rmsnorm: the residual's addition, the root-mean-square norm in
            front of the layer, its output in bf16 and / or in MXFP8
  norm_bwd  add_rmsnorm_backward
  ffn       gated_ffn: the shared expert beside the routed ones
  ffn_bwd   gated_ffn_backward
  adamw     adamw_step: one optimiser step over several tensors

With ``own`` false a pass is computed by elementary torch operations in 32
bits; with ``own`` true by the library's entry points.  ``exact`` computes the
same outputs in 64 bits, before their last rounding.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6
ADAM = dict(lr=3e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
SEED = 1234          # of the stochastic roundings
DEV = "cuda"


def listed():
    return [
        # one decoded token of a DeepSeek-V3-shaped layer: latency of the launch
        dict(name="norm 1x7168 both", op="norm", T=1, d=7168, residual="bf16", bf16=True, mxfp8=True),
        # the same layer's tokens of one training step (6 x 4096), quantised for the MXFP8 GEMMs only
        dict(name="norm 24576x7168 mxfp8", op="norm", T=24576, d=7168, residual="bf16", bf16=False, mxfp8=True),
        # fine-grained layer in training, a ragged number of tokens, residual stream in bf16
        dict(name="norm_bwd 16385x2048", op="norm_bwd", T=16385, d=2048, residual="bf16", dres=True),
        # Mixtral-shaped layer in training with the residual stream kept in fp32
        dict(name="norm_bwd 4096x4096 f32", op="norm_bwd", T=4096, d=4096, residual="f32", dres=True),
        # shared expert of a DeepSeek-V3-shaped layer, one token: the weights are read once
        dict(name="ffn 1 7168 2048", op="ffn", T=1, d=7168, f=2048, residual=True, keep=False),
        # the same for a decode batch of an odd size
        dict(name="ffn 181 7168 2048", op="ffn", T=181, d=7168, f=2048, residual=True, keep=False),
        # prefill / training of the same, with what the backward needs
        dict(name="ffn 16384 7168 2048 keep", op="ffn", T=16384, d=7168, f=2048, residual=False, keep=True),
        # fine-grained layer: backward of a short micro-batch
        dict(name="ffn_bwd 1000 2048 768", op="ffn_bwd", T=1000, d=2048, f=768),
        # DeepSeek-V3-shaped layer: backward of one micro-batch of 4096 tokens
        dict(name="ffn_bwd 4096 7168 2048", op="ffn_bwd", T=4096, d=7168, f=2048),
        # the norms, biases and router of a small layer: many launches' worth of tiny tensors
        dict(name="adamw 14 small f32 states", op="adamw", count=14, largest=8 * 4096, shrink=1.6, bits=32, master=True,
             grad="f32"),
        # the weights of four experts of a DeepSeek-V3-shaped layer, fp32 states and master weights
        dict(name="adamw 4 experts f32 states", op="adamw", count=4, largest=4096 * 7168, shrink=1.0, bits=32,
             master=True, grad="bf16"),
        # the same with 8-bit states and bf16 weights alone
        dict(name="adamw 4 experts 8-bit", op="adamw", count=4, largest=4096 * 7168, shrink=1.0, bits=8, master=False,
             grad="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "ffn", "ffn", "ffn_bwd", "adamw"])
    if op in ("norm", "norm_bwd"):
        mx = op == "norm" and rng.random() < 0.5
        d = 32 * _log(rng, 1, 256) if mx else rng.choice([8 * _log(rng, 4, 1024), _log(rng, 33, 8192)])
        T = min(_log(rng, 1, 24576), 24576 * 7168 // d)
        res = rng.choice(["none", "bf16", "f32"])
        if op == "norm":
            return dict(op=op, T=T, d=d, residual=res, bf16=(not mx) or rng.random() < 0.5, mxfp8=mx)
        return dict(op=op, T=T, d=d, residual=res, dres=rng.random() < 0.7)
    if op == "ffn":
        d, f = 8 * _log(rng, 16, 896), 8 * _log(rng, 16, 1024)
        T = min(_log(rng, 1, 16384), 16384 * 7168 * 2048 // (d * f))
        return dict(op=op, T=T, d=d, f=f, residual=rng.random() < 0.5, keep=rng.random() < 0.4)
    if op == "ffn_bwd":
        d, f = 64 * _log(rng, 2, 112), 64 * _log(rng, 2, 64)
        T = min(_log(rng, 1, 8192), 4096 * 7168 * 2048 // (d * f))
        return dict(op=op, T=T, d=d, f=f)
    bits = rng.choice([32, 8])
    count = rng.randint(1, 11)
    largest = min(_log(rng, 1, 1 << 26), 4 * 4096 * 7168 // count)
    return dict(op=op, count=count, largest=largest, shrink=rng.choice([1.0, 1.3, 3.0]), bits=bits,
                master=rng.random() < 0.5, grad=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------ inputs

def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=F32) * scale).to(dtype)


def _sizes(c):
    return [max(1, int(c["largest"] / c["shrink"] ** i) - 37 * i) for i in range(c["count"])]


def _blocks(v):
    """[n] fp32 in rows of 32, the last one filled up with zeros."""
    return torch.nn.functional.pad(v, (0, -v.numel() % 32)).view(-1, 32)


def _state_scale(amax):
    """The smallest e with amax <= 448 * 2^e (-127 for zeros) of each block."""
    m, ex = torch.frexp(amax)          # amax = 2m * 2^(ex - 1), 2m in [1, 2)
    e = ex - 1 - 8 + (m > 0.875).int()
    return torch.where(amax > 0, e, -127).clamp(-127, 127)


def _pow2(e):
    return torch.ldexp(torch.ones((), device=e.device, dtype=F32), e)


def prepare(case, seed):
    c, g = dict(case), torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=c)
    if c["op"] in ("norm", "norm_bwd"):
        T, d = c["T"], c["d"]
        rt = F32 if c["residual"] == "f32" else BF16
        chan = torch.exp(_normal(g, (d,), F32, 0.5))          # channels of unequal size, as trained ones are
        x = (_normal(g, (T, d), F32) * chan).to(BF16)
        st["w"] = (1 + _normal(g, (d,), F32, 0.2)).to(BF16)
        if c["op"] == "norm":
            st["x"] = x
            st["r"] = None if c["residual"] == "none" else (_normal(g, (T, d), F32, 2.0) * chan).to(rt)
        else:
            s = (x.float() * 2).to(rt)
            st.update(s=s, rstd=(s.double().square().mean(-1) + EPS).rsqrt().float(), dy=_normal(g, (T, d), BF16, 1e-2))
            st["dres"] = _normal(g, (T, d), rt, 1e-2) if c["dres"] else None
    elif c["op"] in ("ffn", "ffn_bwd"):
        T, d, f = c["T"], c["d"], c["f"]
        st.update(x=_normal(g, (T, d), BF16), w1p=_normal(g, (2 * f, d), BF16, d ** -0.5),
                  w2=_normal(g, (d, f), BF16, f ** -0.5))
        if c["op"] == "ffn":
            st["r"] = _normal(g, (T, d), BF16) if c["residual"] else None
        else:
            gu = (st["x"].float() @ st["w1p"].float().t()).to(BF16)
            a, u = gu[:, :f].float(), gu[:, f:].float()
            st.update(gu=gu, h=(a * torch.sigmoid(a) * u).to(BF16), dy=_normal(g, (T, d), BF16))
    else:
        ns = _sizes(c)
        gt = F32 if c["grad"] == "f32" else BF16
        p = [_normal(g, (n,), F32, 0.02) for n in ns]
        m = [_normal(g, (n,), F32, 1e-3) for n in ns]
        rv = [torch.exp(_normal(g, (n,), F32)) * 1e-3 for n in ns]    # sqrt(v)
        st.update(p=[v.to(BF16) for v in p], master=p if c["master"] else None, g=[_normal(g, (n,), gt, 2e-3) for n in ns],
                  step=torch.full((1,), 999, dtype=torch.int32, device=DEV), gs=torch.full((1,), 0.7, device=DEV))
        if c["bits"] == 32:
            st.update(m=m, v=[v * v for v in rv], ms=None, vs=None)
        else:
            for k, t in (("m", m), ("v", rv)):
                e = [_state_scale(_blocks(v).abs().amax(1)) for v in t]
                st[k] = [(_blocks(v) * _pow2(-q)[:, None]).to(F8).view(-1)[:v.numel()].clone() for v, q in zip(t, e)]
                st[k + "s"] = [(q + 127).to(torch.uint8).view(E8) for q in e]
    return st


# ------------------------------------------------------------------ plain forms

def _plain_norm(st, c):
    x, r, w = st["x"], st["r"], st["w"]
    s = x if r is None else (x.float() + r.float()).to(r.dtype)
    sf = s.float()
    rstd = (sf.square().mean(-1) + EPS).rsqrt()
    y = (sf * rstd[:, None] * w.float()).to(BF16)
    out = dict(rstd=rstd)
    if r is not None:
        out["s"] = s
    if c["bf16"]:
        out["y"] = y
    if c["mxfp8"]:
        yb = y.float().view(c["T"], -1, 32)
        amax = yb.abs().amax(-1)
        _, ex = torch.frexp(amax)                              # floor(log2 amax) = ex - 1
        e = torch.where(amax > 0, ex - 1 - 8, -127).clamp(-127, 127)
        out["q"] = (yb * _pow2(-e)[..., None]).clamp(-448, 448).to(F8).view(c["T"], c["d"])
        out["scale"] = (e + 127).to(torch.uint8).view(E8)
    return out


def _plain_norm_bwd(st, c):
    s, w, dy = st["s"].float(), st["w"].float(), st["dy"].float()
    rstd = st["rstd"][:, None]
    xh = s * rstd
    wdy = w * dy
    ds = rstd * (wdy - xh * (wdy * xh).mean(-1, keepdim=True))
    if st["dres"] is not None:
        ds = ds + st["dres"].float()
    out = dict(dx=ds.to(BF16), dweight=(dy * xh).sum(0, dtype=F64).float())
    if st["s"].dtype == F32:
        out["ds"] = ds
    return out


def _plain_ffn(st, c):
    f = c["f"]
    gu = st["x"].float() @ st["w1p"].float().t()
    a, u = gu[:, :f], gu[:, f:]
    h = a * torch.sigmoid(a) * u
    y = h @ st["w2"].float().t()
    if st["r"] is not None:
        y = y + st["r"].float()
    return dict(y=y.to(BF16), h=h.to(BF16), gu=gu.to(BF16)) if c["keep"] else dict(y=y.to(BF16))


def _plain_ffn_bwd(st, c):
    f = c["f"]
    dy, w1p = st["dy"].float(), st["w1p"].float()
    a, u = st["gu"][:, :f].float(), st["gu"][:, f:].float()
    dh = dy @ st["w2"].float()
    sg = torch.sigmoid(a)
    dgu = torch.cat([dh * u * sg * (1 + a * (1 - sg)), dh * a * sg], 1)
    return dict(dx=(dgu @ w1p).to(BF16), dw1p=(dgu.t() @ st["x"].float()).to(BF16),
                dw2=(dy.t() @ st["h"].float()).to(BF16))


M32 = 0xFFFFFFFF


def _mix(v):
    """A 32-bit mixer of integers held in int64."""
    v = ((v ^ (v >> 16)) * 0x7FEB352D) & M32
    v = ((v ^ (v >> 15)) * 0x846CA68B) & M32
    return v ^ (v >> 16)


def _random(step, index, n):
    """32 random bits for each of a tensor's n < 2^32 elements: a function of (SEED, step, tensor, element)."""
    k = _mix(_mix(_mix(torch.full_like(step, SEED)) ^ step) ^ index)
    return _mix((torch.arange(n, device=DEV, dtype=torch.int64) + _mix(k)) & M32)


def _round_bits(v, add, keep):
    """fp32 with random bits added below its kept ones, and cut there."""
    return ((v.view(torch.int32) + add.int()) & ~((1 << keep) - 1)).view(F32)


def _state_codes(v, rnd):
    """fp32 [n] -> E4M3 codes and E8M0 scales, rounded up or down by 16 random bits each."""
    b = _blocks(v)
    e = _state_scale(b.abs().amax(1))
    a = (b * _pow2(-e)[:, None]).view(-1)[:v.numel()]
    mag = a.abs()
    low = mag < 2.0 ** -6
    cut = _round_bits(torch.where(low, mag + 2.0 ** -6, mag), rnd << 4, 20)
    return torch.copysign(torch.where(low, cut - 2.0 ** -6, cut), a).to(F8), (e + 127).to(torch.uint8).view(E8)


def _plain_adamw(st, c):
    (b1, b2), lr = ADAM["betas"], ADAM["lr"]
    st["step"] += 1
    t = st["step"].double()
    c1, c2 = (1 - b1 ** t).float(), (1 - b2 ** t).float()
    for i in range(c["count"]):
        g = st["g"][i].float() * st["gs"]
        p = st["p"][i].float() if st["master"] is None else st["master"][i]
        n = p.numel()
        if c["bits"] == 32:
            m, v = st["m"][i], st["v"][i]
        else:
            wide = lambda k: (_blocks(st[k][i].float()) * st[k + "s"][i].float()[:, None]).view(-1)[:n]  # noqa: E731
            m, v = wide("m"), wide("v").square()
            rnd = _random(st["step"].long(), i, n)
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        p = p - lr * (ADAM["weight_decay"] * p + (m / c1) / ((v / c2).sqrt() + ADAM["eps"]))
        if c["bits"] == 32:
            st["m"][i].copy_(m)
            st["v"][i].copy_(v)
        else:
            for k, x, r in (("m", m, rnd & 0xFFFF), ("v", v.sqrt(), rnd >> 16)):
                q, e = _state_codes(x, r)
                st[k][i].copy_(q)
                st[k + "s"][i].copy_(e)
        if st["master"] is None:
            rnd = _mix((_random(st["step"].long(), i, n) + 0x9E3779B9) & M32) & 0xFFFF
            st["p"][i].copy_(_round_bits(p, rnd, 16))
        else:
            st["master"][i].copy_(p)
            st["p"][i].copy_(p)
    return {k: st[k] for k in ("p", "master", "m", "v", "ms", "vs") if st[k] is not None}


# ------------------------------------------------------------------ the library's calls

def _own(st, c):
    from dropless_moe_expert_amd import ops
    if c["op"] == "norm":
        o = ops.add_rmsnorm(st["x"], st["w"], st["r"], eps=EPS, bf16=c["bf16"], mxfp8=c["mxfp8"], keep_rstd=True)
        out = dict(rstd=o["rstd"])
        if st["r"] is not None:
            out["s"] = o["s"]
        if c["bf16"]:
            out["y"] = o["y"]
        if c["mxfp8"]:
            out.update(q=o["q"].view(F8), scale=o["scale"].view(E8))
        return out
    if c["op"] == "norm_bwd":
        o = ops.add_rmsnorm_backward(st["dy"], st["s"], st["w"], st["rstd"], dresidual=st["dres"])
        out = dict(dx=o["dx"], dweight=o["dweight"])
        if st["s"].dtype == F32:
            out["ds"] = o["ds"]
        return out
    if c["op"] == "ffn":
        if not c["keep"]:
            return dict(y=ops.gated_ffn(st["x"], st["w1p"], st["w2"], st["r"]))
        y, saved = ops.gated_ffn(st["x"], st["w1p"], st["w2"], st["r"], keep=True)
        return dict(y=y, h=saved["h"], gu=saved["gu"])
    if c["op"] == "ffn_bwd":
        o = ops.gated_ffn_backward(st["dy"], st["x"], dict(gu=st["gu"], h=st["h"]), st["w1p"], st["w2"])
        return dict(dx=o["dx"], dw1p=o["dw1p"], dw2=o["dw2"])
    ops.adamw_step(st["p"], st["g"], st["m"], st["v"], st["step"], masters=st["master"], exp_avg_scale=st["ms"],
                   exp_avg_sq_scale=st["vs"], grad_scale=st["gs"], seed=SEED, **ADAM)
    return {k: st[k] for k in ("p", "master", "m", "v", "ms", "vs") if st[k] is not None}


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "ffn": _plain_ffn, "ffn_bwd": _plain_ffn_bwd,
            "adamw": _plain_adamw}[c["op"]](state, c)


def work(case):
    c = dict(case)
    if c["op"] in ("norm", "norm_bwd"):
        T, d = c["T"], c["d"]
        rb = 4 if c["residual"] == "f32" else 2
        if c["op"] == "norm":
            row = 2 * d + (0 if c["residual"] == "none" else 2 * rb * d) + 4
            row += (2 * d if c["bf16"] else 0) + (d + d // 32 if c["mxfp8"] else 0)
            return dict(bytes=T * row + 2 * d, flops=6 * T * d)
        row = 2 * d + rb * d + 4 + (rb * d if c["dres"] else 0) + 2 * d + (4 * d if rb == 4 else 0)
        return dict(bytes=T * row + 6 * d, flops=10 * T * d)
    if c["op"] == "ffn":
        T, d, f = c["T"], c["d"], c["f"]
        return dict(bytes=6 * d * f + 4 * T * d + (2 * T * d if c["residual"] else 0) + (6 * T * f if c["keep"] else 0),
                    flops=6 * T * d * f)
    if c["op"] == "ffn_bwd":
        T, d, f = c["T"], c["d"], c["f"]
        return dict(bytes=6 * T * d + 6 * T * f + 12 * d * f, flops=12 * T * d * f)
    n = sum(_sizes(c))
    per = (4 if c["grad"] == "f32" else 2) + (10 if c["master"] else 4) + (16 if c["bits"] == 32 else 4 + 4 / 32)
    return dict(bytes=n * per, flops=16 * n)


# ------------------------------------------------------------------ 64 bits

def _chunks(T, fn):
    """fn over blocks of rows, its outputs joined: 64-bit temporaries of a few rows at a time."""
    parts = [fn(slice(a, min(T, a + 4096))) for a in range(0, T, 4096)]
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def exact(case, seed):
    c = dict(case)
    st = prepare(case, seed)
    if c["op"] == "norm":
        def rows(i):
            s = st["x"][i].double()
            if st["r"] is not None:
                s = s + st["r"][i].double()
            o = dict(s=s)
            s = s.to(st["r"].dtype).double() if st["r"] is not None else s     # the norm is that of the stored sum
            var = torch.einsum("td,td->t", s, s) / c["d"]
            o["rstd"] = 1 / torch.sqrt(var + EPS)
            o["y"] = s * o["rstd"][:, None] * st["w"].double()
            if c["mxfp8"]:
                top = o["y"].to(BF16).double().abs().view(len(s), -1, 32).amax(-1, keepdim=True)
                e = (torch.floor(torch.log2(top)) - 8).clamp(-127, 127)
                o["q"] = (o["y"].view(len(s), -1, 32) * torch.exp2(-e)).clamp(-448, 448).view(len(s), -1)
            return o
        o = _chunks(c["T"], rows)
        out = dict(rstd=o["rstd"])
        if st["r"] is not None:
            out["s"] = o["s"]
        if c["bf16"]:
            out["y"] = o["y"]
        if c["mxfp8"]:
            # the scale has no such value: on which side of a power of two a
            # block's largest element falls is decided by its rounding
            out.update(q=o["q"], scale=None)
        return out
    if c["op"] == "norm_bwd":
        w, dw = st["w"].double(), torch.zeros(c["d"], dtype=F64, device=DEV)

        def rows(i):
            s, dy, k = st["s"][i].double(), st["dy"][i].double(), st["rstd"][i].double()
            dot = torch.einsum("td,td,d->t", s, dy, w)
            ds = k[:, None] * dy * w - s * (k ** 3 * dot / c["d"])[:, None]
            dw.add_(torch.einsum("td,td,t->d", s, dy, k))
            return dict(ds=ds if st["dres"] is None else ds + st["dres"][i].double())
        o = _chunks(c["T"], rows)
        out = dict(dx=o["ds"], dweight=dw)
        if c["residual"] == "f32":
            out["ds"] = o["ds"]
        return out
    if c["op"] == "ffn":
        f, w1, w2 = c["f"], st["w1p"].double(), st["w2"].double()

        def rows(i):
            gu = torch.mm(st["x"][i].double(), w1.t())
            h = gu[:, :f] / (1 + torch.exp(-gu[:, :f])) * gu[:, f:]
            y = torch.mm(h, w2.t())
            return dict(y=y if st["r"] is None else y + st["r"][i].double(), h=h, gu=gu)
        o = _chunks(c["T"], rows)
        return o if c["keep"] else dict(y=o["y"])
    if c["op"] == "ffn_bwd":
        f, w1, w2 = c["f"], st["w1p"].double(), st["w2"].double()
        dw1, dw2 = torch.zeros_like(w1), torch.zeros_like(w2)

        def rows(i):
            dy, gu = st["dy"][i].double(), st["gu"][i].double()
            e = 1 / (1 + torch.exp(-gu[:, :f]))
            dh = torch.mm(dy, w2)
            dgu = torch.cat([dh * gu[:, f:] * (e + gu[:, :f] * e * (1 - e)), dh * gu[:, :f] * e], 1)
            dw1.addmm_(dgu.t(), st["x"][i].double())
            dw2.addmm_(dy.t(), st["h"][i].double())
            return dict(dx=torch.mm(dgu, w1))
        return dict(dx=_chunks(c["T"], rows)["dx"], dw1p=dw1, dw2=dw2)
    # the optimiser: values before their last rounding.  Codes are given as
    # value / scale; the scales of the 8-bit states have no such value (as above).
    (b1, b2), t, out = ADAM["betas"], 1000, dict(p=[], m=[], v=[])
    for i, n in enumerate(_sizes(c)):
        g = st["g"][i].double() * st["gs"].double()
        p = st["p"][i].double() if st["master"] is None else st["master"][i].double()
        m, v = st["m"][i].double(), st["v"][i].double()
        if c["bits"] == 8:
            m = m * torch.repeat_interleave(st["ms"][i].double(), 32)[:n]
            v = (v * torch.repeat_interleave(st["vs"][i].double(), 32)[:n]) ** 2
        m, v = m + (1 - b1) * (g - m), v + (1 - b2) * (g * g - v)
        step = (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + ADAM["eps"])
        out["p"].append(p * (1 - ADAM["lr"] * ADAM["weight_decay"]) - ADAM["lr"] * step)
        if c["bits"] == 8:
            def scaled(a):
                b = torch.nn.functional.pad(a, (0, -n % 32)).view(-1, 32)
                top = b.float().double().abs().amax(1, keepdim=True)
                return (b * torch.exp2(-torch.ceil(torch.log2(top / 448)).clamp(-127, 127))).view(-1)[:n]
            m, v = scaled(m), scaled(torch.sqrt(v))
        out["m"].append(m)
        out["v"].append(v)
    if st["master"] is not None:
        out["master"] = out["p"]
    if c["bits"] == 8:
        out.update(ms=[None] * c["count"], vs=[None] * c["count"])
    return out
