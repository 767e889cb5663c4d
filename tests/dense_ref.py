"""Plain 64-bit forms of the dense operators (numpy), their formulas written
out, for the tests; no library code."""
import numpy as np

U32 = np.uint32
ULP32 = 2.0 ** -24      # half a step of fp32, relative
ULP16 = 2.0 ** -8       # of bf16
ULP8 = 2.0 ** -4        # of E4M3


def f64(t):
    """A torch tensor's values in float64."""
    return t.detach().to("cpu").double().numpy()


# ------------------------------------------------------------------ norm

def rmsnorm(s, w, eps):
    rstd = 1.0 / np.sqrt((s * s).mean(-1) + eps)
    return s * rstd[:, None] * w, rstd


def rmsnorm_backward(dy, s, w, rstd, dres=None):
    xh = s * rstd[:, None]
    wdy = w * dy
    ds = rstd[:, None] * (wdy - xh * (wdy * xh).mean(-1, keepdims=True))
    return (ds if dres is None else ds + dres), (dy * xh).sum(0)


# ------------------------------------------------------------------ gated block

def silu(g):
    return g / (1.0 + np.exp(-g))


def ffn(x, w1p, w2, res=None):
    f = w2.shape[1]
    gu = x @ w1p.T
    h = silu(gu[:, :f]) * gu[:, f:]
    y = h @ w2.T
    return (y if res is None else y + res), h, gu


def dswiglu(gu, dh):
    f = dh.shape[1]
    g, u = gu[:, :f], gu[:, f:]
    s = 1.0 / (1.0 + np.exp(-g))
    return np.concatenate([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1)


def ffn_backward(dy, x, gu, h, w1p, w2):
    dgu = dswiglu(gu, dy @ w2)
    return dgu @ w1p, dgu.T @ x, dy.T @ h, dgu


# ------------------------------------------------------------------ optimiser

def mix(v):
    v = np.asarray(v, dtype=np.uint64) & 0xFFFFFFFF
    v = ((v ^ (v >> np.uint64(16))) * np.uint64(0x7FEB352D)) & np.uint64(0xFFFFFFFF)
    v = ((v ^ (v >> np.uint64(15))) * np.uint64(0x846CA68B)) & np.uint64(0xFFFFFFFF)
    return v ^ (v >> np.uint64(16))


def random_bits(seed, t, index, n):
    """r of elements 0 .. n - 1 (n < 2^32)."""
    key = mix(mix(mix(seed) ^ np.uint64(t)) ^ np.uint64(index))
    return mix(np.arange(n, dtype=np.uint64) + mix(key))


def bf16_random(p, r16):
    """p (finite) rounded to bf16 up or down: r16 added below its 16 kept bits, the rest cut."""
    b = np.asarray(p, np.float32).view(U32).astype(np.uint64) + np.asarray(r16, np.uint64)
    return (b & np.uint64(0xFFFF0000)).astype(U32).view(np.float32).astype(np.float64)


def e4m3_random(a, r16):
    """|a| <= 448 rounded to the E4M3 grid by 16 random bits."""
    mag = np.abs(a)
    low = mag < 2.0 ** -6
    base = np.where(low, mag + 2.0 ** -6, mag).astype(np.float32)
    b = (base.view(U32).astype(np.uint64) + (np.asarray(r16, np.uint64) << np.uint64(4))) & np.uint64(0xFFF00000)
    cut = b.astype(U32).view(np.float32).astype(np.float64)
    return np.copysign(np.where(low, cut - 2.0 ** -6, cut), a)


def blocks(v):
    return np.pad(v, (0, -len(v) % 32)).reshape(-1, 32)


def state_exponent(amax):
    """The smallest e with amax <= 448 * 2^e, in [-127, 127]; -127 for 0."""
    m, ex = np.frexp(amax)      # amax = 2m * 2^(ex - 1)
    return np.where(amax > 0, np.clip(ex - 1 - 8 + (2 * m > 1.75), -127, 127), -127)


def decode(codes, scale):
    """E4M3 codes and E8M0 scale bytes (torch tensors) -> float64 values."""
    import torch
    q = codes.detach().cpu().reshape(-1).view(torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    e = scale.detach().cpu().view(torch.uint8).numpy().astype(np.float64) - 127
    return (blocks(q) * np.exp2(e)[:, None]).reshape(-1)[:len(q)]


def adamw(p, g, m, v, t, lr, b1, b2, eps, wd, gs=1.0):
    """-> (p, m, v) after step t."""
    g = g * gs
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    upd = (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p - lr * (wd * p + upd), m, v
