"""AdamW step with fp32 or 8-bit block states (CPU oracle).

step32 / step8 follow the stated sequence of binary32 operations (one rounding each), so the
library's results equal theirs bit for bit; step64 is the textbook update in float64.  The
8-bit states are E4M3 codes of m and sqrt(v) with an fp32 scale per 256 elements,
stochastically rounded with 16 bits of a hash.

Pins: step32 against step64 within a bound derived from its operation count, E4M3 values
against torch.float8_e4m3fn, the stochastic rounding's neighbours and mean by brute force.
"""

import numpy as np

BLOCK = 256
F = np.float32


def mix(x):
    """The 32-bit hash of the stochastic rounding (numpy uint32, or a Python int)."""
    x = np.asarray(x, np.uint32)
    with np.errstate(over="ignore"):
        x = x ^ (x >> np.uint32(16))
        x = x * np.uint32(0x7FEB352D)
        x = x ^ (x >> np.uint32(15))
        x = x * np.uint32(0x846CA68B)
        return x ^ (x >> np.uint32(16))


def power(b, t):
    r = 1.0
    while t > 0:
        if t & 1:
            r *= b
        b *= b
        t >>= 1
    return r


def update(p, g, m, v, lr, step, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """(p', m', v', sqrt(v')) in binary32, the stated order."""
    size = F(lr / (1.0 - power(beta1, step)))
    root = F(1.0 / np.sqrt(1.0 - power(beta2, step)))
    keep = F(1.0 - lr * weight_decay)
    g = g.astype(F) * F(grad_scale)
    m = m * F(beta1) + g * F(1.0 - beta1)
    v = v * F(beta2) + (g * F(1.0 - beta2)) * g
    r = np.sqrt(v)
    p = p * keep - (m / (r * root + F(eps))) * size
    return p, m, v, r


def e4m3_values():
    """The 256 values of the E4M3 codes (NaN for 0x7F and 0xFF)."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 0x7F) == 0x7F] = np.nan
    return np.where(c >= 128, -v, v).astype(F)


def encode(x, rnd, lift):
    """(codes, scales) of a 1-D tensor x (binary32) with rnd 16-bit random numbers."""
    n = x.size
    blocks = -(-n // BLOCK)
    xp = np.zeros(blocks * BLOCK, F)
    xp[:n] = x
    rp = np.zeros(blocks * BLOCK, np.uint32)
    rp[:n] = rnd
    xp, rp = xp.reshape(blocks, BLOCK), rp.reshape(blocks, BLOCK)
    top = np.abs(xp).max(1) if n else np.zeros(0, F)
    live = top >= F(2.0 ** -100)
    scale = np.where(live, top * F(1.0 / 448.0), F(0)).astype(F)
    inv = np.where(live, F(1) / np.where(live, scale, F(1)), F(0)).astype(F)
    y = np.minimum(np.abs(xp) * inv[:, None], F(448))
    small = np.floor(y * F(512) + rp.astype(F) * F(2.0 ** -16)).astype(np.int64)
    large = ((y.view(np.uint32) + (rp << np.uint32(4))) >> np.uint32(20)).astype(np.int64) - 960
    code = np.where(y < F(2.0 ** -6), small, large)
    if lift:
        code = np.where((y > 0) & (code < 1), 1, code)
    code = code + np.where(np.signbit(xp), 128, 0)
    return code.reshape(-1)[:n].astype(np.uint8), scale


def decode(codes, scales):
    return e4m3_values()[codes] * np.repeat(scales, BLOCK)[:codes.size]


def step32(p, g, m, v, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0):
    return update(p, g, m, v, lr, step, beta1, beta2, eps, weight_decay, grad_scale)[:3]


def step8(p, g, mc, ms, vc, vs, lr, step, seed, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0):
    """(p', m codes, m scales, v codes, v scales)."""
    r = decode(vc, vs)
    p, m, _, r = update(p, g, decode(mc, ms), r * r, lr, step, beta1, beta2, eps, weight_decay, grad_scale)
    key = mix(np.uint32(seed) ^ mix(step & 0xFFFFFFFF))
    with np.errstate(over="ignore"):
        h = mix(np.arange(p.size, dtype=np.uint32) + key)
    mc, ms = encode(m, h & np.uint32(0xFFFF), False)
    vc, vs = encode(r, h >> np.uint32(16), True)
    return p, mc, ms, vc, vs


def step64(p, g, m, v, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0):
    """(p', m', v') in float64 by the textbook formula."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v
