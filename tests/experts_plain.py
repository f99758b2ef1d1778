"""Plain 64-bit numpy forms of the operators around the experts (routing, its
gradient, MX FP4, the grouped product), written from the formulas in
include/moe_experts.h; the tests' reference."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------------ routing

def scores(logits, sigmoid):
    """(scores, masked) of one token's logits."""
    x = np.asarray(logits, dtype=np.float64)
    masked = np.isnan(x) | (x == -np.inf)
    s = np.zeros_like(x)
    if sigmoid:
        with np.errstate(over="ignore"):
            s[~masked] = 1.0 / (1.0 + np.exp(-x[~masked]))
    elif not masked.all():
        top = x[~masked].max()
        with np.errstate(invalid="ignore"):
            e = np.where(x[~masked] == top, 1.0, np.exp(x[~masked] - top))
        s[~masked] = e / e.sum()
    return s, masked


def keys(logits, bias, sigmoid, top2):
    s, masked = scores(logits, sigmoid)
    if bias is not None:
        key = s + np.asarray(bias, dtype=np.float64)
    else:
        key = s.copy() if top2 else np.asarray(logits, dtype=np.float64).copy()
    key[masked | np.isnan(key)] = -np.inf
    return s, key


def group_values(key, groups, top2):
    out = []
    for part in key.reshape(groups, -1):
        best = np.sort(part)[::-1]
        v = best[0]
        if top2 and len(best) > 1 and best[1] != -np.inf:
            v = v + best[1]
        out.append(v)
    return np.array(out)


def route_token(logits, bias, K, G, KG, sigmoid, top2, renorm, scaling):
    s, key = keys(logits, bias, sigmoid, top2)
    allowed = np.ones(len(key), dtype=bool)
    if G > 1:
        v = group_values(key, G, top2)
        opened = sorted(range(G), key=lambda g: (-v[g], g))[:KG]
        allowed = np.isin(np.arange(len(key)) // (len(key) // G), opened)
    order = sorted(np.flatnonzero(allowed), key=lambda e: (-key[e], e))[:K]
    w = s[order]
    if renorm:
        w = w / w.sum() if w.sum() > 0 else np.zeros(K)
    return np.array(order, dtype=np.int32), w * scaling


def weights_of(logits, ids, sigmoid, renorm, scaling):
    """The weights of given picks (the choice held fixed)."""
    s, _ = scores(logits, sigmoid)
    w = s[ids]
    if renorm:
        w = w / w.sum() if w.sum() > 0 else np.zeros(len(ids))
    return w * scaling


def route_gradient(logits, ids, grad, sigmoid, renorm, scaling):
    s, _ = scores(logits, sigmoid)
    g = np.zeros(len(s))
    g[ids] = np.asarray(grad, dtype=np.float64) * scaling
    chosen = np.zeros(len(s), dtype=bool)
    chosen[ids] = True
    if renorm:
        total = s[chosen].sum()
        r = np.where(chosen, s, 0.0) / total if total > 0 else np.zeros(len(s))
        d = r * (g - (g * r).sum())
        return d * (1.0 - s) if sigmoid else d
    if sigmoid:
        return g * s * (1.0 - s)
    return s * (g - (g * s).sum())


# ------------------------------------------------------------------ MX FP4

def nearest_code(m):
    """E2M1 code of magnitudes m: the nearest value, ties to the even code, saturating."""
    m = np.asarray(m, dtype=np.float64)
    code = np.zeros(m.shape, dtype=np.uint8)
    for c in range(7):  # past the middle between codes c and c + 1; the middle itself goes to the even one
        middle = (MAGNITUDES[c] + MAGNITUDES[c + 1]) / 2
        code += m >= middle if c % 2 else m > middle
    return code


def quantize(x):
    """Unpacked codes [..., cols] and scale bytes [..., ceil(cols / 32)]."""
    x = np.asarray(x, dtype=np.float64)
    cols = x.shape[-1]
    B = -(-cols // 32)
    v = np.zeros(x.shape[:-1] + (B * 32,))
    v[..., :cols] = x
    v = v.reshape(x.shape[:-1] + (B, 32))
    amax = np.abs(v).max(-1)
    exponent = np.full(amax.shape, -127)
    some = amax > 0
    exponent[some] = np.clip(np.frexp(amax[some])[1] - 1 - 2, -127, 127)
    code = nearest_code(np.abs(v) * np.exp2(-exponent.astype(np.float64))[..., None])
    code = code + 8 * np.signbit(v).astype(np.uint8)
    return code.reshape(x.shape[:-1] + (B * 32,))[..., :cols], (exponent + 127).astype(np.uint8)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), dtype=np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def values(codes, scale_bytes):
    """The numbers that unpacked codes and scale bytes stand for."""
    v = np.where(codes & 8, -1.0, 1.0) * MAGNITUDES[codes & 7]
    f = np.exp2(scale_bytes.astype(np.float64) - 127.0)
    return v * np.repeat(f, 32, axis=-1)[..., :codes.shape[-1]]


def tile_scales(s):
    """Scales [E][rows][B] in tiles of 128 rows x 4 blocks (zeros beyond the edges)."""
    E, rows, B = s.shape
    out = np.zeros((E, -(-rows // 128), -(-B // 4), 512), dtype=np.uint8)
    for r in range(rows):
        for b in range(B):
            out[:, r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = s[:, r, b]
    return out


# ------------------------------------------------------------------ the product

def silu_gate(z):
    g, u = z[..., 0::2], z[..., 1::2]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
