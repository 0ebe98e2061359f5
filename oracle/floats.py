"""CPU oracle of the floating-point operations around the DFP-8 products:
the Linear layer's epilogue and its backward pass, the gated layer, layer norm,
the norms around a block, Muon, AdamW and the DFP-8 and E4M3 conversions, each the definition written out in numpy.  Test
infrastructure only.

Everything is in float64 except AdamW, whose definition fixes the rounding of
every operation to float32 and is therefore reproduced bit for bit.
"""
import math

import numpy as np

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
ADAMW_BLOCK = 256
_erfc = np.vectorize(math.erfc, otypes=[np.float64])
_K = math.sqrt(2.0 / math.pi)


def _sigmoid(w):
    return 1.0 / (1.0 + np.exp(-np.clip(w, -700.0, 700.0)))


def act(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(_K * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z * _sigmoid(z)
    assert kind == "none"
    return z.copy()


def act_grad(z, kind):
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = np.tanh(_K * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _K * (1.0 + 3 * 0.044715 * z * z)
    if kind == "silu":
        p = _sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    assert kind == "none"
    return np.ones_like(z)


def dfp8(x):
    """(mantissas, exponent) of a tensor: max |x| = f 2^q, E = q - 6."""
    x = np.asarray(x, np.float64)
    top = float(np.max(np.abs(x))) if x.size else 0.0
    e = math.frexp(top)[1] - 7 if top else 0
    return np.clip(np.rint(np.ldexp(x, -e)), -128, 127).astype(np.int8), e


def product(A, B):
    """sum_k A[m][k] B[n][k], exact (every partial sum is below 2^53)."""
    assert A.shape[1] * 2 ** 14 < 2 ** 53
    return (A.astype(np.float64) @ B.astype(np.float64).T).astype(np.int64)


def linear_fwd(X, eX, W, eW, bias, kind, residual):
    """(y, z) in float64."""
    z = np.ldexp(product(X, W).astype(np.float64), eX + eW)
    if bias is not None:
        z = z + bias.astype(np.float64)
    y = act(z, kind)
    if residual is not None:
        y = y + residual.astype(np.float64)
    return y, z


def gated_fwd(X, eX, W, eW, bias, kind):
    """(y, z) in float64; W: the gate's rows and then the up projection's."""
    z = np.ldexp(product(X, W).astype(np.float64), eX + eW)
    if bias is not None:
        z = z + bias.astype(np.float64)
    H = W.shape[0] // 2
    return act(z[:, :H], kind) * z[:, H:], z


def gated_error(dY, Z, kind):
    """The error of z, in float64."""
    H = Z.shape[1] // 2
    g, u = np.asarray(Z[:, :H], np.float64), np.asarray(Z[:, H:], np.float64)
    return np.concatenate([dY * u * act_grad(g, kind), dY * act(g, kind)], 1)


def layer_norm_fwd(x, gamma, beta, eps):
    """(y, mean, rstd) in float64."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(np.square(x - mean[:, None]).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * gamma.astype(np.float64)
    if beta is not None:
        y = y + beta.astype(np.float64)
    return y, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, gamma, dres):
    """(dx, dgamma, dbeta) in float64."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    h = (x - np.asarray(mean, np.float64)[:, None]) * rstd
    d = dy if gamma is None else dy * gamma.astype(np.float64)
    dx = rstd * (d - d.mean(1, keepdims=True) - h * (d * h).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, (dy * h).sum(0), dy.sum(0)


def _norm(v, kind, gamma, beta, eps):
    """(output, mean, rstd, normalised rows); kind "none": the rows themselves."""
    if kind == "none":
        return v, None, None, v
    mean = v.mean(1) if kind == "layer" else np.zeros(len(v))
    rstd = 1.0 / np.sqrt(np.square(v - mean[:, None]).mean(1) + eps)
    h = (v - mean[:, None]) * rstd[:, None]
    out = h if gamma is None else h * gamma.astype(np.float64)
    return out if beta is None else out + beta.astype(np.float64), mean, rstd, h


def _per_row(gate, gate_rows, rows):
    if gate is None:
        return 1.0
    return gate.astype(np.float64)[np.arange(rows) // (gate_rows if 0 < gate_rows < rows else max(rows, 1))]


def residual_norm_fwd(a, x, norm_a, gamma_a, beta_a, gate, gate_rows, alpha, norm_y, gamma_y, beta_y, eps):
    """{y, n, mean_a, rstd_a, mean_y, rstd_y} in float64."""
    y = alpha * np.asarray(x, np.float64)
    mean_a = rstd_a = None
    if a is not None:
        p, mean_a, rstd_a, _ = _norm(np.asarray(a, np.float64), norm_a, gamma_a, beta_a, eps)
        y = y + _per_row(gate, gate_rows, len(y)) * p
    n, mean_y, rstd_y, _ = _norm(y, norm_y, gamma_y, beta_y, eps)
    return dict(y=y, n=n, mean_a=mean_a, rstd_a=rstd_a, mean_y=mean_y, rstd_y=rstd_y)


def residual_norm_bwd(dy, dn, a, y, norm_a, gamma_a, beta_a, gate, gate_rows, alpha, norm_y, gamma_y, mean_a, rstd_a,
                      mean_y, rstd_y):
    """{dx, da, dgate, dgamma_a, dbeta_a, dgamma_y, dbeta_y} in float64, from the given statistics."""
    wide = lambda v: None if v is None else np.asarray(v, np.float64)  # noqa: E731
    one = lambda v: 1.0 if v is None else wide(v)  # noqa: E731

    def rows(v, kind, mean, rstd):
        return v if kind == "none" else (v - (0.0 if kind == "rms" else wide(mean)[:, None])) * wide(rstd)[:, None]

    def back(d, h, kind, rstd):
        if kind == "none":
            return d
        off = h * (d * h).mean(1, keepdims=True) + (d.mean(1, keepdims=True) if kind == "layer" else 0.0)
        return wide(rstd)[:, None] * (d - off)

    out = {}
    t = 0.0 if dy is None else wide(dy)
    if norm_y != "none":
        hy = rows(wide(y), norm_y, mean_y, rstd_y)
        t = t + back(wide(dn) * one(gamma_y), hy, norm_y, rstd_y)
        out.update(dgamma_y=(wide(dn) * hy).sum(0), dbeta_y=wide(dn).sum(0))
    out["dx"] = alpha * t
    if a is not None:
        ha = rows(wide(a), norm_a, mean_a, rstd_a)
        e = t * _per_row(gate, gate_rows, len(t))
        out["da"] = back(e * one(gamma_a), ha, norm_a, rstd_a)
        out.update(dgamma_a=(e * ha).sum(0), dbeta_a=e.sum(0))
        if gate is not None:
            p = ha * one(gamma_a) + (0.0 if beta_a is None else wide(beta_a))
            out["dgate"] = np.zeros(gate.shape)
            np.add.at(out["dgate"], np.arange(len(t)) // (gate_rows if 0 < gate_rows < len(t) else max(len(t), 1)), t * p)
    return out


NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def newton_schulz(x, steps, rounded=None):
    """steps times x = a x + (b A + c A A) x, A = x x^T, the shorter side first.
    rounded(product, terms): a model of a product's rounding, for tolerances."""
    a, b, c = NEWTON_SCHULZ
    rounded = rounded or (lambda p, q: p @ q)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(steps):
        A = rounded(x, x.T)
        x = a * x + rounded(b * A + c * rounded(A, A), x)
    return x.T if tall else x


def muon_step(P, G, M, lr, momentum, nesterov, eps, weight_decay, steps, scale=None, rounded=None):
    """(P, M, X) in float64."""
    P, G, M = (np.asarray(t, np.float64) for t in (P, G, M))
    M = momentum * M + G
    u = G + momentum * M if nesterov else M
    norm = np.sqrt(np.square(u).sum()) + eps
    x = newton_schulz(u / norm if norm else u, steps, rounded)
    if scale is None:
        scale = math.sqrt(max(1.0, P.shape[0] / P.shape[1]))
    return P * (1 - lr * weight_decay) - lr * scale * x, M, x


# ---- 8-bit optimiser states --------------------------------------------------

def e4m3_table():
    """The value of each E4M3 code (sign 1, exponent 4 with bias 7, mantissa 3; 0x7f and 0xff: NaN)."""
    c = np.arange(256)
    ex, m = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, m * 2.0 ** -9, (8 + m) * np.exp2(ex - 10.0))
    v[(c & 0x7f) == 0x7f] = np.nan
    return np.where(c & 0x80, -v, v)


_TABLE = e4m3_table()


def e4m3_encode(x):
    """Codes of the nearest values, ties to the even code; not finite: NaN (0x7f).  |x| <= 448 or not finite."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    pos = _TABLE[:0x7f]
    hi = np.searchsorted(pos, a).clip(0, 0x7e)
    lo = np.maximum(hi - 1, 0)
    d = (a - pos[lo]) - (pos[hi] - a)
    c = np.where(d > 0, hi, np.where(d < 0, lo, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(np.isfinite(x), c | np.where(np.signbit(x), 0x80, 0), 0x7f)
    return c.astype(np.uint8)


def block_exponents(x):
    """One exponent per block of 256 (float32 x): of the largest finite magnitude."""
    n = x.size
    a = np.zeros(-(-n // ADAMW_BLOCK) * ADAMW_BLOCK)
    a[:n] = np.where(np.isfinite(x), np.abs(x.astype(np.float64)), 0.0)
    top = a.reshape(-1, ADAMW_BLOCK).max(1)
    f, q = np.frexp(top)  # f in [0.5, 1)
    e = np.where(top > 0, np.maximum(q - 1 - 8 + (2 * f > 1.75), -126), 0)
    return e.astype(np.int8)


def state_encode(x, positive):
    """(codes, exponents) of a float32 state; positive: a value above 0 keeps at least code 1."""
    e = block_exponents(x)
    c = e4m3_encode(np.ldexp(x.astype(np.float64), -e.astype(np.int64).repeat(ADAMW_BLOCK)[:x.size]))
    if positive:
        c = np.where((c == 0) & (x > 0), 1, c).astype(np.uint8)
    return c, e


def state_decode(c, e):
    """float32 values (exact)."""
    return np.ldexp(_TABLE[c], e.astype(np.int64).repeat(ADAMW_BLOCK)[:c.size]).astype(np.float32)


def draws(n, t):
    """One of the numbers (k + 1/2) / 65536 for each
    element of a tensor at step t: a fixed hash of the step and the index of
    the four elements that share it, in 32-bit arithmetic, two elements from
    the halves of each of two words."""
    u = np.uint32
    h = np.arange(-(-n // 4), dtype=u) * u(0x9E3779B9) + u((t * 0x6C8E9CF5) & 0xffffffff)
    h ^= h >> u(16)
    h *= u(0x5B8D2E35)
    h ^= h >> u(15)
    h *= u(0xC6A4F30B)
    a = h ^ (h >> u(16))
    h = a * u(0x2D9A73E7)
    b = h ^ (h >> u(15))
    k = np.stack([a & u(0xffff), a >> u(16), b & u(0xffff), b >> u(16)], 1).reshape(-1)[:n]
    return (k.astype(np.float32) + np.float32(0.5)) * np.float32(2.0 ** -16)


def _scaled(x):
    """float32 x over its block's power of two, and the exponents."""
    e = block_exponents(x)
    return np.ldexp(x, -e.astype(np.int32).repeat(ADAMW_BLOCK)[:x.size]), e


def _grid(a):
    """The largest E4M3 value that is not above a >= 0, and the distance to the next one (float32, exact)."""
    f = np.float32
    step = np.maximum(np.ldexp(f(1.0), np.frexp(a)[1] - 4), f(2.0 ** -9)).astype(f)
    return np.floor(a / step) * step, step


def mean_encode(m, draw):
    """(codes, exponents) of a float32 mean: the E4M3 value on either side of
    it, with its expectation kept."""
    f = np.float32
    s, e = _scaled(m)
    with np.errstate(all="ignore"):
        a = np.abs(np.where(np.isfinite(s), s, f(0)))
        lo, step = _grid(a)
        q = np.copysign(np.where(a - lo > draw * step, lo + step, lo), s)
    return e4m3_encode(np.where(np.isfinite(s), q, s)), e


def root_encode(r, draw):
    """(codes, exponents) of a float32 root r >= 0: the E4M3 value below or
    above it, above with the probability that keeps the expectation of r^2."""
    f = np.float32
    s, e = _scaled(r)
    with np.errstate(all="ignore"):
        fin = np.where(np.isfinite(s), s, f(0))
        lo, step = _grid(fin)
        up = (fin - lo) * (fin + lo) > draw * (step * (lo + lo + step))
        q = np.where(up, lo + step, lo)
    q = np.where((r > 0) & (q < f(2.0 ** -9)), f(2.0 ** -9), q)
    return e4m3_encode(np.where(np.isfinite(s), q, s)), e


_REST = np.float32(1.0 / 254.0)


def root_encode_carried(r, draw):
    """(codes, remainders, exponents): the nearest E4M3 code (not 0 for a
    positive r), and what is left of r in 254ths of the code's step, one of
    the two whole numbers around it with its expectation kept."""
    f = np.float32
    s, _ = _scaled(r)
    c, e = state_encode(r, True)
    v = _TABLE[c].astype(f)
    with np.errstate(all="ignore"):
        x = (s - v) * (f(254.0) / _grid(np.where(np.isnan(v), f(0), v))[1])
        q = np.clip(np.floor(x + draw), -127, 127)
    return c, np.where(np.isfinite(s), q, 0).astype(np.int8), e


def root_decode_carried(c, rest, e):
    f = np.float32
    v = _TABLE[c].astype(f)
    v = v + (rest.astype(f) * _grid(np.where(np.isnan(v), f(0), v))[1]) * _REST
    return np.ldexp(v, e.astype(np.int32).repeat(ADAMW_BLOCK)[:c.size])


def adamw_step(p, g, m, v, t, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0, exps=None, rest=None):
    """(p, m, v[, exps[, rest]]) after one step of one tensor.  v: the second
    moment (float32), or with exps (int8 [blocks][2]) m and v are E4M3 codes
    of m and of the root of the second moment.  The step reads the codes;
    rest, where it is given, carries what they leave of the root, for the next
    codes."""
    f = np.float32
    b1, c1, b2, c2 = f(beta1), f(1.0 - beta1), f(beta2), f(1.0 - beta2)
    rs2 = f(1.0 / math.sqrt(1.0 - beta2 ** t))
    decay, size = f(1.0 - lr * weight_decay), f(lr / (1.0 - beta1 ** t))
    with np.errstate(all="ignore"):
        g = g.astype(f) * f(grad_scale)
        if exps is not None:
            m = state_decode(m, exps[:, 0])
            r = state_decode(v, exps[:, 1])
            whole = None if rest is None else root_decode_carried(v, rest, exps[:, 1])
            v = r * r
        m = b1 * m + c1 * g
        v = b2 * v + (c2 * g) * g
        r = np.sqrt(v)
        u = m / (r * rs2 + f(eps))
        p = p * decay - size * u
    assert p.dtype == m.dtype == v.dtype == f
    if exps is None:
        return p, m, v
    draw = draws(p.size, t)
    if beta1 <= 0.9375:
        cm, em = state_encode(m, False)
    else:  # (the number of the element two on, or back, among its four)
        other = draws(-(-p.size // 4) * 4, t).reshape(-1, 4)[:, [2, 3, 0, 1]].reshape(-1)[:p.size]
        cm, em = mean_encode(m, other)
    if rest is None:
        cr, er = root_encode(r, draw)
        return p, cm, cr, np.stack([em, er], 1)
    with np.errstate(all="ignore"):
        r = np.sqrt(b2 * (whole * whole) + (c2 * g) * g)
    cr, rest, er = root_encode_carried(r, draw)
    return p, cm, cr, np.stack([em, er], 1), rest
