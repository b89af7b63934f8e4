"""The norm and rotation of queries and keys, cached states and the verification of
drafts in fp64 numpy, with bounds on what an fp32 evaluation may be off by (as
layer_ref has them: u = 2^-24 for a rounding, sums of magnitudes for the values'
own)."""
import numpy as np

from layer_ref import U

D = 128


# ------------------------------------------------------------------ norm and rotation
def angles(positions, inv_freq, pair_axis):
    """[T, pairs]: the product of an int32 and an fp32 number is within 2^-53 of itself in fp64, both here and there."""
    pos = np.atleast_2d(positions).astype(np.float64)
    axis = np.zeros(len(inv_freq), int) if pair_axis is None else np.clip(pair_axis, 0, len(pos) - 1)
    return pos[axis].T * inv_freq


def turn(x, e, angle, rot, interleaved, sign=1.0):
    """x [T, H, d] with bounds e, turned.  A cosine in fp32 is off by the rounding of the reduced angle (below 2^2: 2 u), the
    angle's own 2^-52 of itself, and two units in the last place (4 u)."""
    y, ey = x.copy(), e.copy()
    if not rot:
        return y, ey
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    c, s = np.cos(angle)[:, None], sign * np.sin(angle)[:, None]
    ec = 6 * U + 2.0 ** -52 * np.abs(angle)[:, None]
    a, b, ea, eb = x[..., ia], x[..., ib], e[..., ia], e[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag = np.abs(a) + np.abs(b)
    ey[..., ia] = ey[..., ib] = ea + eb + mag * (ec + 3 * U)      # (two products and a sum)
    return y, ey


def inverse(x, norm, eps):
    """1 / sqrt(...) and its relative error: a sum of d squares, 1 / d, eps, the root, the quotient."""
    d = x.shape[-1]
    if norm == "none":
        return np.ones(x.shape[:-1] + (1,)), 0.0
    ss = (x * x).sum(-1, keepdims=True) * (1.0 / d if norm == "rms" else 1.0)
    return 1 / np.sqrt(ss + eps), (d / 2 + 5) * U


def qknorm(x, weight, norm, eps, scale, angle, rot, interleaved):
    """out and its bound, for heads x [T, H, d]."""
    inv, rel = inverse(x, norm, eps)
    y = x * inv * scale * (1.0 if weight is None else weight)
    return turn(y, np.abs(y) * (rel + 3 * U), angle, rot, interleaved)


def qknorm_backward(x, weight, norm, eps, scale, angle, rot, interleaved, dout):
    """dx, dw and their bounds."""
    d = x.shape[-1]
    inv, rel = inverse(x, norm, eps)
    w = np.ones(d) if weight is None else weight
    e, ee = turn(dout * scale, np.abs(dout * scale) * U, angle, rot, interleaved, -1.0)
    m = {"rms": 1.0 / d, "l2": 1.0, "none": 0.0}[norm]
    dn, edn = e * w, ee * np.abs(w) + U * np.abs(e * w)
    dot = (dn * x).sum(-1, keepdims=True)
    edot = (edn * np.abs(x)).sum(-1, keepdims=True) + (d + 1) * U * np.abs(dn * x).sum(-1, keepdims=True)
    along = dot * inv * inv * m
    ealong = edot * inv * inv * m + np.abs(along) * (2 * rel + 5 * U)
    inner = dn - along * x
    einner = edn + ealong * np.abs(x) + 2 * U * (np.abs(dn) + np.abs(along * x))
    dx, edx = inv * inner, inv * einner + (rel + U) * np.abs(inv * inner)
    n = x * inv
    terms = e * n
    dw = terms.sum((0, 1))
    edw = (ee * np.abs(n)).sum((0, 1)) + (rel + 2 * U + x.shape[0] * x.shape[1] * U) * np.abs(terms).sum((0, 1))
    return dx, edx, dw, edw


# ------------------------------------------------------------------ codes
NUMBERS = {"fp8": np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                           [(8 + m) / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]),
           "int8": np.arange(128) / 64.0, "fp4": np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])}


def scale_bytes(amax, fmt):
    """The smallest power of two with amax / scale at most the largest number, as e8m0."""
    top = NUMBERS[fmt][-1]
    e = np.full(amax.shape, -127)
    with np.errstate(invalid="ignore", over="ignore"):
        for _ in range(254):
            e = np.where((amax > top * 2.0 ** e.astype(float)) & (e < 127), e + 1, e)
    return np.where(np.isfinite(amax), np.where(amax > 0, e + 127, 127), 255)


def quantise(x, fmt):
    """Rows [n, elems] as codes (one an element) and scale bytes, by the definition."""
    n, elems = x.shape
    nb = -(-elems // 32)
    v = np.zeros((n, nb * 32))
    v[:, :elems] = x
    v = v.reshape(n, nb, 32)
    with np.errstate(invalid="ignore"):
        sc = scale_bytes(np.abs(v).max(-1), fmt)     # (a NaN is the largest)
    steps = NUMBERS[fmt]
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.minimum(np.abs(v) / 2.0 ** (sc[..., None] - 127.0), steps[-1])
        a = np.where(np.isfinite(a), a, 0.0)
    up = np.minimum(np.searchsorted(steps, a), len(steps) - 1)
    down = np.maximum(up - 1, 0)
    hi, lo = steps[up] - a, a - steps[down]
    mag = np.where((hi < lo) | ((hi == lo) & (up % 2 == 0)), up, down)
    neg = np.signbit(v)
    code = np.where(neg, (256 - mag) % 256, mag) if fmt == "int8" else mag + np.where(neg, 128 if fmt == "fp8" else 8, 0)
    code = np.where(sc[..., None] == 255, 0, code)
    return code.reshape(n, -1)[:, :elems].astype(np.uint8), sc.astype(np.uint8)


def pack(code, fmt):
    if fmt != "fp4":
        return code
    code = np.pad(code, ((0, 0), (0, code.shape[1] % 2)))
    return code[:, 0::2] | code[:, 1::2] << 4


def numbers(cache, fmt, elems):
    """Rows of packed codes as numbers."""
    if fmt == "int8":
        return cache.view(np.int8)[:, :elems] / 64.0
    if fmt == "fp4":
        c = np.stack((cache & 15, cache >> 4), -1).reshape(len(cache), -1)[:, :elems]
        return np.where(c & 8, -1, 1) * NUMBERS["fp4"][c & 7]
    m = cache & 127
    return np.where(cache & 128, -1, 1) * np.where(m == 127, np.nan, NUMBERS["fp8"][np.minimum(m, 126)])


def dequantise(cache, scales, fmt, elems):
    sc = scales.astype(np.float64)
    down = np.where(sc == 255, np.nan, 2.0 ** (sc - 127))
    return numbers(cache, fmt, elems) * np.repeat(down, 32, 1)[:, :elems]


# ------------------------------------------------------------------ the recurrence from a state
def decode(q, k, v, g, beta, state):
    """Tokens [t, 128] of one head from a state: outputs, the state after them, and the bounds of both.  A decay is within
    an exponential's unit in the last place (2 u) and a product."""
    S, E = state.astype(np.float64), np.zeros((D, D))
    outs, eouts = [], []
    for t in range(len(q)):
        decay = np.exp(g[t])[:, None]
        S, E = decay * S, decay * E + 4 * U * np.abs(decay * S)
        kk, qq = k[t][:, None], q[t][:, None]
        a, b = (S * kk).sum(0), (S * qq).sum(0)
        ea = (E * np.abs(kk)).sum(0) + (D + 1) * U * np.abs(S * kk).sum(0)
        eb = (E * np.abs(qq)).sum(0) + (D + 1) * U * np.abs(S * qq).sum(0)
        qk, eqk = (q[t] * k[t]).sum(), (D + 1) * U * np.abs(q[t] * k[t]).sum()
        off = beta[t] * (v[t] - a)
        eoff = np.abs(beta[t]) * (ea + U * (np.abs(v[t]) + np.abs(a))) + U * np.abs(off)
        outs.append(b + qk * off)
        eouts.append(eb + np.abs(qk) * eoff + eqk * np.abs(off) + 2 * U * (np.abs(b) + np.abs(qk * off)))
        S, E = S + kk * off, E + np.abs(kk) * eoff + 2 * U * (np.abs(S) + np.abs(kk * off))
    return np.array(outs).reshape(-1, D), S, np.array(eouts).reshape(-1, D), E


# ------------------------------------------------------------------ verification
def verify(target, draft, tokens, cu, accept, sample):
    """num_tokens and next_token, in fp64, one sequence after the other."""
    clean = lambda p: np.where(p > 0, p, 0.0)                       # noqa: E731  (NaN is not above zero)
    V, counts, nexts = target.shape[1], [], []
    for n in range(len(cu) - 1):
        if cu[n + 1] <= cu[n]:
            counts.append(0)
            nexts.append(-1)
            continue
        row = cu[n]
        while True:
            p = clean(target[row])
            w = p
            if row + 1 == cu[n + 1]:
                break
            x = int(tokens[row + 1])
            inside = 0 <= x < V
            if draft is not None:
                q = clean(draft[row + 1])
            else:
                q = np.zeros(V)
                if inside:
                    q[x] = 1.0
            if inside and accept[row + 1] * q[x] < p[x]:
                row += 1
                continue
            if draft is None:
                w = np.where(np.arange(V) == x, 0.0, p)
            else:
                w = np.maximum(p - q, 0.0)
            if not w.sum() > 0:
                w = p
            break
        counts.append(1 + row - cu[n])
        c = np.cumsum(w)
        some = np.flatnonzero(w > 0)
        hit = some[c[some] > sample[n] * c[-1]]
        nexts.append(int(hit[0]) if len(hit) else int(some[-1]) if len(some) else -1)
    return counts, nexts
