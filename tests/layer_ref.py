"""The layer operators in fp64 numpy, token by token, with bounds on what an
fp32 evaluation of them may be off by.

Every bound is a first-order running error analysis.  u = 2^-24 is half a step
of fp32 relative to the value: one rounding of an fp32 operation.  Products and
sums of magnitudes stand for the values' own, so that cancellation is counted.
A bound is used with a factor 1.01 for the terms of second order, and a stored
value of a narrower type may be off by half a step of that type on top.
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"fp32": U, "bf16": 2.0 ** -8}


def close(got, ref, bound, dtype, what):
    """|got - ref| <= bound, plus half a step of the stored type at the larger magnitude."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not got.size:
        return
    tol = 1.01 * bound + HALF_STEP[dtype] * (np.abs(ref) + 1.01 * bound) + 1e-37
    off = np.abs(got - ref)
    worst = float(np.max(off / tol))
    print("%-28s max off %.3g of its bound" % (what, worst), flush=True)
    assert np.all(np.isfinite(got)) and worst <= 1.0, (what, worst, np.unravel_index(int(np.argmax(off / tol)), off.shape))


# ------------------------------------------------------------------ gated linear recurrence
# A step h = a h + x in fp32: expf within one unit in the last place (2 u), the
# product and the sum one rounding each.  Evaluated over pieces that are joined,
# a piece's decay is a product of the same factors (one more rounding a token)
# and a join is a product and a sum, on at most a few levels and once in eight
# tokens or more: less than 2 u a token of the state's magnitude.
STEP = 8 * U


def scan(x, g, init, cu, tile=128):
    """h, final, carried = exp(g) h_{t-1}, checkpoints and the bounds (of h, final, carried)."""
    T, D = x.shape
    N = len(cu) - 1
    h, p = np.zeros((T, D)), np.zeros((T, D))
    eh, ep, ah, ap = (np.zeros((T, D)) for _ in range(4))
    fin = np.zeros((N, D)) if init is None else init.astype(np.float64).copy()
    efin = np.zeros((N, D))
    chk = np.full((-(-T // tile), D), np.nan)
    echk = np.zeros_like(chk)
    for n in range(N):
        s = fin[n].copy()
        A, E = np.abs(s), np.zeros(D)
        for t in range(cu[n], cu[n + 1]):
            if t % tile == 0 and t > cu[n]:
                chk[t // tile], echk[t // tile] = s, E
            a = np.exp(g[t])
            p[t] = a * s
            ap[t] = a * A
            ep[t] = a * E + STEP * ap[t]
            s = p[t] + x[t]
            A = ap[t] + np.abs(x[t])
            E = ep[t] + U * A
            h[t], ah[t], eh[t] = s, A, E
        fin[n], efin[n] = s, E
    return dict(h=h, final=fin, carried=p, chk=chk, e_h=eh, e_final=efin, e_carried=ep, a_carried=ap, e_chk=echk)


def scan_backward(x, g, init, cu, dout, dfinal):
    f = scan(x, g, init, cu)
    T, D = x.shape
    N = len(cu) - 1
    dx, dg, ex, eg = (np.zeros((T, D)) for _ in range(4))
    dinit, einit = np.zeros((N, D)), np.zeros((N, D))
    for n in range(N):
        e = np.zeros(D) if dfinal is None else dfinal[n].astype(np.float64)
        A, E = np.abs(e), np.zeros(D)
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            dh = dout[t] + e
            Adh = np.abs(dout[t]) + A
            Edh = E + U * Adh
            dx[t], ex[t] = dh, Edh
            dg[t] = dh * f["carried"][t]
            eg[t] = Edh * f["a_carried"][t] + Adh * f["e_carried"][t] + U * Adh * f["a_carried"][t]
            a = np.exp(g[t])
            e, A, E = a * dh, a * Adh, a * Edh + STEP * a * Adh
        dinit[n], einit[n] = e, E
    return dict(dx=dx, dg=dg, dinit=dinit, e_dx=ex, e_dg=eg, e_dinit=einit, fwd=f)


# ------------------------------------------------------------------ short convolution
# pre: width products and sums, one rounding each, and the bias: (width + 2) u of
# the sum of magnitudes.  SiLU: exp(-p) within (|p| + 4) u, the sum, the quotient
# and the product one rounding each; its slope lies within 1.1 of zero and the
# slope's own within 0.51.
def _silu(p):
    sig = 1 / (1 + np.exp(-p))
    return p * sig, sig * (1 + p * (1 - sig))


def _rows(x, init, cu, n, W, D):
    lead = np.zeros((W - 1, D)) if init is None else init[n].astype(np.float64)
    return np.concatenate([lead, x[cu[n]:cu[n + 1]].astype(np.float64)])


def conv(x, w, b, init, cu, silu):
    T, D = x.shape
    W, N = w.shape[1], len(cu) - 1
    pre, mag = np.zeros((T, D)), np.zeros((T, D))
    fin = np.zeros((N, W - 1, D))
    for n in range(N):
        rows = _rows(x, init, cu, n, W, D)
        fin[n] = rows[len(rows) - (W - 1):]
        for p in range(cu[n + 1] - cu[n]):
            t = cu[n] + p
            pre[t] = (rows[p:p + W] * w.T).sum(0) + (0 if b is None else b)
            mag[t] = (np.abs(rows[p:p + W] * w.T)).sum(0) + (0 if b is None else np.abs(b))
    e_pre = (W + 2) * U * mag
    out, e = pre, e_pre
    if silu:
        out = _silu(pre)[0]
        e = 1.1 * e_pre + (np.abs(pre) + 8) * U * np.abs(out)
    return dict(out=out, final=fin, pre=pre, e_pre=e_pre, e_out=e)


def conv_backward(x, w, b, init, cu, silu, dout, dfinal):
    T, D = x.shape
    W, N = w.shape[1], len(cu) - 1
    f = conv(x, w, b, init, cu, silu)
    d = dout.astype(np.float64)
    ed = np.zeros((T, D))
    if silu:
        slope = _silu(f["pre"])[1]
        ed = np.abs(d) * (0.51 * f["e_pre"] + (np.abs(f["pre"]) + 8) * 3 * U * 1.1)
        d = d * slope
    dx, edx = np.zeros((T, D)), np.zeros((T, D))
    dinit, edinit = np.zeros((N, W - 1, D)), np.zeros((N, W - 1, D))
    dw, edw, aw = np.zeros((D, W)), np.zeros((D, W)), np.zeros((D, W))
    for n in range(N):
        rows = _rows(x, init, cu, n, W, D)
        dr, er, ar = np.zeros_like(rows), np.zeros_like(rows), np.zeros_like(rows)
        L = cu[n + 1] - cu[n]
        if dfinal is not None:
            dr[L:] += dfinal[n]
            ar[L:] += np.abs(dfinal[n])
        for j in range(W):
            s = slice(cu[n], cu[n + 1])
            dr[j:j + L] += d[s] * w[:, j]
            ar[j:j + L] += np.abs(d[s] * w[:, j])
            er[j:j + L] += ed[s] * np.abs(w[:, j])
            dw[:, j] += (d[s] * rows[j:j + L]).sum(0)
            aw[:, j] += np.abs(d[s] * rows[j:j + L]).sum(0)
            edw[:, j] += (ed[s] * np.abs(rows[j:j + L])).sum(0)
        er += (W + 2) * U * ar
        dinit[n], edinit[n] = dr[:W - 1], er[:W - 1]
        dx[cu[n]:cu[n + 1]], edx[cu[n]:cu[n + 1]] = dr[W - 1:], er[W - 1:]
    # a sum of T terms in any order: T - 1 roundings at most, of partial sums within the sum of magnitudes
    return dict(dx=dx, e_dx=edx, dinit=dinit, e_dinit=edinit, dweight=dw, e_dweight=edw + (T + 2) * U * aw,
                dbias=d.sum(0), e_dbias=ed.sum(0) + (T + 2) * U * np.abs(d).sum(0), fwd=f)


# ------------------------------------------------------------------ residual and norm
# The sum of D squares in fp32 is off by at most D u of itself in any order (all
# terms are positive); its root, reciprocal and the division by D take 5 u more,
# half of the sum's.
def rmsnorm(x, res, w, eps):
    x = x.astype(np.float64)
    r = x if res is None else x + res
    e_r = np.zeros_like(r) if res is None else U * np.abs(r)
    D = r.shape[1]
    rstd = 1 / np.sqrt((r * r).sum(1, keepdims=True) / D + eps)
    y = r * rstd * (1 if w is None else w)
    rel = (D / 2 + 10) * U
    return dict(r=r, e_r=e_r, y=y, rstd=rstd, e_y=rel * np.abs(y))


def rmsnorm_backward(x, w, dout, dres, eps):
    x, dout = x.astype(np.float64), dout.astype(np.float64)
    D = x.shape[1]
    w = np.ones(D) if w is None else w.astype(np.float64)
    rstd = 1 / np.sqrt((x * x).sum(1, keepdims=True) / D + eps)
    rel = (D / 2 + 10) * U
    dw_rows = dout * x * rstd
    wd = dout * w
    k = (wd * x).sum(1, keepdims=True) / D * rstd ** 2
    ak = np.abs(wd * x).sum(1, keepdims=True) / D * rstd ** 2
    ek = (D + 2) * U * ak + 2 * rel * np.abs(k)
    dx = rstd * (wd - k * x)
    e = rel * np.abs(dx) + rstd * (3 * U * (np.abs(wd) + np.abs(k * x)) + ek * np.abs(x))
    if dres is not None:
        dx = dx + dres
        e = e + U * np.abs(dx)
    R = x.shape[0]
    return dict(dx=dx, e_dx=e, dweight=dw_rows.sum(0), e_dweight=(rel + (R + 3) * U) * np.abs(dw_rows).sum(0))
