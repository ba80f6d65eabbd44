"""fp64 references of the operators around the recurrence (numpy), each with a
per-element bound on the kernel's fp32 arithmetic error.

Errors are counted in units of u = 2^-24, the half step of fp32 (one rounding is
off by at most u relative to its result).  A function returns (value, E): the exact
value and E such that a computation in fp32 in the kernels' manner is within E u
of it: a sum of n terms carries at most n roundings of the sum of the terms'
magnitudes; exp2, rcp and rsq are off by one step (2 u); e^x by the product with
log2(e) adds |x| log2(e) < 1.5 |x| to its relative error.  The counts are rounded
up, never down.  An output then adds its own rounding, finfo(dtype).eps / 2 of the
value (`close`)."""
import numpy as np

U = 2.0 ** -24


def close(got, ref, err, dtype, label=""):
    """Every element of `got` within its bound of the exact value."""
    import torch

    x = got.detach().double().cpu().numpy()
    assert x.shape == ref.shape, "%s: shape %s, not %s" % (label, x.shape, ref.shape)
    tol = err * U
    tol = tol + float(torch.finfo(dtype).eps) / 2 * (np.abs(ref) + tol) + 1e-36
    bad = ~(np.abs(x - ref) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isfinite(x), np.abs(x - ref) / tol, np.inf)), x.shape)
        raise AssertionError("%s: %d of %d out of bounds, worst at %s: got %r, exact %r, allowed %.3g" % (
            label, bad.sum(), bad.size, i, x[i], ref[i], tol[i]))


def sig(z):
    return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


# ---- convolution ----


def conv(x, w, b, s0, docs, silu):
    """dict: y, st, z and the rows of each document with its carried-in rows before it."""
    T, C = x.shape
    W = w.shape[1]
    z, Sz = np.zeros((T, C)), np.zeros((T, C))
    st = np.zeros((len(docs), W - 1, C))
    ext, t0 = [], 0
    for n, L in enumerate(docs):
        X = np.concatenate([s0[n] if s0 is not None else np.zeros((W - 1, C)), x[t0:t0 + L]])
        for i in range(W):
            z[t0:t0 + L] += X[i:i + L] * w[:, i]
            Sz[t0:t0 + L] += np.abs(X[i:i + L] * w[:, i])
        st[n] = X[L:]
        ext.append(X)
        t0 += L
    z, Sz = z + b, Sz + np.abs(b)
    Ez = (W + 1) * Sz
    y = z * sig(z) if silu else z
    # SiLU' <= 1.1; sigma's relative error: e^-z (1.5 |z| + 2), the sum, the quotient, the product
    Ey = 1.1 * Ez + np.abs(y) * (1.5 * np.abs(z) + 8) if silu else Ez
    return dict(y=y, Ey=Ey, st=st, z=z, Ez=Ez, ext=ext)


def conv_grad(f, x, w, docs, dy, dst, silu):
    T, C = x.shape
    W = w.shape[1]
    z = f["z"]
    s = sig(z)
    dz = dy * s * (1 + z * (1 - s)) if silu else dy
    # |SiLU''| <= 0.5; sigma is off by at most 2 |z| + 6 absolutely weighted with z and 1
    Edz = np.abs(dy) * (0.5 * f["Ez"] + 3 * np.abs(z) + 16) if silu else 0 * dy
    dx, Edx = np.zeros((T, C)), np.zeros((T, C))
    ds0, Eds0 = np.zeros((len(docs), W - 1, C)), np.zeros((len(docs), W - 1, C))
    dw, Edw = np.zeros((C, W)), np.zeros((C, W))
    t0 = 0
    for n, L in enumerate(docs):
        span = slice(t0, t0 + L)
        dX, E, M = (np.zeros((L + W - 1, C)) for _ in range(3))
        for i in range(W):
            X = f["ext"][n][i:i + L]
            dX[i:i + L] += dz[span] * w[:, i]
            E[i:i + L] += Edz[span] * np.abs(w[:, i])
            M[i:i + L] += np.abs(dz[span] * w[:, i])
            dw[:, i] += (dz[span] * X).sum(0)
            Edw[:, i] += (Edz[span] * np.abs(X) + (T + 4) * np.abs(dz[span] * X)).sum(0)
        if dst is not None:
            dX[L:] += dst[n]
            M[L:] += np.abs(dst[n])
        E += (W + 1) * M
        ds0[n], Eds0[n], dx[span], Edx[span] = dX[:W - 1], E[:W - 1], dX[W - 1:], E[W - 1:]
        t0 += L
    db, Edb = dz.sum(0), (Edz + (T + 4) * np.abs(dz)).sum(0)
    return dict(dx=dx, Edx=Edx, dw=dw, Edw=Edw, db=db, Edb=Edb, ds0=ds0, Eds0=Eds0)


# ---- gate ----


def gate(x, a, b, kind, floor):
    """x, b: [T, H, D] and [H, D]; a: [H]."""
    A = np.exp(a)[:, None]
    u = x + b
    Eu = np.abs(u)
    if kind == "softplus":
        raw = -A * np.logaddexp(u, 0)
        return np.maximum(raw, floor), A * sig(u) * Eu + np.abs(raw) * (1.5 * np.abs(np.log(A)) + 20)
    s = sig(A * u)
    return floor * s, np.abs(floor) * (s * (1 - s) * np.abs(A * u) * (1.5 * np.abs(np.log(A)) + 8) + s * 8)


def gate_grad(x, a, b, kind, floor, dg):
    T = x.shape[0]
    A = np.exp(a)[:, None]
    u = x + b
    la = 1.5 * np.abs(np.log(A))
    if kind == "softplus":
        raw = -A * np.logaddexp(u, 0)
        live = raw >= floor
        du, da = np.where(live, -A * sig(u), 0), np.where(live, raw, 0)
        Edu, Eda = A * (sig(u) * (la + 20) + 0.25 * np.abs(u)), np.abs(da) * (la + 20) + A * sig(u) * np.abs(u)
    else:
        s = sig(A * u)
        du = floor * A * s * (1 - s)
        da = du * u
        # s (1 - s) moves by at most itself times the error of A u
        Edu = np.abs(du) * (np.abs(A * u) * (la + 8) + la + 20)
        Eda = Edu * np.abs(u) + 2 * np.abs(da)
    dx, Edx = dg * du, np.abs(dg) * (Edu + np.abs(du))
    t = dg * da
    return dict(dx=dx, Edx=Edx, db=dx.sum(0), Edb=(Edx + (T + 8) * np.abs(dx)).sum(0),
                da=t.sum((0, 2)), Eda=(np.abs(dg) * Eda + (T + 200) * np.abs(t)).sum((0, 2)))


# ---- single-token recurrence ----


def step(q, k, v, g, beta, state, docs, slots, scale, norm, sigm):
    """In place on `state` and its error `E`; returns (o, Eo, state, E).  Rows of o that no live sequence covers are NaN."""
    T, Hv = v.shape[0], v.shape[1]
    rep = Hv // q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    if norm:
        q, k = (t / np.sqrt((t * t).sum(-1, keepdims=True) + 1e-6) for t in (q, k))
    if sigm:
        beta = sig(beta)
    dec = np.exp(g)[..., None] if g.ndim == 3 else np.exp(g)[..., None, None]
    E = np.zeros_like(state)
    o, Eo = np.full(v.shape, np.nan), np.zeros(v.shape)
    n_terms = 40  # 16 products in a lane, 3 lane groups, and a norm's relative error of at most 16
    t0 = 0
    for n, L in enumerate(docs):
        m = slots[n]
        for t in range(t0, t0 + L):
            if not 0 <= m < len(state):
                continue
            Sd = dec[t] * state[m]
            Ed = dec[t] * E[m] + 12 * np.abs(Sd)
            kt, qt = k[t][..., None], q[t][..., None]
            r, p, kq = (kt * Sd).sum(-2), (qt * Sd).sum(-2), (k[t] * q[t]).sum(-1)[..., None]
            Er = (np.abs(kt) * (Ed + n_terms * np.abs(Sd))).sum(-2)
            c = beta[t][..., None] * (v[t] - r)
            Ec = np.abs(beta[t])[..., None] * (Er + (20 + 12 * 1.5) * (np.abs(v[t]) + np.abs(r)))
            state[m] = Sd + kt * c[..., None, :]
            E[m] = Ed + np.abs(kt) * Ec[..., None, :] + 20 * np.abs(kt * c[..., None, :]) + np.abs(state[m])
            o[t] = scale * (p + kq * c)
            Eo[t] = scale * ((np.abs(qt) * (Ed + n_terms * np.abs(Sd))).sum(-2) + np.abs(kq) * Ec
                             + n_terms * (np.abs(k[t] * q[t])).sum(-1)[..., None] * np.abs(c) + 8 * (np.abs(p) + np.abs(kq * c)))
        t0 += L
    return o, Eo, state, E


# ---- norm ----


def _act(z, kind):
    if z is None:
        return 1.0, 0.0, 0.0, 0.0
    s = sig(z)
    rel = 1.5 * np.abs(z) + 8  # relative error of sigma, as above
    if kind == "silu":
        return z * s, np.abs(z * s) * rel, s * (1 + z * (1 - s)), 3 * np.abs(z) + 16
    return s, s * rel, s * (1 - s), s * (1.5 * np.abs(z) + 16)


def norm(x, w, z, res, place, act, alpha, eps):
    D = x.shape[-1]
    depth = min(D, 64) + 16  # squares in a lane, then across lanes; all positive, so relative to the sum
    u, Eu = x, 0 * x
    if place == "before":
        u, Eu = res + alpha * x, 2 * (np.abs(res) + np.abs(alpha * x))
    ms = (u * u).mean(-1, keepdims=True) + eps
    rs = 1 / np.sqrt(ms)
    Ers = rs * (depth / 2 + 8 + ((np.abs(u) * Eu).mean(-1, keepdims=True) / ms))
    a, Ea, _, _ = _act(z, act)
    y = u * rs * w * a
    Ey = np.abs(w) * (np.abs(a) * (rs * Eu + np.abs(u) * Ers) + np.abs(u) * rs * Ea) + 6 * np.abs(y)
    if place == "after":
        Ey = np.abs(alpha) * Ey + 2 * (np.abs(alpha * y) + np.abs(res))
        y = res + alpha * y
    return dict(y=y, Ey=Ey, s=u, Es=Eu)


def norm_grad(u, w, z, dy, ds, place, act, alpha, eps):
    """u: the normed row as the backward reads it (x, or the stored stream)."""
    D = u.shape[-1]
    rows = u.size // D
    depth = min(D, 64) + 16
    rs = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    rel = depth / 2 + 8  # of rs
    a, Ea, da, Eda = _act(z, act)
    t = dy * (alpha if place == "after" else 1.0)
    v = t * a * w
    Ev = np.abs(t * w) * Ea + 4 * np.abs(v)
    m = rs * rs * (v * u).mean(-1, keepdims=True)
    Em = rs * rs * ((Ev + (depth + 2 * rel + 4) * np.abs(v)) * np.abs(u)).mean(-1, keepdims=True)
    d = rs * (v - u * m)
    Ed = rs * (Ev + np.abs(u) * Em + (rel + 4) * (np.abs(v) + np.abs(u * m)))
    out = dict()
    dn = t * a * u * rs
    Edn = np.abs(t * u * rs) * Ea + (rel + 6) * np.abs(dn)
    axes = tuple(range(u.ndim - 1))
    out["dw"], out["Edw"] = dn.sum(axes), (Edn + (rows + 8) * np.abs(dn)).sum(axes)
    if z is not None:
        out["dz"] = t * w * u * rs * da
        out["Edz"] = np.abs(t * w * u * rs) * Eda + (rel + 8) * np.abs(out["dz"])
    if place == "before":
        add = ds if ds is not None else 0.0
        d, Ed = d + add, Ed + np.abs(d) + np.abs(add)
        out["dres"], out["Edres"] = d, Ed
        d, Ed = alpha * d, np.abs(alpha) * Ed + np.abs(alpha * d)
    out["dx"], out["Edx"] = d, Ed
    return out
