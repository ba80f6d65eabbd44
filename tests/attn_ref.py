"""fp64 references of the attention layers' operators, with bounds on what a kernel
that rounds as the library's do may be off by, element for element.

u = 2^-24 is fp32's half step, B = 2^-8 bf16's.  Scores are fp32 sums of 128 products:
each is off by at most 128 u times the sum of the products' magnitudes, and by a few
roundings of itself and of the log-sum-exp; a probability's relative error is that plus the
hardware's 2^t (a few u).  Probabilities and dS are rounded to bf16 (B of themselves),
and sums of them are off by the sum of the terms' errors; outputs are rounded once."""
import math

import numpy as np
import torch

U, B = 2.0 ** -24, 2.0 ** -8
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def seen_mask(Lq, Lk, causal, window, device):
    p = torch.arange(Lq, device=device)[:, None] + Lk - Lq
    j = torch.arange(Lk, device=device)[None]
    seen = j <= p if causal else torch.ones(Lq, Lk, dtype=torch.bool, device=device)
    return seen & (j > p - window) if window else seen


def attention(q, k, v, cu_q, cu_k, causal=True, window=0, scale=None, dout=None):
    """{name: (value, bound)} in fp64; gradients with dout."""
    q, k, v = q.double(), k.double(), v.double()
    Hq, Hkv, D = q.shape[1], k.shape[1], q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    z = torch.zeros_like
    o, eo, dq, eq, dk, ek, dv, ev = z(q), z(q), z(q), z(q), z(k), z(k), z(v), z(v)
    lse = torch.full((Hq, q.shape[0]), -math.inf, dtype=torch.float64, device=q.device)
    el = torch.zeros_like(lse)
    for n in range(len(cu_q) - 1):
        r, c = slice(cu_q[n], cu_q[n + 1]), slice(cu_k[n], cu_k[n + 1])
        Lq, Lk = r.stop - r.start, c.stop - c.start
        if Lq == 0 or Lk == 0:
            continue
        seen = seen_mask(Lq, Lk, causal, window, q.device)
        some = seen.any(1, keepdim=True)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            Q, K, V = q[r, h], k[c, g], v[c, g]
            S = (Q @ K.t() * scale).masked_fill(~seen, -math.inf)
            L = torch.logsumexp(S, 1, keepdim=True)
            P = torch.exp(S - L.masked_fill(~some, 0.0)).masked_fill(~seen, 0.0)
            off = 130 * U * scale * (Q.abs() @ K.abs().t()) + 4 * U * S.abs().masked_fill(~seen, 0.0)
            lse[h, r] = L[:, 0]
            # the largest score's error, the sum's and the logarithm's own
            el[h, r] = (off.masked_fill(~seen, 0.0).amax(1) + 8 * U * (1 + L[:, 0].abs()) + (Lk + 16) * U).masked_fill(~some[:, 0], 0.0)
            rel = off + off.amax(1, keepdim=True) + (Lk + 40) * U
            O = P @ V
            o[r, h] = O
            PV = P @ V.abs()
            eo[r, h] = B * O.abs() + (B * PV + (P * rel) @ V.abs()) * 1.01 + 1e-30
            if dout is None:
                continue
            G = dout[r, h].double()
            dP = G @ V.t()
            delta = (G * O).sum(1, keepdim=True)
            dS = P * (dP - delta)
            dv[c, g] += P.t() @ G
            dq[r, h] = dS @ K * scale
            dk[c, g] += dS.t() @ Q * scale
            edelta = (G.abs() * eo[r, h]).sum(1, keepdim=True) + 130 * U * (G * O).abs().sum(1, keepdim=True)
            rel = rel + el[h, r][:, None] + 4 * U * L.abs().masked_fill(~some, 0.0)
            eS = 1.01 * (B * dS.abs() + P * (edelta + 130 * U * (G.abs() @ V.abs().t())) + rel * P * (dP.abs() + delta.abs())) + 1e-30
            eS = eS.masked_fill(~seen, 0.0)
            ev[c, g] += (1.01 * B * P + rel * P).t() @ G.abs()
            eq[r, h] = eS @ K.abs() * scale
            ek[c, g] += eS.t() @ Q.abs() * scale
    out = {"o": (o, eo), "lse": (lse, el)}
    if dout is not None:
        out.update(dq=(dq, eq + B * dq.abs() + 1e-30), dk=(dk, 1.01 * ek + B * dk.abs() + 1e-30), dv=(dv, 1.01 * ev + B * dv.abs() + 1e-30))
    return out


def rope(x, positions, freqs, layout_half, magnitude=1.0, back=False):
    """(value, bound): x [T, H, D] turned by positions x freqs (turns, fp64)."""
    y = x.double().clone()
    R = 2 * freqs.shape[0]
    turns = positions.double()[:, None] * freqs.double().to(x.device)
    angle = 2 * math.pi * (turns - torch.round(turns)) * (-1 if back else 1)
    cos, sin = torch.cos(angle)[:, None] * magnitude, torch.sin(angle)[:, None] * magnitude
    i = torch.arange(R // 2, device=x.device)
    first, second = (i, i + R // 2) if layout_half else (2 * i, 2 * i + 1)
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    # sine and cosine to 2^-22, their argument to pi 2^-24, the magnitude's product and two roundings of the sum
    e = torch.zeros_like(y)
    e[..., first] = e[..., second] = (a.abs() + b.abs()) * abs(magnitude) * 2.0 ** -20
    return y, e + (B if x.dtype == torch.bfloat16 else U) * y.abs() * (y != x.double()) + 1e-37


def to_4bit(x):
    """numpy fp64 [..., 128] -> (stored values, scale bytes [..., 4], codes [..., 64]) by comparing with every value."""
    b = x.reshape(x.shape[:-1] + (4, 32))
    bad = ~np.isfinite(b).all(-1)
    top = np.abs(np.where(np.isfinite(b), b, 0)).max(-1)
    e = np.full(top.shape, -126)
    for k in range(-125, 128):
        e = np.where(top > 6.0 * 2.0 ** (k - 1), k, e)
    y = np.abs(np.where(np.isfinite(b), b, 0)) * 2.0 ** -e[..., None].astype(np.float64)
    code, best = np.zeros(y.shape, int), np.full(y.shape, np.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they keep the ties
        d = np.where((e[..., None] == 126) & (c > 5), np.inf, np.abs(y - E2M1[c]))  # 4 2^126 is past bf16
        code, best = np.where(d < best, c, code), np.minimum(best, d)
    value = np.where(bad[..., None], np.nan, np.sign(b) * E2M1[code] * 2.0 ** e[..., None].astype(np.float64))
    code = code + 8 * np.signbit(b)
    flat = code.reshape(x.shape)
    scale = np.where(bad, 255, e + 127)
    return value.reshape(x.shape), scale, flat[..., 0::2] | flat[..., 1::2] << 4


def check(name, got, want, bound):
    got = got.double()
    assert torch.isfinite(got).eq(torch.isfinite(want)).all(), "%s: finite in other places" % name
    fine = torch.isfinite(want)
    assert got[~fine].equal(want[~fine]) or torch.isnan(want[~fine]).any(), name
    d, b = (got - want)[fine].abs(), bound[fine]
    if d.numel():
        worst = (d / b.clamp_min(1e-300)).max().item()
        assert worst <= 1.0, "%s: %.3g times its bound (max error %.3g)" % (name, worst, d.max().item())
