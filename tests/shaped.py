"""Plain 64-bit forms of the shaped-score attention and of rotary positions, with error bounds.

The bounds follow the kernels' arithmetic.  u = 2^-8 is half a step of bf16, the most one
rounding to it can be off (relative).
  scores   products of bf16 are exact in fp32; their sum over D terms is off by at most
           D * 2^-24 * sum |q_d k_d|, and the tanh, the penalty and the scale by 2^-20 of the
           parts they add up: delta per score;
  weights  P = exp(z - lse) is off by exp(delta of z + delta of lse) and the exponential's own
           error, together below a relative w = 3 * (largest delta of the row) + 2^-18;
  out      P is rounded to bf16 before P V (u of each term) and the sum once more (u):
           (2 u + w) * (P |V|);
  D        dO . out from the rounded out: |dO| . (bound of out);
  dS       w + u of itself (its rounding), plus P f times the errors of dP (D * 2^-24 sum
           |dO V|) and of D, and 2^-19 of P (|dP| + |D|) for the cap's factor f = 1 - tanh^2;
  dq, dk   scale times |dS's error| against |K| or |Q|, and u for the final rounding;
  dv       (2 u + w) * (P^T |dO|).
Sums over the query heads of a kv head add their bounds.
"""

import math

import torch

U = 2.0 ** -8


def head(q, k, v, mask, distance, scale, cap, slope, dout=None):
    """One head: q (n, D), k, v (m, D) any float type; mask (n, m).  Results and bounds as dicts of double tensors."""
    q, k, v = q.double(), k.double(), v.double()
    D = q.shape[1]
    raw = q @ k.t() * scale
    t = torch.tanh(raw / cap) if cap else None
    z = cap * t if cap else raw
    size = q.abs() @ k.abs().t() * scale
    delta = D * 2.0 ** -24 * size + 2.0 ** -20 * z.abs()
    if slope is not None:
        z = z - float(slope) * distance.double()
        delta = delta + 2.0 ** -20 * abs(float(slope)) * distance.double()
    z = z.masked_fill(~mask, -math.inf)
    delta = delta.masked_fill(~mask, 0.0)
    lse = torch.logsumexp(z, 1)
    P = torch.exp(z - lse.masked_fill(lse == -math.inf, 0.0)[:, None])
    # a score far below the row's maximum weighs nothing, whatever its error
    d_row = (delta * (P > 1e-12)).amax(1, keepdim=True) if delta.shape[1] else delta.sum(1, keepdim=True)
    w = 3 * d_row + 2.0 ** -18
    out = P @ v
    b_out = (2 * U + w) * (P @ v.abs()) + 1e-9
    res = dict(out=out, lse=lse)
    bound = dict(out=b_out, lse=(d_row.squeeze(1) + 2.0 ** -20 * (1 + lse.abs().masked_fill(lse == -math.inf, 0.0))))
    if dout is not None:
        dout = dout.double()
        dP = dout @ v.t()
        Dv = (dout * out).sum(1, keepdim=True)
        f = 1 - t * t if cap else torch.ones_like(P)
        dS = P * f * (dP - Dv)
        e_dP = D * 2.0 ** -24 * (dout.abs() @ v.abs().t())
        e_D = (dout.abs() * b_out).sum(1, keepdim=True)
        e_dS = (w + U) * dS.abs() + P * f * (e_dP + e_D) + 2.0 ** -19 * P * (dP.abs() + Dv.abs())
        res.update(dq=dS @ k * scale, dk=dS.t() @ q * scale, dv=P.t() @ dout)
        bound.update(dq=scale * (e_dS @ k.abs()) + U * res["dq"].abs() + 1e-9,
                     dk=scale * (e_dS.t() @ q.abs()) + U * res["dk"].abs() + 1e-9,
                     dv=(P * (2 * U + w)).t() @ dout.abs() + 1e-9)
    return res, bound


def batch(q, k, v, mask_of, scale=None, cap=None, slopes=None, dout=None, distance=None):
    """(B, S, H, D) tensors; mask_of(b, kv head) -> (Sq, Sk) bool on the same device."""
    B, Sq, H, D = q.shape
    Sk, Hkv = k.shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    if distance is None:
        distance = (torch.arange(Sq, device=q.device)[:, None] - torch.arange(Sk, device=q.device)).abs()
    names = ("out", "dq", "dk", "dv") if dout is not None else ("out",)
    like = dict(out=q, dq=q, dk=k, dv=k)
    res = {n: torch.zeros(like[n].shape, dtype=torch.float64, device=q.device) for n in names}
    bnd = {n: torch.zeros_like(res[n]) for n in names}
    res["lse"] = torch.zeros(B, H, Sq, dtype=torch.float64, device=q.device)
    bnd["lse"] = torch.zeros_like(res["lse"])
    for b in range(B):
        for h in range(H):
            kh = h // (H // Hkv)
            r, e = head(q[b, :, h], k[b, :, kh], v[b, :, kh], mask_of(b, kh), distance, scale, cap,
                        None if slopes is None else slopes[h], None if dout is None else dout[b, :, h])
            for n in names:
                at = kh if n in ("dk", "dv") else h
                res[n][b, :, at] += r[n]
                bnd[n][b, :, at] += e[n]
            res["lse"][b, h], bnd["lse"][b, h] = r["lse"], e["lse"]
    return res, bnd


def close(got, want, bound, name):
    """Every value of ``got`` within its own bound of ``want`` (infinities alike)."""
    got, want = got.double(), want.to(got.device)
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got) & (got < 0), inf & (want < 0)), f"{name}: -inf in other places"
    err = (got - want).masked_fill(inf, 0.0).abs()
    bound = bound.to(got.device).masked_fill(inf, 1.0)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound).nan_to_num(1e9).max()):.2f} "
                           f"of its bound, first at {bad.nonzero()[0].tolist()}")


def rotate(x, positions, inv_freq, interleaved, amplitude, inverse):
    """x (..., H, D) and positions (...): rotary positions in 64 bits."""
    r = 2 * inv_freq.numel()
    angle = positions.double()[..., None, None] * inv_freq * (-1.0 if inverse else 1.0)
    c, s = torch.cos(angle) * amplitude, torch.sin(angle) * amplitude
    y = x.double().clone()
    a, b = (y[..., 0:r:2].clone(), y[..., 1:r:2].clone()) if interleaved else (y[..., :r // 2].clone(),
                                                                              y[..., r // 2:r].clone())
    first, second = a * c - b * s, a * s + b * c
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = first, second
    else:
        y[..., :r // 2], y[..., r // 2:r] = first, second
    return y


def rotate_bound(x, want, amplitude):
    """bf16's rounding of the result, and 2^-21 of the two values that meet (cos and sin in fp32)."""
    return U * want.abs() + 2.0 ** -21 * 2 * abs(amplitude) * x.double().abs().amax(-1, keepdim=True) + 1e-30
