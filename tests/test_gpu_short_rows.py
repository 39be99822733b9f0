"""Gradients of rows that attend few keys, with shaped scores.

Where a row's weight lies on few keys, dP - D nearly cancels, and D = dO . O from the output
that was rounded to bf16 twice is most of what is left.  Rows of one or two key tiles therefore
take D from the scores themselves, whatever else is in the call.

The bound of dS is that of tests/shaped.py with another error of D.  With D0 = dO . O (off by
|dO| . bound of out) and the kernel's weights P (1 + e), |e| <= w, the refined value is
  D0 + sum P (1 + e) (dP + e_dP - D0)  =  D + sum P e (dP - D0) + sum P (1 + e) e_dP,
D = sum P dP, since sum P = 1.  So
  e_D = w sum P (|dP - D| + |dO| . bound of out) + (1 + w) sum P e_dP + 2^-18 sum P |dP - D0|,
the last for the sums in fp32 (at most 256 terms, each product and sum off by 2^-24 of the sum of
magnitudes, below 2^-18 with those of the dropped second-order terms), and 2^-24 |D| for its storage.
"""

import numpy as np
import pytest
import torch

import shaped

pytestmark = pytest.mark.gpu

bfa = pytest.importorskip("mask_skipping_flashattention_b200")

SHAPES = [(30.0, False), (None, True), (8.0, True)]


def _rand(shape, seed, by=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * by).to(torch.bfloat16).cuda()


def _slopes(H):
    return torch.pow(2.0, -8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).cuda()


def _inputs(T, H, Hkv, D, seed, by):
    return (_rand((T, H, D), seed, by), _rand((T, Hkv, D), seed + 1), _rand((T, Hkv, D), seed + 2),
            _rand((T, H, D), seed + 3))


def refined_bounds(q, k, v, dout, mask, distance, scale, cap, slope):
    """(dq, dk) of one head in 64 bits and their bounds where every row's D is refined."""
    _, bound = shaped.head(q, k, v, mask, distance, scale, cap, slope, dout)
    q, k, v, dout = q.double(), k.double(), v.double(), dout.double()
    D = q.shape[1]
    raw = q @ k.t() * scale
    t = torch.tanh(raw / cap) if cap else None
    z = cap * t if cap else raw
    delta = D * 2.0 ** -24 * (q.abs() @ k.abs().t() * scale) + 2.0 ** -20 * z.abs()
    if slope is not None:
        z = z - float(slope) * distance.double()
        delta = delta + 2.0 ** -20 * abs(float(slope)) * distance.double()
    P = torch.softmax(z.masked_fill(~mask, -torch.inf), 1)
    w = 3 * (delta * mask * (P > 1e-12)).amax(1, keepdim=True) + 2.0 ** -18
    f = 1 - t * t if cap else torch.ones_like(P)
    dP = dout @ v.t()
    Dv = (P * dP).sum(1, keepdim=True)
    e_dP = D * 2.0 ** -24 * (dout.abs() @ v.abs().t())
    e_out = (dout.abs() * bound["out"]).sum(1, keepdim=True)
    apart = (P * ((dP - Dv).abs() + e_out)).sum(1, keepdim=True)
    e_D = (w + 2.0 ** -18) * apart + (1 + w) * (P * e_dP).sum(1, keepdim=True) + 2.0 ** -24 * Dv.abs()
    dS = P * f * (dP - Dv)
    e_dS = (w + shaped.U) * dS.abs() + P * f * (e_dP + e_D) + 2.0 ** -19 * P * (dP.abs() + Dv.abs())
    dq, dk = dS @ k * scale, dS.t() @ q * scale
    return ((dq, scale * (e_dS @ k.abs()) + shaped.U * dq.abs() + 1e-9),
            (dk, scale * (e_dS.t() @ q.abs()) + shaped.U * dk.abs() + 1e-9))


def _check_block(q, k, v, dout, dq, dk, mask, distance, cap, slopes, name):
    """dq and dk (n, heads, D) of one block of tokens against the refined bounds (H = Hkv)."""
    for h in range(q.shape[1]):
        (wq, bq), (wk, bk) = refined_bounds(q[:, h], k[:, h], v[:, h], dout[:, h], mask, distance, q.shape[2] ** -0.5,
                                            cap, None if slopes is None else slopes[h])
        shaped.close(dq[:, h], wq, bq, f"dq of {name}, head {h}")
        shaped.close(dk[:, h], wk, bk, f"dk of {name}, head {h}")


def _causal(n):
    d = torch.arange(n, device="cuda")[:, None] - torch.arange(n, device="cuda")
    return d >= 0, d.abs()


def _documents(lens):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, bfa.plan_blockids(cu_seqlens_q=torch.from_numpy(cu).cuda(), max_q=max(lens), max_k=max(lens))


def _step(plan, q, k, v, dout, shape):
    out, lse = bfa.fwd(plan, q, k, v, **shape)
    return (out, lse) + bfa.bwd(plan, q, k, v, out, dout, lse, **shape)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES)
@pytest.mark.parametrize("neighbour", [0, 2100])
def test_short_documents_of_peaked_scores(D, cap, with_slopes, neighbour):
    lens = [2, 30, 7, 1, 19, 130, 3, 256, 12] + ([neighbour] if neighbour else [])
    cu, plan = _documents(lens)
    H = 2
    slopes = _slopes(H) if with_slopes else None
    q, k, v, dout = _inputs(int(cu[-1]), H, H, D, 61, 8.0)
    _, _, dq, dk, _ = _step(plan, q, k, v, dout, dict(softcap=cap, slopes=slopes))
    for a, b in zip(cu[:9], cu[1:10]):
        _check_block(q[a:b], k[a:b], v[a:b], dout[a:b], dq[a:b], dk[a:b], *_causal(b - a), cap, slopes,
                     f"document {a}:{b}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES)
def test_a_long_neighbour_changes_no_bit_of_a_short_document(D, cap, with_slopes):
    lens, H = [20, 130, 3, 256, 64, 300], 2
    slopes = _slopes(H) if with_slopes else None
    cu, alone = _documents(lens)
    _, beside = _documents([2100] + lens)  # in front: what follows the documents stays the same
    x = _inputs(2100 + int(cu[-1]), H, H, D, 67, 4.0)
    bfa.set_bwd_deterministic(True)  # the form whose results repeat bit for bit
    try:
        want = _step(alone, *(t[2100:].contiguous() for t in x), dict(softcap=cap, slopes=slopes))
        got = _step(beside, *x, dict(softcap=cap, slopes=slopes))
    finally:
        bfa.set_bwd_deterministic(False)
    for name, a, b in zip(("out", "lse", "dq", "dk", "dv"), got, want):
        assert torch.equal(a[:, 2100:] if name == "lse" else a[2100:], b), name


# masks over a grid of more than 16 key tiles whose rows list one or two
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES)
@pytest.mark.parametrize("form", ["dense", "blockids", "predicate", "window", "window, more queries than keys"])
def test_short_rows_of_a_wide_grid(D, cap, with_slopes, form):
    H, S, n = 2, 2304, 32
    Sk = S
    i = torch.arange(S, device="cuda")
    d = i[:, None] - i
    if form.startswith("window"):
        mask = (d >= 0) & (d < 6)
        if form != "window":
            Sk, mask = 2100, mask[:, :2100]
        plan = bfa.plan_blockids(B=1, Sq=S, Sk=Sk, window_left=6)
    else:
        mask = (d >= 0) & (i[:, None] // n == i // n)  # documents of 32 tokens
        if form == "dense":
            plan = bfa.plan_dense(mask)
        elif form == "predicate":
            mask = (d >= 0) & (d <= 3)
            plan = bfa.plan_predicate([dict(diag_lo=0, diag_hi=3)], B=1, Sq=S, Sk=S)
        else:  # the first key block is seen by every query, the others (invalid) by none
            valid = (i < 5)[None]
            ids = (i[None] // 5).to(torch.int32)
            mask = (i < 5)[None].expand(S, S)
            plan = bfa.plan_blockids(ids, ids, torch.ones_like(valid), valid)
    slopes = _slopes(H) if with_slopes else None
    q, k, v, dout = _inputs(S, H, H, D, 71, 8.0)
    k, v = k[:Sk], v[:Sk]
    _, _, dq, dk, _ = _step(plan, q[None], k[None], v[None], dout[None], dict(softcap=cap, slopes=slopes))
    some = mask.any(1)
    assert not dq[0][~some].any()
    _check_block(q[some], k, v, dout[some], dq[0][some], dk[0], mask[some], d[:, :Sk].abs()[some], cap, slopes, form)
