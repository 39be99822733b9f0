"""Shaped scores (tanh cap, distance penalty) on the GPU, forward and backward, over the plan forms,
against the 64-bit form of tests/shaped.py with its bounds."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import shaped

pytestmark = pytest.mark.gpu

bfa = pytest.importorskip("mask_skipping_flashattention_b200")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPES = [(30.0, False), (None, True), (8.0, True)]


def _rand(shape, seed, by=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * by).to(torch.bfloat16).cuda()


def _slopes(H):
    return torch.pow(2.0, -8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).cuda()


def _check(plan, q, k, v, dout, mask_of, cap, slopes, scale=None):
    shape = dict(softcap=cap, slopes=slopes, scale=scale)
    out, lse = bfa.fwd(plan, q, k, v, **shape)
    dq, dk, dv = bfa.bwd(plan, q, k, v, out, dout, lse, **shape)
    torch.cuda.synchronize()
    plan.device_status()
    got = dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)
    want, bound = shaped.batch(q, k, v, mask_of, scale, cap, slopes, dout)
    for n in got:
        assert got[n].shape == want[n].shape
        shaped.close(got[n], want[n], bound[n], n)
    return got


def _inputs(B, Sq, Sk, H, Hkv, D, seed, by=2.0):
    return (_rand((B, Sq, H, D), seed, by), _rand((B, Sk, Hkv, D), seed + 1), _rand((B, Sk, Hkv, D), seed + 2),
            _rand((B, Sq, H, D), seed + 3))


def _causal(Sq, Sk, window=0):
    d = torch.arange(Sq, device="cuda")[:, None] - torch.arange(Sk, device="cuda")
    m = d >= 0
    return m & (d < window) if window else m


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES)
@pytest.mark.parametrize("Sq,Sk,density", [(300, 300, 0.3), (129, 257, 0.9), (1, 1, 1.0), (5, 700, 0.02)])
def test_dense_masks_with_empty_rows(D, cap, with_slopes, Sq, Sk, density):
    rng = np.random.default_rng(Sq + Sk + D)
    M = torch.from_numpy(rng.random((Sq, Sk)) < density).cuda()
    if Sq > 3:
        M[2] = False
        M[:, Sk // 2] = False
    q, k, v, dout = _inputs(1, Sq, Sk, 2, 1, D, 100 + Sq)
    got = _check(bfa.plan_dense(M), q, k, v, dout, lambda b, h: M, cap, _slopes(2) if with_slopes else None)
    if Sq > 3:  # what attends nothing, or is attended by nothing, is exactly 0
        assert got["out"][:, 2].abs().max() == 0 and got["dq"][:, 2].abs().max() == 0
        assert got["dk"][:, Sk // 2].abs().max() == 0 and got["dv"][:, Sk // 2].abs().max() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES)
@pytest.mark.parametrize("H,Hkv,window", [(4, 2, 0), (3, 1, 0), (4, 4, 100)])
def test_causal_batches(D, cap, with_slopes, H, Hkv, window):
    B, S = 2, 333
    q, k, v, dout = _inputs(B, S, S, H, Hkv, D, 7 * H + D)
    plan = bfa.plan_blockids(B=B, Sq=S, Sk=S, window_left=window or -1)
    M = _causal(S, S, window)
    _check(plan, q, k, v, dout, lambda b, h: M, cap, _slopes(H) if with_slopes else None)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES)
def test_prefix_in_front_of_a_causal_text(D, cap, with_slopes):
    S, P = 500, 200
    q, k, v, dout = _inputs(1, S, S, 2, 2, D, 31)
    M = _causal(S, S) | (torch.arange(S, device="cuda") < P)[None, :]
    plan = bfa.plan_predicate([dict(diag_lo=0), dict(k_hi=P)], B=1, Sq=S, Sk=S)
    _check(plan, q, k, v, dout, lambda b, h: M, cap, _slopes(2) if with_slopes else None, scale=0.2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES)
def test_packed_documents(D, cap, with_slopes):
    lens = [130, 0, 1, 257, 128, 64]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T, H, Hkv = int(cu[-1]), 4, 2
    q, k, v, dout = (x[0] for x in _inputs(1, T, T, H, Hkv, D, 53))
    plan = bfa.plan_blockids(cu_seqlens_q=torch.from_numpy(cu).cuda(), max_q=max(lens), max_k=max(lens))
    shape = dict(softcap=cap, slopes=_slopes(H) if with_slopes else None)
    out, lse = bfa.fwd(plan, q, k, v, **shape)
    dq, dk, dv = bfa.bwd(plan, q, k, v, out, dout, lse, **shape)
    torch.cuda.synchronize()
    plan.device_status()
    for a, b in zip(cu[:-1], cu[1:]):
        if a == b:
            continue
        M = _causal(b - a, b - a)
        want, bound = shaped.batch(q[None, a:b], k[None, a:b], v[None, a:b], lambda *_: M, None, cap,
                                   shape["slopes"], dout[None, a:b])
        got = dict(out=out[None, a:b], lse=lse[None, :, a:b], dq=dq[None, a:b], dk=dk[None, a:b], dv=dv[None, a:b])
        for n in got:
            shaped.close(got[n], want[n], bound[n], f"{n} of document {a}:{b}")


def test_block_ids_with_cross_columns():
    B, N, C, H, D = 2, 200, 60, 2, 128
    pad = torch.ones(B, N, dtype=torch.bool)
    pad[1, 150:] = False
    att = torch.zeros(B, N, dtype=torch.bool)
    att[:, [0, 40, 41, 130]] = True
    cross = torch.ones(B, C, dtype=torch.bool)
    cross[0, 10:20] = False
    ids = bfa.make_att_block_ids(pad.cuda(), att.cuda(), C, cross.cuda())
    qb, kb, qv, kv = ids
    M = qv[:, :, None] & kv[:, None, :] & (kb[:, None, :] <= qb[:, :, None])
    q, k, v, dout = _inputs(B, N, N + C, H, H, D, 71)
    _check(bfa.plan_blockids(*ids), q, k, v, dout, lambda b, h: M[b], 20.0, _slopes(H))


def test_block_sparse_routing():
    B, S, H, Hkv, D = 1, 512, 4, 2, 64
    indptr = torch.tensor([[[0, 1, 3, 5, 8], [8, 9, 10, 12, 14]]], dtype=torch.int32).cuda()
    indices = torch.tensor([0, 0, 1, 0, 2, 0, 1, 3, 0, 1, 1, 2, 0, 3], dtype=torch.int32).cuda()
    plan = bfa.plan_bsr(indptr, indices, S, S, causal=True)
    M = torch.zeros(Hkv, S, S, dtype=torch.bool, device="cuda")
    for h in range(Hkv):
        for r in range(4):
            for c in indices[indptr[0, h, r]:indptr[0, h, r + 1]].tolist():
                M[h, 128 * r:128 * r + 128, 128 * c:128 * c + 128] = True
    M &= _causal(S, S)
    q, k, v, dout = _inputs(B, S, S, H, Hkv, D, 81)
    _check(plan, q, k, v, dout, lambda b, h: M[h], 15.0, _slopes(H))
    packed = bfa.plan_bsr_packed(indptr, indices, S, S, H // Hkv, causal=True)
    with pytest.raises(bfa.BfaError) as e:
        bfa.fwd(packed, q, k, v, softcap=15.0)
    assert e.value.status == "BFA_ERR_UNSUPPORTED"


@pytest.mark.parametrize("D", [64, 128])
def test_scores_far_beyond_the_cap(D):
    # products up to some 2000 under a cap of 3: the tanh is flat nearly everywhere
    S = 260
    q, k, v, dout = _inputs(1, S, S, 2, 2, D, 91, by=40.0)
    M = _causal(S, S)
    _check(bfa.plan_blockids(B=1, Sq=S, Sk=S), q, k, v, dout, lambda b, h: M, 3.0, None, scale=1.0)


@pytest.mark.parametrize("cap", [1e-3, 1e6])
def test_the_caps_at_the_ends_of_their_range(cap):
    S, D = 200, 64
    q, k, v, dout = _inputs(1, S, S, 2, 2, D, 93)
    M = _causal(S, S)
    _check(bfa.plan_blockids(B=1, Sq=S, Sk=S), q, k, v, dout, lambda b, h: M, cap, None)


def test_slopes_of_any_sign_and_none():
    S, D, H = 300, 128, 4
    slopes = torch.tensor([0.0, -0.05, 3.0, 0.5], device="cuda")
    q, k, v, dout = _inputs(2, S, S, H, H, D, 95)
    M = torch.ones(S, S, dtype=torch.bool, device="cuda")
    _check(bfa.plan_dense(M), q, k, v, dout, lambda b, h: M, None, slopes)


@pytest.mark.parametrize("cap,with_slopes", SHAPES)
def test_two_pass_form_at_128(cap, with_slopes):
    S, D, H = 400, 128, 4
    q, k, v, dout = _inputs(1, S, S, H, 2, D, 97)
    M = _causal(S, S)
    plan = bfa.plan_blockids(B=1, Sq=S, Sk=S)
    bfa.set_bwd_deterministic(True)
    try:
        a = _check(plan, q, k, v, dout, lambda b, h: M, cap, _slopes(H) if with_slopes else None)
        b = _check(plan, q, k, v, dout, lambda b, h: M, cap, _slopes(H) if with_slopes else None)
        assert all(torch.equal(a[n], b[n]) for n in a)
    finally:
        bfa.set_bwd_deterministic(False)


def test_strides_and_given_results():
    B, S, H, D = 2, 190, 2, 64
    M = _causal(S, S)
    plan = bfa.plan_blockids(B=B, Sq=S, Sk=S)
    qkv = _rand((B, S, 3, H, D), 101)  # one projection's output, token-major
    q, k, v = qkv.unbind(2)
    dout = _rand((B, H, S, D), 102).transpose(1, 2)  # head-major storage
    want, bound = shaped.batch(q, k, v, lambda *_: M, None, 9.0, _slopes(H), dout)
    wide = torch.full((B, S, H, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = bfa.fwd(plan, q, k, v, softcap=9.0, slopes=_slopes(H), out=wide[..., :D])
    grads = torch.full((3, B, S, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    dq, dk, dv = bfa.bwd(plan, q, k, v, out, dout, lse, softcap=9.0, slopes=_slopes(H), dq=grads[0], dk=grads[1],
                         dv=grads[2])
    torch.cuda.synchronize()
    assert (wide[..., D:] == 7).all() and dq.data_ptr() == grads.data_ptr()
    for n, got in dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv).items():
        shaped.close(got, want[n], bound[n], n)


def test_another_stream_and_a_captured_step():
    B, S, H, D = 1, 300, 2, 64  # the reproducible form: equal bit for bit
    plan = bfa.plan_blockids(B=B, Sq=S, Sk=S)
    q, k, v, dout = _inputs(B, S, S, H, H, D, 111)
    shape = dict(softcap=12.0, slopes=_slopes(H))

    def step(stream=None):
        out, lse = bfa.fwd(plan, q, k, v, stream=stream, **shape)
        return (out, lse) + bfa.bwd(plan, q, k, v, out, dout, lse, stream=stream, **shape)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    q2 = _rand(q.shape, 999)
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    eager = step()
    assert all(torch.equal(a, b) for a, b in zip(captured, eager))
    assert not torch.equal(captured[0], want[0])


def test_long_rows_in_a_later_tile():
    # the row maxima move late, and the penalty changes direction inside a tile
    S, D = 2100, 128
    q, k, v, dout = _inputs(1, S, S, 2, 1, D, 121)
    k[:, 1500:] *= 3
    M = torch.ones(S, S, dtype=torch.bool, device="cuda")
    _check(bfa.plan_dense(M), q, k, v, dout, lambda b, h: M, 50.0, torch.tensor([0.01, 0.002], device="cuda"))


CHECKED = ["test_dense_masks_with_empty_rows", "test_causal_batches", "test_packed_documents",
           "test_block_sparse_routing", "test_two_pass_form_at_128"]


def test_the_checked_build_finds_no_index_out_of_bounds():
    if os.environ.get("BFA_LIBRARY") == "checked":
        pytest.skip("already the checked build")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu", "-p", "no:cacheprovider"] +
                       [f"tests/test_gpu_shaped.py::{n}" for n in CHECKED],
                       cwd=ROOT, env=dict(os.environ, BFA_LIBRARY="checked"), capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES)
def test_a_row_with_a_single_key_has_no_query_gradient(D, cap, with_slopes):
    # its weight is 1 whatever the query, so dP - D must cancel: D of such rows comes from the same
    # products as dP, and what is left is the weights' error (2^-18) of |dP|, not the output's rounding
    lens = [1, 5, 1, 300, 2]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    T, H = sum(lens), 2
    q, k, v, dout = (x[0] for x in _inputs(1, T, T, H, H, D, 17, by=4.0))
    plan = bfa.plan_blockids(cu_seqlens_q=cu, max_q=300, max_k=300)
    shape = dict(softcap=cap, slopes=_slopes(H) if with_slopes else None)
    out, lse = bfa.fwd(plan, q, k, v, **shape)
    dq = bfa.bwd(plan, q, k, v, out, dout, lse, **shape)[0]
    first = cu[:-1].long()
    dp = (dout[first].double().abs() * v[first].double().abs()).sum(-1, keepdim=True)
    bound = D ** -0.5 * k[first].double().abs() * dp * 2.0 ** -18
    shaped.close(dq[first], torch.zeros_like(bound), bound + 1e-9, "dq of the first tokens")


def test_repeated_data_is_refused():
    # an expanded tensor has a stride of 0, which the tensor maps cannot hold
    S, H, D = 130, 4, 64
    q, k, v, dout = _inputs(2, S, S, H, H, D, 131)
    plan = bfa.plan_blockids(B=2, Sq=S, Sk=S)
    out, lse = bfa.fwd(plan, q, k, v, softcap=9.0)
    for bad in (k[:, :, :1].expand(2, S, H, D), k[:1].expand(2, S, H, D), k[:, :1].expand(2, S, H, D)):
        with pytest.raises(bfa.BfaError) as e:
            bfa.fwd(plan, q, bad, v, softcap=9.0)
        assert e.value.status == "BFA_ERR_UNSUPPORTED"
    with pytest.raises(bfa.BfaError) as e:
        bfa.bwd(plan, q, k, v, out, dout[:, :1].expand(2, S, H, D), lse, softcap=9.0)
    assert e.value.status == "BFA_ERR_UNSUPPORTED"


@pytest.mark.parametrize("by", [1.0, 80.0])  # scores inside the polynomials' range, and far past it
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES)
def test_nan_reaches_every_row_that_attends_it(by, D, cap, with_slopes):
    S, H, row, key = 200, 2, 70, 150
    q, k, v, _ = _inputs(1, S, S, H, H, D, 31, by)
    slopes = _slopes(H) if with_slopes else None
    plan = bfa.plan_blockids(B=1, Sq=S, Sk=S)
    q[0, row, 0, 3] = float("nan")
    k[0, key, 1, 5] = float("nan")
    out, _ = bfa.fwd(plan, q, k, v, softcap=cap, slopes=slopes)
    nan = out[0].isnan()
    want = torch.zeros(S, H, dtype=torch.bool, device="cuda")
    want[row, 0] = True
    want[key:, 1] = True  # causal: the rows from the key on
    assert torch.equal(nan.all(-1), want) and torch.equal(nan.any(-1), want)


# few columns: a kv head's query heads are shared between CTAs, evenly or not
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,B,S", [(2, 1, 1, 130), (3, 1, 2, 77), (5, 1, 1, 300), (16, 2, 1, 200), (8, 4, 1, 2100)])
def test_query_heads_shared_between_blocks(D, H, Hkv, B, S):
    q, k, v, dout = _inputs(B, S, S, H, Hkv, D, 51 + H)
    plan = bfa.plan_blockids(B=B, Sq=S, Sk=S)
    _check(plan, q, k, v, dout, lambda b, h: _causal(S, S), 30.0, _slopes(H))


@pytest.mark.parametrize("D", [64, 128])
def test_shared_query_heads_into_strided_results_and_empty_columns(D):
    B, S, H, Hkv = 1, 300, 7, 1
    q, k, v, dout = _inputs(B, S, S, H, Hkv, D, 61)
    mask = torch.zeros(S, S, dtype=torch.bool, device="cuda")
    mask[:, 140:200] = True  # the first and the last key tile are attended by no query
    mask[17] = False
    plan = bfa.plan_dense(mask)
    out, lse = bfa.fwd(plan, q, k, v, softcap=30.0)
    want = bfa.bwd(plan, q, k, v, out, dout, lse, softcap=30.0)
    wide = [torch.full((B, S, 3, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dk, dv = (w[:, :, 1:2, D:] for w in wide)
    bfa.bwd(plan, q, k, v, out, dout, lse, softcap=30.0, dk=dk, dv=dv)
    assert torch.equal(dk, want[1]) and torch.equal(dv, want[2])  # the shares are added in one order
    for w, name in zip(wide, ("dk", "dv")):
        w[:, :, 1:2, D:] = 7.0
        assert (w == 7.0).all(), name
    for g in want[1:]:
        assert not g[:, :140].any() and not g[:, 200:].any() and g[:, 140:200].any()
    _check(plan, q, k, v, dout, lambda b, h: mask, 30.0, None)


def _nan_inputs(D, H=2, S=300):
    q, k, v, dout = _inputs(1, S, S, H, H, D, 33)
    return q, k, v, dout, bfa.plan_blockids(B=1, Sq=S, Sk=S)


@pytest.mark.parametrize("two_pass", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,with_slopes", SHAPES + [(None, False)])
def test_a_nan_score_shows_in_the_lse_and_in_every_gradient(two_pass, D, cap, with_slopes):
    # an lse of -inf is a row that attends nothing, and the backward takes it for that
    S, H, row, key = 300, 2, 70, 200
    q, k, v, dout, plan = _nan_inputs(D, H, S)
    shape = dict(softcap=cap, slopes=_slopes(H) if with_slopes else None)
    q[0, row, 0, 3] = float("nan")
    k[0, key, 1, 5] = float("nan")
    out, lse = bfa.fwd(plan, q, k, v, **shape)
    bad = torch.zeros(H, S, dtype=torch.bool, device="cuda")
    bad[0, row] = True
    bad[1, key:] = True  # causal: the rows from the key on
    assert torch.equal(lse[0].isnan(), bad) and torch.isfinite(lse[0][~bad]).all()
    bfa.set_bwd_deterministic(two_pass)
    try:
        dq, dk, dv = bfa.bwd(plan, q, k, v, out, dout, lse, **shape)
    finally:
        bfa.set_bwd_deterministic(False)
    assert torch.equal(dq[0, :, 0].isnan().all(-1), bad[0]) and torch.equal(dq[0, :, 0].isnan().any(-1), bad[0])
    assert dq[0, key:, 1].isnan().all() and torch.isfinite(dq[0, :128, 1].float()).all()
    # every key that such a row attends
    assert dv[0, :row + 1, 0].isnan().all() and dk[0, :row + 1, 0].isnan().all()
    assert dv[0, :, 1].isnan().all() and dk[0, :, 1].isnan().all()
    # key tiles that head 0's poisoned row does not reach
    assert torch.isfinite(dv[0, 128:, 0].float()).all() and torch.isfinite(dk[0, 128:, 0].float()).all()


@pytest.mark.parametrize("D", [64, 128])
def test_an_infinite_score_is_no_empty_row(D):
    S, H, key = 300, 2, 200
    q, k, v, dout, plan = _nan_inputs(D, H, S)
    q[0, :, 1, 5], k[0, key, 1, 5] = 1.0, float("inf")  # a score of +inf in head 1
    lse = bfa.fwd(plan, q, k, v, slopes=_slopes(H))[1]
    assert not torch.isneginf(lse).any()
    assert torch.isfinite(lse[0, 0]).all() and torch.isfinite(lse[0, 1, :key]).all()
    assert not torch.isfinite(lse[0, 1, key:]).any()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq,Sk,window", [(256, 8192, 0), (8192, 8192, 200)])
def test_short_columns_are_not_shared_between_blocks(D, Sq, Sk, window):
    # 256 columns of two or three query tiles: sharing their heads costs more than it gives.  With the
    # batch doubled there are too many columns to share any, so equal bits are one share's order of sums
    H, Hkv = 8, 4
    q, k, v, dout = _inputs(1, Sq, Sk, H, Hkv, D, 141)
    slopes, grads = _slopes(H), []
    for B in (1, 2):
        if window:
            plan = bfa.plan_blockids(B=B, Sq=Sq, Sk=Sk, window_left=window)
        else:
            plan = bfa.plan_predicate([dict(k_lo=0)], B=B, Sq=Sq, Sk=Sk)
        x = [t.repeat(B, 1, 1, 1) for t in (q, k, v, dout)]
        out, lse = bfa.fwd(plan, *x[:3], softcap=30.0, slopes=slopes)
        grads.append(bfa.bwd(plan, *x[:3], out, x[3], lse, softcap=30.0, slopes=slopes))
    assert torch.equal(grads[0][1][0], grads[1][1][0]) and torch.equal(grads[0][2][0], grads[1][2][0])
