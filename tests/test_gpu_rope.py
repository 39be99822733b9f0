"""Rotary positions and the paged cache's writer, and the operators run together as a model runs them."""

import numpy as np
import pytest
import torch

import shaped

pytestmark = pytest.mark.gpu

bfa = pytest.importorskip("mask_skipping_flashattention_b200")


def _rand(shape, seed, by=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * by).to(torch.bfloat16)


def _close(got, x, positions, f, interleaved, amplitude, inverse, name="rope"):
    want = shaped.rotate(x, positions, f, interleaved, amplitude, inverse)
    shaped.close(got, want, shaped.rotate_bound(x, want, amplitude), name)


@pytest.mark.parametrize("D,rotary", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 80)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(D, rotary, interleaved, inverse):
    f = bfa.rope_frequencies(rotary)
    for B, S, H, first in ((1, 1, 1, 0), (2, 77, 3, 5), (3, 130, 32, 999_000)):
        x = _rand((B, S, H, D), S)
        p = first + torch.arange(B * S, device="cuda").reshape(B, S)
        y = bfa.rope(x, p, f, interleaved=interleaved, inverse=inverse, amplitude=1.2)
        _close(y, x, p, f, interleaved, 1.2, inverse)
        assert torch.equal(y[..., rotary:], x[..., rotary:])


def test_rope_forms_of_the_arguments():
    f = bfa.rope_frequencies(64, 500000.0, factor=8.0, ramp=(8192, 1.0, 32.0))
    x = _rand((2, 50, 3, 4, 64), 3)[:, :, 1]  # a slice of a fused projection
    p = torch.randint(-50, 10 ** 6, (2, 50), device="cuda", dtype=torch.int32)
    _close(bfa.rope(x, p, f), x, p, f, False, 1.0, False)
    # one row of positions for every batch row, packed tokens, positions beyond 32 bits
    _close(bfa.rope(x, p[0], f), x, p[0].expand(2, 50), f, False, 1.0, False)
    t = x[0]
    far = p[0].long() + 2 ** 33
    want = shaped.rotate(t, far, f, False, 1.0, False)
    # the angle itself: 2^33 in 53 bits leaves 2^33 * 2^-53 * 2^2 of a radian
    shaped.close(bfa.rope(t, far, f), want, shaped.rotate_bound(t, want, 1.0) + 2.0 ** -16, "far")
    y = x.clone()
    assert bfa.rope(y, p, f, out=y) is y
    assert torch.equal(y, bfa.rope(x, p, f))
    wide = torch.full((2, 50, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    bfa.rope(x, p, f, out=wide[..., :64])
    assert torch.equal(wide[..., :64], y) and (wide[..., 64:] == 9).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = bfa.rope(x, p, f, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(z, y)
    assert bfa.rope(x[:, :0], p[:, :0], f).shape == (2, 0, 4, 64)
    for rotary in (24, 62):
        with pytest.raises(bfa.BfaError) as e:
            bfa.rope(x, p, bfa.rope_frequencies(rotary))
        assert e.value.status == "BFA_ERR_UNSUPPORTED"


def test_rope_gradient_is_the_transpose():
    # <rope x, g> = <x, rope^-1 g>: both sides from bf16 results, each value off by 2^-8 of itself
    f = bfa.rope_frequencies(64)
    x, g = _rand((1, 200, 4, 64), 1), _rand((1, 200, 4, 64), 2)
    p = torch.arange(200, device="cuda")[None]
    y, dx = bfa.rope(x, p, f, amplitude=1.1), bfa.rope(g, p, f, amplitude=1.1, inverse=True)
    a, b = (y.double() * g.double()).sum(), (x.double() * dx.double()).sum()
    room = shaped.U * ((y.double() * g.double()).abs().sum() + (x.double() * dx.double()).abs().sum())
    assert abs(float(a - b)) <= float(room)


def _cache_case(lens, kv, page, Hkv, D, seed):
    pages = [-(-n // page) for n in kv]
    rng = np.random.default_rng(seed)
    order = rng.permutation(sum(pages) + 2).astype(np.int32)
    table = np.full((len(kv), max(pages)), -1, np.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n]
        at += n
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    caches = torch.full((2, sum(pages) + 2, page, Hkv, D), 4.0, dtype=torch.bfloat16, device="cuda")
    return torch.from_numpy(table).cuda(), cu, torch.tensor(kv, dtype=torch.int32, device="cuda"), caches[0], caches[1]


@pytest.mark.parametrize("D,rotary,interleaved", [(64, 64, False), (128, 48, True), (128, 128, False), (64, 0, False)])
@pytest.mark.parametrize("page", [8, 128])
@pytest.mark.parametrize("with_q", [True, False])
def test_append(D, rotary, interleaved, page, with_q):
    lens, kv, H, Hkv, pad = [1, 0, 30, 7, 129], [200, 9, 30, 5, 400], 6, 2, 5  # the fourth: two tokens before position 0
    table, cu, used, kc, vc = _cache_case(lens, kv, page, Hkv, D, page)
    T = sum(lens) + pad
    k, v, q = _rand((T, Hkv, D), 1), _rand((T, Hkv, D), 2), _rand((T, H, D), 3)
    f = bfa.rope_frequencies(rotary) if rotary else None
    k0, v0 = kc.clone(), vc.clone()
    q_out = torch.full_like(q, 6.0)
    got = bfa.append_paged(k, v, kc, vc, table, cu, used, q=q if with_q else None, q_out=q_out if with_q else None,
                           inv_freq=f, interleaved=interleaved, amplitude=0.9)
    torch.cuda.synchronize()
    pos = torch.cat([torch.arange(n - l, n) for l, n in zip(lens, kv)]).cuda()
    n = sum(lens)
    none = torch.zeros(0, dtype=torch.float64, device="cuda")
    if with_q:
        assert got is q_out and (q_out[n:] == 6).all()
        _close(q_out[:n], q[:n], pos, f if rotary else none, interleaved, 0.9, False, "q")
    else:
        assert got is None
    want_k = shaped.rotate(k[:n], pos, f if rotary else none, interleaved, 0.9, False)
    at = 0
    for s, (l, m) in enumerate(zip(lens, kv)):
        for t in range(l):
            p = m - l + t
            if p >= 0:
                page_id, row = int(table[s, p // page]), p % page
                shaped.close(kc[page_id, row], want_k[at + t], shaped.rotate_bound(k[at + t], want_k[at + t], 0.9), "k")
                assert torch.equal(vc[page_id, row], v[at + t])
                k0[page_id, row], v0[page_id, row] = kc[page_id, row], v[at + t]
        at += l
    assert torch.equal(kc, k0) and torch.equal(vc, v0)  # nothing else was written


def test_append_leaves_out_places_that_do_not_exist():
    table, cu, used, kc, vc = _cache_case([4, 4], [40, 40], 16, 2, 64, 1)
    table[0, 2] = kc.shape[0]  # a page the cache does not have
    used[1] = 10 ** 6  # keys beyond the table
    k0 = kc.clone()
    k = _rand((8, 2, 64), 1)
    bfa.append_paged(k, k, kc, vc, table, cu, used)
    torch.cuda.synchronize()
    assert torch.equal(kc, k0) and torch.equal(vc, k0)


def test_a_captured_append_follows_the_lengths():
    table, cu, used, kc, vc = _cache_case([1, 1], [64, 64], 16, 2, 64, 1)
    k, v, q = _rand((2, 2, 64), 1), _rand((2, 2, 64), 2), _rand((2, 4, 64), 3)
    f = bfa.rope_frequencies(64)
    bfa.append_paged(k, v, kc, vc, table, cu, used, q=q, inv_freq=f)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = bfa.append_paged(k, v, kc, vc, table, cu, used, q=q, inv_freq=f)
    used.copy_(torch.tensor([3, 33]))
    g.replay()
    torch.cuda.synchronize()
    pos = torch.tensor([2, 32], device="cuda")
    _close(out, q, pos, f, False, 1.0, False)
    assert torch.equal(vc[int(table[0, 0]), 2], v[0]) and torch.equal(vc[int(table[1, 2]), 0], v[1])


@pytest.mark.parametrize("D,cap,with_slopes", [(64, None, False), (128, 20.0, True)])
def test_serving_in_steps_equals_the_whole_prompt(D, cap, with_slopes):
    """append_paged and fwd_chunk over pieces of two prompts, then single tokens, against rope and fwd with a
    causal plan over the whole of each: the same attention, so each is within its bounds of the 64-bit form."""
    H, Hkv, page, total = 8, 2, 16, [210, 97]
    q = [_rand((n, H, D), 1 + s, 1.5) for s, n in enumerate(total)]
    k = [_rand((n, Hkv, D), 11 + s) for s, n in enumerate(total)]
    v = [_rand((n, Hkv, D), 21 + s) for s, n in enumerate(total)]
    f = bfa.rope_frequencies(D)
    slopes = torch.pow(2.0, -torch.arange(1, H + 1, dtype=torch.float32)).cuda() if with_slopes else None
    table, _, _, kc, vc = _cache_case(total, total, page, Hkv, D, 7)
    steps = [[130, 0], [40, 60], [1, 1], [30, 30]] + [[1, 1]] * 6 + [[3, 0]]
    assert [sum(x) for x in zip(*steps)] == total
    done, outs, lses = [0, 0], [[], []], [[], []]
    for lens in steps:
        cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
        starts, done = done, [d + n for d, n in zip(done, lens)]
        used = torch.tensor(done, dtype=torch.int32, device="cuda")
        cut = lambda x: torch.cat([x[s][starts[s]:done[s]] for s in (0, 1)])  # noqa: E731
        qr = bfa.append_paged(cut(k), cut(v), kc, vc, table, cu, used, q=cut(q), inv_freq=f)
        o, l = bfa.fwd_chunk(qr, kc, vc, table, cu, used, max_q=max(lens), softcap=cap, slopes=slopes)
        outs[0].append(o[:lens[0]])
        outs[1].append(o[lens[0]:])
        lses[0].append(l[:, :lens[0]])
        lses[1].append(l[:, lens[0]:])
    for s, n in enumerate(total):
        p = torch.arange(n, device="cuda")
        qr, kr = bfa.rope(q[s], p, f)[None], bfa.rope(k[s], p, f)[None]
        plan = bfa.plan_blockids(B=1, Sq=n, Sk=n)
        out, lse = bfa.fwd(plan, qr, kr, v[s][None], softcap=cap, slopes=slopes)
        M = p[:, None] >= p
        want, bound = shaped.batch(qr, kr, v[s][None], lambda *_: M, None, cap, slopes)
        shaped.close(out, want["out"], bound["out"], "whole out")
        shaped.close(torch.cat(outs[s])[None], want["out"], bound["out"], "stepped out")
        shaped.close(torch.cat(lses[s], 1)[None], want["lse"], bound["lse"], "stepped lse")


def test_a_training_step_through_positions_and_scores():
    """rope, shaped attention, and the gradients of q and k before rope, against autograd in 64 bits; the
    bound of dq and dk turns with them (a turned value adds two)."""
    S, H, Hkv, D, cap = 150, 4, 2, 64, 10.0
    q, k, v, dout = _rand((1, S, H, D), 1), _rand((1, S, Hkv, D), 2), _rand((1, S, Hkv, D), 3), _rand((1, S, H, D), 4)
    f, p = bfa.rope_frequencies(D), torch.arange(S, device="cuda")
    plan = bfa.plan_blockids(B=1, Sq=S, Sk=S)
    qr, kr = bfa.rope(q, p, f), bfa.rope(k, p, f)
    out, lse = bfa.fwd(plan, qr, kr, v, softcap=cap)
    dqr, dkr, dv = bfa.bwd(plan, qr, kr, v, out, dout, lse, softcap=cap)
    dq, dk = bfa.rope(dqr, p, f, inverse=True), bfa.rope(dkr, p, f, inverse=True)
    leaf = lambda x: x.double().requires_grad_()  # noqa: E731
    a, b, c = leaf(qr), leaf(kr), leaf(v)
    s = torch.einsum("bihd,bjhd->bhij", a, b.repeat_interleave(H // Hkv, 2)) * D ** -0.5
    s = (cap * torch.tanh(s / cap)).masked_fill(p[:, None] < p, -float("inf"))
    torch.einsum("bhij,bjhd->bihd", s.softmax(-1), c.repeat_interleave(H // Hkv, 2)).backward(dout.double())
    M = p[:, None] >= p
    _, bound = shaped.batch(qr, kr, v, lambda *_: M, None, cap, None, dout)
    shaped.close(dqr, a.grad, bound["dq"], "dq of the turned q")
    shaped.close(dkr, b.grad, bound["dk"], "dk of the turned k")
    shaped.close(dv, c.grad, bound["dv"], "dv")
    for got, turned, e in ((dq, a.grad, bound["dq"]), (dk, b.grad, bound["dk"])):
        want = shaped.rotate(turned, p[None], f, False, 1.0, True)
        two = e[..., :D // 2] + e[..., D // 2:]
        shaped.close(got, want, torch.cat((two, two), -1) + shaped.rotate_bound(turned, want, 1.0), "before rope")
