"""The plain 64-bit forms the shaped-score and rotary tests compare with, against differences
and closed forms (CPU)."""

import math

import pytest
import torch

import shaped


def _case(n, m, D, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    mask = torch.rand(n, m, generator=g) < 0.7
    mask[0] = False  # a row that attends nothing
    mask[1:, 0] = True
    distance = (torch.arange(n)[:, None] - torch.arange(m)).abs()
    return 2 * r(n, D), r(m, D), r(m, D), mask, distance, r(n, D)


@pytest.mark.parametrize("cap,slope", [(None, None), (2.0, None), (None, 0.3), (1.5, 0.2), (5.0, -0.1)])
def test_gradients_match_differences(cap, slope):
    q, k, v, mask, distance, dout = _case(5, 7, 4, 3)
    loss = lambda q, k, v: float((shaped.head(q, k, v, mask, distance, 0.5, cap, slope)[0]["out"] * dout).sum())  # noqa: E731
    got, _ = shaped.head(q, k, v, mask, distance, 0.5, cap, slope, dout)
    h = 1e-6
    for n, name in enumerate(("dq", "dk", "dv")):
        base = [q, k, v]
        for i in range(base[n].shape[0]):
            for j in range(base[n].shape[1]):
                up, down = [t.clone() for t in base], [t.clone() for t in base]
                up[n][i, j] += h
                down[n][i, j] -= h
                # central differences: error h^2 times the third derivative, and 1e-16 / h
                assert abs((loss(*up) - loss(*down)) / (2 * h) - float(got[name][i, j])) < 1e-7


def test_the_shapes_do_what_they_say():
    q, k, v, mask, distance, _ = _case(6, 6, 4, 5)
    plain = shaped.head(q, k, v, mask, distance, 0.5, None, None)[0]
    wide = shaped.head(q, k, v, mask, distance, 0.5, 1e6, None)[0]
    assert torch.allclose(plain["out"], wide["out"], atol=1e-9)
    tight = shaped.head(q, k, v, mask, distance, 1e6, 1e-3, None)[0]  # every score is +-1e-3
    n = mask.sum(1)
    assert torch.allclose(tight["lse"][1:], torch.log(n[1:].double()), atol=2e-3)
    steep = shaped.head(q, k, v, torch.ones_like(mask), distance, 0.5, None, 1e4)[0]
    assert torch.allclose(steep["out"], v[:6], atol=1e-9)  # only the key at distance 0 is left
    assert torch.isneginf(plain["lse"][0]) and plain["out"][0].abs().max() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation(interleaved):
    x = torch.randn(3, 2, 8, dtype=torch.float64)
    f = torch.tensor([1.0, 0.25, 0.01], dtype=torch.float64)
    p = torch.tensor([0, 1, 1000])
    y = shaped.rotate(x, p, f, interleaved, 1.0, False)
    assert torch.equal(y[0], x[0]) and torch.equal(y[..., 6:], x[..., 6:])
    assert torch.allclose(y[..., :6].norm(dim=-1), x[..., :6].norm(dim=-1))
    assert torch.allclose(shaped.rotate(y, p, f, interleaved, 1.0, True), x, atol=1e-12)
    # the inverse is the transpose: <rotate x, g> = <x, rotate^-1 g>
    g = torch.randn(3, 2, 8, dtype=torch.float64)
    a = (shaped.rotate(x, p, f, interleaved, 1.3, False) * g).sum() - (x[..., 6:] * g[..., 6:]).sum()
    b = (x * shaped.rotate(g, p, f, interleaved, 1.3, True)).sum() - (x[..., 6:] * g[..., 6:]).sum()
    assert math.isclose(float(a), float(b), rel_tol=1e-12)
    one = shaped.rotate(torch.tensor([[[1.0, 0.0]]], dtype=torch.float64), torch.tensor([1]),
                        torch.tensor([math.pi / 2], dtype=torch.float64), interleaved, 2.0, False)
    assert torch.allclose(one, torch.tensor([[[0.0, 2.0]]], dtype=torch.float64), atol=1e-12)
