"""Calls that the shaped-score, chunk, rotary and append entry points refuse (CPU: nothing is launched)."""

import pytest
import torch

import mask_skipping_flashattention_b200 as bfa

BF = torch.bfloat16


class FakePlan:
    """What the argument checks read of a plan."""

    def __init__(self, **info):
        self.info = dict(dict(varlen=0, batch=1, sq=8, sk=8, heads_per_kv=1), **info)
        self.handle = None


def _qkv(S=8, H=4, Hkv=2, D=64):
    return torch.zeros(1, S, H, D, dtype=BF), torch.zeros(1, S, Hkv, D, dtype=BF), torch.zeros(1, S, Hkv, D, dtype=BF)


def _cache(pages=4, page=16, Hkv=2, D=64):
    c = torch.zeros(pages, page, Hkv, D, dtype=BF)
    return c, c.clone(), torch.zeros(1, 4, dtype=torch.int32)


CU, USED = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([10], dtype=torch.int32)


@pytest.mark.parametrize("change,error", [
    (dict(slopes=torch.zeros(4, dtype=torch.float64)), TypeError),
    (dict(slopes=torch.zeros(3)), ValueError),
    (dict(slopes=torch.zeros(1, 4)), ValueError),
    (dict(softcap=30.0, softmax_threshold=5.0), ValueError),
    (dict(softcap=30.0, out=torch.zeros(1, 8, 4, 64)), ValueError),
    (dict(softcap=30.0, out=torch.zeros(1, 8, 2, 64, dtype=BF)), ValueError),
    (dict(softcap=30.0, lse=torch.zeros(4, 8)), ValueError),
])
def test_shaped_forward_refuses(change, error):
    with pytest.raises(error):
        bfa.fwd(FakePlan(), *_qkv(), stream=0, **change)


def test_shaped_forward_refuses_other_shapes_than_the_plan():
    q, k, v = _qkv()
    for plan in (FakePlan(sq=9), FakePlan(sk=7), FakePlan(varlen=1)):
        with pytest.raises(ValueError):
            bfa.fwd(plan, q, k, v, softcap=30.0, stream=0)
    for bad in ((q.float(), k, v), (q, k[:, :, :, :32], v), (q, k, v[:, :, :1]), (q[0], k, v)):
        with pytest.raises((TypeError, ValueError)):
            bfa.fwd(FakePlan(), *bad, softcap=30.0, stream=0)


def test_shaped_backward_refuses():
    q, k, v = _qkv()
    lse = torch.zeros(1, 4, 8)
    for change in (dict(lse=torch.zeros(1, 8, 4)), dict(dout=q[:, :4]), dict(out=q.float()), dict(lse=lse.double())):
        args = dict(dict(out=q, dout=q, lse=lse), **change)
        with pytest.raises((TypeError, ValueError)):
            bfa.bwd(FakePlan(), q, k, v, args["out"], args["dout"], args["lse"], softcap=30.0, stream=0)


@pytest.mark.parametrize("cap", [-1.0, 1e-4, 1e7, float("nan"), float("inf")])
def test_softcap_out_of_range(cap):
    k, v, bt = _cache()
    with pytest.raises(bfa.BfaError) as e:
        bfa.fwd_chunk(torch.zeros(3, 4, 64, dtype=BF), k, v, bt, CU, USED, softcap=cap, stream=0)
    assert e.value.status == "BFA_ERR_INVALID_ARG"


@pytest.mark.parametrize("change,error", [
    (dict(q=torch.zeros(3, 4, 64)), TypeError),
    (dict(q=torch.zeros(3, 4, 128, dtype=BF)), ValueError),
    (dict(q=torch.zeros(1, 3, 4, 64, dtype=BF)), ValueError),
    (dict(q=torch.zeros(3, 5, 64, dtype=BF)), "BFA_ERR_INVALID_ARG"),  # 5 heads on 2 kv heads
    (dict(cu=torch.tensor([0, 1, 3], dtype=torch.int32)), ValueError),
    (dict(cu=torch.tensor([0.0, 3.0])), TypeError),
    (dict(bt=torch.zeros(2, 4, dtype=torch.int32)), ValueError),
    (dict(bt=torch.zeros(4, dtype=torch.int32)), ValueError),
    (dict(window_left=0), "BFA_ERR_INVALID_ARG"),
    (dict(window_left=-2), "BFA_ERR_INVALID_ARG"),
    (dict(page=24), "BFA_ERR_INVALID_ARG"),
    (dict(page=4), "BFA_ERR_INVALID_ARG"),
    (dict(D=32), "BFA_ERR_UNSUPPORTED"),
    (dict(), "BFA_ERR_NOT_DEVICE"),
])
def test_chunk_refuses(change, error):
    D = change.pop("D", 64)
    k, v, bt = _cache(page=change.pop("page", 16), D=D)
    q = change.pop("q", torch.zeros(3, 4, D, dtype=BF))
    cu, bt = change.pop("cu", CU), change.pop("bt", bt)
    if isinstance(error, str):
        with pytest.raises(bfa.BfaError) as e:
            bfa.fwd_chunk(q, k, v, bt, cu, USED, stream=0, **change)
        assert e.value.status == error
    else:
        with pytest.raises(error):
            bfa.fwd_chunk(q, k, v, bt, cu, USED, stream=0, **change)


def test_chunk_refuses_other_caches():
    k, v, bt = _cache()
    q = torch.zeros(3, 4, 64, dtype=BF)
    for kc, vc in ((k, v[:2]), (k.float(), v.float()), (k, v.transpose(1, 2).contiguous().transpose(1, 2)), (k[0], v[0])):
        with pytest.raises((TypeError, ValueError)):
            bfa.fwd_chunk(q, kc, vc, bt, CU, USED, stream=0)


def test_chunk_workspace_sizes():
    size = lambda *a: bfa._L.bfa_fwd_chunk_workspace(*a)  # noqa: E731
    # few rows need the row kernel's places, more of them the tile kernel's, a mixed batch both
    one, long, mixed = size(1, 1, 1, 32, 8, 128), size(600, 1, 600, 32, 8, 128), size(600, 2, 600, 32, 8, 128)
    assert 0 < one < long < mixed and mixed == one + long and size(64, 64, 1, 32, 8, 128) == one
    assert size(600, 1, 0, 32, 8, 128) == long  # an unknown max_q is the longest it can be
    assert size(1, 1, 1, 32, 8, 96) == -1 and size(1, 1, 1, 30, 8, 64) == -1 and size(-1, 1, 1, 8, 8, 64) == -1


@pytest.mark.parametrize("change,error", [
    (dict(x=torch.zeros(2, 4, 64)), TypeError),
    (dict(x=torch.zeros(4, 64, dtype=BF)), ValueError),
    (dict(p=torch.zeros(2)), TypeError),
    (dict(p=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(f=torch.zeros(32)), TypeError),
    (dict(f=torch.zeros(31, dtype=torch.float64)), "BFA_ERR_UNSUPPORTED"),  # 62 values
    (dict(f=torch.zeros(40, dtype=torch.float64)), "BFA_ERR_UNSUPPORTED"),  # 80 of 64
    (dict(x=torch.zeros(2, 4, 48, dtype=BF)), "BFA_ERR_UNSUPPORTED"),
    (dict(out=torch.zeros(2, 4, 64)), ValueError),
    (dict(), "BFA_ERR_NOT_DEVICE"),
])
def test_rope_refuses(change, error):
    x = change.pop("x", torch.zeros(2, 4, 64, dtype=BF))
    p = change.pop("p", torch.zeros(2, dtype=torch.int32))
    f = change.pop("f", torch.zeros(32, dtype=torch.float64))
    if error in ("BFA_ERR_UNSUPPORTED", "BFA_ERR_NOT_DEVICE"):
        with pytest.raises(bfa.BfaError) as e:
            bfa.rope(x, p, f, stream=0, **change)
        # pointers are looked at before the rotary size, so a CPU tensor may be named first
        assert e.value.status in (error, "BFA_ERR_NOT_DEVICE")
    else:
        with pytest.raises(error):
            bfa.rope(x, p, f, stream=0, **change)


def test_append_refuses():
    kc, vc, bt = _cache()
    k = torch.zeros(3, 2, 64, dtype=BF)
    for kk, vv, extra in ((k[:, :1], k[:, :1], {}), (k, k[:2], {}), (k.float(), k, {}),
                          (k, k, dict(q=torch.zeros(2, 4, 64, dtype=BF))), (k, k, dict(q_out=k)),
                          (k, k, dict(inv_freq=torch.zeros(32)))):
        with pytest.raises((TypeError, ValueError)):
            bfa.append_paged(kk, vv, kc, vc, bt, CU, USED, stream=0, **extra)
    for extra in (dict(inv_freq=torch.zeros(33, dtype=torch.float64)), dict()):
        with pytest.raises(bfa.BfaError):
            bfa.append_paged(k, k, kc, vc, bt, CU, USED, stream=0, **extra)


def test_frequencies():
    f = bfa.rope_frequencies(8, 100.0, device="cpu")
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64))
    assert torch.allclose(bfa.rope_frequencies(8, 100.0, factor=4.0, device="cpu"), f / 4)
    turns = 1000 * f / (2 * torch.pi)  # 159, 50.3, 15.9, 5.03
    got = bfa.rope_frequencies(8, 100.0, factor=4.0, ramp=(1000, 10.0, 100.0), device="cpu")
    keep = ((turns - 10) / 90).clamp(0, 1)
    assert keep[0] == 1 and keep[3] == 0 and 0 < keep[2] < 1
    assert torch.allclose(got, f * keep + f / 4 * (1 - keep))
    for bad in (dict(rotary=7), dict(rotary=0), dict(rotary=8, factor=0.0), dict(rotary=8, base=-1.0),
                dict(rotary=8, ramp=(0, 1, 2)), dict(rotary=8, ramp=(10, 2, 2))):
        with pytest.raises(ValueError):
            bfa.rope_frequencies(device="cpu", **bad)


def _refused(call, status):
    with pytest.raises(bfa.BfaError) as e:
        call()
    assert e.value.status == status


def test_results_that_repeat_an_axis_are_refused():
    k, v, bt = _cache()
    f = torch.zeros(16, dtype=torch.float64)
    q, kn = torch.zeros(3, 4, 64, dtype=BF), torch.zeros(3, 2, 64, dtype=BF)
    x = torch.zeros(2, 3, 4, 64, dtype=BF)
    at = torch.arange(3)
    for out in (torch.zeros(1, 4, 64, dtype=BF).expand(3, 4, 64), torch.zeros(3, 1, 64, dtype=BF).expand(3, 4, 64)):
        _refused(lambda: bfa.fwd_chunk(q, k, v, bt, CU, USED, out=out, stream=0), "BFA_ERR_INVALID_ARG")
        _refused(lambda: bfa.append_paged(kn, kn, k, v, bt, CU, USED, q=q, q_out=out, stream=0), "BFA_ERR_INVALID_ARG")
        _refused(lambda: bfa.rope(q, at, f, out=out, stream=0), "BFA_ERR_INVALID_ARG")
    _refused(lambda: bfa.rope(x, at, f, out=torch.zeros(1, 3, 4, 64, dtype=BF).expand(2, 3, 4, 64), stream=0), "BFA_ERR_INVALID_ARG")
    # an axis of one entry has no stride of its own
    one = torch.zeros(1, 4, 64, dtype=BF)
    _refused(lambda: bfa.rope(one, at[:1], f, out=one.clone().as_strided((1, 4, 64), (0, 64, 1)), stream=0), "BFA_ERR_NOT_DEVICE")


def test_windows_beyond_32_bits_do_not_wrap():
    k, v, bt = _cache()
    q = torch.zeros(3, 4, 64, dtype=BF)
    _refused(lambda: bfa.fwd_chunk(q, k, v, bt, CU, USED, window_left=5 - 2 ** 32, stream=0), "BFA_ERR_INVALID_ARG")
    _refused(lambda: bfa.fwd_chunk(q, k, v, bt, CU, USED, window_left=2 ** 32, stream=0), "BFA_ERR_NOT_DEVICE")


def test_a_workspace_that_is_not_one_run_of_bytes_is_refused():
    # its bytes are counted by its values, so a view with gaps or repeats has less room than it seems to
    k, v, bt = _cache()
    q = torch.zeros(3, 4, 64, dtype=BF)
    need = bfa._L.bfa_fwd_chunk_workspace(3, 1, 0, 4, 2, 64)
    for ws in (torch.zeros(need, 2, dtype=torch.uint8)[:, 0], torch.zeros(64, 128, dtype=torch.uint8)[:, :64],
               torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            bfa.fwd_chunk(q, k, v, bt, CU, USED, workspace=ws, stream=0)
    _refused(lambda: bfa.fwd_chunk(q, k, v, bt, CU, USED, workspace=torch.zeros(need, dtype=torch.uint8), stream=0),
             "BFA_ERR_NOT_DEVICE")


def test_rope_without_frequencies_is_a_type_error():
    x, p = torch.zeros(2, 4, 64, dtype=BF), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="inv_freq"):
        bfa.rope(x, p, None, stream=0)
