"""Attention of new tokens over a paged cache, against the 64-bit form of tests/shaped.py."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import shaped

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

bfa = pytest.importorskip("mask_skipping_flashattention_b200")


def _rand(shape, seed, by=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * by).to(torch.bfloat16)


def _slopes(H):
    return torch.pow(2.0, -8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).cuda()


class Batch:
    """A ragged batch over a shuffled page pool; everything that is no key of a sequence is NaN."""

    def __init__(self, q_lens, kv_lens, H, Hkv, D, page, seed=0, spare=2, pad_rows=0, by=1.5):
        self.q_lens, self.kv_lens, self.H, self.Hkv, self.D, self.page = q_lens, kv_lens, H, Hkv, D, page
        rng = np.random.default_rng(seed)
        pages = [-(-kv // page) for kv in kv_lens]
        total = sum(pages) + spare
        order = rng.permutation(total)
        self.k_cache = torch.full((total, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v_cache = self.k_cache.clone()
        table = np.full((len(kv_lens), max(max(pages), 1) + 1), 10 ** 9, np.int32)  # unused entries: nonsense
        self.k, self.v, at = [], [], 0
        for s, n in enumerate(pages):
            ids = order[at:at + n]
            at += n
            table[s, :n] = ids
            k, v = _rand((kv_lens[s], Hkv, D), seed + 10 * s + 1), _rand((kv_lens[s], Hkv, D), seed + 10 * s + 2)
            self.k.append(k)
            self.v.append(v)
            for i, p in enumerate(ids):
                m = min(page, kv_lens[s] - i * page)
                self.k_cache[p, :m] = k[i * page:i * page + m]
                self.v_cache[p, :m] = v[i * page:i * page + m]
        self.table = torch.from_numpy(table).cuda()
        cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.cu, self.used = torch.from_numpy(cu).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda()
        self.cu_h = cu
        self.q = _rand((int(cu[-1]) + pad_rows, H, D), seed + 5, by)
        self.pad_rows = pad_rows

    def call(self, **kw):
        kw.setdefault("max_q", max(self.q_lens))
        q = kw.pop("q", self.q)
        return bfa.fwd_chunk(q, self.k_cache, self.v_cache, self.table, self.cu, self.used, **kw)

    def check(self, out, lse, window=0, cap=None, slopes=None, scale=None):
        torch.cuda.synchronize()
        G = self.H // self.Hkv
        scale = self.D ** -0.5 if scale is None else scale
        for s, (n, kv) in enumerate(zip(self.q_lens, self.kv_lens)):
            a = int(self.cu_h[s])
            if n == 0:
                continue
            d = (kv - n + torch.arange(n, device="cuda"))[:, None] - torch.arange(kv, device="cuda")
            mask = d >= 0
            if window:
                mask &= d < window
            if kv == 0:
                assert out[a:a + n].abs().max() == 0 and torch.isneginf(lse[:, a:a + n]).all()
                continue
            for h in range(self.H):
                want, bound = shaped.head(self.q[a:a + n, h], self.k[s][:, h // G], self.v[s][:, h // G], mask, d.abs(),
                                          scale, cap, None if slopes is None else slopes[h])
                shaped.close(out[a:a + n, h], want["out"], bound["out"], f"out of sequence {s}, head {h}")
                shaped.close(lse[h, a:a + n], want["lse"], bound["lse"], f"lse of sequence {s}, head {h}")


SHAPES = [(None, False, 0), (20.0, False, 100), (None, True, 0), (6.0, True, 37)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 64, 256])
@pytest.mark.parametrize("cap,with_slopes,window", SHAPES)
def test_single_tokens(D, page, cap, with_slopes, window):
    kv = [0, 1, 2, 7, 8, 9, 63, 64, 65, 127, 500, 1025]
    b = Batch([1] * len(kv), kv, 8, 2, D, page, seed=page + D)
    slopes = _slopes(8) if with_slopes else None
    b.check(*b.call(softcap=cap, slopes=slopes, window_left=window or -1), window, cap, slopes)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (5, 5), (16, 1), (20, 4), (40, 1), (64, 2)])
def test_head_layouts(H, Hkv):
    for q_lens, kv in (([1, 1, 1], [300, 1, 77]), ([3, 0, 5], [300, 12, 5])):
        b = Batch(q_lens, kv, H, Hkv, 64, 32, seed=H)
        b.check(*b.call())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128, 384])
@pytest.mark.parametrize("cap,with_slopes,window", SHAPES)
def test_chunks_of_all_lengths(D, page, cap, with_slopes, window):
    # decoding, nothing new, a whole prompt, pieces behind a context, more new tokens than keys
    q_lens, kv = [1, 0, 130, 257, 64, 5, 9], [400, 50, 130, 700, 65, 5, 4]
    b = Batch(q_lens, kv, 6, 2, D, page, seed=page + D)
    slopes = _slopes(6) if with_slopes else None
    b.check(*b.call(softcap=cap, slopes=slopes, window_left=window or -1), window, cap, slopes)


@pytest.mark.parametrize("q_len", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 300])
@pytest.mark.parametrize("G", [1, 4])
def test_lengths_around_the_tiles(q_len, G):
    b = Batch([q_len, q_len], [q_len, q_len + 128], 2 * G, 2, 64, 64, seed=q_len)
    b.check(*b.call())
    b.check(*b.call(max_q=0))
    b.check(*b.call(max_q=1))  # understated: only the tiles change


def test_rows_behind_the_last_sequence_stay():
    for q_lens in ([1, 1], [70, 200]):
        b = Batch(q_lens, [300, 301], 8, 2, 64, 16, pad_rows=11)
        out = torch.full_like(b.q, 3.0)
        lse = torch.full((8, b.q.shape[0]), 3.0, device="cuda")
        b.call(out=out, lse=lse)
        b.check(out, lse)
        n = sum(q_lens)
        assert (out[n:] == 3).all() and (lse[:, n:] == 3).all()


def test_long_context_is_cut_into_pieces():
    b = Batch([1, 1, 200], [70001, 3, 20000], 4, 1, 128, 128, seed=3)
    out, lse = b.call()
    b.check(out, lse)
    again, lse2 = b.call()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_pages_that_do_not_exist_read_as_zeros():
    for n in (1, 150):
        b = Batch([n], [320], 4, 2, 64, 32)
        b.table[0, 3] = b.k_cache.shape[0]
        b.table[0, 5] = -1
        for i in (3, 5):
            b.k[0][32 * i:32 * i + 32] = 0
            b.v[0][32 * i:32 * i + 32] = 0
        b.check(*b.call())


def test_lengths_beyond_the_table_count_as_its_room():
    for n in (1, 140):
        b = Batch([n], [256], 4, 2, 64, 64)
        b.table = b.table[:, :4].contiguous()
        out, lse = b.call()
        b.used.fill_(10 ** 6)
        # 256 keys as before: the last new token stands at the last of them
        out2, lse2 = b.call()
        assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_strides_scale_and_given_results():
    for n in (1, 150):
        b = Batch([n, n], [200, 333], 4, 2, 128, 16)
        wide = _rand((2 * n, 4, 3, 128), 77)
        b.q = wide[:, :, 1]
        room = torch.full((2 * n, 6, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        out, lse = b.call(out=room[:, 1:5], scale=0.3)
        b.check(out, lse, scale=0.3)
        assert (room[:, 0] == 5).all() and (room[:, 5] == 5).all()
        assert bfa.fwd_chunk(b.q, b.k_cache, b.v_cache, b.table, b.cu, b.used, return_lse=False)[1] is None


def test_a_cache_with_wider_rows():
    # keys and values side by side in one buffer: token and head strides of their own
    b = Batch([1, 140], [200, 333], 4, 2, 64, 64)
    both = torch.stack((b.k_cache, b.v_cache), dim=3).flatten(3)  # (pages, page, Hkv, 2 D)
    b.k_cache, b.v_cache = both[..., :64], both[..., 64:]
    b.check(*b.call())


def test_infinities_reach_only_rows_that_see_them():
    for n in (1, 150):
        b = Batch([n, n], [200, 201], 4, 2, 64, 16)
        want, lse_w = b.call()
        p = int(b.table[1, 0])
        b.v_cache[p, 3] = float("inf")
        out, lse = b.call()
        assert torch.equal(out[:n], want[:n]) and torch.equal(lse, lse_w)
        assert not torch.isfinite(out[n:].float()).all()


def test_streams_and_two_captured_calls():
    big = Batch([1, 1, 1], [900, 40, 2000], 8, 2, 128, 16, seed=5)
    small = Batch([160, 1], [400, 77], 8, 2, 128, 16, seed=6)
    want = [b.call() for b in (big, small)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [b.call(stream=side) for b in (big, small)]
    torch.cuda.current_stream().wait_stream(side)
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
    graphs, results = [], []
    for b in (big, small):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(b.call())
        graphs.append(g)
    for _ in range(3):  # in turn, and at once on two streams
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(results, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
    # a replay follows the lengths on the device
    big.used.copy_(torch.tensor([300, 41, 1]))
    graphs[0].replay()
    torch.cuda.synchronize()
    o, l = big.call()
    # bit for bit: the second sequence now has a key that was never written (NaN)
    assert torch.equal(results[0][0].view(torch.int16), o.view(torch.int16))
    assert torch.equal(results[0][1].view(torch.int32), l.view(torch.int32))


def test_a_given_workspace_with_anything_in_it():
    b = Batch([1, 1], [3000, 800], 8, 2, 64, 16)
    need = bfa._L.bfa_fwd_chunk_workspace(2, 2, 1, 8, 2, 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    want = b.call()
    got = b.call(workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(bfa.BfaError) as e:
        b.call(workspace=ws[:need - 16])
    assert e.value.status == "BFA_ERR_CAPACITY"


def test_offsets_past_31_bits():
    # a cache of 2.2 * 10^9 values each; the sequence lies at its far end
    page, Hkv, D = 64, 8, 128
    pages = 34000
    k_cache = torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v_cache = torch.empty_like(k_cache)
    for n in (1, 160):
        b = Batch([n], [500], 16, Hkv, D, page)
        last = pages - b.k_cache.shape[0]
        k_cache[last:] = b.k_cache
        v_cache[last:] = b.v_cache
        b.table = torch.where(b.table < 10 ** 8, b.table + last, b.table)
        b.k_cache, b.v_cache = k_cache, v_cache
        b.check(*b.call())


def test_many_sequences():
    rng = np.random.default_rng(9)
    kv = rng.integers(0, 90, 700).tolist()
    b = Batch([1] * 700, kv, 4, 2, 64, 16, seed=2)
    b.check(*b.call())


def test_empty_calls():
    b = Batch([0, 0], [10, 0], 4, 2, 64, 16)
    out, lse = b.call(max_q=1)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    b = Batch([0, 0], [10, 0], 4, 2, 64, 16, pad_rows=3)
    out = torch.full_like(b.q, 2.0)
    b.call(out=out, max_q=1)
    torch.cuda.synchronize()
    assert (out == 2).all()


def test_a_short_wait_bound_is_reported_and_leaves_nothing_behind():
    b = Batch([300, 1], [5000, 3000], 8, 2, 128, 64)
    want = b.call()
    torch.cuda.synchronize()
    bfa.chunk_device_status()
    bfa.set_wait_timeout_ns(1000)  # the first wait for scores outlasts it
    try:
        b.call()
        with pytest.raises(bfa.BfaError) as e:
            bfa.chunk_device_status()
        assert e.value.status == "BFA_ERR_TIMEOUT"
    finally:
        bfa.set_wait_timeout_ns(0)
    got = b.call()
    bfa.chunk_device_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_other_integer_types_and_strides_on_another_stream():
    # they are copied where the launch's stream is current, behind what that stream has queued
    b = Batch([1, 70], [200, 333], 8, 2, 64, 16)
    slopes = torch.stack((_slopes(8), _slopes(8)), 1)[:, 0]
    want = b.call(slopes=slopes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        table, cu, used = b.table.long() + 0, b.cu.long() + 0, b.used.long() + 0
    wide = torch.stack((table, table), 2)[:, :, 0]
    side.wait_stream(torch.cuda.current_stream())
    got = bfa.fwd_chunk(b.q, b.k_cache, b.v_cache, wide, cu, used, max_q=70, slopes=slopes, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the raw handle of a stream, too
    raw = bfa.fwd_chunk(b.q, b.k_cache, b.v_cache, b.table, b.cu, b.used, max_q=70, slopes=slopes,
                        stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(raw[0], want[0])


FIRST_CALLS = """
import torch
import mask_skipping_flashattention_b200 as bfa
BF = torch.bfloat16
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
kc, vc, q, k, v = r(40, 16, 2, 64), r(40, 16, 2, 64), r(101, 8, 64), r(101, 2, 64), r(101, 2, 64)
table = torch.arange(40, dtype=torch.int32, device="cuda").reshape(2, 20)
cu = torch.tensor([0, 1, 101], dtype=torch.int32, device="cuda")
used = torch.tensor([200, 300], dtype=torch.int32, device="cuda")
f = torch.pow(100.0, -torch.arange(32, dtype=torch.float64, device="cuda"))
p = torch.arange(101, dtype=torch.int32, device="cuda")

def step():
    qr = bfa.append_paged(k, v, kc, vc, table, cu, used, q=q, inv_freq=f)
    out, lse = bfa.fwd_chunk(qr, kc, vc, table, cu, used, max_q=100, softcap=20.0)
    return out, lse, bfa.rope(out, p, f, inverse=True)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = step()
graph.replay()
torch.cuda.synchronize()
eager = step()
assert all(torch.equal(a, b) for a, b in zip(captured, eager))
bfa.chunk_device_status()
print("same")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-1000:] + r.stderr[-2000:]


def test_a_single_kv_head_may_have_any_stride():
    b = Batch([1, 70], [200, 333], 4, 1, 64, 16)
    want = b.call()
    flat_k, flat_v = b.k_cache[:, :, 0], b.v_cache[:, :, 0]
    b.k_cache = torch.as_strided(flat_k, (*flat_k.shape[:2], 1, 64), (16 * 64, 64, 0, 1))
    b.v_cache = torch.as_strided(flat_v, (*flat_v.shape[:2], 1, 64), (16 * 64, 64, 0, 1))
    got = b.call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("by", [1.0, 80.0])  # scores inside the polynomials' range, and far past it
@pytest.mark.parametrize("cap,with_slopes", [(None, False), (30.0, False), (30.0, True)])
def test_nan_in_a_query_reaches_its_row_alone(by, cap, with_slopes):
    for n in (1, 150):  # row kernel, tile kernel
        b = Batch([n, n], [200, 201], 4, 2, 64, 16, by=by)
        b.q[n + n // 2, 1, 7] = float("nan")
        out, _ = b.call(softcap=cap, slopes=_slopes(4) if with_slopes else None)
        nan = out.isnan()
        want = torch.zeros(2 * n, 4, dtype=torch.bool, device="cuda")
        want[n + n // 2, 1] = True
        assert torch.equal(nan.all(-1), want) and torch.equal(nan.any(-1), want)


def test_a_window_beyond_31_bits_is_no_window():
    b = Batch([1, 3], [200, 30], 4, 2, 64, 16)
    want = b.call()[0]
    for w in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5):
        assert torch.equal(b.call(window_left=w)[0], want)


@pytest.mark.parametrize("by", [1.0, 80.0])
@pytest.mark.parametrize("cap,with_slopes", [(None, False), (30.0, False), (30.0, True)])
@pytest.mark.parametrize("n,kv", [(1, 201), (1, 70001), (9, 9000), (150, 400), (150, 20001), (300, 70001)])
def test_the_lse_of_a_row_that_attends_a_nan_is_nan(by, cap, with_slopes, n, kv):
    # whole units and units in a few, in some and in hundreds of pieces, of both kernels
    b = Batch([n, n], [n + 40, kv], 4, 2, 64, 16, by=by)
    shape = dict(softcap=cap, slopes=_slopes(4) if with_slopes else None)
    hk, key = 1, kv - n + n // 2  # the key of a new token: the later ones attend it
    b.k_cache[int(b.table[1, key // 16]), key % 16, hk, 7] = float("nan")
    out, lse = b.call(**shape)
    bad = torch.zeros(2 * n, 4, dtype=torch.bool, device="cuda")
    bad[n + n // 2:, 2:] = True
    assert torch.equal(lse.isnan(), bad.t()) and torch.equal(out.isnan().any(-1), bad)
    assert torch.isfinite(lse[~bad.t()]).all()
