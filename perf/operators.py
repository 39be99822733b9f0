"""The cases that the attention operators around positions and the paged cache are measured on.

Four operators, in the kinds of a case:

- ``train``   attention over a tile plan with shaped scores (a tanh cap, a penalty linear in the
              distance), forward and, with ``grad``, its gradients;
- ``chunk``   a chunk of new tokens of each sequence over a paged cache, single tokens included;
- ``rope``    rotary positions and, with ``inverse``, their gradient;
- ``append``  new keys and values into the paged cache, rotated on the way, with the queries.

``run`` computes them from elementary torch operations in 32 bits (angles in 64), or, with ``own``
set, through the package.
"""

import math
import random

import torch

own = False


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one short batch of a small model: launch latency and ragged tiles
        dict(name="train_small", kind="train", grad=True, layout="causal", B=2, S=77, H=2, Hkv=2, D=64, cap=30.0,
             slopes=True, window=0, prefix=0, lens_seed=0),
        # scoring with a bidirectional prefix in front of a causal text, capped scores: forward only
        dict(name="prefix_cap_fwd", kind="train", grad=False, layout="prefix", B=4, S=4096, H=16, Hkv=4, D=128,
             cap=50.0, slopes=False, window=0, prefix=768, lens_seed=0),
        # documents packed into one row, each attending to itself, distance penalty, 64-wide heads
        dict(name="train_docs_slopes", kind="train", grad=True, layout="docs", B=5, S=1500, H=16, Hkv=16, D=64,
             cap=0.0, slopes=True, window=0, prefix=0, lens_seed=1),
        # the long training row: grouped heads, cap and distance penalty together
        dict(name="train_long", kind="train", grad=True, layout="causal", B=1, S=8192, H=16, Hkv=4, D=128, cap=30.0,
             slopes=True, window=0, prefix=0, lens_seed=0),
        # one user's next token, short context: latency
        dict(name="decode_one", kind="chunk", B=1, q_max=1, kv_max=500, H=32, Hkv=8, D=128, page=16, cap=0.0,
             slopes=False, window=0, lens_seed=2),
        # next tokens of a full serving batch with ragged contexts
        dict(name="decode_batch", kind="chunk", B=64, q_max=1, kv_max=8192, H=32, Hkv=8, D=128, page=64, cap=0.0,
             slopes=False, window=0, lens_seed=3),
        # a scheduler step that mixes next tokens with pieces of prompts; window, cap and penalty
        dict(name="chunk_mixed", kind="chunk", B=12, q_max=700, kv_max=6000, H=16, Hkv=4, D=64, page=32, cap=50.0,
             slopes=True, window=1024, lens_seed=4),
        # one piece of a long prompt behind a long context
        dict(name="chunk_long", kind="chunk", B=1, q_max=2048, kv_max=16384, H=32, Hkv=8, D=128, page=128, cap=0.0,
             slopes=False, window=0, lens_seed=5),
        # the queries of a training batch, pairs in the two halves of the head
        dict(name="rope_train", kind="rope", B=4, S=4096, H=32, D=128, rotary=128, interleaved=False, far=0,
             amplitude=1.0, inverse=False),
        # the gradient for a part of the head in interleaved pairs, far positions, odd length
        dict(name="rope_part_grad", kind="rope", B=3, S=1001, H=16, D=64, rotary=32, interleaved=True, far=900000,
             amplitude=1.2, inverse=True),
        # the new token of every sequence of a serving batch
        dict(name="append_decode", kind="append", B=64, q_max=1, kv_max=1024, H=32, Hkv=8, D=128, page=64,
             rotary=128, interleaved=False, amplitude=1.0, lens_seed=6),
        # pieces of prompts of several sequences
        dict(name="append_chunk", kind="append", B=16, q_max=1024, kv_max=2048, H=32, Hkv=8, D=128, page=16,
             rotary=64, interleaved=False, amplitude=1.0, lens_seed=7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["train", "train", "chunk", "chunk", "chunk", "rope", "append"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    shape = rng.choice([(0.0, True), (50.0, False), (30.0, True), (20.0, False)])
    if kind == "train":
        layout = rng.choice(["causal", "prefix", "docs"])
        H = min(Hkv * G, 16)
        Hkv = H if H % Hkv else Hkv
        S = _log_int(rng, 64, 4096)
        B = max(1, min(rng.randint(1, 6), 8192 // S))
        if layout == "docs":
            S = max(16, S // B)
        return dict(kind="train", grad=rng.random() < 0.7, layout=layout, B=B, S=S, H=H, Hkv=Hkv, D=D, cap=shape[0],
                    slopes=shape[1], window=rng.choice([0, 0, max(1, S // 3)]) if layout == "causal" else 0,
                    prefix=rng.randint(1, S) if layout == "prefix" else 0, lens_seed=rng.randint(0, 10 ** 6))
    if kind == "chunk":
        q_max = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 1024)])
        kv_max = max(q_max, _log_int(rng, 100, 12000))
        B = _log_int(rng, 1, 48) if q_max <= 8 else _log_int(rng, 1, max(1, 12000 // max(q_max, kv_max // 4)))
        if rng.random() < 0.4:
            shape = (0.0, False)
        return dict(kind="chunk", B=B, q_max=q_max, kv_max=kv_max, H=Hkv * G, Hkv=Hkv, D=D,
                    page=rng.choice([8, 16, 32, 64, 128, 256]), cap=shape[0], slopes=shape[1],
                    window=rng.choice([0, 0, rng.randint(1, kv_max)]), lens_seed=rng.randint(0, 10 ** 6))
    rotary = rng.choice([D, D // 2, 32, 48])
    if kind == "rope":
        S = _log_int(rng, 1, 4096)
        return dict(kind="rope", B=rng.randint(1, 4), S=S, H=rng.choice([1, 3, 8, 32]), D=D, rotary=rotary,
                    interleaved=rng.random() < 0.5, far=rng.choice([0, 5000, 900000]),
                    amplitude=rng.choice([1.0, 1.2]), inverse=rng.random() < 0.5)
    q_max = rng.choice([1, _log_int(rng, 2, 1024)])
    return dict(kind="append", B=_log_int(rng, 1, 16 if q_max > 1 else 64), q_max=q_max,
                kv_max=max(q_max, _log_int(rng, 64, 2048)), H=Hkv * G, Hkv=Hkv, D=D,
                page=rng.choice([8, 16, 32, 64, 128, 256]), rotary=rotary, interleaved=rng.random() < 0.5,
                amplitude=rng.choice([1.0, 1.2]), lens_seed=rng.randint(0, 10 ** 6))


# ---------------------------------------------------------------------------------------- inputs
def _doc_lens(c):
    """Lengths of the packed documents of a ``docs`` case: odd and even, around S."""
    r = random.Random(c["lens_seed"])
    return [r.randint(max(1, c["S"] // 2), c["S"]) for _ in range(c["B"])]


def _seq_lens(c):
    """(new tokens, keys after them) of each sequence: every second one of a mixed batch decodes."""
    r = random.Random(c["lens_seed"])
    pairs = []
    for s in range(c["B"]):
        n = c["q_max"] if s == 0 else (1 if s % 2 else r.randint(1, c["q_max"]))
        pairs.append((n, c["kv_max"] if s == 0 else r.randint(n, max(n, c["kv_max"]))))
    return pairs


def _cumulated(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def _frequencies(rotary):
    return torch.pow(10000.0, -torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)


def _slopes(H):
    return torch.pow(2.0, -8.0 * torch.arange(1, H + 1, dtype=torch.float32, device="cuda") / H)


def _term(prefix):
    """A causal text whose first ``prefix`` keys every query attends."""
    return [dict(diag_lo=0), dict(k_hi=prefix)]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * by).to(torch.bfloat16)

    st = dict(case=c)
    if c["kind"] == "train":
        by = 4.0 if c["cap"] else 1.0  # a cap is there for scores that grow large
        lead = (sum(_doc_lens(c)),) if c["layout"] == "docs" else (c["B"], c["S"])
        st.update(q=normal(*lead, c["H"], c["D"], by=by), k=normal(*lead, c["Hkv"], c["D"]),
                  v=normal(*lead, c["Hkv"], c["D"]), dout=normal(*lead, c["H"], c["D"]),
                  slopes=_slopes(c["H"]) if c["slopes"] else None)
        if c["layout"] == "docs":
            st["cu"] = torch.tensor(_cumulated(_doc_lens(c)), dtype=torch.int32, device="cuda")
        if own:  # the tile plan is made once for a mask and kept, as every user of the package does
            import mask_skipping_flashattention_b200 as bfa

            if c["layout"] == "docs":
                st["plan"] = bfa.plan_blockids(cu_seqlens_q=st["cu"], max_q=c["S"], max_k=c["S"])
            elif c["layout"] == "prefix":
                st["plan"] = bfa.plan_predicate(_term(c["prefix"]), B=c["B"], Sq=c["S"], Sk=c["S"])
            else:
                st["plan"] = bfa.plan_blockids(B=c["B"], Sq=c["S"], Sk=c["S"], window_left=c["window"] or -1)
        return st
    if c["kind"] == "rope":
        first = torch.randint(0, c["far"] + 1, (c["B"], 1), generator=g, device="cuda")
        st.update(x=normal(c["B"], c["S"], c["H"], c["D"]), inv_freq=_frequencies(c["rotary"]),
                  positions=(first + torch.arange(c["S"], device="cuda")).to(torch.int32).contiguous())
        return st
    pairs = _seq_lens(c)
    pages = [-(-kv // c["page"]) for _, kv in pairs]
    per_seq = max(pages)
    order = torch.randperm(sum(pages) + 3, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(c["B"], per_seq, dtype=torch.int32, device="cuda")
    for s, (n, at) in enumerate(zip(pages, _cumulated(pages))):
        table[s, :n] = order[at:at + n]
    total = sum(n for n, _ in pairs)
    st.update(k_cache=normal(sum(pages) + 3, c["page"], c["Hkv"], c["D"]),
              v_cache=normal(sum(pages) + 3, c["page"], c["Hkv"], c["D"]), block_table=table,
              cu=torch.tensor(_cumulated([n for n, _ in pairs]), dtype=torch.int32, device="cuda"),
              kv_len=torch.tensor([kv for _, kv in pairs], dtype=torch.int32, device="cuda"))
    if c["kind"] == "chunk":
        st.update(q=normal(total, c["H"], c["D"], by=4.0 if c["cap"] else 1.0),
                  slopes=_slopes(c["H"]) if c["slopes"] else None)
    else:
        st.update(q=normal(total, c["H"], c["D"]), k=normal(total, c["Hkv"], c["D"]),
                  v=normal(total, c["Hkv"], c["D"]), inv_freq=_frequencies(c["rotary"]))
    return st


# ---------------------------------------------------------------------------------------- plain forms
def _heads_first(x, Hkv):
    """(B, S, H, D) -> (B, Hkv, H / Hkv, S, D) in 32 bits."""
    B, S, H, D = x.shape
    return x.float().reshape(B, S, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)


def _tokens_first(x):
    """(B, Hkv, G, S, D) -> (B, S, H, D) in bf16."""
    B, Hkv, G, S, D = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(B, S, Hkv * G, D).to(torch.bfloat16)


def _scores(q, k, scale, cap, slopes, distance, mask):
    """Shaped scores and the tanh values of the cap; q, k heads first."""
    s = (q @ k.transpose(-1, -2)) * scale
    t = None
    if cap:
        t = torch.tanh(s / cap)
        s = cap * t
    if slopes is not None:
        s = s - slopes.reshape(1, k.shape[1], -1, 1, 1) * distance
    return s.masked_fill(~mask, -math.inf), t


def _softmax(s):
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), (torch.log(total) + m).squeeze(-1)


def _train_plain(st):
    c = st["case"]
    Hkv, scale = c["Hkv"], c["D"] ** -0.5
    packed = c["layout"] == "docs"
    q, k, v, dout = (_heads_first(x.unsqueeze(0) if packed else x, Hkv)
                     for x in (st["q"], st["k"], st["v"], st["dout"]))
    S = q.shape[-2]
    i = torch.arange(S, device="cuda")
    mask = i[:, None] >= i[None, :]
    if packed:
        doc = torch.searchsorted(st["cu"][1:].long(), i, right=True)
        mask = mask & (doc[:, None] == doc[None, :])
    if c["prefix"]:
        mask = mask | (i[None, :] < c["prefix"])
    if c["window"]:
        mask = mask & (i[:, None] - i[None, :] < c["window"])
    distance = (i[:, None] - i[None, :]).abs().float()
    s, t = _scores(q, k, scale, c["cap"], st["slopes"], distance, mask)
    p, lse = _softmax(s)
    del s
    out = p @ v
    lse = lse.flatten(1, 2)
    heads = lambda x: _tokens_first(x).squeeze(0) if packed else _tokens_first(x)  # noqa: E731
    result = dict(out=heads(out), lse=lse.squeeze(0) if packed else lse)
    if not c["grad"]:
        return result
    dp = dout @ v.transpose(-1, -2)
    ds = p * (dp - (dout * out).sum(-1, keepdim=True))
    if t is not None:
        ds = ds * (1 - t * t)
    dq = (ds @ k) * scale
    dk = (ds.transpose(-1, -2) @ q).sum(2, keepdim=True) * scale
    dv = (p.transpose(-1, -2) @ dout).sum(2, keepdim=True)
    result.update(dq=heads(dq), dk=heads(dk), dv=heads(dv))
    return result


def _padded_positions(st):
    """Of a ragged batch: (sequence, place in it, position) of each token."""
    c, cu, kv = st["case"], st["cu"].long(), st["kv_len"].long()
    token = torch.arange(st["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:], token, right=True)
    place = token - cu[seq]
    return seq, place, kv[seq] - (cu[seq + 1] - cu[seq]) + place


def _chunk_plain(st):
    c = st["case"]
    B, H, Hkv, D = c["B"], c["H"], c["Hkv"], c["D"]
    seq, place, position = _padded_positions(st)
    q = torch.zeros(B, c["q_max"], H, D, device="cuda", dtype=torch.bfloat16)
    q[seq, place] = st["q"]
    at = torch.full((B, c["q_max"]), -1, device="cuda")
    at[seq, place] = position
    keys = _heads_first(st["k_cache"][st["block_table"].long()].flatten(1, 2), Hkv)
    values = _heads_first(st["v_cache"][st["block_table"].long()].flatten(1, 2), Hkv)
    j = torch.arange(keys.shape[-2], device="cuda")
    mask = (j <= at[..., None]) & (j < st["kv_len"].long()[:, None, None])
    distance = at[..., None] - j
    if c["window"]:
        mask = mask & (distance < c["window"])
    s, _ = _scores(_heads_first(q, Hkv), keys, D ** -0.5, c["cap"], st["slopes"],
                   distance[:, None, None].float() if c["slopes"] else None, mask[:, None, None])
    p, lse = _softmax(s)
    out = _tokens_first(p @ values)
    return dict(out=out[seq, place], lse=lse.flatten(1, 2)[seq, :, place].t().contiguous())


def _rotated(x, positions, inv_freq, interleaved, amplitude, inverse):
    """x (..., H, D) with positions (...): the first 2 * len(inv_freq) values of each head turned."""
    angle = positions.double()[..., None, None] * inv_freq
    cos, sin = (torch.cos(angle) * amplitude).float(), (torch.sin(angle) * amplitude).float()
    if inverse:
        sin = -sin
    r = 2 * inv_freq.numel()
    y = x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    first, second = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((first, second), -1).flatten(-2) if interleaved else torch.cat((first, second), -1)
    return torch.cat((turned, y[..., r:]), -1).to(torch.bfloat16)


def _append_plain(st):
    c = st["case"]
    seq, _, position = _padded_positions(st)
    how = (st["inv_freq"], c["interleaved"], c["amplitude"], False)
    page = st["block_table"].long()[seq, position // c["page"]]
    st["k_cache"][page, position % c["page"]] = _rotated(st["k"], position, *how)
    st["v_cache"][page, position % c["page"]] = st["v"]
    return dict(q=_rotated(st["q"], position, *how), k_cache=st["k_cache"], v_cache=st["v_cache"])


# ---------------------------------------------------------------------------------------- one pass
def _own(st):
    import mask_skipping_flashattention_b200 as bfa

    c = st["case"]
    if c["kind"] == "train":
        shape = dict(softcap=c["cap"] or None, slopes=st["slopes"])
        out, lse = bfa.fwd(st["plan"], st["q"], st["k"], st["v"], **shape)
        result = dict(out=out, lse=lse)
        if c["grad"]:
            dq, dk, dv = bfa.bwd(st["plan"], st["q"], st["k"], st["v"], out, st["dout"], lse, **shape)
            result.update(dq=dq, dk=dk, dv=dv)
        return result
    if c["kind"] == "chunk":
        out, lse = bfa.fwd_chunk(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["cu"], st["kv_len"],
                                 max_q=c["q_max"], window_left=c["window"] or -1, softcap=c["cap"] or None,
                                 slopes=st["slopes"])
        return dict(out=out, lse=lse)
    if c["kind"] == "rope":
        return bfa.rope(st["x"], st["positions"], st["inv_freq"], interleaved=c["interleaved"],
                        amplitude=c["amplitude"], inverse=c["inverse"])
    q = bfa.append_paged(st["k"], st["v"], st["k_cache"], st["v_cache"], st["block_table"], st["cu"], st["kv_len"],
                         q=st["q"], inv_freq=st["inv_freq"], interleaved=c["interleaved"], amplitude=c["amplitude"])
    return dict(q=q, k_cache=st["k_cache"], v_cache=st["v_cache"])


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "train":
        return _train_plain(state)
    if kind == "chunk":
        return _chunk_plain(state)
    if kind == "append":
        return _append_plain(state)
    c = state["case"]
    return _rotated(state["x"], state["positions"], state["inv_freq"], c["interleaved"], c["amplitude"], c["inverse"])


# ---------------------------------------------------------------------------------------- work
def _causal_pairs(first, n, window, keys):
    """Attended pairs of n queries at positions first, first + 1, ... over ``keys`` keys."""
    pairs = 0
    for p in range(first, first + n):
        hi = min(p + 1, keys)
        pairs += max(0, hi - (max(0, p - window + 1) if window else 0))
    return pairs


def work(case):
    c = case
    D = c["D"]
    if c["kind"] == "train":
        H, Hkv = c["H"], c["Hkv"]
        if c["layout"] == "docs":
            lens = _doc_lens(c)
            tokens, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
        else:
            tokens = c["B"] * c["S"]
            one = _causal_pairs(0, c["S"], c["window"], c["S"])
            if c["prefix"]:  # the keys of the prefix behind a query
                one += c["prefix"] * (c["prefix"] - 1) // 2
            pairs = c["B"] * one
        flops = 4.0 * D * pairs * H * (3.5 if c["grad"] else 1.0)
        size = tokens * D * 2 * (2 * H + 2 * Hkv) + tokens * H * 4
        if c["grad"]:  # dout in; dq, dk, dv out
            size += tokens * D * 2 * (2 * H + 2 * Hkv)
        return dict(bytes=float(size), flops=flops)
    if c["kind"] == "rope":
        elements = c["B"] * c["S"] * c["H"] * D
        return dict(bytes=4.0 * elements + 4.0 * c["B"] * c["S"], flops=3.0 * elements)
    lens = _seq_lens(c)
    tokens = sum(n for n, _ in lens)
    if c["kind"] == "append":  # q, k, v in; q and the new rows of the caches out
        elements = tokens * D * (c["H"] + 2 * c["Hkv"])
        return dict(bytes=4.0 * elements, flops=3.0 * tokens * D * (c["H"] + c["Hkv"]))
    pairs = sum(_causal_pairs(kv - n, n, c["window"], kv) for n, kv in lens)
    keys = sum(kv - (max(0, kv - n - c["window"] + 1) if c["window"] else 0) for n, kv in lens)
    size = keys * c["Hkv"] * D * 4 + tokens * c["H"] * (D * 4 + 4)
    return dict(bytes=float(size), flops=4.0 * D * pairs * c["H"])


# ---------------------------------------------------------------------------------------- 64 bits
def _exact_row_block(q, k, v, allowed, distance, cap, slope, dout=None):
    """One head of one sequence: q (n, D), k, v (m, D) in 64 bits; rows that attend nothing give 0 and -inf."""
    raw = q.mm(k.t()).div(math.sqrt(q.shape[1]))
    bent = torch.tanh(raw / cap) if cap else None
    z = cap * bent if cap else raw
    if slope is not None:
        z = z - float(slope) * distance
    z = torch.where(allowed, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, 1)
    w = torch.exp(z - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[:, None])
    o = w.mm(v)
    if dout is None:
        return o, lse
    g = w * (dout.mm(v.t()) - (dout * o).sum(1)[:, None])
    if cap:
        g = g * (1 - bent.square())
    g = g / math.sqrt(q.shape[1])
    return o, lse, g.mm(k), g.t().mm(q), w.t().mm(dout)


def _exact_train(st):
    c = st["case"]
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    packed = c["layout"] == "docs"
    starts = _cumulated(_doc_lens(c)) if packed else [b * c["S"] for b in range(c["B"] + 1)]
    q, k, v, dout = (st[n].reshape(-1, st[n].shape[-2], D).double() for n in ("q", "k", "v", "dout"))
    out, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.zeros(H, q.shape[0], dtype=torch.float64, device="cuda")
    for a, b in zip(starts, starts[1:]):
        i = torch.arange(b - a, device="cuda")
        behind = i[:, None] - i[None, :]
        allowed = behind >= 0
        if c["window"]:
            allowed = allowed & (behind < c["window"])
        if c["prefix"]:
            allowed = allowed | (i < c["prefix"])[None, :]
        for h in range(H):
            kh = h * Hkv // H
            got = _exact_row_block(q[a:b, h], k[a:b, kh], v[a:b, kh], allowed, behind.abs().double(), c["cap"],
                                   st["slopes"][h] if c["slopes"] else None, dout[a:b, h] if c["grad"] else None)
            out[a:b, h], lse[h, a:b] = got[0], got[1]
            if c["grad"]:
                dq[a:b, h] = got[2]
                dk[a:b, kh] += got[3]
                dv[a:b, kh] += got[4]
    shaped = (lambda x: x) if packed else (lambda x: x.reshape(c["B"], c["S"], -1, D))
    result = dict(out=shaped(out), lse=lse if packed else lse.reshape(H, c["B"], c["S"]).transpose(0, 1))
    if c["grad"]:
        result.update(dq=shaped(dq), dk=shaped(dk), dv=shaped(dv))
    return result


def _exact_chunk(st):
    c = st["case"]
    q = st["q"].double()
    out = torch.zeros_like(q)
    lse = torch.zeros(c["H"], q.shape[0], dtype=torch.float64, device="cuda")
    at = 0
    for s, (n, kv) in enumerate(_seq_lens(c)):
        used = st["block_table"][s, :-(-kv // c["page"])].long()
        behind = torch.arange(kv - n, kv, device="cuda")[:, None] - torch.arange(kv, device="cuda")
        allowed = behind >= 0
        if c["window"]:
            allowed = allowed & (behind < c["window"])
        for kh in range(c["Hkv"]):
            k = st["k_cache"][used, :, kh].flatten(0, 1)[:kv].double()
            v = st["v_cache"][used, :, kh].flatten(0, 1)[:kv].double()
            G = c["H"] // c["Hkv"]
            for h in range(kh * G, kh * G + G):
                out[at:at + n, h], lse[h, at:at + n] = _exact_row_block(
                    q[at:at + n, h], k, v, allowed, behind.double(), c["cap"],
                    st["slopes"][h] if c["slopes"] else None)
        at += n
    return dict(out=out, lse=lse)


def _exact_turn(x, positions, c, inverse):
    """Rotation as a product of complex numbers."""
    r = c["rotary"]
    turns = torch.polar(torch.full((r // 2,), float(c["amplitude"]), dtype=torch.float64, device="cuda"),
                        torch.zeros(r // 2, dtype=torch.float64, device="cuda"))
    exponent = torch.arange(r // 2, dtype=torch.float64, device="cuda") * (-2.0 / r)
    angle = positions.double().unsqueeze(-1) * torch.exp(exponent * math.log(10000.0))
    turns = turns * torch.exp(1j * (-angle if inverse else angle))
    y = x.double().clone()
    if c["interleaved"]:
        z = torch.view_as_complex(y[..., :r].reshape(*y.shape[:-1], r // 2, 2).contiguous()) * turns.unsqueeze(-2)
        y[..., :r] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * turns.unsqueeze(-2)
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def _exact_append(st):
    c = st["case"]
    k_cache, v_cache, q_out = st["k_cache"].double(), st["v_cache"].double(), []
    at = 0
    for s, (n, kv) in enumerate(_seq_lens(c)):
        position = torch.arange(kv - n, kv, device="cuda")
        q_out.append(_exact_turn(st["q"][at:at + n], position, c, False))
        page, row = st["block_table"][s].long()[position // c["page"]], position % c["page"]
        k_cache[page, row] = _exact_turn(st["k"][at:at + n], position, c, False)
        v_cache[page, row] = st["v"][at:at + n].double()
        at += n
    return dict(q=torch.cat(q_out), k_cache=k_cache, v_cache=v_cache)


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "train":
        return _exact_train(st)
    if case["kind"] == "chunk":
        return _exact_chunk(st)
    if case["kind"] == "append":
        return _exact_append(st)
    return _exact_turn(st["x"], st["positions"], case, case["inverse"])
