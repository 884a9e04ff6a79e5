"""Workloads of the serving operators around the q8 decode: rotary positions on the way into
the cache, decode with the log-sum-exp of its rows, accumulated attention weights, eviction
by those weights, and verification of drafted tokens.

Each case is a dict of plain values. ``prepare`` draws its inputs on the GPU, ``run`` makes
one pass (the plain torch form, or the library's call where ``own`` is set), ``exact`` gives
the result in 64 bits, ``work`` the bytes and operations a pass cannot do without.

Cached K and V codes are compared as the int8 numbers they are, next to their scales: both
forms follow the same fp32 quantisation rule, so the codes are equal, not merely near.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
DEVICE = "cuda"
INV127 = 1.0 / 127.0


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a mid-size batch: one new token per sequence, text positions
        dict(name="rope_decode_step", op="rope", tokens=64, hq=32, hk=8, d=128, rot=128, axes=1,
             adjacent=False, dtype="bf16", bs=64),
        # a prompt with an image: time, height and width positions, odd token count
        dict(name="rope_image_prompt", op="rope", tokens=4999, hq=32, hk=8, d=128, rot=128, axes=3,
             adjacent=False, dtype="bf16", bs=64),
        # a long prompt filled at once from fp32 projections
        dict(name="rope_long_prompt", op="rope", tokens=32768, hq=32, hk=8, d=128, rot=128, axes=3,
             adjacent=False, dtype="fp32", bs=128),
        # the GQA decode batch of the benchmark, with its row statistics
        dict(name="lse_gqa_batch", op="lse", batch=16, hq=32, hk=8, length=4096, ragged=False,
             queries=1, bs=64),
        # four drafted tokens per sequence, ragged lengths
        dict(name="lse_draft_ragged", op="lse", batch=24, hq=64, hk=8, length=8192, ragged=True,
             queries=4, bs=128),
        # the smallest call: one short sequence
        dict(name="mass_tiny", op="mass", batch=1, hq=8, hk=8, length=256, ragged=False, queries=1,
             bs=16, decay=1.0),
        # the GQA decode batch: weights of one step added to the running sums
        dict(name="mass_gqa_batch", op="mass", batch=16, hq=32, hk=8, length=4096, ragged=False,
             queries=1, bs=64, decay=1.0),
        # a large ragged batch with decaying sums
        dict(name="mass_ragged_decay", op="mass", batch=48, hq=64, hk=8, length=16384, ragged=True,
             queries=1, bs=128, decay=0.9),
        # a few chats that passed their budget at different lengths
        dict(name="evict_chat", op="evict", batch=3, hk=8, d=128, length=2500, ragged=True,
             keep=1024, sink=4, recent=256, bs=16),
        # a batch of long contexts cut to a quarter
        dict(name="evict_long", op="evict", batch=16, hk=8, d=128, length=16384, ragged=False,
             keep=4096, sink=16, recent=1024, bs=64),
        # one user, a short draft
        dict(name="verify_single", op="verify", batch=1, drafts=4, vocab=32000, dtype="fp32"),
        # a large batch, a vocabulary that is no multiple of a vector
        dict(name="verify_batch", op="verify", batch=128, drafts=5, vocab=131075, dtype="fp32"),
    ]


HEADS = [(8, 8), (32, 8), (32, 4), (64, 8), (16, 4), (40, 8), (28, 4), (4, 1)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "lse", "mass", "evict", "verify"])
    if op == "rope":
        hq, hk = rng.choice(HEADS)
        d = rng.choice([64, 128, 128, 256])
        rot = rng.choice([d, d, d // 2])
        most = max(1, 32768 * 48 * 128 // ((hq + 2 * hk) * d))
        return dict(op=op, tokens=_log(rng, 1, min(most, 32768)), hq=hq, hk=hk, d=d, rot=rot,
                    axes=rng.randint(1, 4), adjacent=rng.random() < 0.3,
                    dtype=rng.choice(["fp32", "bf16", "fp16"]), bs=rng.choice([16, 32, 64, 128]))
    if op in ("lse", "mass"):
        hq, hk = rng.choice(HEADS)
        batch = _log(rng, 1, 64)
        most = 100_000 if op == "lse" else 390_000  # tokens in all
        length = _log(rng, 16, min(131072, max(16, most * 8 // hk // batch)))
        queries = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        if queries * hq // hk > 32:  # the plain form's score table grows with it
            queries = 1
        c = dict(op=op, batch=batch, hq=hq, hk=hk, length=length + rng.randint(0, 7),
                 ragged=rng.random() < 0.6, queries=queries, bs=rng.choice([16, 32, 64, 128, 256]))
        if op == "mass":
            c["decay"] = rng.choice([1.0, 1.0, 0.9, 0.0])
        return c
    if op == "evict":
        hk = rng.choice([1, 2, 4, 8, 3])
        batch = _log(rng, 1, 32)
        length = _log(rng, 64, min(131072, 16 * 16384 * 8 // (batch * hk))) + rng.randint(0, 9)
        keep = max(8, min(int(length * rng.uniform(0.1, 0.9)), 16 * 4096 * 8 // (batch * hk)))
        sink, recent = rng.randint(0, keep // 8), rng.randint(0, keep // 2)
        return dict(op=op, batch=batch, hk=hk, d=rng.choice([64, 128, 128, 256]) if length < 8192
                    else 128, length=length, ragged=rng.random() < 0.5, keep=keep, sink=sink,
                    recent=recent, bs=rng.choice([16, 32, 64, 128]))
    vocab = _log(rng, 1000, 200_000) + rng.randint(0, 3)
    batch = _log(rng, 1, min(128, max(1, 128 * 131075 // vocab)))
    drafts = rng.randint(0, 8)
    while drafts > 1 and batch * vocab * drafts > 128 * 131075 * 5:
        drafts -= 1
    return dict(op="verify", batch=batch, drafts=drafts, vocab=vocab,
                dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]))


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _lengths(case):
    """Lengths are part of the case (what a pass has to read follows from them): equal, or
    spread evenly over [1, length] by a fixed stream, with the longest present."""
    n, top = case["batch"], case["length"]
    if not case["ragged"]:
        return [top] * n
    r = random.Random(7919 * n + top)
    return [top] + [r.randint(1, top) for _ in range(n - 1)]


def _table(lens, bs, g, spare=2):
    """A permuted block table (entries past a sequence's blocks -1) and the pool's size."""
    need = [-(-n // bs) for n in lens]
    width = max(1, max(need))
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pool, perm[at:]


def _rows(shape, g):
    """Codes and scales of normal rows, as the cache write stores them."""
    codes = torch.empty(shape, dtype=torch.int8, device=DEVICE)
    scales = torch.empty(shape[:-1], dtype=torch.float32, device=DEVICE)
    step = max(1, (64 << 20) // math.prod(shape[1:]))
    for i in range(0, shape[0], step):
        x = torch.randn((min(step, shape[0] - i),) + tuple(shape[1:]), generator=g, device=DEVICE)
        top = x.abs().amax(-1, keepdim=True)
        scales[i:i + step] = (top * INV127)[..., 0]
        codes[i:i + step] = (x * (torch.full_like(top, 127.0) / top)).round().clamp(-127, 127)
    return codes, scales


def _prepare_cache(case, g, v):
    lens = _lengths(case)
    bs, hk, d = case["bs"], case["hk"], case.get("d", 128)
    table, pool, free = _table(lens, bs, g)
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE))
    s["k"], s["ks"] = _rows((pool, bs, hk, d), g)
    if v:
        s["v"], s["vs"] = _rows((pool, bs, hk, d), g)
    return s


def _prepare_rope(case, seed):
    g = _gen(seed)
    n, hq, hk, d, rot, axes = (case[k] for k in ("tokens", "hq", "hk", "d", "rot", "axes"))
    dt = DTYPES[case["dtype"]]
    # q, k and v are slices of one fused projection
    qkv = torch.randn((n, (hq + 2 * hk) * d), generator=g, device=DEVICE).to(dt)
    q = qkv[:, :hq * d].view(n, hq, d)
    k = qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
    v = qkv[:, (hq + hk) * d:].view(n, hk, d)
    top = 32768
    inv = 10000.0 ** (-torch.arange(rot // 2, device=DEVICE, dtype=torch.float64) * 2 / rot)
    angle = torch.arange(top, device=DEVICE, dtype=torch.float64)[:, None] * inv
    table = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    # text: the axes agree; image patches: rows and columns of a grid under one time step
    t = torch.arange(n, device=DEVICE) % top
    side = max(1, math.isqrt(n // 2 + 1))
    image = (t >= n // 4) & (t < 3 * n // 4)
    place = (t - n // 4).clamp(min=0)
    rows = [t, torch.where(image, n // 4 + place // side % side, t),
            torch.where(image, n // 4 + place % side, t), torch.where(image, t // 2, t)]
    pos = torch.stack([rows[a].clamp(0, top - 1) for a in range(axes)]).to(torch.int32).contiguous()
    pairs = rot // 2
    if axes == 1:
        axis = None
    elif seed % 2:  # axes take turns over the frequencies
        axis = [i % axes for i in range(pairs)]
    else:  # one run of frequencies per axis, a quarter for time and the rest shared
        first = max(1, pairs // 4)
        axis = [0 if i < first else 1 + (i - first) * (axes - 1) // (pairs - first)
                for i in range(pairs)]
    bs = case["bs"]
    pool = -(-n // bs) + 1
    t = torch.arange(n, device=DEVICE)
    slots = torch.randperm(pool, generator=g, device=DEVICE)[t // bs] * bs + t % bs
    if n > 8:
        slots[torch.randperm(n, generator=g, device=DEVICE)[:n // 64 + 1]] = -1  # padding
    s = dict(case=case, q=q, k_new=k, v_new=v, table=table, pos=pos, axis=axis, slots=slots,
             q_out=torch.empty((n, hq, d), device=DEVICE))
    # the axis of each pair, as the plain form indexes with it
    s["axis_index"] = torch.tensor(axis or [0] * pairs, device=DEVICE)
    for a in ("k", "v"):
        s[a] = torch.zeros((pool, bs, hk, d), dtype=torch.int8, device=DEVICE)
        s[a + "s"] = torch.zeros((pool, bs, hk), device=DEVICE)
    return s


def _prepare_lse(case, seed):
    g = _gen(seed)
    s = _prepare_cache(case, g, True)
    shape = (case["batch"], case["queries"], case["hq"], 128)
    s["q"] = torch.randn(shape, generator=g, device=DEVICE)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(shape[:3], device=DEVICE)
    s["scale"] = 128 ** -0.5
    return s


def _prepare_mass(case, seed):
    g = _gen(seed)
    s = _prepare_cache(case, g, False)
    b, hk = case["batch"], case["hk"]
    s["q"] = torch.randn((b, case["queries"], case["hq"], 128), generator=g, device=DEVICE)
    s["scale"] = 128 ** -0.5
    cap = s["table"].shape[1] * case["bs"]
    # running sums of a few earlier steps, of the size of one step's weights
    s["mass"] = torch.empty((b, hk, cap), device=DEVICE).exponential_(1.0, generator=g) * \
        (4.0 * case["hq"] / hk / case["length"])
    s["lse"] = torch.empty((b, case["queries"], case["hq"]), device=DEVICE)
    for i in range(b):  # the statistics that the decode of the same step left
        one = dict(s, q=s["q"][i:i + 1], table=s["table"][i:i + 1], lens=s["lens"][i:i + 1])
        s["lse"][i] = _scores(one).double().logsumexp(-1).permute(0, 3, 1, 2).reshape(
            case["queries"], case["hq"]).float()
    return s


def _prepare_evict(case, seed):
    g = _gen(seed)
    lens = _lengths(case)
    bs, hk, d, keep = case["bs"], case["hk"], case["d"], case["keep"]
    width = -(-keep // bs)
    table, pool, free = _table(lens, bs, g, spare=2 + width * len(lens))
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE),
             new_table=free[:width * len(lens)].view(len(lens), width).contiguous())
    s["k"], s["ks"] = _rows((pool, bs, hk, d), g)
    s["v"], s["vs"] = _rows((pool, bs, hk, d), g)
    b = len(lens)
    # sums of many softmax weights: heavy tailed, and zero where nothing ever looked
    mass = torch.randn((b, hk, table.shape[1] * bs), generator=g, device=DEVICE)
    mass = (2.0 * mass - 6.0).exp()
    mass[torch.rand(mass.shape, generator=g, device=DEVICE) < 0.05] = 0.0
    s["mass"] = mass
    s["new_mass"] = torch.empty((b, hk, width * bs), device=DEVICE)
    s["kept"] = torch.empty((b, hk, keep), dtype=torch.int32, device=DEVICE)
    s["new_lens"] = torch.empty((b,), dtype=torch.int32, device=DEVICE)
    return s


def _prepare_verify(case, seed):
    g = _gen(seed)
    b, n, v = case["batch"], case["drafts"], case["vocab"]
    dt = DTYPES[case["dtype"]]
    logits = torch.randn((b, n + 1, v), generator=g, device=DEVICE) * 2.5
    target = logits.softmax(-1).to(dt)
    logits = logits[:, :n] + 0.6 * torch.randn((b, n, v), generator=g, device=DEVICE)
    draft = logits.softmax(-1).to(dt)
    # the draft model's own samples
    noise = torch.empty((b, n, v), device=DEVICE).exponential_(1.0, generator=g)
    tokens = (draft.float() / noise).argmax(-1).to(torch.int32) if n else \
        torch.zeros((b, 0), dtype=torch.int32, device=DEVICE)
    return dict(case=case, target=target, draft=draft, drafted=tokens,
                uniforms=torch.rand((b, n + 1), generator=g, device=DEVICE),
                accepted=torch.empty((b,), dtype=torch.int32, device=DEVICE),
                tokens=torch.empty((b, n + 1), dtype=torch.int32, device=DEVICE))


def prepare(case, seed):
    return {"rope": _prepare_rope, "lse": _prepare_lse, "mass": _prepare_mass,
            "evict": _prepare_evict, "verify": _prepare_verify}[case["op"]](case, seed)


# ------------------------------------------------------------------------------- plain forms

def _quantise(x, block):
    """int8 codes of blocks of the last dimension (as fp32 numbers) and the blocks' scales."""
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // block, block))
    top = y.abs().amax(-1, keepdim=True)
    top = torch.where(top < 1e-6, torch.ones_like(top), top)
    codes = (y * (torch.full_like(top, 127.0) / top)).round().clamp(-127, 127)
    return codes, (top * INV127)[..., 0]


def _slots(s):
    """Physical slot of every position of every sequence, and whether it holds a token."""
    bs, cap = s["case"]["bs"], s["table"].shape[1] * s["case"]["bs"]
    t = torch.arange(cap, device=DEVICE)
    slot = s["table"].long().clamp(min=0)[:, t // bs] * bs + t % bs
    return slot, t[None] < s["lens"][:, None]


def _scores(s):
    """Softmax scores [sequence][KV head][head in its group][query][position], -inf at the
    positions that the query does not see."""
    b, nq, hq, d = s["q"].shape
    hk = s["k"].shape[2]
    codes, qs = _quantise(s["q"], 32)
    codes = codes.reshape(b, nq, hk, hq // hk, d // 32, 32)
    qs = qs.reshape(b, nq, hk, hq // hk, d // 32)
    slot, inside = _slots(s)
    k = s["k"].reshape(-1, hk, d)[slot].float().reshape(b, -1, hk, d // 32, 32)
    dots = torch.einsum("bnhgjc,bthjc->bhgnjt", codes, k)
    dots = (dots * qs.permute(0, 2, 3, 1, 4)[..., None]).sum(4)
    ks = s["ks"].reshape(-1, hk)[slot].permute(0, 2, 1)
    t = torch.arange(slot.shape[1], device=DEVICE)
    sees = s["lens"][:, None] - (nq - 1 - torch.arange(nq, device=DEVICE))
    seen = t < sees[..., None]  # [b][nq][t]
    x = dots * ks[:, :, None, None] * s["scale"]
    return x.masked_fill(~seen[:, None, None], -math.inf)


def _run_rope(s):
    c = s["case"]
    n, rot, pairs = c["tokens"], c["rot"], c["rot"] // 2
    row = s["table"][s["pos"].long()]  # [axes][n][rot]
    pick = s["axis_index"][None, None].expand(1, n, pairs)
    cos = row[..., :pairs].gather(0, pick)[0][:, None]
    sin = row[..., pairs:].gather(0, pick)[0][:, None]

    def rotate(x):
        x = x.float()
        if c["adjacent"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :pairs], x[..., pairs:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1)

    live = (s["slots"] >= 0).nonzero()[:, 0]
    at = s["slots"][live]
    for name, x in (("k", rotate(s["k_new"])), ("v", s["v_new"].float())):
        codes, scale = _quantise(x[live], c["d"])
        s[name].view(-1, c["hk"], c["d"])[at] = codes[..., 0, :].to(torch.int8)
        s[name + "s"].view(-1, c["hk"])[at] = scale[..., 0]
    return {"q": rotate(s["q"]), "k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"]}


def _run_lse(s):
    x = _scores(s)  # [b][hk][g][nq][t]
    b, hk, g, nq, _ = x.shape
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = (x - top).exp()
    total = w.sum(-1)
    slot, inside = _slots(s)
    d = s["v"].shape[3]
    v = s["v"].reshape(-1, hk, d)[slot].float() * s["vs"].reshape(-1, hk)[slot][..., None]
    v = v.masked_fill(~inside[..., None, None], 0.0)
    out = torch.einsum("bhgnt,bthd->bnhgd", w, v)
    total = total.permute(0, 3, 1, 2)
    out = torch.where(total[..., None] > 0, out / total[..., None], torch.zeros_like(out))
    lse = total.log() + top[..., 0].permute(0, 3, 1, 2)
    return {"out": out.reshape(b, nq, hk * g, d), "lse": lse.reshape(b, nq, hk * g)}


def _run_mass(s):
    x = _scores(s)
    b, hk, g, nq, _ = x.shape
    lse = s["lse"].reshape(b, nq, hk, g).permute(0, 2, 3, 1)[..., None]
    w = torch.where(x == -math.inf, torch.zeros_like(x), (x - lse).exp()).sum((2, 3))
    _, inside = _slots(s)
    old = s["mass"] * s["case"]["decay"]
    s["mass"].copy_(torch.where(inside[:, None], old + w, s["mass"]))
    return s["mass"]


def _run_evict(s):
    c = s["case"]
    keep, sink, recent, bs, hk, d = (c[k] for k in ("keep", "sink", "recent", "bs", "hk", "d"))
    lens = s["lens"].long()
    cap = s["mass"].shape[2]
    t = torch.arange(cap, device=DEVICE)
    inside = t < lens[:, None]
    held = ((t < sink) | (t >= lens[:, None] - recent) | (lens[:, None] <= keep)) & inside
    key = torch.where(held[:, None], math.inf, s["mass"])
    key = torch.where(inside[:, None], key, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True)[1][..., :min(keep, cap)]
    new = lens.clamp(max=keep)
    j = torch.arange(keep, device=DEVICE)
    taken = torch.full((c["batch"], hk, keep), cap, device=DEVICE)
    taken[..., :order.shape[-1]] = order
    taken = torch.where(j < new[:, None, None], taken, cap).sort(dim=-1)[0]
    live = taken < cap
    src = taken.clamp(max=cap - 1)
    where = s["table"].long().clamp(min=0)
    from_slot = where.gather(1, (src // bs).flatten(1)).view_as(src) * bs + src % bs
    to_slot = (s["new_table"].long()[:, j // bs] * bs + j % bs)[:, None].expand_as(src)
    head = torch.arange(hk, device=DEVICE)[None, :, None].expand_as(src)
    a, b, h = from_slot[live], to_slot[live], head[live]
    for name in ("k", "v"):
        rows, scale = s[name].view(-1, hk, d), s[name + "s"].view(-1, hk)
        rows[b, h] = rows[a, h]
        scale[b, h] = scale[a, h]
    s["new_mass"].zero_()
    s["new_mass"][..., :keep] = torch.where(live, s["mass"].gather(2, src), 0.0)
    s["kept"].copy_(torch.where(live, taken, -1))
    s["new_lens"].copy_(new)
    return {k: s[k] for k in ("k", "v", "ks", "vs", "new_mass", "kept", "new_lens")}


def _run_verify(s):
    c = s["case"]
    b, n, v = c["batch"], c["drafts"], c["vocab"]
    at = s["drafted"].long()[..., None]
    p = s["target"][:, :n].gather(2, at)[..., 0].double()
    q = s["draft"].gather(2, at)[..., 0].double()
    good = s["uniforms"][:, :n].double() * q < p
    count = good.long().cumprod(1).sum(1)
    every = torch.arange(b, device=DEVICE)
    row = s["target"][every, count].double()
    if n:
        other = s["draft"][every, count.clamp(max=n - 1)].double()
        rest = (row - other).clamp(min=0.0)
        rest = torch.where((count == n)[:, None] | (rest.sum(1, keepdim=True) <= 0), row, rest)
    else:
        rest = row
    c = rest.cumsum(1)
    goal = s["uniforms"][:, n:].double() * c[:, -1:]
    last = (rest > 0).long().cumsum(1).argmax(1)  # the last token of any weight
    token = torch.minimum((c <= goal).sum(1), last)
    j = torch.arange(n + 1, device=DEVICE)
    padded = torch.cat([s["drafted"].long(), token[:, None]], 1)
    tokens = torch.where(j < count[:, None], padded, -1)
    tokens = torch.where(j == count[:, None], token[:, None], tokens)
    return {"accepted": count.int(), "tokens": tokens.int()}


# ------------------------------------------------------------------------------- the library

def _own(s):
    import decode_attention_int8_b200 as q8

    c = s["case"]
    if c["op"] == "rope":
        q8.q8kv_rope_cache_write(s["q_out"], s["k"], s["v"], s["ks"], s["vs"], s["q"], s["k_new"],
                                 s["v_new"], s["slots"], s["pos"], s["table"], pair_axis=s["axis"],
                                 adjacent=c["adjacent"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"]}
    if c["op"] == "lse":
        q8.q8kv_decode_attn_lse(s["out"], s["lse"], s["q"], s["k"], s["v"], s["ks"], s["vs"],
                                s["table"], s["lens"], s["scale"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "mass":
        q8.q8kv_attn_mass(s["mass"], s["q"], s["lse"], s["k"], s["ks"], s["table"], s["lens"],
                          s["scale"], decay=c["decay"])
        return s["mass"]
    if c["op"] == "evict":
        q8.q8kv_evict(s["k"], s["v"], s["ks"], s["vs"], s["new_mass"], s["kept"], s["new_lens"],
                      s["mass"], s["table"], s["lens"], s["new_table"], sink=c["sink"],
                      recent=c["recent"])
        return {k: s[k] for k in ("k", "v", "ks", "vs", "new_mass", "kept", "new_lens")}
    q8.q8kv_verify_draft(s["accepted"], s["tokens"], s["target"], s["draft"], s["drafted"],
                         s["uniforms"])
    return {"accepted": s["accepted"], "tokens": s["tokens"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _run_rope, "lse": _run_lse, "mass": _run_mass, "evict": _run_evict,
            "verify": _run_verify}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "rope":
        n, hq, hk, d = (case[k] for k in ("tokens", "hq", "hk", "d"))
        size = 4 if case["dtype"] == "fp32" else 2
        read = n * ((hq + 2 * hk) * d * size + 8 + 4 * case["axes"])
        write = n * (hq * d * 4 + 2 * hk * (d + 4))
        rows = min(n, 32768)  # table rows that some token names
        return {"bytes": read + write + rows * case["rot"] * 4, "flops": n * (hq + hk) * case["rot"] * 3}
    if op == "verify":
        b, n, v = case["batch"], case["drafts"], case["vocab"]
        size = 4 if case["dtype"] == "fp32" else 2
        # about three drafts in four are taken: a row of the target for each sequence, and one
        # of the draft for those that refuse a token
        refuse = 1.0 - 0.75 ** n
        return {"bytes": b * (v * size * (1 + refuse) + n * (2 * size + 8) + 4 * (n + 2)),
                "flops": b * v * (1 + 2 * refuse)}
    lens, hk, bs = _lengths(case), case["hk"], case["bs"]
    units = sum(lens) * hk
    blocks = sum(-(-n // bs) for n in lens)
    if op == "evict":
        d = case["d"]
        rows = sum(min(n, case["keep"]) for n in lens) * hk
        return {"bytes": units * 4 + rows * (2 * (2 * d + 8) + 8) + 4 * (blocks + 2 * len(lens)),
                "flops": units}
    heads = case["batch"] * case["queries"] * case["hq"]
    group = case["queries"] * case["hq"] // hk
    if op == "lse":
        return {"bytes": units * 264 + heads * (1024 + 4) + 4 * (blocks + len(lens)),
                "flops": units * group * 4 * 128}
    old = 4 if case["decay"] else 0
    return {"bytes": units * (132 + 4 + old) + heads * (512 + 4) + 4 * (blocks + len(lens)),
            "flops": units * group * 2 * 128}


# ------------------------------------------------------------------------------- 64 bits

def _exact_codes(q):
    """The query's codes and block scales by the rule of the decode (fp32 decides them)."""
    import numpy as np

    x = q.cpu().numpy().reshape(-1, 32)
    top = np.abs(x).max(1, keepdims=True)
    top = np.where(top < np.float32(1e-6), np.float32(1), top)
    codes = np.clip(np.rint(x * (np.float32(127) / top)), -127, 127)
    scale = np.broadcast_to(top * np.float32(1 / 127), x.shape)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE).double().view(q.shape)
    return to(codes), to(scale)


def _exact_rows(s):
    """For each sequence: (scores [nq][hk][g][t], slots of its positions), in 64 bits."""
    b, nq, hq, d = s["q"].shape
    hk, bs = s["k"].shape[2], s["case"]["bs"]
    codes, scale = _exact_codes(s["q"])
    q = (codes * scale).view(b, nq, hk, hq // hk, d)
    for i, n in enumerate(s["lens"].tolist()):
        t = torch.arange(n, device=DEVICE)
        slot = s["table"][i].long()[t // bs] * bs + t % bs
        k = s["k"].view(-1, hk, d)[slot].double() * s["ks"].view(-1, hk)[slot].double()[..., None]
        x = torch.matmul(q[i].transpose(0, 1).reshape(hk, -1, d), k.permute(1, 2, 0))
        x = x.view(hk, nq, hq // hk, n).transpose(0, 1) * s["scale"]
        for j in range(nq):
            x[j, :, :, max(0, n - (nq - 1 - j)):] = -math.inf
        yield i, x, slot


def _exact_attention(case, seed):
    s = prepare(case, seed)
    b, nq, hq, d = s["q"].shape
    hk = case["hk"]
    if case["op"] == "mass":
        mass = s["mass"].double()
        for i, x, slot in _exact_rows(s):
            lse = s["lse"][i].double().view(nq, hk, hq // hk, 1)
            w = torch.where(x == -math.inf, 0.0, torch.exp(x - lse)).sum((0, 2))
            mass[i, :, :x.shape[-1]] = mass[i, :, :x.shape[-1]] * case["decay"] + w
        return mass
    out = torch.zeros((b, nq, hk, hq // hk, d), dtype=torch.float64, device=DEVICE)
    lse = torch.full((b, nq, hk, hq // hk), -math.inf, dtype=torch.float64, device=DEVICE)
    for i, x, slot in _exact_rows(s):
        v = s["v"].view(-1, hk, d)[slot].double() * s["vs"].view(-1, hk)[slot].double()[..., None]
        lse[i] = torch.logsumexp(x, -1)
        w = torch.exp(x - lse[i][..., None])
        w = torch.where(torch.isnan(w), 0.0, w)
        out[i] = torch.einsum("nhgt,thd->nhgd", w, v)
    return {"out": out.view(b, nq, hq, d), "lse": lse.view(b, nq, hq)}


def _exact_rope(case, seed):
    s = prepare(case, seed)
    rot, pairs = case["rot"], case["rot"] // 2
    axis = s["axis"] or [0] * pairs
    table, pos = s["table"].double(), s["pos"].long()

    def rotate(x):
        y = x.double().clone()
        for i in range(pairs):
            cos = table[pos[axis[i]], i][:, None]
            sin = table[pos[axis[i]], pairs + i][:, None]
            m, n = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + pairs)
            a, b = x[..., m].double(), x[..., n].double()
            y[..., m] = a * cos - b * sin
            y[..., n] = a * sin + b * cos
        return y

    live = s["slots"] >= 0
    got = {"q": rotate(s["q"]), "k": None, "v": None}
    for name, x in (("ks", rotate(s["k_new"])), ("vs", s["v_new"].double())):
        scale = s[name].double().view(-1, case["hk"])
        top = x[live].abs().amax(-1)
        scale[s["slots"][live]] = torch.where(top < 1e-6, 1.0, top) / 127.0
        got[name] = scale.view(s[name].shape)
    return got


def _exact_evict(case, seed):
    import numpy as np

    s = prepare(case, seed)
    keep, sink, recent, bs = (case[k] for k in ("keep", "sink", "recent", "bs"))
    mass, table, new_table = (s[k].cpu().numpy() for k in ("mass", "table", "new_table"))
    b, hk, _ = mass.shape
    new_mass = np.zeros(tuple(s["new_mass"].shape))
    ks, vs = (s[k].cpu().numpy().astype(np.float64).reshape(-1, hk) for k in ("ks", "vs"))
    old = {"ks": ks.copy(), "vs": vs.copy()}
    for i, n in enumerate(s["lens"].tolist()):
        for h in range(hk):
            if n <= keep:
                took = np.arange(n)
            else:
                middle = np.arange(sink, n - recent)
                best = middle[np.lexsort((middle, -mass[i, h, middle]))]
                took = np.sort(np.concatenate([np.arange(sink), np.arange(n - recent, n),
                                               best[:keep - sink - recent]])).astype(np.int64)
            j = np.arange(len(took))
            a = table[i, took // bs].astype(np.int64) * bs + took % bs
            to = new_table[i, j // bs].astype(np.int64) * bs + j % bs
            ks[to, h], vs[to, h] = old["ks"][a, h], old["vs"][a, h]
            new_mass[i, h, :len(took)] = mass[i, h, took]
    return {"k": None, "v": None, "ks": ks.reshape(s["ks"].shape), "vs": vs.reshape(s["vs"].shape),
            "new_mass": new_mass, "kept": None, "new_lens": None}


def exact(case, seed):
    if case["op"] in ("lse", "mass"):
        return _exact_attention(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, seed)
    return None  # verification answers in whole numbers
