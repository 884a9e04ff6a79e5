"""Plain numpy references of the serving operators (rotary cache write, decode log-sum-exp,
attention mass, eviction, draft verification), in 64 bits except where the operator fixes an
fp32 operation because it decides whole numbers (quantised codes). They share no code with the
library."""
import numpy as np

F32 = np.float32
EPS = 2.0 ** -24  # half a step of fp32, relative


# ------------------------------------------------------------------ rotary positions

def rotate(x, positions, table, pair_axis, adjacent, dtype):
    """Rows x [n][heads][D] rotated with every operation rounded to `dtype` (np.float32: the
    operator's arithmetic; np.float64: the mathematics)."""
    x = np.asarray(x).astype(dtype)
    rot = table.shape[1]
    pairs = rot // 2
    y = x.copy()
    n = np.arange(x.shape[0])
    top = table.shape[0] - 1
    for p in range(pairs):
        pos = np.clip(positions[pair_axis[p] if pair_axis is not None else 0], 0, top)[n]
        c = table[pos, p].astype(dtype)[:, None]
        s = table[pos, pairs + p].astype(dtype)[:, None]
        i, j = (2 * p, 2 * p + 1) if adjacent else (p, p + pairs)
        a, b = x[..., i], x[..., j]
        y[..., i] = a * c - b * s
        y[..., j] = b * c + a * s
    return y


def quantise_rows(x):
    """The q8 cache write's row rule in fp32: codes int8 and scales; non-finite rows give codes
    0 and a NaN scale."""
    x = np.asarray(x, F32)
    bad = ~np.isfinite(x).all(-1)
    z = np.where(bad[..., None], F32(0), x)
    top = np.abs(z).max(-1)
    top = np.where(top < F32(1e-6), F32(1), top)
    codes = np.clip(np.rint(z * (F32(127) / top)[..., None]), -127, 127).astype(np.int8)
    scale = (top * F32(1 / 127)).astype(F32)
    codes[bad] = 0
    scale[bad] = np.nan
    return codes, scale


# ------------------------------------------------------------------ scores and their statistics

def query_codes(q):
    """Codes and block scales of query rows (fp32 decides the codes), as float64."""
    x = np.asarray(q, F32).reshape(q.shape[:-1] + (q.shape[-1] // 32, 32))
    top = np.abs(x).max(-1, keepdims=True)
    top = np.where(top < F32(1e-6), F32(1), top)
    codes = np.clip(np.rint(x * (F32(127) / top)), -127, 127)
    return codes.astype(np.float64), (top * F32(1 / 127))[..., 0].astype(np.float64)


def scores(q, k, ks, table, L, scale):
    """For one sequence: scores [nq][Hq][L] (-inf outside a query's view or in a block whose
    table entry is no block) and the sum of the magnitudes of each score's four terms."""
    nq, Hq, D = q.shape
    P, bs, Hk, _ = k.shape
    G = Hq // Hk
    codes, qs = query_codes(q)
    t = np.arange(L)
    blk = table[t // bs].astype(np.int64)
    ok = (blk >= 0) & (blk < P)
    blk = np.where(ok, blk, 0)
    rows = k[blk, t % bs].astype(np.float64).reshape(L, Hk, D // 32, 32)
    sc = ks[blk, t % bs].astype(np.float64)
    x = np.empty((nq, Hq, L))
    mag = np.empty((nq, Hq, L))
    for h in range(Hq):
        dots = np.einsum("njc,tjc->njt", codes[:, h], rows[:, h // G]) * qs[:, h][..., None]
        m = sc[:, h // G] * scale
        x[:, h] = dots.sum(1) * m
        mag[:, h] = np.abs(dots).sum(1) * np.abs(m)
    for i in range(nq):
        x[i, :, max(0, L - (nq - 1 - i)):] = -np.inf
    x[:, :, ~ok] = -np.inf
    return x, mag, ok


def lse_rows(x):
    """ln sum exp over the last axis, -inf for rows that see nothing."""
    top = x.max(-1, keepdims=True)
    top = np.where(np.isneginf(top), 0.0, top)
    with np.errstate(divide="ignore"):
        return (np.log(np.exp(x - top).sum(-1, keepdims=True)) + top)[..., 0]


def decode_lse(q, k, v, ks, vs, table, lens, scale):
    """out [B][nq][Hq][D], lse [B][nq][Hq] and a bound on the error of an fp32 lse."""
    B, nq, Hq, D = q.shape
    P, bs, Hk, _ = k.shape
    G = Hq // Hk
    out = np.zeros((B, nq, Hq, D))
    lse = np.full((B, nq, Hq), -np.inf)
    bound = np.zeros((B, nq, Hq))
    cap = table.shape[1] * bs
    for b in range(B):
        L = int(min(max(lens[b], 0), cap))
        if L == 0:
            continue
        x, mag, ok = scores(q[b], k, ks, table[b], L, scale)
        lse[b] = lse_rows(x)
        t = np.arange(L)
        blk = np.where(ok, table[b, t // bs], 0).astype(np.int64)
        w = np.where(np.isneginf(x), 0.0, np.exp(x - np.where(np.isneginf(lse[b]), 0.0,
                                                              lse[b])[..., None]))
        for h in range(Hq):
            vv = v[blk, t % bs, h // G].astype(np.float64) * \
                vs[blk, t % bs, h // G].astype(np.float64)[:, None]
            out[b, :, h] = w[:, h] @ vv
        # A score: 4 products and sums, the product with two rounded scales: 10 roundings of
        # its terms' magnitudes. An exponential: 2 steps of fp32 (2^-22) and the rounding of
        # its argument. The sum: a lane adds at most L / 8 + 64 terms and rescaled partial sums.
        # The logarithm's product and sum: 4 roundings of the result and of the maximum.
        m = np.where(np.isneginf(x), 0.0, mag).max(-1)
        bound[b] = 10 * EPS * m + 2.0 ** -21 + (L / 8 + 64) * EPS + \
            4 * EPS * (np.where(np.isneginf(lse[b]), 0.0, np.abs(lse[b])) + m)
    return out, lse, bound


def attn_mass(mass, q, lse, k, ks, table, lens, scale, decay):
    """The updated mass (float64, [B][Hk][cap]) and a bound on the error of an fp32 update."""
    B, nq, Hq, D = q.shape
    P, bs, Hk, _ = k.shape
    G = Hq // Hk
    cap = table.shape[1] * bs
    new = np.asarray(mass, np.float64).copy()
    bound = np.zeros_like(new)
    for b in range(B):
        L = int(min(max(lens[b], 0), cap))
        if L == 0:
            continue
        x, mag, ok = scores(q[b], k, ks, table[b], L, scale)
        ls = np.asarray(lse[b], np.float64)[..., None]
        with np.errstate(invalid="ignore"):
            p = np.where(np.isneginf(x), 0.0, np.exp(x - ls))
        # score: 10 roundings of its terms; the argument score - lse in base 2: 3 of lse and
        # one of the difference; the exponential 2^-22; the sum over nq G rows and the update
        ls = np.where(np.isneginf(ls), 0.0, ls)  # (rows that see nothing weigh nothing)
        rel = 10 * EPS * mag + 4 * EPS * np.abs(ls) + 2.0 ** -21 + (nq * G + 4) * EPS
        for h in range(Hk):
            w = p[:, h * G:(h + 1) * G].sum((0, 1))
            e = (p * rel)[:, h * G:(h + 1) * G].sum((0, 1))
            old = new[b, h, :L] * decay if decay else np.zeros(L)
            new[b, h, :L] = np.where(ok, old + w, new[b, h, :L])
            bound[b, h, :L] = e + 2 * EPS * (np.abs(old) + w)
    return new, bound


# ------------------------------------------------------------------ eviction

def evict(k, v, ks, vs, mass, table, lens, new_table, keep, sink, recent):
    """(k, v, ks, vs after the move, new_mass, kept, new_lens)."""
    P, bs, Hk, D = k.shape
    B, cap = table.shape[0], table.shape[1] * bs
    src = [a.copy() for a in (k, v, ks, vs)]
    dst = [a.copy() for a in (k, v, ks, vs)]
    new_mass = np.zeros((B, Hk, new_table.shape[1] * bs), F32)
    kept = np.full((B, Hk, keep), -1, np.int32)
    new_lens = np.zeros(B, np.int32)
    for b in range(B):
        L = int(min(max(lens[b], 0), cap))
        new_lens[b] = min(L, keep)
        for h in range(Hk):
            if L <= keep:
                took = list(range(L))
            else:
                held = list(range(sink)) + list(range(L - recent, L))
                value = lambda t: -np.inf if np.isnan(mass[b, h, t]) else float(mass[b, h, t])
                middle = sorted(range(sink, L - recent), key=lambda t: (-value(t), t))
                took = sorted(held + middle[:keep - sink - recent])
            for j, t in enumerate(took):
                kept[b, h, j] = t
                new_mass[b, h, j] = mass[b, h, t]
                a, z = table[b, t // bs], new_table[b, j // bs]
                if 0 <= a < P and 0 <= z < P:
                    for s, d in zip(src, dst):
                        d[z, j % bs, h] = s[a, t % bs, h]
    return (*dst, new_mass, kept, new_lens)


# ------------------------------------------------------------------ draft verification

def verify(target, draft, drafted, uniforms, n_drafts=None):
    """n_accepted [B], tokens [B][n + 1], by running sums in float64."""
    B, n1, V = target.shape
    accepted = np.zeros(B, np.int32)
    tokens = np.full((B, n1), -1, np.int32)
    for b in range(B):
        n = n1 - 1 if n_drafts is None else int(min(max(n_drafts[b], 0), n1 - 1))
        a = 0
        while a < n:
            x = int(drafted[b, a])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[b, a, x])
            if not float(uniforms[b, a]) * q < float(target[b, a, x]):
                break
            a += 1
        w = target[b, a].astype(np.float64)
        plain = w
        if a < n:
            if draft is None:
                w = w.copy()
                if 0 <= drafted[b, a] < V:
                    w[drafted[b, a]] = 0.0
            else:
                w = w - draft[b, a].astype(np.float64)
        w = np.where(w > 0, w, 0.0)
        if a < n and not w.sum() > 0:
            w = np.where(plain > 0, plain, 0.0)
        accepted[b] = a
        tokens[b, :a] = drafted[b, :a]
        run = np.cumsum(w)
        if run[-1] > 0 and np.isfinite(run[-1]):
            over = np.nonzero(run > float(uniforms[b, -1]) * run[-1])[0]
            tokens[b, a] = over[0] if len(over) else np.nonzero(w)[0][-1]
    return accepted, tokens
