"""Host side of the serving operators: bad arguments are refused before any CUDA call (fake,
never dereferenced pointers), and the numpy references agree with independent statements."""
import ctypes

import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8
import serving_ref as ref

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = lambda x: None if x is None else ctypes.c_void_p(x)


def ptrs(n):
    return [0x100000 * (i + 1) for i in range(n)]


# ---- q8kv_decode_attn_lse

LSE_SIZES = dict(B=2, nq=2, Hq=8, Hk=2, D=128, bs=16, mbps=4, P=8, scale=0.1)


def call_lse(a=None, **over):
    a = a or ptrs(9)
    s = dict(LSE_SIZES, **over)
    return q8.lib().q8kv_decode_attn_lse(*map(P, a), s["B"], s["nq"], s["Hq"], s["Hk"], s["D"],
                                         s["bs"], s["mbps"], s["P"], s["scale"], None, 0, None)


@pytest.mark.parametrize("i", range(9))
def test_lse_null_pointers(i):
    a = ptrs(9)
    a[i] = None
    assert call_lse(a) == INVALID


@pytest.mark.parametrize("over", [dict(B=0), dict(nq=0), dict(nq=-1), dict(Hq=9), dict(Hk=0),
                                  dict(D=100), dict(bs=0), dict(mbps=0), dict(P=0),
                                  dict(scale=float("nan"))])
def test_lse_bad_sizes(over):
    assert call_lse(**over) == INVALID


def test_lse_alignment():
    a = ptrs(9)
    a[1] += 2
    assert call_lse(a) == INVALID


# ---- q8kv_attn_mass

MASS_SIZES = dict(B=2, nq=2, Hq=8, Hk=2, D=128, bs=16, mbps=4, P=8, scale=0.1, decay=1.0)


def call_mass(a=None, **over):
    a = a or ptrs(7)
    s = dict(MASS_SIZES, **over)
    return q8.lib().q8kv_attn_mass(*map(P, a), s["B"], s["nq"], s["Hq"], s["Hk"], s["D"], s["bs"],
                                   s["mbps"], s["P"], s["scale"], s["decay"], None)


@pytest.mark.parametrize("i", range(7))
def test_mass_null_pointers(i):
    a = ptrs(7)
    a[i] = None
    assert call_mass(a) == INVALID


@pytest.mark.parametrize("over", [dict(B=0), dict(nq=0), dict(Hq=9), dict(Hk=-1), dict(D=100),
                                  dict(bs=0), dict(mbps=0), dict(P=0), dict(scale=float("inf")),
                                  dict(decay=-0.1), dict(decay=1.5), dict(decay=float("nan"))])
def test_mass_bad_sizes(over):
    assert call_mass(**over) == INVALID


@pytest.mark.parametrize("over", [dict(D=64), dict(bs=8), dict(bs=24), dict(bs=512),
                                  dict(nq=33), dict(B=16385), dict(P=1 << 27), dict(mbps=1 << 26)])
def test_mass_unsupported(over):
    assert call_mass(**over) == UNSUPPORTED


@pytest.mark.parametrize("i,off", [(0, 2), (1, 4), (2, 2), (3, 8), (4, 2), (5, 2), (6, 1)])
def test_mass_alignment(i, off):
    a = ptrs(7)
    a[i] += off
    assert call_mass(a) == INVALID


# ---- q8kv_evict

EVICT_SIZES = dict(B=2, Hk=2, D=128, bs=16, mbps=4, nmbps=2, P=8, keep=32, sink=4, recent=8)


def call_evict(a=None, **over):
    a = a or ptrs(11)
    s = dict(EVICT_SIZES, **over)
    return q8.lib().q8kv_evict(*map(P, a), s["B"], s["Hk"], s["D"], s["bs"], s["mbps"], s["nmbps"],
                               s["P"], s["keep"], s["sink"], s["recent"], None)


@pytest.mark.parametrize("i", range(11))
def test_evict_null_pointers(i):
    a = ptrs(11)
    a[i] = None
    assert call_evict(a) == INVALID


@pytest.mark.parametrize("over", [dict(B=0), dict(Hk=0), dict(D=100), dict(bs=0), dict(mbps=0),
                                  dict(nmbps=0), dict(P=0), dict(keep=0), dict(sink=-1),
                                  dict(recent=-1), dict(sink=20, recent=13), dict(keep=33)])
def test_evict_bad_sizes(over):
    assert call_evict(**over) == INVALID


@pytest.mark.parametrize("over", [dict(D=96), dict(D=32), dict(B=16385), dict(P=1 << 27),
                                  dict(mbps=1 << 26), dict(nmbps=1 << 26),
                                  dict(nmbps=1 << 25, keep=1 << 29, Hk=8)])
def test_evict_unsupported(over):
    assert call_evict(**over) == UNSUPPORTED


def test_evict_aliases_and_alignment():
    a = ptrs(11)
    assert call_evict(a[:6] + [a[9]] + a[7:]) == INVALID  # new_lens is seq_lens
    assert call_evict(a[:4] + [a[7]] + a[5:]) == INVALID  # new_mass is mass
    for i, off in [(0, 8), (1, 4), (2, 2), (4, 1), (5, 2), (7, 2)]:
        b = list(a)
        b[i] += off
        assert call_evict(b) == INVALID


# ---- q8kv_rope_cache_write

ROPE_SIZES = dict(n=4, axes=3, Hq=4, Hk=2, D=128, rot=128, adj=0, top=100, dt=0, bs=16, P=8, qs=0,
                  kvs=0)


def call_rope(a=None, axis=None, **over):
    a = a or ptrs(11)
    s = dict(ROPE_SIZES, **over)
    return q8.lib().q8kv_rope_cache_write(*map(P, a), axis, s["n"], s["axes"], s["Hq"], s["Hk"],
                                          s["D"], s["rot"], s["adj"], s["top"], s["dt"], s["bs"],
                                          s["P"], s["qs"], s["kvs"], None)


@pytest.mark.parametrize("i", range(11))
def test_rope_null_pointers(i):
    a = ptrs(11)
    a[i] = None
    assert call_rope(a) == INVALID


@pytest.mark.parametrize("over", [dict(n=-1), dict(axes=0), dict(Hq=0), dict(Hk=0), dict(D=100),
                                  dict(rot=0), dict(rot=136), dict(rot=12), dict(top=0),
                                  dict(dt=3), dict(dt=-1), dict(bs=0), dict(P=0), dict(qs=511),
                                  dict(qs=514), dict(kvs=252), dict(kvs=258), dict(dt=1, qs=516),
                                  dict(axis=bytes([3] * 64)), dict(axis=bytes([0] * 63 + [7]))])
def test_rope_bad_sizes(over):
    assert call_rope(**over) == INVALID


@pytest.mark.parametrize("over", [dict(D=96, rot=96), dict(D=512), dict(axes=5), dict(Hq=4097)])
def test_rope_unsupported(over):
    assert call_rope(**over) == UNSUPPORTED


def test_rope_no_tokens_in_place_and_alignment():
    a = ptrs(11)
    assert call_rope([None] + a[1:5] + [None] * 6, n=0) == OK
    b = [a[5]] + a[1:]  # q_out is q_new: only fp32 rows without gaps
    assert call_rope(b, dt=1) == INVALID
    assert call_rope(b, qs=1024) == INVALID
    for i, off in [(0, 4), (1, 8), (3, 2), (5, 4), (6, 8), (7, 4), (8, 4), (9, 2), (10, 8)]:
        c = list(a)
        c[i] += off
        assert call_rope(c) == INVALID, i


# ---- q8kv_verify_draft

VERIFY_SIZES = dict(B=2, n=3, V=100, ts=0, ds=0, dt=0)


def call_verify(a=None, **over):
    a = a or ptrs(7)
    s = dict(VERIFY_SIZES, **over)
    return q8.lib().q8kv_verify_draft(*map(P, a), s["B"], s["n"], s["V"], s["ts"], s["ds"],
                                      s["dt"], None)


@pytest.mark.parametrize("i", [0, 1, 2, 4, 6])  # (draft_probs and n_drafts may be null)
def test_verify_null_pointers(i):
    a = ptrs(7)
    a[i] = None
    assert call_verify(a) == INVALID


@pytest.mark.parametrize("over", [dict(B=-1), dict(n=-1), dict(V=0), dict(ts=99), dict(ds=99),
                                  dict(dt=3)])
def test_verify_bad_sizes(over):
    assert call_verify(**over) == INVALID


@pytest.mark.parametrize("over", [dict(n=1025), dict(B=(1 << 24) + 1), dict(V=(1 << 30) + 1)])
def test_verify_unsupported(over):
    assert call_verify(**over) == UNSUPPORTED


def test_verify_empty_batch_and_alignment():
    assert call_verify([None] * 7, B=0) == OK
    for i, off in [(0, 2), (1, 2), (2, 2), (3, 1), (4, 2), (5, 2), (6, 2)]:
        a = ptrs(7)
        a[i] += off
        assert call_verify(a) == INVALID


# ---- the binding refuses tensors that disagree (CPU tensors never reach the library)

def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    with pytest.raises(ValueError):
        q8.q8kv_attn_mass(z(1, 2, 64), z(1, 1, 4, 128), z(1, 1, 4),
                          z(4, 16, 2, 128, dtype=torch.int8), z(4, 16, 2),
                          z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError):
        q8.q8kv_verify_draft(z(1, dtype=torch.int32), z(1, 2, dtype=torch.int32), z(1, 2, 10),
                             z(1, 1, 10), z(1, 1, dtype=torch.int32), z(1, 2))


# ---- the references

def test_reference_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    angle = rng.standard_normal((50, 16))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    x = rng.standard_normal((7, 3, 64))
    pos = rng.integers(0, 50, (2, 7))
    axis = [i % 2 for i in range(16)]
    for adjacent in (False, True):
        y = ref.rotate(x, pos, table, axis, adjacent, np.float64)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))  # lengths stay
        assert np.array_equal(y[..., 32:], x[..., 32:])         # past rotary_dim
        # complex form: (a + ib) e^(i angle)
        a, b = (x[..., 0:32:2], x[..., 1:32:2]) if adjacent else (x[..., :16], x[..., 16:32])
        z = (a + 1j * b) * np.exp(1j * angle[pos[axis], :][np.arange(16), :, np.arange(16)].T[:, None])
        u, w = (y[..., 0:32:2], y[..., 1:32:2]) if adjacent else (y[..., :16], y[..., 16:32])
        assert np.allclose(u, z.real) and np.allclose(w, z.imag)


def test_reference_mass_adds_up_to_the_rows():
    rng = np.random.default_rng(2)
    q = rng.standard_normal((2, 3, 4, 128)).astype(np.float32)
    k = rng.integers(-127, 128, (6, 16, 2, 128)).astype(np.int8)
    ks = rng.random((6, 16, 2)).astype(np.float32) * 0.02
    v, vs = k, ks
    table = np.array([[0, 1, 2], [3, 4, 5]], np.int32)
    lens = np.array([40, 2])
    out, lse, _ = ref.decode_lse(q, k, v, ks, vs, table, lens, 0.1)
    mass, _ = ref.attn_mass(np.zeros((2, 2, 48)), q, lse, k, ks, table, lens, 0.1, 1.0)
    assert np.allclose(mass[0].sum(-1), 6)  # 3 queries x 2 heads of the group
    assert np.allclose(mass[1].sum(-1), 4)  # of two tokens, query 0 sees none
    assert np.isneginf(lse[1, 0]).all() and np.isfinite(lse[1, 1:]).all()


def test_reference_verification_keeps_the_target_distribution():
    """Speculative sampling's own property: whatever the draft, the first token follows the
    target's distribution (exactly, over a grid of uniforms for a two-token vocabulary)."""
    p, q = np.array([0.3, 0.7]), np.array([0.6, 0.4])
    m = 400
    grid = (np.arange(m) + 0.5) / m
    count = np.zeros(2)
    for x in range(2):
        for u in grid:
            for s in grid[::10]:
                a, t = ref.verify(np.stack([p, p])[None], q[None, None], np.array([[x]]),
                                  np.array([[u, s]]))
                count[t[0, 0]] += q[x]
    assert np.allclose(count / count.sum(), p, atol=2e-3)
