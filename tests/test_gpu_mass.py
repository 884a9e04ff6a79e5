"""q8kv_decode_attn_lse and q8kv_attn_mass against the softmax in 64 bits on the same
quantised data. Tolerances count roundings (serving_ref.decode_lse, attn_mass)."""
import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8
import serving_ref as ref
from decode_attention_int8_b200 import inputs
from gpu_util import assert_close

pytestmark = pytest.mark.gpu


def make(B, Hq, Hk, lens, bs, nq, seed, **kw):
    w = inputs.make_custom(B, Hq, Hk, 128, lens, bs, seed=seed, **kw)
    q = inputs.multi_queries(B, nq, Hq, 128, seed=seed)
    return w, np.ascontiguousarray(q, np.float32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_lse(w, q, workspace=None):
    d = [dev(a) for a in (w.k, w.v, w.ks, w.vs, w.block_table, w.seq_lens)]
    qd = dev(q)
    out = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    q8.q8kv_device_errors(clear=True)
    q8.q8kv_decode_attn_lse(out, lse, qd, *d, w.scale, workspace=workspace)
    err = q8.q8kv_device_errors(clear=True)
    return out, lse, err, d, qd


SHAPES = [  # B, Hq, Hk, lens, bs, nq
    (1, 8, 8, [256], 16, 1),
    (3, 8, 2, [1, 300, 1000], 64, 1),
    (2, 32, 4, [700, 33], 128, 1),
    (4, 16, 4, [0, 17, 500, 1], 32, 1),
    (2, 32, 1, [130, 999], 16, 1),
    (3, 8, 2, [1, 2, 400], 16, 3),
    (2, 32, 8, [600, 5], 64, 2),
    (2, 32, 8, [900, 3], 64, 4),
    (2, 64, 8, [513, 260], 128, 4),
    (1, 28, 4, [300], 256, 3),
    (2, 40, 4, [64, 129], 16, 4),
    (2, 12, 3, [100, 77], 16, 1),
    (1, 5, 5, [90], 16, 2),
    (2, 18, 9, [40, 200], 16, 1),
    (40, 4, 1, list(range(0, 200, 5)), 16, 1),
]
# head counts that the decode's tiling does not take (q8kv_attn_mass has no such rule)
NO_DECODE = {(12, 3), (5, 5), (18, 9)}


def decodes(Hq, Hk, nq):
    return (Hq, Hk) not in NO_DECODE


@pytest.mark.parametrize("B,Hq,Hk,lens,bs,nq", [s for s in SHAPES if decodes(s[1], s[2], s[5])])
def test_lse(B, Hq, Hk, lens, bs, nq):
    w, q = make(B, Hq, Hk, lens, bs, nq, seed=B + Hq)
    out, lse, err, d, qd = run_lse(w, q)
    ro, rl, bound = ref.decode_lse(q, w.k, w.v, w.ks, w.vs, w.block_table, w.seq_lens, w.scale)
    got = lse.cpu().numpy().astype(np.float64)
    assert err == 0
    assert np.array_equal(np.isneginf(got), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert (np.abs(got[fin] - rl[fin]) <= bound[fin]).all()
    assert_close(out.cpu().numpy(), ro)
    # the output is the decode's: bit for bit, but for the finer weights of the tcgen05 path
    again = torch.empty_like(out)
    q8.q8kv_decode_attn_multi(again, qd, *d, w.scale)
    tcgen05 = nq > 1 and 9 <= nq * Hq // Hk <= 32 and (Hk == 1 or Hk % 4 == 0)
    assert torch.equal(out, again) or tcgen05
    if tcgen05:  # 2^-22 of the largest weight per token instead of 2^-19
        mine, other = (np.linalg.norm(x.cpu().numpy() - ro) for x in (out, again))
        assert mine <= other


def test_lse_split_over_many_blocks():
    """A long sequence split over every SM (merged statistics), and one empty neighbour."""
    w, q = make(2, 8, 4, [20000, 0], 64, 1, seed=5, k_dist="student_t3")
    out, lse, err, d, qd = run_lse(w, q)
    ro, rl, bound = ref.decode_lse(q, w.k, w.v, w.ks, w.vs, w.block_table, w.seq_lens, w.scale)
    got = lse.cpu().numpy()
    assert np.isneginf(got[1]).all() and (np.abs(got[0] - rl[0]) <= bound[0]).all()
    assert err == 0


def test_lse_of_no_tokens_at_all():
    w, q = make(2, 8, 4, [16, 16], 16, 2, seed=5)
    w.seq_lens[:] = 0
    out, lse, err, d, qd = run_lse(w, q)
    assert (out == 0).all() and torch.isneginf(lse).all() and err == 0


def test_lse_with_the_callers_workspace():
    w, q = make(2, 32, 8, [3000, 1000], 64, 2, seed=6)
    out, lse, _, d, qd = run_lse(w, q)
    n = q8.q8kv_workspace_bytes(2, 2 * 32, 8, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o2, l2, _, _, _ = run_lse(w, q, workspace=ws)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    with pytest.raises(q8.Q8KVError) as e:
        run_lse(w, q, workspace=ws[:256])
    assert e.value.status == 4


def mass_case(B, Hq, Hk, lens, bs, nq, decay, seed, change=None, want_err=0, **kw):
    w, q = make(B, Hq, Hk, lens, bs, nq, seed=seed, **kw)
    cap = w.block_table.shape[1] * bs
    rng = np.random.default_rng(seed)
    mass = (rng.random((B, Hk, cap)) * 0.1).astype(np.float32)
    if change:
        change(w, q, mass)
    # statistics in 64 bits, rounded: what the decode leaves, up to its own rounding
    _, lse, _ = ref.decode_lse(q, w.k, w.v, w.ks, w.vs, w.block_table, w.seq_lens, w.scale)
    lse = lse.astype(np.float32)
    d = dev(mass)
    q8.q8kv_device_errors(clear=True)
    q8.q8kv_attn_mass(d, dev(q), dev(lse), dev(w.k), dev(w.ks), dev(w.block_table),
                      dev(w.seq_lens), w.scale, decay=decay)
    err = q8.q8kv_device_errors(clear=True)
    want, bound = ref.attn_mass(mass, q, lse, w.k, w.ks, w.block_table, w.seq_lens, w.scale, decay)
    got = d.cpu().numpy().astype(np.float64)
    off = np.abs(got - want) - bound
    assert not np.isnan(got).any() or np.isnan(mass).any()
    assert (off[~np.isnan(want)] <= 0).all(), off[~np.isnan(want)].max()
    for b in range(B):  # entries past the sequence stay as they were, bit for bit
        L = max(0, min(int(w.seq_lens[b]), cap))
        assert np.array_equal(d.cpu().numpy()[b, :, L:], mass[b, :, L:], equal_nan=True)
    assert err == want_err
    return w, got, mass


@pytest.mark.parametrize("B,Hq,Hk,lens,bs,nq", SHAPES)
@pytest.mark.parametrize("decay", [1.0, 0.9])
def test_mass(B, Hq, Hk, lens, bs, nq, decay):
    mass_case(B, Hq, Hk, lens, bs, nq, decay, seed=B + Hq)


@pytest.mark.parametrize("Hq,Hk,nq", [(64, 2, 1), (16, 1, 8), (48, 4, 5), (128, 1, 1), (6, 2, 7)])
def test_mass_many_query_rows(Hq, Hk, nq):
    mass_case(2, Hq, Hk, [150, 33], 16, nq, 1.0, seed=Hq + nq)


@pytest.mark.parametrize("Hk", [1, 2, 3, 5, 7, 8, 9, 16, 17, 33])
def test_mass_head_counts(Hk):
    mass_case(2, 2 * Hk, Hk, [70, 130], 32, 1, 1.0, seed=Hk)


def test_mass_long_and_ragged():
    mass_case(6, 8, 2, [5000, 1, 16, 17, 2047, 640], 64, 1, 1.0, seed=4, k_dist="student_t3")


def test_mass_wide_scores():
    """Scores in the hundreds: nearly all the weight on a few tokens."""
    def wide(w, q, mass):
        q *= 20.0
    mass_case(2, 8, 2, [400, 90], 16, 2, 0.5, seed=5, change=wide)


def test_mass_without_decay_does_not_read_the_buffer():
    def poison(w, q, mass):
        mass[:] = np.nan
    w, got, _ = mass_case(2, 8, 2, [100, 40], 16, 1, 0.0, seed=6, change=poison)
    for b, L in enumerate([100, 40]):
        assert np.isfinite(got[b, :, :L]).all()
        assert np.allclose(got[b, :, :L].sum(-1), 4, rtol=1e-5)


def test_mass_bad_table_entries_keep_their_tokens():
    def holes(w, q, mass):
        w.block_table[0, 1] = -1
        w.block_table[1, 3] = 1 << 30
    mass_case(2, 8, 4, [100, 128], 16, 1, 0.5, seed=7, change=holes,
              want_err=q8.DEVERR_BLOCK_TABLE)


def test_mass_stored_lengths_out_of_range():
    def lengths(w, q, mass):
        w.seq_lens[0], w.seq_lens[1] = -3, 9999
    mass_case(2, 8, 4, [64, 128], 16, 1, 1.0, seed=8, change=lengths,
              want_err=q8.DEVERR_SEQ_LEN, max_blocks_per_seq=8)


def test_mass_large_batch():
    rng = np.random.default_rng(9)
    mass_case(300, 4, 2, rng.integers(0, 60, 300).tolist(), 16, 1, 1.0, seed=9)
