"""q8kv_evict against the numpy reference: kept positions, moved rows, masses and lengths are
copies or whole numbers and have to be equal; rows that are nobody's stay as they were."""
import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8
import serving_ref as ref

pytestmark = pytest.mark.gpu


def make(B, Hk, D, bs, lens, keep, seed, spare=3, width=None):
    rng = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lens]
    mbps = max(1, max(need)) if width is None else width
    nmbps = -(-keep // bs)
    P = sum(need) + B * nmbps + spare
    perm = rng.permutation(P).astype(np.int32)
    table = np.full((B, mbps), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    new_table = perm[at:at + B * nmbps].reshape(B, nmbps).copy()
    k, v = (rng.integers(-127, 128, (P, bs, Hk, D)).astype(np.int8) for _ in range(2))
    ks, vs = (rng.random((P, bs, Hk)).astype(np.float32) for _ in range(2))
    mass = np.exp(2 * rng.standard_normal((B, Hk, mbps * bs)) - 4).astype(np.float32)
    return [k, v, ks, vs], mass, table, np.array(lens, np.int32), new_table


def call(pools, mass, table, lens, new_table, keep, sink, recent):
    Hk, bs, B = pools[0].shape[2], pools[0].shape[1], len(lens)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a).copy()).cuda()
    d = [t(a) for a in pools]
    nm = torch.full((B, Hk, new_table.shape[1] * bs), float("nan"), device="cuda")
    kept = torch.full((B, Hk, keep), -5, dtype=torch.int32, device="cuda")
    nl = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    q8.q8kv_device_errors(clear=True)
    q8.q8kv_evict(*d, nm, kept, nl, t(mass), t(table), t(lens), t(new_table), sink=sink,
                  recent=recent)
    err = q8.q8kv_device_errors(clear=True)
    return [x.cpu().numpy() for x in (*d, nm, kept, nl)], err


def check(B, Hk, D, bs, lens, keep, sink, recent, seed, change=None, want_err=0, **kw):
    pools, mass, table, ln, new_table = make(B, Hk, D, bs, lens, keep, seed, **kw)
    if change:
        change(mass, table, ln, new_table)
    got, err = call(pools, mass, table, ln, new_table, keep, sink, recent)
    want = ref.evict(*pools, mass, table, ln, new_table, keep, sink, recent)
    for name, g, w in zip(("k", "v", "ks", "vs", "new_mass", "kept", "new_lens"), got, want):
        if name == "kept":
            assert np.array_equal(g, w), (name, np.argwhere(g != w)[:3])
        else:
            assert np.array_equal(g, w, equal_nan=g.dtype == np.float32), name
    assert err == want_err
    return got


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [16, 64, 24])
def test_head_dims_and_blocks(D, bs):
    check(3, 2, D, bs, [200, 37, 90], 50, 3, 11, seed=D + bs)


@pytest.mark.parametrize("Hk", [1, 3, 8])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (40, 0, 0),
                                              (40, 40, 0), (40, 0, 40), (40, 13, 27), (99, 1, 1)])
def test_budgets(Hk, keep, sink, recent):
    check(2, Hk, 64, 16, [100, 101], keep, sink, recent, seed=keep + Hk)


@pytest.mark.parametrize("lens", [[0, 5, 1], [49, 50, 51], [1000, 2049, 1025], [4100, 31, 0]])
def test_lengths(lens):
    check(3, 2, 64, 16, lens, 50, 2, 9, seed=sum(lens))


@pytest.mark.parametrize("L,B,Hk,bs", [(70000, 1, 2, 128), (20000, 20, 1, 256), (3000, 90, 4, 64),
                                       (500000, 1, 1, 1024)])
def test_long_and_many(L, B, Hk, bs):
    """Masses over several blocks' shared memory, in one block, and past what eight hold."""
    rng = np.random.default_rng(L)
    lens = [L] + rng.integers(1, L + 1, B - 1).tolist()
    # (small rows: what grows here is the number of positions)
    check(B, Hk, 64, bs, lens, 700, 10, 100, seed=L, spare=1)


def test_equal_masses_go_to_the_lowest_positions():
    def same(mass, *_):
        mass[0] = 0.5
        mass[1, 0] = 0.0
        mass[1, 1] = np.where(np.arange(mass.shape[2]) % 3 == 0, 2.0, 1.0)
    got = check(2, 2, 64, 16, [3000, 2900], 1000, 5, 50, seed=1, change=same)
    assert got[5][0, 0, :950].tolist() == list(range(950))


def test_special_masses():
    """Infinities, NaN (lowest), negative values, both zeros (equal), subnormals."""
    def special(mass, *_):
        v = np.array([np.inf, -np.inf, np.nan, -1.0, -0.0, 0.0, 1e-45, -1e-45, 3e38], np.float32)
        rng = np.random.default_rng(3)
        mass[0] = v[rng.integers(0, len(v), mass.shape[1:])]
        mass[1] = np.nan
        mass[2] = -np.abs(mass[2])
    check(3, 2, 64, 16, [400, 300, 350], 120, 4, 16, seed=2, change=special)


@pytest.mark.parametrize("keep", [90, 200])
def test_stored_lengths_out_of_range(keep):
    def lengths(mass, table, lens, new_table):
        lens[0], lens[1] = -4, 100000
    check(3, 2, 64, 16, [96, 128, 64], keep, 2, 8, seed=6, change=lengths,
          want_err=q8.DEVERR_SEQ_LEN, width=8)


def test_bad_table_entries_skip_their_rows():
    def tables(mass, table, lens, new_table):
        table[0, 2] = 9999
        table[1, 0] = -7
        new_table[0, 1] = -1
        new_table[1, 0] = 1 << 30
    check(2, 2, 64, 16, [128, 100], 50, 2, 8, seed=7, change=tables,
          want_err=q8.DEVERR_BLOCK_TABLE)


def test_a_sequence_within_budget_may_keep_its_blocks():
    pools, mass, table, lens, new_table = make(2, 2, 64, 16, [60, 300], 64, seed=8)
    new_table[0, :4] = table[0, :4]
    got, err = call(pools, mass, table, lens, new_table, 64, 2, 8)
    want = ref.evict(*pools, mass, table, lens, new_table, 64, 2, 8)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert err == 0


@pytest.mark.parametrize("bs,L", [(7, 1000), (5, 20001), (1, 77), (33, 4099)])
def test_rows_of_masses_that_start_anywhere(bs, L):
    """Block sizes that leave the rows of mass unaligned: no 16-byte loads."""
    check(2, 3, 64, bs, [L, L - 1], L // 3, 2, L // 9, seed=bs)


@pytest.mark.parametrize("B,Hk,L", [(1, 1, 40000), (1, 2, 66000), (2, 4, 33000)])
def test_clusters(B, Hk, L):
    """Two, four and eight blocks per row, with ties on the threshold across blocks."""
    def coarse(mass, *_):
        mass[:] = np.round(mass * 50) / 50
    check(B, Hk, 64, 64, [L] * B, 5000, 100, 900, seed=L, change=coarse)


@pytest.mark.parametrize("B,L", [(14, 70000), (18, 70000), (40, 34000), (80, 17000)])
def test_as_many_clusters_as_run_at_once(B, L):
    """Around the numbers of rows from which a row gets fewer blocks."""
    rng = np.random.default_rng(B)
    lens = [L] + (L - rng.integers(0, L // 4, B - 1)).tolist()
    check(B, 1, 64, 64, lens, 300, 10, 100, seed=B, spare=1)


def test_twice_is_the_same():
    """Old blocks are read only: the same call again gives the same answer."""
    pools, mass, table, lens, new_table = make(2, 4, 128, 32, [700, 900], 300, seed=9)
    a, _ = call(pools, mass, table, lens, new_table, 300, 4, 64)
    b, _ = call(a[:4], mass, table, lens, new_table, 300, 4, 64)
    for x, y in zip(a, b):
        assert np.array_equal(x, y)
