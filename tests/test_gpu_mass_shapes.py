"""q8kv_attn_mass in the launch shapes of larger calls: blocks of three and four heads (with idle
ones in the last), and blocks that go through many sequences."""
import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8
import serving_ref as ref

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("Hk", [3, 4, 5, 8])
@pytest.mark.parametrize("nq,group", [(1, 4), (1, 1), (2, 3), (1, 8)])
@pytest.mark.parametrize("decay", [0.75, 0.0])
def test_mass_with_a_wide_table(nq, group, Hk, decay):
    """Short ragged sequences under a table that could hold 16384 tokens of 4 sequences (as many
    tiles as take four heads to a block); 1100 sequences in all."""
    mass_case(1100, nq, group * Hk, Hk, bs=16, width=14, longest=50, decay=decay, seed=Hk)


@pytest.mark.parametrize("Hk,nq,group", [(4, 1, 4), (8, 1, 8), (5, 2, 3)])
def test_mass_of_blocks_that_go_through_many_sequences(Hk, nq, group):
    """Every warp's ring is drained and filled again dozens of times, each time after a few tiles:
    lengths of one tile up to a ring and a half."""
    mass_case(6000, nq, group * Hk, Hk, bs=16, width=7, longest=100, decay=1.0, seed=3)


def mass_case(B, nq, Hq, Hk, bs, width, longest, decay, seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, B).astype(np.int32)
    need = -(-lens // bs)
    P = 600  # blocks, shared by many sequences
    table = np.full((B, width), -1, np.int32)
    for b in range(B):
        table[b, :need[b]] = rng.integers(0, P, need[b])
    k = rng.integers(-127, 128, (P, bs, Hk, D)).astype(np.int8)
    ks = (rng.random((P, bs, Hk)) * 0.02).astype(np.float32)
    q = rng.standard_normal((B, nq, Hq, D)).astype(np.float32)
    lse = (2 + 3 * rng.random((B, nq, Hq))).astype(np.float32)
    mass = rng.random((B, Hk, width * bs)).astype(np.float32)
    t = lambda a: torch.from_numpy(a.copy()).cuda()
    d, args = t(mass), [t(a) for a in (q, lse, k, ks, table, lens)]
    q8.q8kv_device_errors(clear=True)
    q8.q8kv_attn_mass(d, *args, 0.088, decay=decay)
    got = d.cpu().numpy()
    assert q8.q8kv_device_errors(clear=True) == 0
    past = np.arange(width * bs) >= lens[:, None, None]
    assert np.array_equal(np.where(past, got, 0), np.where(past, mass, 0))
    some = rng.permutation(B)[:120]  # the reference's share: the same inputs, fewer sequences
    want, bound = ref.attn_mass(mass[some], q[some], lse[some], k, ks, table[some], lens[some],
                                0.088, decay)
    assert (np.abs(got[some] - want) <= bound).all()
    # and every sequence by itself gives the same bits (24 of them)
    for b in some[:24]:
        one = t(mass[b:b + 1])
        q8.q8kv_attn_mass(one, *(a[b:b + 1] for a in args[:2]), args[2], args[3],
                          *(a[b:b + 1] for a in args[4:]), 0.088, decay=decay)
        assert np.array_equal(one.cpu().numpy()[0], got[b])
