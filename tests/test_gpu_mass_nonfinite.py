"""A query row or a statistic that is not finite reaches the masses: q8kv_attn_mass gives NaN to
every token that the row sees, and changes nothing else."""
import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8
from decode_attention_int8_b200 import inputs

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# (changed buffer, value): one channel of a query row, or the row's log-sum-exp
CHANGES = [("q", NAN), ("q", INF), ("q", -INF), ("lse", NAN), ("lse", INF)]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("nq,Hq,Hk", [(1, 8, 2), (2, 6, 3), (2, 12, 3), (3, 24, 2)])
@pytest.mark.parametrize("what,value", CHANGES)
def test_a_row_that_is_not_finite(nq, Hq, Hk, what, value):
    lens = [200, 77]
    w = inputs.make_custom(2, Hq, Hk, 128, lens, 16, seed=nq + Hq)
    q = dev(np.asarray(inputs.multi_queries(2, nq, Hq, 128, seed=Hq), np.float32))
    k, ks, table, seq = (dev(a) for a in (w.k, w.ks, w.block_table, w.seq_lens))
    g = torch.Generator(device="cuda").manual_seed(5)
    lse = 2.0 + torch.rand((2, nq, Hq), generator=g, device="cuda")
    start = torch.rand((2, Hk, w.block_table.shape[1] * 16), generator=g, device="cuda")
    clean = start.clone()
    q8.q8kv_attn_mass(clean, q, lse, k, ks, table, seq, w.scale, decay=0.5)
    for i in range(nq):
        for h, channel in ((0, 0), (Hq // 2, 77), (Hq - 1, 127)):
            bad_q, bad_lse, got = q.clone(), lse.clone(), start.clone()
            if what == "q":
                bad_q[0, i, h, channel] = value
            else:
                bad_lse[0, i, h] = value
            q8.q8kv_attn_mass(got, bad_q, bad_lse, k, ks, table, seq, w.scale, decay=0.5)
            kv, sees = h // (Hq // Hk), lens[0] - (nq - 1 - i)
            assert torch.isnan(got[0, kv, :sees]).all()
            want = clean.clone()
            want[0, kv, :sees] = NAN
            assert torch.equal(got.nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))
    assert q8.q8kv_device_errors(clear=True) == 0


@pytest.mark.parametrize("nq,Hq,Hk", [(1, 8, 2), (2, 6, 3), (2, 12, 3), (3, 24, 2)])
def test_a_scale_of_nan(nq, Hq, Hk):
    """A token whose key row was not finite: NaN for it, and for no other token."""
    lens = [200, 77]
    w = inputs.make_custom(2, Hq, Hk, 128, lens, 16, seed=nq + Hq)
    q = dev(np.asarray(inputs.multi_queries(2, nq, Hq, 128, seed=Hq), np.float32))
    k, ks, table, seq = (dev(a) for a in (w.k, w.ks, w.block_table, w.seq_lens))
    g = torch.Generator(device="cuda").manual_seed(5)
    lse = 2.0 + torch.rand((2, nq, Hq), generator=g, device="cuda")
    start = torch.rand((2, Hk, w.block_table.shape[1] * 16), generator=g, device="cuda")
    clean, got = start.clone(), start.clone()
    q8.q8kv_attn_mass(clean, q, lse, k, ks, table, seq, w.scale)
    for t in (0, 100, 198, 199):
        ks[int(w.block_table[0, t // 16]), t % 16, Hk - 1] = NAN
        clean[0, Hk - 1, t] = NAN
    q8.q8kv_attn_mass(got, q, lse, k, ks, table, seq, w.scale)
    assert torch.equal(got.nan_to_num(nan=-1.0), clean.nan_to_num(nan=-1.0))


@pytest.mark.parametrize("nq,Hq,Hk", [(1, 8, 2), (1, 32, 2), (2, 16, 4), (4, 32, 4)])
def test_the_decode_of_such_rows(nq, Hq, Hk):
    """The statistics call: a NaN channel counts as zero (it has no part in its block's maximum and
    its code is 0), an infinite one gives a NaN log-sum-exp; other rows keep their bits."""
    w = inputs.make_custom(2, Hq, Hk, 128, [300, 40], 16, seed=Hq)
    q = dev(np.asarray(inputs.multi_queries(2, nq, Hq, 128, seed=Hq), np.float32))
    args = [dev(a) for a in (w.k, w.v, w.ks, w.vs, w.block_table, w.seq_lens)]

    def run(x):
        out, lse = torch.empty_like(x), torch.empty(x.shape[:3], device="cuda")
        q8.q8kv_decode_attn_lse(out, lse, x, *args, w.scale)
        return out, lse

    zero, nan, inf = q.clone(), q.clone(), q.clone()
    zero[0, nq - 1, 1, 5], nan[0, nq - 1, 1, 5], inf[0, nq - 1, 1, 5] = 0.0, NAN, INF
    (zo, zl), (no, nl), (io, il) = run(zero), run(nan), run(inf)
    assert torch.equal(zo, no) and torch.equal(zl, nl)
    assert torch.isnan(il[0, nq - 1, 1])
    io[0, nq - 1, 1], il[0, nq - 1, 1] = zo[0, nq - 1, 1], zl[0, nq - 1, 1]
    assert torch.equal(io, zo) and torch.equal(il, zl)
