"""q8kv_rope_cache_write against the numpy reference: queries, codes and scales bit for bit (the
operator fixes every fp32 operation), and the queries against the rotation in 64 bits."""
import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8
import serving_ref as ref

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def angles(top, rot, rng):
    a = rng.uniform(-np.pi, np.pi, (top, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def run(n, Hq, Hk, D, rot, axes, dtype, adjacent, seed, bs=16, top=50, fused=False, axis="mixed",
        bad_pos=False, values=None, in_place=False):
    rng = np.random.default_rng(seed)
    rows = rng.standard_normal((n, Hq + 2 * Hk, D)).astype(np.float32)
    if values is not None:
        rows = values(rows, rng)
    t = torch.from_numpy(rows).cuda().to(DT[dtype])
    if fused:  # slices of one projection: a token stride above the rows
        q, k, v = t[:, :Hq], t[:, Hq:Hq + Hk], t[:, Hq + Hk:]
    else:
        q, k, v = (x.contiguous() for x in (t[:, :Hq], t[:, Hq:Hq + Hk], t[:, Hq + Hk:]))
    pos = rng.integers(0, top, (axes, n)).astype(np.int32)
    if bad_pos:
        pos[0, 0], pos[-1, -1] = -5, top + 7
    table = angles(top, rot, rng)
    pair_axis = None if axis is None else rng.integers(0, axes, rot // 2).tolist()
    if axis == "runs":
        pair_axis = sorted(pair_axis)
    P = -(-n // bs) + 2
    slots = rng.permutation(P * bs)[:n].astype(np.int64)
    if n > 3:
        slots[1] = -1
        slots[3] = -9
    pools = [np.full((P, bs, Hk, D), 77, np.int8), np.full((P, bs, Hk, D), -77, np.int8),
             np.full((P, bs, Hk), 5.5, np.float32), np.full((P, bs, Hk), 6.5, np.float32)]
    d = [torch.from_numpy(a.copy()).cuda() for a in pools]
    qin = q.float().cpu().numpy()
    out = q if in_place else torch.full((n, Hq, D), float("nan"), device="cuda")
    q8.q8kv_device_errors(clear=True)
    q8.q8kv_rope_cache_write(out, *d, q, k, v, torch.from_numpy(slots).cuda(),
                             torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(),
                             pair_axis=pair_axis, adjacent=adjacent)
    err = q8.q8kv_device_errors(clear=True)
    # references: the operator's fp32 steps, and the mathematics
    live = slots >= 0
    with np.errstate(invalid="ignore", over="ignore"):
        q32 = ref.rotate(qin, pos, table, pair_axis, adjacent, np.float32)
        kr = ref.rotate(k.float().cpu().numpy(), pos, table, pair_axis, adjacent, np.float32)
    for i, x in enumerate((kr, v.float().cpu().numpy())):
        codes, scale = ref.quantise_rows(x)
        pools[i].reshape(-1, Hk, D)[slots[live]] = codes[live]
        pools[2 + i].reshape(-1, Hk)[slots[live]] = scale[live]
    got = out.cpu().numpy()
    assert np.array_equal(got, q32, equal_nan=True)
    for a, b in zip(d, pools):
        a = a.cpu().numpy()
        assert np.array_equal(a, b, equal_nan=a.dtype == np.float32)
    if values is None:
        q64 = ref.rotate(qin, pos, table.astype(np.float64), pair_axis, adjacent, np.float64)
        # two products and a sum, each off by half a step: 2 EPS of the products' magnitudes
        mag = np.abs(qin).max(-1, keepdims=True) * 2.0
        assert (np.abs(got - q64) <= 2.001 * ref.EPS * mag).all()
    return err


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (64, 8), (128, 128), (128, 64), (128, 96),
                                   (256, 256), (256, 128), (256, 40)])
@pytest.mark.parametrize("adjacent", [False, True])
def test_shapes_and_types(dtype, D, rot, adjacent):
    assert run(37, 6, 3, D, rot, 3, dtype, adjacent, seed=D + rot) == 0


@pytest.mark.parametrize("n", [1, 2, 5, 64, 333])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (32, 8), (7, 7), (40, 5)])
def test_token_and_head_counts(n, Hq, Hk):
    assert run(n, Hq, Hk, 128, 128, 1, "bf16", False, seed=n, fused=True, axis=None) == 0


@pytest.mark.parametrize("axes,axis", [(1, "mixed"), (2, "runs"), (3, "runs"), (3, "mixed"),
                                       (4, "mixed")])
def test_axes(axes, axis):
    assert run(50, 8, 2, 128, 128, axes, "fp32", False, seed=axes, axis=axis) == 0


def test_many_tokens_take_a_warp_each():
    assert run(5000, 4, 2, 64, 64, 2, "fp32", False, seed=9, bs=64) == 0


def test_bad_positions_are_clamped_and_flagged():
    assert run(20, 4, 2, 128, 64, 2, "fp32", False, seed=3, bad_pos=True) == q8.DEVERR_POSITION


@pytest.mark.parametrize("rot,adjacent", [(128, False), (64, False), (96, False), (128, True)])
def test_in_place(rot, adjacent):
    assert run(40, 8, 2, 128, rot, 2, "fp32", adjacent, seed=4, in_place=True) == 0


def test_special_values():
    """Zero rows, rows below the quantiser's guard, infinities and NaN, the largest values."""
    def values(x, rng):
        x[0] = 0.0
        x[1] *= 1e-8
        x[2, :, 5] = np.inf
        x[4, :, 9] = np.nan
        x[5] *= 1e37
        return x
    assert run(12, 4, 2, 128, 128, 1, "fp32", False, seed=5, values=values) == \
        q8.DEVERR_NONFINITE


def test_slot_past_the_pool_is_skipped():
    t = lambda *s: torch.zeros(*s, device="cuda")
    pool = [torch.zeros((2, 16, 1, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
    sc = [t(2, 16, 1) for _ in range(2)]
    q8.q8kv_device_errors(clear=True)
    ones = torch.ones((2, 1, 64), device="cuda")
    q8.q8kv_rope_cache_write(t(2, 1, 64), *pool, *sc, ones, ones, ones,
                             torch.tensor([32, 31], device="cuda"),
                             torch.zeros((1, 2), dtype=torch.int32, device="cuda"),
                             torch.ones((1, 64), device="cuda"))
    assert q8.q8kv_device_errors(clear=True) == q8.DEVERR_SLOT
    assert sc[1].count_nonzero() == 1 and sc[1][1, 15, 0] > 0


def test_matches_the_cache_write_at_position_zero():
    """With angle zero nothing turns: the same pools as q8kv_cache_write of the same rows."""
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((100, 8, 128), generator=g, device="cuda") for _ in range(2))
    slots = torch.randperm(160, generator=g, device="cuda")[:100]
    table = torch.cat([torch.ones(4, 64), torch.zeros(4, 64)], 1).cuda()
    a, b = ([torch.zeros((10, 16, 8, 128), dtype=torch.int8, device="cuda") for _ in range(2)] +
            [torch.zeros((10, 16, 8), device="cuda") for _ in range(2)] for _ in range(2))
    q = torch.randn((100, 8, 128), generator=g, device="cuda")
    out = torch.empty_like(q)
    q8.q8kv_rope_cache_write(out, *a, q, k, v, slots,
                             torch.zeros((1, 100), dtype=torch.int32, device="cuda"), table)
    q8.q8kv_cache_write(*b, k, v, slots)
    assert torch.equal(out, q)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
