"""The serving operators at the ends of their ranges: pools and tables whose offsets pass 32
bits, large batches, the largest row counts, and refusals that need a device."""
import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8
import serving_ref as ref

pytestmark = pytest.mark.gpu

BS, HK, D = 64, 8, 128
BIG = 66000  # blocks: 4.3e9 bytes of K codes, past 2^32


def big_pool():
    k = torch.zeros((BIG, BS, HK, D), dtype=torch.int8, device="cuda")
    return k, torch.zeros((BIG, BS, HK), device="cuda")


def rows(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randint(-127, 128, (n, BS, HK, D), generator=g, device="cuda").to(torch.int8),
            torch.rand((n, BS, HK), generator=g, device="cuda") * 0.02)


def test_offsets_past_32_bits():
    """The same blocks at the far end of a 4.3 GB pool and in a small one: attention mass,
    decode statistics, eviction and rotary write give the same bits."""
    n = 6
    far = torch.tensor([BIG - 1, BIG - 7, 3, BIG - 3, BIG // 2 + 1, BIG - 2], device="cuda")
    k, ks = rows(n, 1)
    v, vs = rows(n, 2)
    bk, bks = big_pool()
    bv, bvs = big_pool()
    for big, small in ((bk, k), (bks, ks), (bv, v), (bvs, vs)):
        big[far] = small
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((1, 2, 16, D), generator=g, device="cuda")
    lens = torch.tensor([4 * BS - 5], dtype=torch.int32, device="cuda")
    near = torch.arange(n, dtype=torch.int32, device="cuda")
    got = []
    for pools, ids in (((k, v, ks, vs), near), ((bk, bv, bks, bvs), far.int())):
        table, new_table = ids[None, :4].contiguous(), ids[None, 4:].contiguous()
        out, lse = torch.empty_like(q), torch.empty((1, 2, 16), device="cuda")
        q8.q8kv_decode_attn_lse(out, lse, q, *pools, table, lens, 0.088)
        mass = torch.zeros((1, HK, 4 * BS), device="cuda")
        q8.q8kv_attn_mass(mass, q, lse, pools[0], pools[2], table, lens, 0.088)
        nm = torch.empty((1, HK, 2 * BS), device="cuda")
        kept = torch.empty((1, HK, 100), dtype=torch.int32, device="cuda")
        nl = torch.empty((1,), dtype=torch.int32, device="cuda")
        q8.q8kv_evict(*pools, nm, kept, nl, mass, table, lens, new_table, sink=3, recent=20)
        # the last slots of the last of these blocks: new rows
        slots = (ids[5].long() * BS + torch.arange(BS - 9, BS, device="cuda"))
        x = torch.randn((9, HK, D), generator=torch.Generator(device="cuda").manual_seed(4),
                        device="cuda")
        qo = torch.empty_like(x)
        angles = torch.ones((10, D), device="cuda") * 0.7
        q8.q8kv_rope_cache_write(qo, *pools, x, x, x, slots,
                                 torch.arange(9, dtype=torch.int32, device="cuda")[None], angles)
        got.append([out, lse, mass, nm, kept, nl, qo] + [p[ids.long()] for p in pools])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert q8.q8kv_device_errors(clear=True) == 0


def test_probability_rows_past_32_bits():
    """2200 rows of a million weights: row offsets beyond 2^31 elements."""
    B, V = 1100, 1 << 20
    target = torch.zeros((B, 2, V), device="cuda")
    b = torch.arange(B, device="cuda")
    at = (b * 977 + 13) % V
    target[b, 0, at] = 0.5
    target[b, 0, V - 1 - at] = 0.5
    target[b, 1, at] = 1.0
    acc = torch.empty((B,), dtype=torch.int32, device="cuda")
    tok = torch.empty((B, 2), dtype=torch.int32, device="cuda")
    uni = torch.full((B, 2), 0.25, device="cuda")
    uni[::2, 0] = 0.75  # refused: the other token of the row remains
    q8.q8kv_verify_draft(acc, tok, target, None, at.int()[:, None], uni)
    odd = (b % 2 == 1)
    assert torch.equal(acc, odd.int())
    assert torch.equal(tok[:, 0], torch.where(odd, at, V - 1 - at).int())
    assert torch.equal(tok[:, 1], torch.where(odd, at, torch.full_like(at, -1)).int())


@pytest.mark.parametrize("B,nq,Hq,Hk", [(3000, 1, 4, 1), (2, 8, 32, 2), (1, 1, 128, 1)])
def test_mass_many_sequences_and_rows(B, nq, Hq, Hk):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 40, B).astype(np.int32)
    need = -(-lens // 16)
    P = int(need.sum()) + 1
    table = np.full((B, 3), -1, np.int32)
    perm, at = rng.permutation(P), 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    k = rng.integers(-127, 128, (P, 16, Hk, D)).astype(np.int8)
    ks = (rng.random((P, 16, Hk)) * 0.02).astype(np.float32)
    q = rng.standard_normal((B, nq, Hq, D)).astype(np.float32)
    _, lse, _ = ref.decode_lse(q, k, k, ks, ks, table, lens, 0.088)
    lse = lse.astype(np.float32)
    mass = rng.random((B, Hk, 48)).astype(np.float32)
    t = lambda a: torch.from_numpy(a.copy()).cuda()
    d = t(mass)
    q8.q8kv_attn_mass(d, t(q), t(lse), t(k), t(ks), t(table), t(lens), 0.088, decay=0.5)
    want, bound = ref.attn_mass(mass, q, lse, k, ks, table, lens, 0.088, 0.5)
    assert (np.abs(d.cpu().numpy() - want) <= bound).all()
    assert q8.q8kv_device_errors(clear=True) == 0


@pytest.mark.parametrize("B,nq,Hq,Hk", [(2, 1, 500, 500), (3, 3, 520, 130), (5, 2, 26, 13)])
def test_mass_many_heads(B, nq, Hq, Hk):
    """More heads than blocks run at once, and numbers of heads that no block size divides."""
    test_mass_many_sequences_and_rows(B, nq, Hq, Hk)


def test_binding_refusals_on_a_device():
    """Shapes, types, devices and strides that disagree never reach the library."""
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
    k, ks = z(4, 16, 2, 128, dt=torch.int8), z(4, 16, 2)
    q, lse, lens = z(1, 1, 4, 128), z(1, 1, 4), z(1, dt=torch.int32)
    table, mass = z(1, 4, dt=torch.int32), z(1, 2, 64)
    ok = dict(mass=mass, q=q, lse=lse, k_blocks=k, kscale=ks, block_table=table, seq_lens=lens)
    for name, bad in [("mass", z(1, 2, 63)), ("mass", mass.double()), ("lse", z(1, 4)),
                      ("kscale", ks.cpu()), ("seq_lens", lens.long()), ("q", q.transpose(2, 3)),
                      ("block_table", z(2, 4, dt=torch.int32)), ("k_blocks", k[:, :, :, :64])]:
        with pytest.raises((ValueError, IndexError)):
            q8.q8kv_attn_mass(**dict(ok, **{name: bad}), scale=0.1)
    with pytest.raises(TypeError):
        q8.q8kv_attn_mass(**dict(ok, mass=3), scale=0.1)
    with pytest.raises(q8.Q8KVError) as e:
        q8.q8kv_attn_mass(**ok, scale=0.1, decay=2.0)
    assert e.value.status == 1
    # rotary write: rows with gaps, token strides that differ, a pair table of another length
    x = z(5, 2, 128)
    rope = dict(q_out=z(5, 2, 128), k_blocks=k, v_blocks=k.clone(), kscale=ks, vscale=ks.clone(),
                q_new=x, k_new=x, v_new=x, slot_mapping=z(5, dt=torch.int64),
                positions=z(1, 5, dt=torch.int32), cos_sin=z(8, 128))
    for change in [dict(q_new=z(5, 4, 128)[:, ::2]), dict(v_new=z(5, 4, 128)[:, :2]),
                   dict(q_new=x.double()), dict(k_new=x.half()), dict(pair_axis=[0] * 63),
                   dict(positions=z(5, dt=torch.int32)), dict(slot_mapping=z(5, dt=torch.int32)),
                   dict(cos_sin=z(8, 128).cpu())]:
        with pytest.raises(ValueError):
            q8.q8kv_rope_cache_write(**dict(rope, **change))
    with pytest.raises(q8.Q8KVError):
        q8.q8kv_rope_cache_write(**dict(rope, pair_axis=[1] * 64))
    # verification: strides that are no rows, types that differ
    ver = dict(n_accepted=z(2, dt=torch.int32), tokens=z(2, 3, dt=torch.int32),
               target_probs=z(2, 3, 10), draft_probs=z(2, 2, 10),
               draft_tokens=z(2, 2, dt=torch.int32), uniforms=z(2, 3))
    for change in [dict(target_probs=z(2, 3, 20)[..., ::2]), dict(draft_probs=z(2, 2, 10).half()),
                   dict(tokens=z(2, 2, dt=torch.int32)), dict(target_probs=z(2, 4, 10)[:, :3]),
                   dict(uniforms=z(2, 2)), dict(n_drafts=z(3, dt=torch.int32))]:
        with pytest.raises(ValueError):
            q8.q8kv_verify_draft(**dict(ver, **change))
    # eviction: lengths in place
    ev = dict(k_blocks=k, v_blocks=k.clone(), kscale=ks, vscale=ks.clone(),
              new_mass=z(1, 2, 16), kept=z(1, 2, 16, dt=torch.int32), new_lens=lens.clone(),
              mass=mass, block_table=table, seq_lens=lens, new_block_table=z(1, 1, dt=torch.int32))
    with pytest.raises(q8.Q8KVError):
        q8.q8kv_evict(**dict(ev, new_lens=lens))
    with pytest.raises(q8.Q8KVError):
        q8.q8kv_evict(**ev, sink=9, recent=8)
    with pytest.raises(q8.Q8KVError):
        q8.q8kv_evict(**dict(ev, kept=z(1, 2, 17, dt=torch.int32)))
    torch.cuda.synchronize()
    assert q8.q8kv_device_errors(clear=True) == 0


def test_expanded_rows_are_refused():
    """A stride of zero (one row expanded over tokens or drafts) is not the library's zero, which
    says that rows have no gap."""
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
    k, ks = z(4, 16, 2, 128, dt=torch.int8), z(4, 16, 2)
    x, one = z(5, 2, 128), z(1, 2, 128).expand(5, 2, 128)
    rope = dict(q_out=z(5, 2, 128), k_blocks=k, v_blocks=k.clone(), kscale=ks, vscale=ks.clone(),
                q_new=x, k_new=x, v_new=x, slot_mapping=z(5, dt=torch.int64) - 1,
                positions=z(1, 5, dt=torch.int32), cos_sin=z(8, 128))
    for change in [dict(q_new=one), dict(k_new=one, v_new=one)]:
        with pytest.raises(ValueError):
            q8.q8kv_rope_cache_write(**dict(rope, **change))
    ver = dict(n_accepted=z(2, dt=torch.int32), tokens=z(2, 3, dt=torch.int32),
               target_probs=z(2, 3, 10), draft_probs=z(2, 2, 10),
               draft_tokens=z(2, 2, dt=torch.int32), uniforms=z(2, 3))
    for change in [dict(target_probs=z(1, 1, 10).expand(2, 3, 10)),
                   dict(draft_probs=z(1, 1, 10).expand(2, 2, 10)),
                   dict(target_probs=z(1, 3, 10).expand(2, 3, 10))]:
        with pytest.raises(ValueError):
            q8.q8kv_verify_draft(**dict(ver, **change))
    ver = dict(ver, tokens=z(2, 1, dt=torch.int32), draft_probs=None, uniforms=z(2, 1),
               draft_tokens=z(2, 0, dt=torch.int32))
    with pytest.raises(ValueError):
        q8.q8kv_verify_draft(**dict(ver, target_probs=z(1, 1, 10).expand(2, 1, 10)))
    q8.q8kv_rope_cache_write(**rope)  # (the call that these differ from)
    torch.cuda.synchronize()
    assert q8.q8kv_device_errors(clear=True) == 0


def test_options_of_the_wrong_kind_are_refused():
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
    k, ks, x = z(4, 16, 2, 128, dt=torch.int8), z(4, 16, 2), z(5, 2, 128)
    rope = dict(q_out=z(5, 2, 128), k_blocks=k, v_blocks=k.clone(), kscale=ks, vscale=ks.clone(),
                q_new=x, k_new=x, v_new=x, slot_mapping=z(5, dt=torch.int64) - 1,
                positions=z(1, 5, dt=torch.int32), cos_sin=z(8, 128))
    for change in [dict(pair_axis=64), dict(adjacent=torch.zeros(2)), dict(stream="first")]:
        with pytest.raises(TypeError):
            q8.q8kv_rope_cache_write(**dict(rope, **change))
