"""The serving operators together, as a speculative server with a bounded cache calls them: the
drafted tokens' rows go in with their positions, the decode scores them, the target's rows
decide which stay, their attention weights are added up, and when the cache is full the
lightest tokens leave it. Also: captured graphs, other streams, two streams at once."""
import math

import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8
import serving_ref as ref
from gpu_util import assert_close

pytestmark = pytest.mark.gpu

B, HQ, HK, D, BS, DRAFTS = 3, 8, 2, 128, 16, 3
SCALE = 1 / math.sqrt(D)


def angles(top):
    inv = 10000.0 ** (-np.arange(0, D, 2) / D)
    a = np.arange(top)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Server:
    """Pools, tables and running masses of a small server, and the same state in numpy."""

    def __init__(self, lens, blocks=120, width=12):
        self.rng = np.random.default_rng(7)
        z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
        self.pools = [z(blocks, BS, HK, D, dt=torch.int8), z(blocks, BS, HK, D, dt=torch.int8),
                      z(blocks, BS, HK), z(blocks, BS, HK)]
        self.free = self.rng.permutation(blocks).tolist()
        self.table = np.array([[self.free.pop() for _ in range(width)] for _ in range(B)], np.int32)
        self.lens = np.zeros(B, np.int32)
        self.next_pos = np.zeros(B, np.int64)  # positions go on counting after an eviction
        self.mass = z(B, HK, width * BS)
        self.angles = angles(1000)
        self.angles_dev = torch.from_numpy(self.angles).cuda()
        for b, n in enumerate(lens):
            self.append([b] * n)

    def append(self, owners):
        """Write one new token for each entry of owners; returns their rotated queries."""
        n = len(owners)
        qkv = torch.from_numpy(self.rng.standard_normal((n, HQ + 2 * HK, D)).astype(np.float32))
        qkv = qkv.cuda()
        slots, pos = [], []
        for b in owners:
            t = int(self.lens[b])
            slots.append(int(self.table[b, t // BS]) * BS + t % BS)
            pos.append(int(self.next_pos[b]))
            self.lens[b] += 1
            self.next_pos[b] += 1
        out = torch.empty((n, HQ, D), device="cuda")
        q8.q8kv_rope_cache_write(out, *self.pools, qkv[:, :HQ], qkv[:, HQ:HQ + HK],
                                 qkv[:, HQ + HK:], torch.tensor(slots, device="cuda"),
                                 torch.tensor([pos], dtype=torch.int32, device="cuda"),
                                 self.angles_dev)
        return out

    def dev(self, a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def test_a_speculative_server_with_a_bounded_cache():
    s = Server([90, 30, 120])
    keep, sink, recent = 64, 2, 16
    vocab = 500
    q8.q8kv_device_errors(clear=True)
    for step in range(3):
        # the drafted tokens (and the last accepted one) of every sequence
        q = torch.stack([s.append([b] * (DRAFTS + 1)) for b in range(B)])
        table, lens = s.dev(s.table), s.dev(s.lens)
        out = torch.empty((B, DRAFTS + 1, HQ, D), device="cuda")
        lse = torch.empty((B, DRAFTS + 1, HQ), device="cuda")
        q8.q8kv_decode_attn_lse(out, lse, q, *s.pools, table, lens, SCALE)
        k, v, ks, vs = (x.cpu().numpy() for x in s.pools)
        ro, rl, bound = ref.decode_lse(q.cpu().numpy(), k, v, ks, vs, s.table, s.lens, SCALE)
        assert_close(out.cpu().numpy(), ro)
        assert (np.abs(lse.cpu().numpy() - rl) <= bound).all()

        before = s.mass.cpu().numpy()
        q8.q8kv_attn_mass(s.mass, q, lse, s.pools[0], s.pools[2], table, lens, SCALE, decay=0.95)
        want, mb = ref.attn_mass(before, q.cpu().numpy(), lse.cpu().numpy(), k, ks, s.table,
                                 s.lens, SCALE, 0.95)
        assert (np.abs(s.mass.cpu().numpy() - want) <= mb).all()

        # which of the drafts stay
        g = torch.Generator(device="cuda").manual_seed(step)
        target = (2 * torch.randn((B, DRAFTS + 1, vocab), generator=g, device="cuda")).softmax(-1)
        draft = (target[:, :DRAFTS].log() +
                 0.5 * torch.randn((B, DRAFTS, vocab), generator=g, device="cuda")).softmax(-1)
        drafted = draft.argmax(-1).int()
        uni = torch.rand((B, DRAFTS + 1), generator=g, device="cuda")
        acc = torch.empty(B, dtype=torch.int32, device="cuda")
        tok = torch.empty((B, DRAFTS + 1), dtype=torch.int32, device="cuda")
        q8.q8kv_verify_draft(acc, tok, target, draft, drafted, uni)
        ra, rt = ref.verify(target.cpu().numpy(), draft.cpu().numpy(), drafted.cpu().numpy(),
                            uni.cpu().numpy())
        assert np.array_equal(acc.cpu().numpy(), ra) and np.array_equal(tok.cpu().numpy(), rt)
        refused = DRAFTS - ra
        for b in range(B):  # refused tokens leave the cache; their masses start again
            s.mass[b, :, s.lens[b] - refused[b]:s.lens[b]] = 0
        s.lens -= refused.astype(np.int32)
        s.next_pos -= refused

        # a full cache loses its lightest tokens
        width = s.table.shape[1]
        new_table = np.array([[s.free.pop() for _ in range(width)] for _ in range(B)], np.int32)
        pools = [x.cpu().numpy() for x in s.pools]
        mass, new_mass = s.mass, torch.empty_like(s.mass)
        kept = torch.empty((B, HK, keep), dtype=torch.int32, device="cuda")
        nl = torch.empty(B, dtype=torch.int32, device="cuda")
        q8.q8kv_evict(*s.pools, new_mass, kept, nl, mass, s.dev(s.table), s.dev(s.lens),
                      s.dev(new_table), sink=sink, recent=recent)
        wantp = ref.evict(*pools, mass.cpu().numpy(), s.table, s.lens, new_table, keep, sink, recent)
        for a, w in zip((*s.pools, new_mass, kept, nl), wantp):
            assert np.array_equal(a.cpu().numpy(), w)
        assert int(nl.max()) == keep
        s.free += s.table.flatten().tolist()
        s.table, s.lens, s.mass = new_table, nl.cpu().numpy().copy(), new_mass
    assert q8.q8kv_device_errors(clear=True) == 0


def step_calls(s, stream=None, workspace=None):
    """One call of each operator on fixed inputs; returns the call and its outputs."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *sh: torch.randn(sh, generator=g, device="cuda")
    n = B
    qkv = r(n, HQ + 2 * HK, D)
    slots = torch.tensor([int(s.table[b, s.lens[b] // BS]) * BS + int(s.lens[b]) % BS
                          for b in range(B)], device="cuda")
    pos = torch.tensor([s.next_pos.tolist()], dtype=torch.int32, device="cuda")
    lens = s.dev(s.lens + 1)
    table = s.dev(s.table)
    q = torch.empty((n, HQ, D), device="cuda")
    out, lse = torch.empty((B, 1, HQ, D), device="cuda"), torch.empty((B, 1, HQ), device="cuda")
    mass = torch.zeros_like(s.mass)
    keep = 40
    new_table = s.dev(np.array([[s.free[3 * b + i] for i in range(3)] for b in range(B)], np.int32))
    new_mass = torch.empty((B, HK, 3 * BS), device="cuda")
    kept = torch.empty((B, HK, keep), dtype=torch.int32, device="cuda")
    nl = torch.empty(B, dtype=torch.int32, device="cuda")
    target, draft = r(B, 3, 700).softmax(-1), r(B, 2, 700).softmax(-1)
    drafted, uni = draft.argmax(-1).int(), torch.rand((B, 3), generator=g, device="cuda")
    acc = torch.empty(B, dtype=torch.int32, device="cuda")
    tok = torch.empty((B, 3), dtype=torch.int32, device="cuda")

    def call():
        q8.q8kv_rope_cache_write(q, *s.pools, qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:],
                                 slots, pos, s.angles_dev, stream=stream)
        q8.q8kv_decode_attn_lse(out, lse, q[:, None], *s.pools, table, lens, SCALE,
                                workspace=workspace, stream=stream)
        q8.q8kv_attn_mass(mass, q[:, None], lse, s.pools[0], s.pools[2], table, lens, SCALE,
                          decay=0.0, stream=stream)
        q8.q8kv_evict(*s.pools, new_mass, kept, nl, mass, table, lens, new_table, sink=2,
                      recent=8, stream=stream)
        q8.q8kv_verify_draft(acc, tok, target, draft, drafted, uni, stream=stream)

    return call, [q, out, lse, mass, new_mass, kept, nl, acc, tok] + s.pools


def test_captured_and_replayed():
    s = Server([70, 20, 100])
    ws = torch.empty(q8.q8kv_workspace_bytes(B, HQ, HK, D), dtype=torch.uint8, device="cuda")
    call, outs = step_calls(s, workspace=ws)
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    for x in outs[:9]:
        x.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for x in outs[:9]:
            x.fill_(7)
        outs[3].zero_()  # (masses past the sequences are not written by any call)
        graph.replay()
    torch.cuda.synchronize()
    for a, w in zip(outs, want):
        assert torch.equal(a, w)


def test_on_another_stream():
    s = Server([70, 20, 100])
    call, outs = step_calls(s)
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    for x in outs[:9]:
        x.zero_()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    call2, outs2 = step_calls(s, stream=other)
    torch.cuda.synchronize()
    call2()
    other.synchronize()
    for a, w in zip(outs2, want):
        assert torch.equal(a, w)


def test_two_streams_at_once():
    """Two servers on two streams, each with its own workspace, give what each gives alone."""
    nbytes = q8.q8kv_workspace_bytes(B, HQ, HK, D)
    streams = [torch.cuda.Stream() for _ in range(2)]
    servers = [Server([70, 20, 100]), Server([33, 150, 5])]
    calls = []
    for st, s in zip(streams, servers):
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        calls.append(step_calls(s, stream=st, workspace=ws))
    torch.cuda.synchronize()
    want = []
    for (call, outs) in calls:
        call()
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
        for x in outs[:9]:
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for call, _ in calls:
            call()
    torch.cuda.synchronize()
    for (_, outs), w in zip(calls, want):
        for a, x in zip(outs, w):
            assert torch.equal(a, x)
