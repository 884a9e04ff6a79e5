"""A captured graph of calls on the library-managed workspace stays valid when a later call needs a
larger one: the graph holds the address of the workspace it was captured with. In a process of its
own, where the workspace starts small."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import numpy as np, torch
import decode_attention_int8_b200 as q8
from decode_attention_int8_b200 import inputs

def case(Hq, Hk, lens, seed):
    w = inputs.make_custom(len(lens), Hq, Hk, 128, lens, 16, seed=seed)
    d = [torch.from_numpy(np.ascontiguousarray(a)).cuda()
         for a in (w.q, w.k, w.v, w.ks, w.vs, w.block_table, w.seq_lens)]
    q = d[0][:, None].contiguous()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    call = lambda: q8.q8kv_decode_attn_lse(out, lse, q, *d[1:], w.scale)
    return call, out, lse

small, out, lse = case(4, 4, [9000, 700], 1)  # split over many blocks
small()
torch.cuda.synchronize()
want = out.clone(), lse.clone()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    small()
sizes = []
for Hq, Hk in ((32, 8), (128, 8), (64, 8)):  # larger workspaces, then a smaller one
    sizes.append(q8.q8kv_workspace_bytes(2, Hq, Hk, 128))
    call, o, l = case(Hq, Hk, [9000, 700], 2)
    call()
    torch.cuda.synchronize()
    again = o.clone()
    out.fill_(9.0), lse.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    call()
    torch.cuda.synchronize()
    assert torch.equal(o, again)
assert q8.q8kv_workspace_bytes(2, 4, 4, 128) < sizes[0] < sizes[1] > sizes[2]
assert q8.q8kv_device_errors(clear=True) == 0
print("replayed")
"""


def test_replay_after_the_workspace_grew():
    got = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert got.returncode == 0 and "replayed" in got.stdout, got.stderr[-2000:]
