"""Launch shapes that only larger calls take: clusters of four blocks in the verification, tiles
of two to four tokens in the rotary write, shared between blocks or with a partial last one."""
import numpy as np
import pytest

import serving_ref as ref
from test_gpu_rope import run as run_rope
from test_gpu_verify import call as call_verify
from test_gpu_verify import draw, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,V", [("fp32", 4099), ("bf16", 5000), ("fp16", 8192)])
@pytest.mark.parametrize("B", [90, 128, 148])
def test_verify_with_clusters_of_four(B, dtype, V):
    target, draft, drafted, uni = draw(B, 3, V, dtype, seed=B)
    a, t, err = call_verify(target, draft, drafted, uni)
    ra, rt = ref.verify(host(target), host(draft), drafted.cpu().numpy(), uni.cpu().numpy())
    assert np.array_equal(a, ra) and np.array_equal(t, rt) and err == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [500, 501, 900, 1337, 1799, 4999])
@pytest.mark.parametrize("rot,adjacent", [(64, False), (32, False), (24, False), (64, True)])
def test_rope_tiles(n, dtype, rot, adjacent):
    assert run_rope(n, 3, 2, 64, rot, 3, dtype, adjacent, seed=n, bs=64, fused=True) == 0


@pytest.mark.parametrize("D,rot,n", [(128, 128, 1801), (128, 96, 1337), (256, 128, 950),
                                     (256, 40, 4999)])
def test_rope_tiles_of_larger_heads(D, rot, n):
    assert run_rope(n, 4, 1, D, rot, 2, "fp16", False, seed=n, bs=32) == 0


@pytest.mark.parametrize("n,dtype", [(501, "fp32"), (900, "fp32"), (1337, "fp32"), (900, "bf16"),
                                     (1337, "bf16"), (1799, "bf16")])
@pytest.mark.parametrize("rot,in_place", [(128, False), (32, False), (128, True), (96, True)])
def test_rope_tiles_shared_by_blocks(n, dtype, rot, in_place):
    """As many heads as give two blocks a part of each tile."""
    assert run_rope(n, 32, 8, 128, rot, 2, dtype, False, seed=n, bs=64,
                    in_place=in_place and dtype == "fp32") == 0


@pytest.mark.parametrize("n", [501, 1799, 4999])
@pytest.mark.parametrize("rot,adjacent", [(64, False), (32, False), (24, False), (64, True)])
def test_rope_tiles_in_place(n, rot, adjacent):
    assert run_rope(n, 3, 2, 64, rot, 2, "fp32", adjacent, seed=n, bs=64, in_place=True) == 0
