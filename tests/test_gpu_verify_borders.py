"""q8kv_verify_draft on long rows whose every weight is rounded the same way: the sums keep fp64's
precision whatever the vocabulary, so a border stays where it is."""
import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8

pytestmark = pytest.mark.gpu


def test_one_sided_roundings_do_not_move_a_border():
    """Both halves of a row of 2^24 weights weigh nearly the same, and the draw is at half their
    total: the token at the border says which half is heavier.

    In the first half p = 1 and q = c 2^-25, so each weight 1 - q is rounded to 1 in fp32 and -q is
    left over, always of one sign. The second half's weights are exact, and its last one makes the
    halves differ by 2 m, m = 3e-6 in 1.7e7 (1.8e-13): above or below the border by that much. An
    fp32 sum of the leftovers of a lane (8192 weights of the row) is off by 1e-12 of the half.
    The largest error of the kernel's sums, 2^-43.3 for the roundings of the pairs and 2^-53 for
    each of the 2^11 sums of a lane's pairs, whose partial sums are short enough to be exact here,
    is 9.2e-14 of the total: half of the distance to the border."""
    half = 1 << 23
    V, m = 2 * half, 3e-6
    target = torch.ones((2, 2, V), device="cuda")
    draft = torch.zeros((2, 1, V), device="cuda")
    drafted = torch.full((2, 1), half + 12345, dtype=torch.int32, device="cuda")
    want = []
    for b, (c, sign) in enumerate([(0.9491, 1), (0.786925, -1)]):
        q = np.float32(c) * np.float32(2.0 ** -25)
        draft[b, 0, :half] = float(q)
        target[b, 0, half + 12345] = 0.0  # the drafted token: refused, and without weight
        last = np.float32(2.0 - half * float(q) - 2 * sign * m)
        target[b, 0, V - 1] = float(last)
        first, second = half - half * float(q), (half - 2) + float(last)  # (exact in fp64)
        margin = (first - second) / 2
        assert sign * margin > 0.8 * m
        want.append(half - 1 if margin > 0 else half)
    acc = torch.empty((2,), dtype=torch.int32, device="cuda")
    tok = torch.empty((2, 2), dtype=torch.int32, device="cuda")
    q8.q8kv_verify_draft(acc, tok, target, draft, drafted,
                         torch.full((2, 2), 0.5, device="cuda"))
    assert acc.tolist() == [0, 0] and tok[:, 0].tolist() == want and (tok[:, 1] == -1).all()
    assert q8.q8kv_device_errors(clear=True) == 0
