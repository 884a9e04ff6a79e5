"""q8kv_verify_draft against running sums in 64 bits: counts and tokens are whole numbers and
have to be equal."""
import numpy as np
import pytest
import torch

import decode_attention_int8_b200 as q8
import serving_ref as ref

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def call(target, draft, drafted, uni, n_drafts=None):
    B, n1, V = target.shape
    acc = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    tok = torch.full((B, n1), -7, dtype=torch.int32, device="cuda")
    nd = None if n_drafts is None else torch.tensor(n_drafts, dtype=torch.int32, device="cuda")
    q8.q8kv_device_errors(clear=True)
    q8.q8kv_verify_draft(acc, tok, target, draft, torch.as_tensor(drafted).int().cuda(),
                         torch.as_tensor(uni).float().cuda(), n_drafts=nd)
    err = q8.q8kv_device_errors(clear=True)
    return acc.cpu().numpy(), tok.cpu().numpy(), err


def host(t):
    return None if t is None else t.float().cpu().numpy()


def draw(B, n, V, dtype, seed, spread=2.0, noise=0.7):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((B, n + 1, V), generator=g, device="cuda") * spread
    target = logits.softmax(-1).to(DT[dtype])
    draft = (logits[:, :n] + noise * torch.randn((B, n, V), generator=g, device="cuda")
             ).softmax(-1).to(DT[dtype])
    e = torch.empty((B, n, V), device="cuda").exponential_(1.0, generator=g)
    drafted = (draft.float() / e).argmax(-1).int() if n else torch.zeros((B, 0)).int().cuda()
    uni = torch.rand((B, n + 1), generator=g, device="cuda")
    return target, draft, drafted, uni


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("B,n,V", [(1, 4, 32000), (3, 0, 1000), (7, 1, 1), (5, 3, 2), (16, 5, 4099),
                                   (2, 8, 65537), (16, 4, 4098), (3, 5, 20006), (64, 3, 777), (300, 2, 513), (700, 1, 64)])
def test_random_rows(dtype, B, n, V):
    target, draft, drafted, uni = draw(B, n, V, dtype, seed=B + V)
    a, t, err = call(target, draft, drafted, uni)
    ra, rt = ref.verify(host(target), host(draft), drafted.cpu().numpy(), uni.cpu().numpy())
    assert np.array_equal(a, ra) and np.array_equal(t, rt) and err == 0
    if n >= 2 and B >= 16:
        assert 0 < a.mean() < n  # both outcomes occur


@pytest.mark.parametrize("B,n,V", [(6, 3, 5000), (200, 2, 130)])
def test_drafts_without_probabilities(B, n, V):
    target, draft, drafted, uni = draw(B, n, V, "fp32", seed=5, spread=4.0)
    drafted = torch.where(torch.rand((B, n), device="cuda") < 0.5, target[:, :n].argmax(-1),
                          drafted.long()).int()
    a, t, err = call(target, None, drafted, uni)
    ra, rt = ref.verify(host(target), None, drafted.cpu().numpy(), uni.cpu().numpy())
    assert np.array_equal(a, ra) and np.array_equal(t, rt) and err == 0
    for b in range(B):  # a refused token is not drawn again
        if a[b] < n:
            assert t[b, a[b]] != drafted[b, a[b]].item()


def test_draft_counts_and_more_than_a_warp_of_drafts():
    B, n, V = 9, 70, 96
    target, draft, drafted, uni = draw(B, n, V, "fp32", seed=11, noise=0.02)
    nd = [0, 1, 31, 32, 33, 64, 69, 70, 5]
    uni[:, :n] *= 0.9  # long accepted runs
    a, t, err = call(target, draft, drafted, uni, nd)
    ra, rt = ref.verify(host(target), host(draft), drafted.cpu().numpy(), uni.cpu().numpy(), nd)
    assert np.array_equal(a, ra) and np.array_equal(t, rt) and err == 0
    assert a.max() > 32


def test_draft_counts_out_of_range_are_clamped_and_flagged():
    target, draft, drafted, uni = draw(2, 2, 50, "fp32", seed=1)
    a, t, err = call(target, draft, drafted, uni, [-3, 9])
    ra, rt = ref.verify(host(target), host(draft), drafted.cpu().numpy(), uni.cpu().numpy(), [0, 2])
    assert np.array_equal(a, ra) and np.array_equal(t, rt) and err == q8.DEVERR_PROBS


def test_draft_token_outside_the_vocabulary_is_refused():
    target, draft, drafted, uni = draw(2, 2, 50, "fp32", seed=2)
    drafted[0, 0], drafted[1, 0] = 50, -1
    a, t, err = call(target, draft, drafted, uni)
    ra, rt = ref.verify(host(target), host(draft), drafted.cpu().numpy(), uni.cpu().numpy())
    assert (a == 0).all() and np.array_equal(t, rt) and err == q8.DEVERR_PROBS
    a, t, err = call(target, None, drafted, uni)
    ra, rt = ref.verify(host(target), None, drafted.cpu().numpy(), uni.cpu().numpy())
    assert (a == 0).all() and np.array_equal(t, rt) and err == q8.DEVERR_PROBS


@pytest.mark.parametrize("V", [8, 40000])
def test_borders_are_exact(V):
    """Dyadic weights: every running sum is exact, so a uniform on a border names the token
    after it, zero names the first token of any weight, and the largest uniform the last."""
    B = 6
    target = torch.zeros((B, 1, V))
    at = [0, 3, V // 2, V - 1] if V > 8 else [0, 3, 4, 7]
    target[:, 0, at] = 0.25
    uni = torch.tensor([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.7499999])[:, None]
    a, t, err = call(target.cuda(), None, torch.zeros((B, 0)), uni)
    assert t[:, 0].tolist() == [at[0], at[1], at[2], at[3], at[3], at[2]] and err == 0
    target[:, 0, 0] = 0.0  # leading zeros
    a, t, err = call(target.cuda(), None, torch.zeros((B, 0)), torch.zeros((B, 1)))
    assert (t[:, 0] == at[1]).all() and err == 0


def test_equal_rows_accept_and_empty_residuals_fall_back():
    """p = q accepts whatever uniform below one; a refusal whose residual is empty (a draft
    more certain than itself allows) draws from the target's row."""
    V = 3000
    p = torch.rand((4, 2, V), generator=torch.Generator().manual_seed(4)).softmax(-1)
    drafted = torch.tensor([[7], [8], [9], [10]])
    q = p[:, :1].clone()
    uni = torch.full((4, 2), 1 - 2.0 ** -24)
    a, t, err = call(p.cuda(), q.cuda(), drafted, uni)
    assert (a == 1).all() and err == 0
    q = 2 * q  # nowhere above the target
    uni = torch.tensor([[0.9, 0.0], [0.9, 0.3], [0.9, 0.8], [0.1, 0.5]])
    a, t, err = call(p.cuda(), q.cuda(), drafted, uni)
    ra, rt = ref.verify(host(p), host(q), drafted.numpy(), uni.numpy())
    assert np.array_equal(a, ra) and np.array_equal(t, rt) and err == 0
    assert a.tolist() == [0, 0, 0, 1]


def test_rows_without_weight_give_no_token():
    target = torch.zeros((3, 2, 20))
    target[1] = float("nan")
    target[2, :, 4] = float("inf")
    draft = torch.full((3, 1, 20), 0.05)
    uni = torch.full((3, 2), 0.5)
    a, t, err = call(target.cuda(), draft.cuda(), torch.tensor([[1], [2], [3]]), uni)
    assert a.tolist() == [0, 0, 0] and (t == -1).all() and err == q8.DEVERR_PROBS


def test_strided_rows_and_unaligned_starts():
    """Rows inside a wider buffer, with strides and starts that 16-byte loads do not fit."""
    B, n, V = 5, 2, 1001
    target, draft, drafted, uni = draw(B, n, V, "fp32", seed=8)
    for off, width in [(0, 1001), (0, 1002), (2, 1006), (0, 1004), (3, 1010), (4, 1024)]:
        wt = torch.full((B, n + 1, width), 9.0, device="cuda")
        wd = torch.full((B, n, width), 9.0, device="cuda")
        if off + V > width:
            continue
        wt[..., off:off + V], wd[..., off:off + V] = target, draft
        a, t, err = call(wt[..., off:off + V], wd[..., off:off + V], drafted, uni)
        ra, rt = ref.verify(host(target), host(draft), drafted.cpu().numpy(), uni.cpu().numpy())
        assert np.array_equal(a, ra) and np.array_equal(t, rt) and err == 0


def test_draws_follow_the_target():
    """Speculative sampling keeps the target's distribution: first tokens of 40000 sequences
    that share one pair of rows, their counts within 6 standard deviations."""
    B, V = 40000, 12
    g = torch.Generator(device="cuda").manual_seed(21)
    p = torch.rand((V,), generator=g, device="cuda").pow(3)
    q = torch.rand((V,), generator=g, device="cuda").pow(3)
    p, q = p / p.sum(), q / q.sum()
    drafted = torch.multinomial(q, B, replacement=True, generator=g).int()[:, None]
    uni = torch.rand((B, 2), generator=g, device="cuda")
    a, t, err = call(p.expand(B, 2, V).contiguous(), q.expand(B, 1, V).contiguous(), drafted, uni)
    n = np.bincount(t[:, 0], minlength=V)
    want = p.double().cpu().numpy() * B
    assert (np.abs(n - want) < 6 * np.sqrt(want) + 6).all() and err == 0


@pytest.mark.parametrize("V", [7, 600, 1024, 5000, 65536])
def test_weights_near_the_largest(V):
    """Rows need not sum to one: weights of which two pass fp32's range still have an fp64 sum."""
    target = torch.zeros((4, 2, V))
    draft = torch.zeros((4, 1, V))
    target[:, 0], target[:, 1] = 3e38, 2.5e38
    target[0, 0, 0] = 1.0
    draft[1] = 1e37
    uni = torch.tensor([[0.5, 0.7], [0.5, 0.31], [0.0, 0.0], [0.5, 1 - 2.0 ** -24]])
    drafted = torch.tensor([[0], [V], [0], [V - 1]]).int()
    drafted[1] = 1
    uni[1, 0] = 1.0
    target[1, 0, 1] = 0.0  # refused: the residual of the others
    target[3, 0, V - 1] = 0.0
    for q in (draft, None):
        a, t, err = call(target.cuda(), None if q is None else q.cuda(), drafted, uni)
        ra, rt = ref.verify(host(target), host(q), drafted.numpy(), uni.numpy())
        assert np.array_equal(a, ra) and np.array_equal(t, rt) and err == 0
