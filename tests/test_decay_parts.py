"""The bf16 chunk products keep fp32 accuracy: weighted rows go to the tensor cores in three bf16 parts.
With one token that is not zero there is nothing to sum, and a state's entries are held to the few
roundings that they meet.  Dropping the third part would show."""
import pytest
import torch

from positive_quadratic_b200 import oal

U = 2.0 ** -24
B, HQ, HKV, SCALE = 2, 4, 2, 0.37


def bound(T):
    """Relative: l^m 6 (CUDA's expf 2 units in the last place, 4 of 2^-24; its correction and the
    product 2), times scale 1, times the row 1, the three parts' sum 2; per further chunk of 128 tokens
    another l^m and the sum, 7.  Parts and products are exact: 8 + 8 + 8 and 8 + 8 digits."""
    return (10 + 7 * ((T + 127) // 128 - 1)) * U


def inputs(T, at):
    """y and z [B, HKV, 64] of the token `at`, and the decays: rates whose powers fill 24 digits."""
    gen = torch.Generator().manual_seed(100 * T + at)
    y, z = (torch.randn(B, HKV, 64, generator=gen).bfloat16() for _ in range(2))
    return y, z, torch.tensor([-0.0137, -0.0291])


CASES = [(100, 0), (100, 57), (128, 3), (300, 5), (300, 140), (300, 290)]


@pytest.mark.parametrize("T,at", CASES)
def test_two_parts_would_not_do(T, at):
    """The same rows in two parts, on the CPU, miss the bound."""
    y, _, g = inputs(T, at)
    n = min(128, T - at // 128 * 128)
    w = torch.exp(g.double() * (n - 1 - at % 128)).float()[None, :, None]
    row = y.float() * w
    hi = row.bfloat16().float()
    mid = (row - hi).bfloat16().float()
    lo = row - hi - mid
    assert torch.equal(hi + (mid + lo.bfloat16().float()), row)
    assert float((lo / row).abs().max()) > bound(T)


def check(got, want, T):
    assert got.shape == want.shape
    worst = ((got.double().cpu() - want).abs() / (bound(T) * want.abs())).max()
    assert worst <= 1, f"{float(worst):.2f} times the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("T,at", CASES)
def test_state_of_one_token(cuda, T, at):
    y, z, g = inputs(T, at)
    k, v = (torch.zeros(B, HKV, T, 64, dtype=torch.bfloat16) for _ in range(2))
    k[:, :, at], v[:, :, at] = y, z
    q = torch.zeros(B, HQ, T, 64, dtype=torch.bfloat16)
    _, state = oal.decay_prefill(q.to(cuda), k.to(cuda), v.to(cuda), g.to(cuda), SCALE)
    left = torch.exp(g.double() * (T - 1 - at))[None, :, None, None]
    check(state, left * (y.double()[..., :, None] * z.double()[..., None, :]), T)


@pytest.mark.gpu
@pytest.mark.parametrize("T,at", CASES)
def test_first_state_gradient_of_one_token(cuda, T, at):
    """In the second head of each group: the heads are summed, some of them in separate blocks."""
    y, z, g = inputs(T, at)
    q, do = (torch.zeros(B, HQ, T, 64, dtype=torch.bfloat16) for _ in range(2))
    q[:, 1::2, at], do[:, 1::2, at] = y, z
    k = torch.zeros(B, HKV, T, 64, dtype=torch.bfloat16).to(cuda)
    got = oal.decay_backward(q.to(cuda), k, k, g.to(cuda), SCALE, do.to(cuda))["dstate"]
    scale = torch.tensor(SCALE).double()  # as the call takes it, in fp32
    far = scale * torch.exp(g.double() * (at + 1))[None, :, None, None]
    check(got, far * (y.double()[..., :, None] * z.double()[..., None, :]), T)
