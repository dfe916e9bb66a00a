"""bf16 outputs and gradients of decayed attention are rounded once, at the end: what lies between (the
decayed scores, the states before the chunks) is carried in two bf16 parts, or in fp32."""
import pytest
import torch

from positive_quadratic_b200 import oal
from tests import _decay_ref as ref
from tests.test_decay_gpu import SCALE, make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def check(name, got, want, size, T):
    """The result's rounding, 2^-8 of the value; two parts leave 2^-8 of 2^-8 of a term; and fp32 as
    in _decay_ref.tolerance."""
    half = 2.0 ** -8
    few = (300 + 1024 + T / 64) * 2.0 ** -24
    live = ~torch.isnan(want)
    err = (got.double().cpu() - want).abs()[live]
    tol = (half * want.abs() + (1 + half) * (half * half + few) * size + 1e-30)[live]
    assert float((err / tol).max()) <= 1.0, f"{name}: {float((err / tol).max()):.2f} times its bound"


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (3, 17, 2, 1), (2, 100, 14, 2), (1, 128, 6, 3)])
def test_scores_of_one_chunk(cuda, B, T, Hq, Hkv):
    q, k, v, g, do, _, _ = make(cuda, B, T, Hq, Hkv, BF, seed=2)
    out, _ = oal.decay_prefill(q, k, v, g, SCALE)
    w = ref.forward(q, k, v, g, SCALE)
    check("out", out, w[0], w[2], T)
    got = oal.decay_backward(q, k, v, g, SCALE, do)
    w = ref.backward(q, k, v, g, SCALE, do)
    for n in ("dq", "dk", "dv"):
        check(n, got[n], *w[n], T)
