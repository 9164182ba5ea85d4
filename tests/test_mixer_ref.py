"""CPU pins of the references that the GPU tests of the mixer operators go by: their
gradients against central differences, and hand-worked values."""
import math

import pytest
import torch

from tests import mixer_ref as R

F64 = torch.float64


def rnd(*s, seed=0):
    return torch.randn(*s, dtype=F64, generator=torch.Generator().manual_seed(seed + sum(s)))


@pytest.mark.parametrize("lens", [None, (2, 0, 3)])
def test_conv_gradients_are_the_differences(lens):
    N = 2 if lens is None else 3
    B = 2 if lens is None else 1
    a = [rnd(B, 5, 3).requires_grad_(), rnd(3, 4).requires_grad_(), rnd(3).requires_grad_(), rnd(N, 3, 3).requires_grad_()]
    assert torch.autograd.gradcheck(lambda *t: R.conv(*t, lens), a)


@pytest.mark.parametrize("lens", [None, (2, 0, 3)])
def test_ssm_gradients_are_the_differences(lens):
    B, N = (2, 2) if lens is None else (1, 3)
    H, n, p = 2, 2, 3
    a = [rnd(B, 5, H, p), rnd(B, 5, H), -rnd(H).abs(), rnd(B, 5, H, n, seed=1), rnd(B, 5, H, n, seed=2), rnd(H, seed=3), rnd(H, seed=4),
         rnd(N, H, n, p)]
    assert torch.autograd.gradcheck(lambda *t: R.ssm(*t, lens), [t.requires_grad_() for t in a])


def test_norm_gradients_are_the_differences():
    a = [rnd(3, 2, 5), rnd(2, 5), rnd(2, 5, seed=1), rnd(3, 2, 5, seed=2)]
    assert torch.autograd.gradcheck(lambda *t: R.norm(*t, 1e-5), [t.requires_grad_() for t in a])


def test_worked_values():
    x = torch.tensor([[[1.0], [2.0], [4.0]]], dtype=F64)
    w = torch.tensor([[10.0, 1.0]], dtype=F64)
    y, fin = R.conv(x, w, None, torch.tensor([[[3.0]]], dtype=F64), None, False)
    assert y.flatten().tolist() == [31.0, 12.0, 24.0] and fin.flatten().tolist() == [4.0]
    one = torch.ones(1, 2, 1, 1, dtype=F64)
    y, h = R.ssm(2 * one, one[..., 0], -math.log(2) * torch.ones(1, dtype=F64), 3 * one, one, torch.ones(1, dtype=F64), None,
                 8 * one[:, :1], None, False)
    # h: 8/2 + 6 = 10, 10/2 + 6 = 11; y = h + 2
    assert torch.allclose(y.flatten(), torch.tensor([12.0, 13.0], dtype=F64)) and abs(float(h) - 11) < 1e-12
    q = torch.ones(1, 1, dtype=F64)
    o, h = R.delta_rule(q, q, 5 * q, torch.zeros(1, dtype=F64), 0.5 * torch.ones(1, dtype=F64), 3 * q[None], 2.0)
    assert float(h) == 4.0 and float(o) == 8.0     # u = 0.5 (5 - 3) = 1
