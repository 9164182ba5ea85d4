"""Arguments out of range raise the ValueError that the binding promises; on the CPU."""
import pytest
import torch

from gated_deltanet_chunked_fwd_amd import mixer as M

BF = torch.bfloat16


def z(*s, dtype=BF):
    return torch.zeros(*s, dtype=dtype)


def ssm(nb=1, H=2, **kw):
    d = dict(x=z(nb, 7, H, 64), dt=z(nb, 7, H), A=z(H), B=z(nb, 7, 1, 64), C=z(nb, 7, 1, 64))
    d.update(kw)
    return M.check_ssm_args(require_cuda=False, **d)


def test_empty_axes():
    for call in (lambda: M.check_conv_args(z(0, 7, 16), z(16, 4), require_cuda=False),
                 lambda: M.check_conv_args(z(2, 7, 0), z(0, 4), require_cuda=False),
                 lambda: M.check_conv_step_args(z(3, 0), z(5, 3, 0), z(0, 4), require_cuda=False),
                 lambda: ssm(nb=0), lambda: ssm(H=0),
                 lambda: M.check_ssm_step_args(z(3, 0, 64), z(3, 0), z(0), z(3, 1, 64), z(3, 1, 64), z(5, 0, 64, 64, dtype=torch.float32),
                                               require_cuda=False),
                 lambda: M.check_delta_step_args(z(3, 0, 64), z(3, 0, 64), z(3, 0, 64), z(3, 0, dtype=torch.float32), z(3, 0),
                                                 z(5, 0, 64, 64, dtype=torch.float32), require_cuda=False)):
        with pytest.raises(ValueError):
            call()
    M.check_conv_args(z(2, 0, 16), z(16, 4), require_cuda=False)      # no tokens: an empty output and the states


@pytest.mark.parametrize("segment_chunks,fine", [(0, True), (2 ** 31 - 1, True), (2 ** 31, False), (2 ** 32 + 1, False), (-1, False)])
def test_segment_chunks(segment_chunks, fine):
    if fine:
        assert ssm(segment_chunks=segment_chunks)[0].segment_chunks == segment_chunks
    else:
        with pytest.raises(ValueError, match="^segment_chunks"):
            ssm(segment_chunks=segment_chunks)


@pytest.mark.parametrize("eps", [0.0, -1.0, 1e-60, 1e39, float("nan"), float("inf")])
def test_eps_is_a_positive_fp32_number(eps):
    with pytest.raises(ValueError, match="^eps"):
        M.check_norm_args(z(6, 32), eps=eps, require_cuda=False)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 1e39])
def test_scale_is_a_finite_fp32_number(scale):
    d = [z(3, 2, 64), z(3, 2, 64), z(3, 2, 64), z(3, 2, dtype=torch.float32), z(3, 2), z(5, 2, 64, 64, dtype=torch.float32)]
    M.check_delta_step_args(*d, scale=0.5, require_cuda=False)
    with pytest.raises(ValueError, match="^scale"):
        M.check_delta_step_args(*d, scale=scale, require_cuda=False)
