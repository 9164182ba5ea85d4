"""The operators of gated_deltanet_chunked_fwd_amd.mixer on the GPU where their bounds are
tight: results whose sums nearly cancel, sizes that take every branch of the kernels, values
that are not finite.  References and tolerances as in test_gpu_mixer.py."""
import pytest
import torch

from gated_deltanet_chunked_fwd_amd import mixer
from tests import mixer_ref as R
from tests.test_gpu_mixer import BF, F32, close, dev, gen, ssm_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seg", [0, 2])
@pytest.mark.parametrize("n,p", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_ssm_outputs_of_a_long_memory(n, p, seg):
    """bf16 outputs that are nearly all C h, with products of both signs: the state enters as a
    bf16 pair, which leaves 2^-8 of 2^-8 of each product, as the pair of the q k products
    does; 128 more fp32 roundings for the sums and the decays."""
    B, T, H = 1, 200, 2
    d = ssm_inputs(n + p, B, T, H, 1, n, p, BF, F32, None, True, F32)
    d["C"] = gen(7)(B, T, 1, n).to(BF)
    d["h0"] = d["h0"] * 100
    d["A"] = torch.tensor([-1e-3, -1e-2])
    w = {k: R.wide(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias", "h0")}
    e = lambda t: t.expand(-1, -1, H, -1)  # noqa: E731
    ref, hr = R.ssm(w["x"], w["dt"], w["A"], e(w["B"]), e(w["C"]), w["D"], w["bias"], w["h0"], None)
    ra, ha = R.ssm(w["x"].abs(), w["dt"], w["A"], e(w["B"]).abs(), e(w["C"]).abs(), w["D"], w["bias"], w["h0"].abs(), None)
    a = tuple(dev(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias"))
    y, h = mixer.ssm_fwd(*a, initial_state=dev(d["h0"]), segment_chunks=seg)
    close(y, ref, ra, 2.0 ** -16 + 128 * 2.0 ** -24, "y")
    close(h, hr, ha, 128 * 2.0 ** -24, "state")
