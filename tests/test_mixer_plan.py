"""How the selective scan splits sequences into segments, seen in the workspace that a call
asks for (the gates of every chunk, and a state and a decay per segment and head); nothing is
launched.  Without a GPU the split is that of 256 CUs."""
import ctypes

import pytest
import torch

from gated_deltanet_chunked_fwd_amd import abi as A
from gated_deltanet_chunked_fwd_amd import mixer
from gated_deltanet_chunked_fwd_amd.binding import lib


def segments(lens, H, B=1, bf16=True, n=128, p=128):
    """Segments over all sequences that gdn_ssm_fwd splits into, 0 if none is split."""
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    host = (ctypes.c_int32 * len(cu))(*cu)
    t = A.GDN_BF16 if bf16 else A.GDN_F32
    dense = B > 1 or len(lens) == 1
    sh = A.GdnSsmShape(B=B, T=lens[0] if dense else cu[-1], H=H, G=1, n=n, p=p, N=B if dense else len(lens), dtype=t, dt_dtype=t,
                       param_dtype=A.GDN_F32, dt_softplus=1, cu_seqlens_host=None if dense else host)
    size = ctypes.c_size_t(0)
    assert lib().gdn_ssm_fwd_workspace_bytes(ctypes.byref(sh), ctypes.byref(size)) == 0
    gates = B * sum((v + 63) // 64 for v in lens) * H * 1024
    states = size.value - gates
    return states // (H * n * p * 4)          # (the decays are less than one state)


@pytest.mark.parametrize("rest", [(), (1,) * 30, (1,) * 31, (1,) * 500, (0,) * 31, (64,) * 31, (0, 1, 200) * 40])
def test_short_sequences_do_not_keep_a_long_one_whole(rest):
    alone = segments((131072,), 16)
    assert alone >= 32
    assert segments((131072,) + rest, 16) >= len(rest) + alone // 2
    assert segments(rest + (131072,), 16) >= len(rest) + alone // 2


@pytest.mark.parametrize("B,T,H", [(31, 4096, 16), (24, 4096, 16), (16, 4096, 16), (31, 1024, 16), (32, 4096, 16), (200, 640, 4)])
def test_equal_sequences_that_nearly_fill_the_gpu_stay_whole(B, T, H):
    assert segments((T,), H, B) == 0


@pytest.mark.parametrize("B,T,H", [(16, 4096, 16), (12, 4096, 16), (10, 2048, 16), (200, 640, 4)])
def test_the_same_of_fp32_tensors(B, T, H):
    assert segments((T,), H, B, bf16=False) == 0


@pytest.mark.parametrize("B,T,H,want", [(4, 4096, 16, 8), (9, 4096, 16, 3), (1, 131072, 4, 128), (1, 512, 16, 4), (1, 256, 16, 0)])
def test_segments_of_equal_length(B, T, H, want):
    assert segments((T,), H, B) == B * want


@pytest.mark.parametrize("N", [3, 64, 65, 500])
def test_sequence_offsets_are_checked(N):
    cu = torch.arange(N + 1, dtype=torch.int32) * 2
    x = torch.zeros(1, 2 * N, 8)
    w = torch.zeros(8, 4)
    assert mixer.check_conv_args(x, w, cu_seqlens=cu, require_cuda=False)[0].N == N
    for at, v in ((0, 1), (N, 2 * N + 1), (N // 2, -1), (1, 2 * N)):
        bad = cu.clone()
        bad[at] = v
        with pytest.raises(ValueError, match="^cu_seqlens"):
            mixer.check_conv_args(x, w, cu_seqlens=bad, require_cuda=False)
