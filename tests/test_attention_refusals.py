"""CPU tests of refusals at the ends of the attention operators' argument types: sums and products of sizes that would pass
64 bits, scales that pass fp32.  And the words of
one.  Nothing is launched."""
import pytest
import torch
from torch.autograd import forward_ad

from linear_spatial_propagation_gspn_amd import attention as A
from test_attention_abi import BF16, F32, SHAPE, UNSUP, refuse


@pytest.fixture(scope="module")
def lib():
    return A.lib()


@pytest.mark.parametrize("kind", ["fwd", "bwd"])
@pytest.mark.parametrize("pairs", [1 << 62, (1 << 62) + 3, (1 << 63) - 1, 1 << 61])
def test_pairs_whose_double_passes_64_bits(lib, kind, pairs):
    refuse(lib, "rotary", kind, SHAPE, pairs=pairs, axes=1, section0=pairs, section1=0)
    refuse(lib, "rotary", kind, SHAPE, dtype=BF16, pairs=pairs, section0=pairs, section1=0)


@pytest.mark.parametrize("kind", ["fwd", "step", "bwd"])
@pytest.mark.parametrize("kv_rows", [(1 << 63) - 1, (1 << 63) - 2, 1 << 62, (1 << 30) + 2])
def test_keys_whose_number_with_the_sequences_passes_64_bits(lib, kind, kv_rows):
    # (128 heads of keys: a count of their workgroups would come round to a small one)
    for heads in (128, 2):
        build = dict(heads=heads, kv_heads=heads, d=2, lse=True)
        refuse(lib, "attn", kind, SHAPE, build=build, kv_rows=kv_rows)
        if kind != "step":
            refuse(lib, "attn", kind, SHAPE, build=dict(build, kv_cu=True), kv_rows=kv_rows)
            refuse(lib, "attn", kind, SHAPE, build=dict(build, cu=True, nseq=1), kv_rows=kv_rows)


@pytest.mark.parametrize("nseq", [(1 << 63) - 1, (1 << 63) - 30, 1 << 62, 1 << 30])
def test_workspaces_of_too_many_sequences(lib, nseq):
    assert lib.gspn_attention_bwd_workspace_bytes(40, nseq, 6, 40, 2, 20) == -1
    assert lib.gspn_attention_bwd_workspace_bytes(1 << 30, nseq, 6, 40, 2, 20) == -1
    if nseq > 1 << 30:
        assert lib.gspn_attention_step_workspace_bytes(nseq, 6, 2, 20, 50) == -1


@pytest.mark.parametrize("kind", ["fwd", "step", "bwd"])
def test_scales_whose_powers_of_two_pass_fp32(lib, kind):
    for scale in (2.4e38, -3.4e38):
        refuse(lib, "attn", kind, SHAPE, scale=scale)
        refuse(lib, "attn", kind, SHAPE, dtype=BF16, scale=scale)
    refuse(lib, "attn", kind, UNSUP, scale=2.3e38, d=129)  # (the scale alone is no reason)


def test_forward_mode_is_not_refused_in_another_operators_name():
    x, pos, freqs = torch.zeros(4, 2, 8), torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for call in (lambda: A.attention(x, dual, x), lambda: A.head_rotary(dual, pos, freqs)):
            with pytest.raises(NotImplementedError, match="over token rows"):
                call()
