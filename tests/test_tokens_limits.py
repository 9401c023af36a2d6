"""Head counts and strides at the ends of their integer types (CPU): refused on
the host, in arithmetic that does not wrap."""
import pytest

import depth_weighted_scatter_amd as dws
from test_tokens_abi import OVERFLOW, attend_call, grad_call, lib, no_gpu_only, rope_call  # noqa: F401

MOST = 2 ** 31 - 1


@no_gpu_only
@pytest.mark.parametrize("kw", [dict(n=0, hq=MOST, hk=MOST), dict(n=0, hq=1, hk=2 ** 30),
                                dict(n=MOST, hq=MOST, hk=MOST), dict(n=2, hq=2 ** 30, hk=2 ** 30)])
def test_heads_past_31_bits(lib, kw):  # noqa: F811
    assert rope_call(lib, **kw) == OVERFLOW
    assert grad_call(lib, **kw) == OVERFLOW
    assert attend_call(lib, **kw) == OVERFLOW


@no_gpu_only
@pytest.mark.parametrize("stride", [2 ** 31 + 8, 2 ** 61, 2 ** 62, 2 ** 63 - 8])
def test_strides_past_63_bits(lib, stride):  # noqa: F811
    assert rope_call(lib, qs=stride) == OVERFLOW
    assert attend_call(lib, os=stride) == OVERFLOW


def test_sizes_of_heads_past_31_bits():
    assert dws.bevpool_qk_norm_rope_backward_workspace_size(0, MOST, MOST, 16) == 0
    assert dws.bevpool_qk_norm_rope_backward_workspace_size(0, 2 ** 30, 2 ** 29, 16) == 0
    assert dws.bevpool_qk_norm_rope_backward_workspace_size(0, 2 ** 30, 0, 16) > 0
    assert dws.bevpool_paged_attention_workspace_size(0, 1, MOST, MOST, 16, 16, 1) == 0
