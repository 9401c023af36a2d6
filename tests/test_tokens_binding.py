"""The token calls' Python signatures (CPU): every argument by name, the first
one among them, and the keyword stream."""
import inspect

import pytest
import torch

import depth_weighted_scatter_amd as dws

CALLS = {"bevpool_qk_norm_rope": "q", "bevpool_qk_norm_rope_backward": "dq_out",
         "bevpool_kv_append": "k", "bevpool_paged_attention": "q"}


@pytest.mark.parametrize("name,first", CALLS.items())
def test_signature(name, first):
    par = inspect.signature(getattr(dws, name)).parameters
    assert next(iter(par)) == first
    assert par["stream"].kind is inspect.Parameter.KEYWORD_ONLY and par["stream"].default is None


@pytest.mark.parametrize("name,first", CALLS.items())
def test_first_argument_by_name(name, first):
    """Without a GPU the call gets as far as the check of its first tensor."""
    call = getattr(dws, name)
    with pytest.raises(TypeError, match=f"{first} must be a GPU tensor"):
        call(**{first: torch.zeros(4, 2, 64)})
    with pytest.raises(TypeError, match=f"{first} must be a GPU tensor"):
        call(torch.zeros(4, 2, 64))
    with pytest.raises(TypeError, match=f"{first} must be a GPU tensor"):
        call(**{first: None})
    with pytest.raises(TypeError, match=f"missing.*{first}"):
        call()
