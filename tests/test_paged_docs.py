"""CPU: the serving calls say how their errors are read."""
import inspect

import pytest

import sparse_attention_mla_gb300 as dsa


@pytest.mark.parametrize("name", ["dsa_paged_slots", "dsa_norm_rope_fwd", "dsa_norm_rope_bwd", "dsa_paged_mla",
                                  "dsa_paged_indexer_topk"])
def test_a_call_with_a_workspace_says_how_its_errors_are_read(name):
    call = getattr(dsa, name)
    assert inspect.signature(call).parameters["workspace"].default is None
    assert "dsa_read_device_status" in call.__doc__ and "paged_workspace_size" in call.__doc__
    if name != "dsa_norm_rope_bwd":  # (which has none)
        assert "zeroed once" in " ".join(call.__doc__.split()) and "dropped" in call.__doc__
