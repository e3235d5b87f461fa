"""append_cache writes the scales of an int8 cache in place, so it takes no
Problem that holds copies of them.  (The refusal comes before any launch.)"""
import pytest
import torch

import block_sparse_attention_index_gb300 as m


def _call(k_scale, v_scale, T=70, H=2):
    pb = m.Problem(H, 2, [(3, 60)], "cpu", cache_tokens=T, k_scale=k_scale, v_scale=v_scale)
    k, v = (torch.zeros(T, H, 128, dtype=torch.int8) for _ in range(2))
    new = torch.zeros(3, H, 128, dtype=torch.bfloat16)
    return pb, lambda: m.append_cache(pb, new, new, k, v)


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("form", ["strided", "float64", "list", "transposed"])
def test_scales_that_are_copied_are_refused(form, which):
    good = torch.ones(70, 2)
    other = {"strided": torch.ones(70, 4)[:, ::2], "float64": torch.ones(70, 2, dtype=torch.float64),
             "list": [[1.0, 1.0]] * 70, "transposed": torch.ones(2, 70).t()}[form]
    pb, call = _call(*((other, good) if which == 0 else (good, other)))
    with pytest.raises(ValueError, match="k_scale and v_scale"):
        call()
    assert pb.k_scale.shape == pb.v_scale.shape == (70, 2)  # (reading them is as before)


def test_scales_given_as_they_are_kept_are_the_problems():
    k_scale, v_scale = torch.ones(70, 2), torch.ones(70, 2)
    pb, _ = _call(k_scale, v_scale)
    assert pb.k_scale is k_scale and pb.v_scale is v_scale and not pb.scales_copied
    view = torch.ones(80, 2)[10:]  # contiguous rows of a larger buffer
    pb, _ = _call(view, v_scale)
    assert pb.k_scale.data_ptr() == view.data_ptr() and not pb.scales_copied
