"""Workspaces are checked like every other tensor of a call, before its address
goes to the library: type, device and layout (no GPU: nothing is enqueued)."""
import pytest
import torch


def _calls(m, pb, ws):
    R, H, G = pb.total_rows, pb.H, pb.G
    q = torch.zeros(R, H * G, 128, dtype=torch.bfloat16)
    iq = torch.zeros(R, H, 64, dtype=torch.bfloat16)
    k = torch.zeros(pb.cache_tokens, H, 128, dtype=torch.bfloat16)
    ik = torch.zeros(pb.cache_tokens, H, 64, dtype=torch.bfloat16)
    new = torch.zeros(R, H, 128, dtype=torch.bfloat16)
    sel, nsel = pb.new_sel()
    return [lambda: m.forward(pb, q, iq, k, k, ik, workspace=ws), lambda: m.attend_decode(pb, q, k, k, sel, nsel, workspace=ws),
            lambda: m.attend_prefill(pb, q, k, k, sel, nsel, workspace=ws), lambda: m.dense_forward(pb, q, k, k, workspace=ws),
            lambda: m.append_cache(pb, new, new, k, k, workspace=ws)]


@pytest.mark.parametrize("call", range(5))
def test_a_workspace_of_another_kind(call):
    import block_sparse_attention_index_gb300 as m
    pb = m.Problem(2, 4, [(1, 100), (2, 300)], "cpu")
    size = max(pb.workspace_size(), pb.dense_workspace_size())
    for ws, error in ((torch.zeros(size, dtype=torch.float32), TypeError), (torch.zeros(2 * size, dtype=torch.uint8)[::2], ValueError),
                      (torch.zeros(size, dtype=torch.uint8, device="meta"), ValueError)):
        with pytest.raises(error, match="workspace must be"):
            _calls(m, pb, ws)[call]()
