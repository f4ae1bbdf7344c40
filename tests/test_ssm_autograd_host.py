"""Host-side behaviour of the state space layer's autograd wrappers (no GPU
needed): they refuse host tensors before anything reaches the library."""
import pytest
import torch

from varlen_depthwise_causal_amd.autograd import group_norm_silu, selective_scan


def test_selective_scan_refuses_host_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, requires_grad=True)  # noqa: E731
    with pytest.raises(ValueError, match="device tensor"):
        selective_scan(bf(5, 8), bf(5, 8), torch.zeros(8, 16, requires_grad=True), bf(5, 16), bf(5, 16),
                       torch.tensor([0, 5], dtype=torch.int32))


def test_group_norm_silu_refuses_host_tensors_and_groups():
    x = torch.zeros(5, 8, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="device tensor"):
        group_norm_silu(x, torch.ones(8), 2)
    with pytest.raises(ValueError, match="groups"):
        group_norm_silu(x, torch.ones(8), 3)
