"""Numbers that the calls between a layer's projections take and give at the ends of their ranges (needs a B200)."""

import pytest
import torch

from hybrid_model_ssm_gdn_b200 import add_rmsnorm, gated_rmsnorm

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def test_numbers_given_as_tensors_are_read_at_each_call(cuda_ok):
    """eps and offset as tensors of one element that change in place between calls, a group as one."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, z = (torch.randn(3, 64, generator=g, device="cuda") for _ in range(2))
    w, eps, offset, group = torch.ones(64, device="cuda"), torch.tensor(0.5), torch.tensor(0.0), torch.tensor(16)
    for e, o, n in ((0.5, 0.0, 16), (2.0, 1.0, 32)):
        eps.fill_(e), offset.fill_(o), group.fill_(n)
        assert torch.equal(add_rmsnorm(x, w, eps=eps, offset=offset), add_rmsnorm(x, w, eps=e, offset=o))
        assert torch.equal(gated_rmsnorm(x, z, w, group=group, eps=eps, offset=offset),
                           gated_rmsnorm(x, z, w, group=n, eps=e, offset=o))
