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


@pytest.mark.parametrize("y_dtype", [BF, F32])
@pytest.mark.parametrize("gate_dtype,out_dtype", [(F32, F32), (BF, F32), (F32, BF), (BF, BF)])
@pytest.mark.parametrize("columns,group", [(256, 256), (512, 512), (2048, 512), (4096, 4096), (16384, 64)])
def test_gates_of_any_size(cuda_ok, y_dtype, gate_dtype, out_dtype, columns, group):
    """SiLU over the whole range in which its value is a number above 0 in fp32: with inputs of +1 and -1 the norm is exactly 1,
    so that the output is the gate's. It is within 2^-20 of its value and the product adds 2^-24, a result below 2^-126 half of
    fp32's least step, a bf16 one half a step more (of its least, 2^-133, too). Only bf16 gates with bf16 outputs may be 0 where SiLU
    is below 2^-119, and take the rounding of z log2(e) along, 2^-23 |z|."""
    z = torch.linspace(-105.0, 95.0, columns, device="cuda").to(gate_dtype)[None]
    y = torch.ones(1, columns, dtype=y_dtype, device="cuda")
    y[:, ::3] = -1
    got = gated_rmsnorm(y, z, torch.ones(columns, device="cuda"), group=group, eps=0.0, out_dtype=out_dtype).double()
    t = z.double()
    want = y.double() * t / (1 + torch.exp(-t))
    bound = want.abs() * 2.0 ** -19.9 + 2.0 ** -149
    if out_dtype == BF:
        bound += want.abs() * 2.0 ** -8 + 2.0 ** -134
        if gate_dtype == BF:
            bound += want.abs() * t.abs() * 2.0 ** -23 + (want.abs() < 2.0 ** -119) * want.abs()
    assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound).max()
