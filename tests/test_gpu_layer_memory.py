"""What a layer's rows of padding hold does not depend on who used the memory before."""
import pytest
import torch

from combine_moe_route_03_gb300 import api
from support import bf16_dev, device_weights, host_experts, host_workload, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["small_masked", "small_contig"])
def test_rows_without_a_token_are_finite_over_used_memory(dev, name):
    cfg, x, W, bias = host_workload(name)
    W, bias, weights, x = to_dev(W), to_dev(bias), device_weights(host_experts(name)), bf16_dev(x)
    sizes = [2 ** n for n in range(10, 27)]
    used = [torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del used                    # NaN in every type, for the allocator to hand out again
    lay = api.MoELayer(cfg, W, bias, weights)
    lay.forward(x)
    Y = lay.Y.clone()
    assert bool(torch.isfinite(Y.float()).all())
    lay.forward(x)
    torch.cuda.synchronize()
    assert api.read_status(lay.status) == 0
    assert torch.equal(lay.Y, Y)


@pytest.mark.parametrize("name", ["small_masked", "small_contig"])
def test_rows_of_earlier_tokens_do_not_reach_later_outputs(dev, name):
    """A call whose routing leaves rows empty that an earlier call filled."""
    cfg, x, W, bias = host_workload(name)
    W, bias, weights, x = to_dev(W), to_dev(bias), device_weights(host_experts(name)), bf16_dev(x)
    same = x[:1].expand_as(x).contiguous()      # every token to the same experts
    lay = api.MoELayer(cfg, W, bias, weights)
    lay.forward(same)
    first = lay.counts.clone()
    out = lay.forward(x).clone()
    torch.cuda.synchronize()
    assert bool((lay.counts < first).any())     # rows that were filled and are empty now
    assert bool(torch.isfinite(lay.Y.float()).all())
    fresh = api.MoELayer(cfg, W, bias, weights)
    assert torch.equal(fresh.forward(x), out)
