"""The longest limit of a group's waits, on the GPU: the kernels add it to a clock of 64 bits."""
import pytest
import torch

from test_gpu_experts import tide  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [2 ** 64 - 1, 2 ** 63, 2 ** 63 - 1])
@pytest.mark.parametrize("variant", [2, 3], ids=["bulk", "tmem"])
def test_the_longest_wait_limit_of_a_group(tide, variant, limit):
    R, params = 4, [(3000, 512), (100, 16), (2048, 1024)]
    g = torch.Generator(device="cuda").manual_seed(0)
    grads = [[torch.randn(r * n, generator=g, device="cuda").bfloat16() for r, n in params] for _ in range(R)]
    results = []
    for ns in (0, limit):
        G = tide.Group(R, params)
        G.set_rs_variant(variant)
        G.set_ag_variant(tide.TIDE_AG_BULK)
        G.set_wait_timeout(ns)
        sums, shards = torch.zeros(R, G.S, device="cuda"), torch.zeros(R, G.S, dtype=torch.bfloat16, device="cuda")
        outs = [torch.zeros(r * n, dtype=torch.bfloat16, device="cuda") for r, n in params]
        for _ in range(20):
            G.reduce_scatter(grads, list(sums))
            shards.copy_(sums)
            G.all_gather(list(shards), outs)
        assert G.device_status() == 0
        results.append([sums, *outs])
        G.close()
    assert all(torch.equal(p, q) for p, q in zip(*results)) and bool(results[0][0].any())
