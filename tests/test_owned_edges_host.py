"""route_*, w8a8_mul_mat_experts and lora_add on the host (no GPU): what the edges need that no launch shows.

Addresses are made up: the file runs only where there is no GPU to launch on."""

import numpy as np
import pytest
import torch

from tests.test_gpu_owned_edges import full_values, in_parts, three_bytes
from tests.test_owned_host import Call, i2s, refused  # noqa: F401 (a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")


def test_flags_of_the_router(i2s):
    for flags in (0, 1, 2, 3, 8, 9, 10, 11):
        c = Call(i2s)
        c.flags = flags
        assert c.topk() in (c.E["I2S_E_CUDA"], c.E["I2S_E_UNSUPPORTED_DEVICE"])   # with and without a bias
        c.bias = 30 << 40
        assert c.topk() in (c.E["I2S_E_CUDA"], c.E["I2S_E_UNSUPPORTED_DEVICE"])
    refused(i2s, "topk", [("BAD_ARG", ("flags", f)) for f in (4, 12, 16, 1 << 31)])
    assert i2s.ROUTE_BIAS_SCORE == 8
    with pytest.raises(ValueError, match="bias_on"):
        i2s.RouteTopk(torch.zeros(4, 4), 2, bias_on="logits")


@pytest.mark.parametrize("items,x_group,N,K", [(32768, 8, 1536, 2048), (20, 2, 64, 48), (1, 1, 32, 16), (256, 1, 4096, 1040)])
def test_workspace_of_the_products_by_form(i2s, items, x_group, N, K):
    """Codes of the rows with the 128 bytes behind the last that a copy may read, scales, and what the form needs besides: the
    gate has no F32 rows, a row of its own per item no places."""
    c = Call(i2s)
    c.w.N, c.w.K, c.plan.items = N, K, items
    need = lambda flags: c.L.w8a8_mul_mat_experts_workspace(c.w, c.plan, x_group, 1, flags)
    least = 256 + items * (2 * K + 4) + 128 + (4 * items if x_group > 1 else 0)
    assert least <= need(1) <= least + 3 * 256
    more = items * (4 * N + 1)
    assert least + more <= need(0) <= least + more + 5 * 256
    c.x_group, c.ws_bytes, c.flags = x_group, need(1) - 1, 1
    c.x.stride, c.y.stride = K, N
    assert c.product() == c.E["I2S_E_WORKSPACE_TOO_SMALL"]


def test_values_that_show_a_missing_part(i2s):
    """The rows of the test of 24 bits come out whole of three bf16 parts, and of two not one in a hundred does."""
    x = full_values(300, 520, 1)
    t = three_bytes(3000, 1).sum(1)
    for v in (x, t):
        assert np.array_equal(in_parts(v, 3), v.astype(np.float64))
        assert (in_parts(v, 2) == v).mean() < 0.01
    assert np.array_equal(in_parts(three_bytes(3000, 1), 1), three_bytes(3000, 1))   # the positions have 8 bits each
