"""route_*, w8a8_mul_mat_experts and lora_add on the host (no GPU): what the edges need that no launch shows.

Addresses are made up: the file runs only where there is no GPU to launch on."""

import pytest
import torch

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
