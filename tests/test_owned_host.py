"""route_*, w8a8_mul_mat_experts and lora_add on the host (no GPU): sizes, and every refusal before any CUDA call.

Addresses are made up: the file runs only where there is no GPU to launch on."""

import ctypes

import pytest
import torch

from int8_quantized_matmul_gb300 import build as libbuild

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")
A = 1 << 40   # dummy addresses, never dereferenced


@pytest.fixture(scope="module")
def i2s():
    libbuild.build()
    from int8_quantized_matmul_gb300 import i2s as mod
    return mod


class Call:
    """Valid arguments of the calls, to be spoiled one at a time."""

    def __init__(self, i2s):
        self.L = i2s.lib
        self.E = {v: k for k, v in i2s.STATUS.items()}
        self.plan = i2s.route_plan_t(A, 2 * A, 20, 4)
        self.owner, self.ws, self.ws_bytes = 3 * A, 4 * A, 1 << 40
        # router: 10 rows, 4 experts, 2 of them
        self.logits = i2s.i2s_rows(5 * A, 4, 0)
        self.rows, self.experts, self.k, self.bias, self.factor, self.flags = 10, 4, 2, None, 1.0, 0
        self.expert, self.weight = 6 * A, 7 * A
        # products: 20 items, two to a row of x
        self.w = i2s.w8a8_experts(8 * A, 9 * A, 64, 48, 4)
        self.x, self.y = i2s.i2s_rows(10 * A, 48, 0), i2s.i2s_rows(11 * A, 64, 0)
        self.x_group, self.y_group, self.gate = 2, 1, None
        # adapters: 20 rows
        self.a = i2s.lora_adapters(12 * A, 13 * A, 14 * A, 64, 30, 8, 4, 2)
        self.lx, self.base, self.out = i2s.i2s_rows(15 * A, 64, 0), i2s.i2s_rows(16 * A, 30, 0), i2s.i2s_rows(17 * A, 30, 0)

    def build(self):
        return self.L.route_plan_build(self.owner, self.plan, self.ws, self.ws_bytes, None)

    def topk(self):
        return self.L.route_topk(self.logits, self.rows, self.experts, self.k, self.bias, self.factor, self.flags, self.expert,
                                 self.weight, self.plan, self.ws, self.ws_bytes, None)

    def product(self):
        return self.L.w8a8_mul_mat_experts(self.w, self.plan, self.x, self.x_group, self.y, self.gate, self.y_group, self.flags,
                                           self.ws, self.ws_bytes, None)

    def lora(self):
        return self.L.lora_add(self.a, self.plan, self.lx, self.base, self.out, self.ws, self.ws_bytes, None)


def spoil(c, path, value):
    *parts, last = path.split(".")
    for p in parts:
        c = getattr(c, p)
    setattr(c, last, value)


def refused(i2s, name, cases):
    for want, *changes in cases:
        c = Call(i2s)
        for path, value in changes:
            spoil(c, path, value)
        assert getattr(c, name)() == c.E["I2S_E_" + want], (want, changes)


def test_valid_calls_reach_the_device_check(i2s):
    for name in ("build", "topk", "product", "lora"):
        c = Call(i2s)
        assert getattr(c, name)() in (c.E["I2S_E_CUDA"], c.E["I2S_E_UNSUPPORTED_DEVICE"]), name


PLAN = [("NULL_PTR", ("plan", None)), ("NULL_PTR", ("plan.start", None)), ("NULL_PTR", ("plan.list", None)),
        ("BAD_SHAPE", ("plan.items", 0)), ("BAD_SHAPE", ("plan.items", (1 << 27) + 1)), ("BAD_SHAPE", ("plan.owners", 0)),
        ("BAD_SHAPE", ("plan.owners", 1025)), ("MISALIGNED", ("plan.start", A + 2)), ("MISALIGNED", ("plan.list", A + 1)),
        ("NULL_PTR", ("ws", None)), ("MISALIGNED", ("ws", 4 * A + 128)), ("WORKSPACE_TOO_SMALL", ("ws_bytes", 255))]


@pytest.mark.parametrize("name", ["build", "topk", "product", "lora"])
def test_plan_and_workspace_refusals(i2s, name):
    cases = PLAN[1:] if name == "topk" else PLAN   # a router needs no plan
    refused(i2s, name, cases)


def test_build_refusals(i2s):
    refused(i2s, "build", [
        ("NULL_PTR", ("owner", None)), ("MISALIGNED", ("owner", 3 * A + 2)), ("BAD_ARG", ("owner", A + 16)),
        ("BAD_ARG", ("owner", 2 * A + 76)), ("BAD_ARG", ("plan.list", A + 16)), ("BAD_ARG", ("ws", 3 * A)), ("BAD_ARG", ("ws", A)),
        ("BAD_ARG", ("plan.list", 4 * A + 1020))])
    assert i2s.lib.route_plan_workspace(20, 4) >= 256
    for items, owners in ((0, 4), (-1, 4), ((1 << 27) + 1, 4), (20, 0), (20, 1025)):
        assert i2s.lib.route_plan_workspace(items, owners) == 0


def test_topk_refusals(i2s):
    refused(i2s, "topk", [
        ("BAD_SHAPE", ("rows", 0)), ("BAD_SHAPE", ("experts", 0)), ("BAD_SHAPE", ("experts", 1025)), ("BAD_SHAPE", ("k", 0)),
        ("BAD_SHAPE", ("k", 5)), ("BAD_SHAPE", ("rows", (1 << 26) + 1)), ("BAD_SHAPE", ("rows", 11)), ("BAD_SHAPE", ("k", 3)),
        ("BAD_SHAPE", ("plan.owners", 5)), ("NULL_PTR", ("expert", None)), ("NULL_PTR", ("weight", None)),
        ("NULL_PTR", ("logits.data", None)), ("NULL_PTR", ("logits", None)), ("BAD_ARG", ("logits.dtype", 3)),
        ("BAD_ARG", ("logits.dtype", -1)), ("BAD_SHAPE", ("logits.stride", -4)), ("BAD_SHAPE", ("logits.stride", 1 << 38)),
        ("MISALIGNED", ("logits.data", 5 * A + 2)), ("BAD_ARG", ("flags", 4)), ("BAD_ARG", ("factor", float("inf"))),
        ("BAD_ARG", ("factor", float("nan"))), ("MISALIGNED", ("bias", A + 2)), ("MISALIGNED", ("expert", 6 * A + 2)),
        ("MISALIGNED", ("weight", 7 * A + 1)), ("BAD_ARG", ("expert", 5 * A + 156)), ("BAD_ARG", ("weight", 6 * A + 76)),
        ("BAD_ARG", ("plan.start", 7 * A + 76)), ("BAD_ARG", ("plan.list", 5 * A)), ("BAD_ARG", ("ws", 6 * A)),
        ("BAD_ARG", ("bias", 6 * A))])
    c = Call(i2s)
    c.plan = c.ws = None   # neither is needed without the other
    assert c.topk() in (c.E["I2S_E_CUDA"], c.E["I2S_E_UNSUPPORTED_DEVICE"])
    c = Call(i2s)
    c.experts = c.plan.owners = 1000
    c.logits.stride, c.k, c.rows = 1000, 17, 1
    c.plan.items = 17
    assert c.topk() == c.E["I2S_E_BAD_SHAPE"]


def test_product_refusals(i2s):
    refused(i2s, "product", [
        ("NULL_PTR", ("w", None)), ("NULL_PTR", ("w.wq", None)), ("NULL_PTR", ("w.bscale", None)), ("BAD_SHAPE", ("w.N", 0)),
        ("BAD_SHAPE", ("w.N", 1 << 29)), ("BAD_SHAPE", ("w.K", 0)), ("BAD_SHAPE", ("w.K", 40)), ("BAD_SHAPE", ("w.K", 65552)),
        ("BAD_SHAPE", ("w.experts", 0)), ("BAD_SHAPE", ("w.experts", 3)), ("BAD_SHAPE", ("w.experts", 1025), ("plan.owners", 1025)),
        ("BAD_SHAPE", ("x_group", 0)), ("BAD_SHAPE", ("x_group", 3)), ("BAD_SHAPE", ("y_group", 0)), ("BAD_SHAPE", ("y_group", 3)),
        ("BAD_SHAPE", ("w.N", 80), ("flags", 1)), ("BAD_ARG", ("y_group", 2)), ("BAD_ARG", ("flags", 2)),
        ("BAD_ARG", ("gate", 18 * A), ("flags", 1)), ("MISALIGNED", ("w.wq", 8 * A + 8)), ("MISALIGNED", ("w.bscale", 9 * A + 2)),
        ("MISALIGNED", ("x.data", 10 * A + 8)), ("MISALIGNED", ("x.stride", 50)), ("MISALIGNED", ("y.data", 11 * A + 2)),
        ("MISALIGNED", ("gate", 18 * A + 1)), ("NULL_PTR", ("x", None)), ("NULL_PTR", ("y.data", None)), ("BAD_ARG", ("x.dtype", 4)),
        ("BAD_ARG", ("y.dtype", -1)), ("BAD_SHAPE", ("x.stride", -48)), ("BAD_SHAPE", ("y.stride", 1 << 39)),
        ("BAD_ARG", ("y.stride", 63)), ("BAD_ARG", ("y.data", 10 * A + 16)), ("BAD_ARG", ("y.data", 8 * A + 64)),
        ("BAD_ARG", ("y.data", 9 * A)), ("BAD_ARG", ("y.data", A - 16)), ("BAD_ARG", ("y.data", 2 * A + 76)),
        ("BAD_ARG", ("y.data", 4 * A + 256)), ("BAD_ARG", ("x.data", 4 * A + 256)), ("BAD_ARG", ("w.wq", 4 * A)),
        ("BAD_ARG", ("gate", 4 * A)), ("BAD_ARG", ("gate", 11 * A + 16), ("y_group", 2)), ("BAD_ARG", ("plan.start", 4 * A + 64))])
    c = Call(i2s)
    need = lambda **kw: c.L.w8a8_mul_mat_experts_workspace(c.w, c.plan, kw.get("x_group", 2), kw.get("y_group", 1), kw.get("flags", 0))
    assert need() > 256 and need(flags=2) == 0 and need(x_group=0) == 0 and need(y_group=3) == 0
    c.ws_bytes = need() - 1
    assert c.product() == c.E["I2S_E_WORKSPACE_TOO_SMALL"]


def test_lora_refusals(i2s):
    refused(i2s, "lora", [
        ("NULL_PTR", ("a", None)), ("NULL_PTR", ("a.A", None)), ("NULL_PTR", ("a.B", None)), ("BAD_SHAPE", ("a.rank", 0)),
        ("BAD_SHAPE", ("a.rank", 12)), ("BAD_SHAPE", ("a.rank", 136)), ("BAD_SHAPE", ("a.K", 4)), ("BAD_SHAPE", ("a.K", 68)),
        ("BAD_SHAPE", ("a.K", 65544)), ("BAD_SHAPE", ("a.N", 0)), ("BAD_SHAPE", ("a.N", (1 << 24) + 1)), ("BAD_SHAPE", ("a.adapters", 5)),
        ("BAD_ARG", ("a.dtype", 0)), ("BAD_ARG", ("a.dtype", 1)), ("BAD_ARG", ("base.dtype", 2)), ("BAD_ARG", ("out.dtype", 1)),
        ("BAD_ARG", ("lx.dtype", 1)), ("MISALIGNED", ("a.A", 12 * A + 8)), ("MISALIGNED", ("a.B", 13 * A + 8)),
        ("MISALIGNED", ("a.scale", 14 * A + 2)), ("MISALIGNED", ("lx.data", 15 * A + 4)), ("MISALIGNED", ("lx.stride", 66)),
        ("MISALIGNED", ("base.data", 16 * A + 2)), ("MISALIGNED", ("out.data", 17 * A + 1)), ("NULL_PTR", ("lx", None)),
        ("NULL_PTR", ("base", None)), ("NULL_PTR", ("out.data", None)), ("BAD_SHAPE", ("base.stride", -30)),
        ("BAD_ARG", ("out.stride", 29)), ("BAD_ARG", ("out.data", 16 * A + 4)), ("BAD_ARG", ("out.data", 16 * A), ("out.stride", 31)),
        ("BAD_ARG", ("out.data", 15 * A)), ("BAD_ARG", ("out.data", 12 * A)), ("BAD_ARG", ("out.data", 13 * A + 64)),
        ("BAD_ARG", ("out.data", 14 * A)), ("BAD_ARG", ("out.data", 2 * A)), ("BAD_ARG", ("out.data", 4 * A)),
        ("BAD_ARG", ("lx.data", 4 * A)), ("BAD_ARG", ("base.data", 4 * A)), ("BAD_ARG", ("a.A", 4 * A))])
    c = Call(i2s)
    c.out = i2s.i2s_rows(16 * A, 30, 0)   # in place
    assert c.lora() in (c.E["I2S_E_CUDA"], c.E["I2S_E_UNSUPPORTED_DEVICE"])
    c = Call(i2s)
    c.ws_bytes = c.L.lora_add_workspace(c.a, c.plan) - 1
    assert c.ws_bytes > 0 and c.lora() == c.E["I2S_E_WORKSPACE_TOO_SMALL"]
    c.a.rank = 9
    assert c.L.lora_add_workspace(c.a, c.plan) == 0


def test_python_refusals(i2s):
    cpu = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        i2s.RouteBuild(cpu, 2)
    with pytest.raises(ValueError):
        i2s.RouteTopk(torch.zeros(4, 4), 2)
    with pytest.raises(ValueError):
        i2s.RoutePlan(4, 2, device="cpu")
    for items, owners in ((0, 2), (4, 0), (4, 2000), ((1 << 27) + 1, 2)):
        with pytest.raises((ValueError, i2s.I2SError)):
            i2s.RoutePlan(items, owners, device="cuda:0")


def test_structures_have_the_sizes_of_the_header(i2s):
    assert [ctypes.sizeof(t) for t in (i2s.route_plan_t, i2s.i2s_rows, i2s.w8a8_experts, i2s.lora_adapters)] == [32, 24, 40, 56]
