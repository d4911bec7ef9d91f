"""Rows that have weights of their own, at the edges: plans rewritten behind calls without work, memory around
outputs and workspaces, what each part of a sum carries, choices by a biased score."""

import numpy as np
import pytest

from tests import owned_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def i2s():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_quantized_matmul_gb300 import build as libbuild
    libbuild.build()
    from int8_quantized_matmul_gb300 import i2s as mod
    assert mod.device_supported() == 1
    return mod


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


# -- a plan without owners, and the next plan in its place -------------------------------------------

@pytest.mark.parametrize("rank", [16, 64, 128])
@pytest.mark.parametrize("graph", [False, True])
def test_lora_plan_of_nobody_then_another(i2s, rank, graph):
    """Steps whose rows all lack an adapter, alternating with others on the same plan, workspace and stream: the plan is
    rewritten right behind each call. Every output is its own plan's (small whole numbers: sums are exact)."""
    rows, adapters, N, K, steps = 200, 9, 300, 512, 40
    rng = np.random.default_rng(rank)
    A = dev(rng.integers(-1, 2, (adapters, rank, K)).astype(np.float32)).bfloat16()
    B = dev(rng.integers(-2, 3, (adapters, N, rank)).astype(np.float32)).bfloat16()
    x = dev(rng.integers(-1, 2, (rows, K)).astype(np.float32))
    owners = rng.integers(0, adapters, (steps, rows)).astype(np.int32)
    owners[::2] = -1                 # nobody
    owners[1::4, rng.random(rows) < 0.5] = -1
    owner = torch.empty(rows, dtype=torch.int32, device="cuda")
    each = dev(owners)
    outs = [torch.full((rows, N), 0.5, device="cuda") for _ in range(steps)]
    base = torch.zeros((rows, N), device="cuda")
    build = i2s.RouteBuild(owner, adapters)
    first = i2s.LoraAdd(A, B, build.plan, x, base, out=outs[0])
    calls = [first] + [i2s.LoraAdd(A, B, build.plan, x, base, out=o, ws=first.ws) for o in outs[1:]]

    def run():
        for i, call in enumerate(calls):
            owner.copy_(each[i])
            build()
            call()

    if graph:
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            run()
        run = g.replay
    for _ in range(3):
        for o in outs:
            o.fill_(0.5)
        run()
        for i, o in enumerate(outs):
            own = torch.from_numpy(owners[i]).long().cuda()
            want = torch.full((rows, N), 0.5, device="cuda")
            for a in range(adapters):
                at = own == a
                want[at] = ((x[at].double() @ A[a].double().T) @ B[a].double().T).float()
            assert torch.equal(o, want), i


# -- the two warps that issue an expert's MMAs --------------------------------------------------------

@pytest.mark.parametrize("K", [16, 128, 144, 1024, 1152, 2176, 8976])
@pytest.mark.parametrize("rows", [7, 250])
def test_experts_stages_of_both_issuers(i2s, rows, K):
    """One stage and many, odd and even counts, few rows (an accumulator for each issuer) and many (one, by turns): sums of
    one sign as large as they come, and random ones, exact and the same in every call."""
    E, N = 3, 520
    rng = np.random.default_rng(K)
    for extreme in (False, True):
        wq = np.full((E, N, K), -128, np.int8) if extreme else rng.integers(-128, 128, (E, N, K)).astype(np.int8)
        x = np.full((rows, K), 3.0, np.float32) if extreme else rng.normal(0, 1, (rows, K)).astype(np.float32)
        bscale = np.exp(rng.normal(0, 0.3, (E, N))).astype(np.float32)
        owner = rng.integers(0, E, rows).astype(np.int32)
        want = torch.from_numpy(ref.dots(wq, bscale, owner, x, 1)).cuda()
        call = i2s.W8A8Experts(dev(wq), dev(bscale), i2s.route_plan(dev(owner), E), dev(x))
        for _ in range(8):
            call.out.fill_(0)
            call()
            assert torch.equal(call.out, want)
        call.check()
