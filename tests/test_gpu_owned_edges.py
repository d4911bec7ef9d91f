"""Rows that have weights of their own, at the edges: plans rewritten behind calls without work, memory around
outputs and workspaces, what each part of a sum carries, choices by a biased score."""

import numpy as np
import pytest

from tests import owned_reference as ref
from tests.test_gpu_guard import Guarded

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


# -- choices by a biased score ------------------------------------------------------------------------

EPS = 2.0 ** -24


def scores(logits, bias, sigmoid):
    """What the bias is added to in 64 bits, the score, how far binary32's steps may be off it, and which experts may be chosen.
    The exponential is within 2 units (2^-22 of its value), its argument of a softmax rounded once (2^-24 of its size), a sum over
    E values takes E/32 + 5 roundings, the sum with one, a quotient and the sum with the bias one each; below binary32's range
    2^-126."""
    with np.errstate(all="ignore"):
        live = (logits > -np.inf) & (logits + bias > -np.inf)
        if sigmoid:
            p = 1 / (1 + np.exp(-logits))
            err = p * (2.0 ** -22 + 2 * EPS)
        else:
            far = np.minimum(np.abs(logits - np.where(live, logits, -np.inf).max(1, keepdims=True)), 110)
            e = np.where(live, np.exp(-far), 0)
            total = e.sum(1, keepdims=True)
            p = e / total
            spread = (e * far).sum(1, keepdims=True) / total
            err = p * ((far + spread) * EPS + 2 * 2.0 ** -22 + (logits.shape[1] / 32 + 7) * EPS)
        score = p + bias
        return score, err + np.abs(score) * EPS + 2.0 ** -126, live & (score > -np.inf)


def check_scored(i2s, logits, k, bias, factor=1.0, sigmoid=False, norm=False):
    call = i2s.RouteTopk(logits, k, bias=dev(bias), bias_on="score", factor=factor, sigmoid=sigmoid, norm=norm)
    call.expert.fill_(77)
    call()
    values = logits.double().cpu().numpy()
    got, weight = call.expert.cpu().numpy(), call.weight.double().cpu().numpy()
    score, err, live = scores(values, bias.astype(np.float64), sigmoid)
    rows, experts = values.shape
    assert ((got >= 0).sum(1) == np.minimum(live.sum(1), k)).all()
    left, at = live.copy(), np.arange(rows)
    for j in range(k):
        e, has = got[:, j], got[:, j] >= 0
        assert (has | ~left.any(1)).all()
        assert left[at[has], e[has]].all()   # live, and not chosen before
        best = np.where(left, score - err, -np.inf).max(1)
        assert (score[at[has], e[has]] + err[at[has], e[has]] >= best[has]).all()
        left[at[has], e[has]] = False
    # the weights are those of the chosen, without the bias
    masked = np.where((values > -np.inf) & (values + bias > -np.inf), values, -np.inf)
    v = np.where(got >= 0, np.take_along_axis(values, np.maximum(got, 0), 1), -np.inf)
    with np.errstate(all="ignore"):
        if sigmoid:
            want = 1 / (1 + np.exp(-v))
            want = want / want.sum(1, keepdims=True) if norm else want
            size = 0
        else:
            base = v if norm else masked
            top = base.max(1, keepdims=True)
            want, size = np.exp(v - top) / np.exp(base - top).sum(1, keepdims=True), np.where(got >= 0, np.abs(v - top), 0)
    want = np.where(got >= 0, want * factor, 0)
    bound = 2 * (size + experts / 32 + k + 24) * EPS * np.abs(want) + 2.0 ** -126
    assert (np.abs(weight - want) <= bound).all()
    start, items = ref.plan(got.reshape(-1), experts)
    assert call.plan.start.cpu().tolist() == start.tolist()
    assert call.plan.list.cpu().tolist()[:len(items)] == items.tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,experts,k", [(1, 8, 2), (7, 33, 4), (48, 128, 8), (130, 60, 16), (300, 256, 8), (65, 1000, 16), (1003, 60, 4)])
def test_route_by_biased_score(i2s, dtype, rows, experts, k):
    rng = np.random.default_rng(rows + experts)
    logits = dev(rng.normal(0, 2, (rows, experts)), dtype)
    for scale in (0.3, 0.01):
        bias = rng.normal(0, scale, experts).astype(np.float32)
        for sigmoid in (False, True):
            for norm in (False, True):
                check_scored(i2s, logits, k, bias, 2.5 if norm else 1.0, sigmoid, norm)


@pytest.mark.parametrize("sigmoid,logits,bias", [(True, [4.0, 1.0], [0.0, 0.5]), (False, [2.0, 1.0], [0.0, 0.5])])
def test_route_where_the_two_choices_differ(i2s, sigmoid, logits, bias):
    """By hand: sigmoid 0.982 + 0 and 0.731 + 0.5; softmax 0.731 + 0 and 0.269 + 0.5. The logits with the bias say the first
    expert, the scores the second."""
    x, b = dev(np.array([logits], np.float32)), dev(np.array(bias, np.float32))
    by = {on: i2s.route_topk(x, 1, bias=b, bias_on=on, sigmoid=sigmoid) for on in ("logit", "score")}
    assert by["logit"][0].tolist() == [[0]] and by["score"][0].tolist() == [[1]]
    want = 1 / (1 + np.exp(-1.0)) if sigmoid else np.exp(1) / (np.exp(2) + np.exp(1))
    assert abs(by["score"][1].item() - want) < 1e-6
    assert by["score"][2].start.tolist() == [0, 0, 1]


@pytest.mark.parametrize("rows", [6, 200])
def test_route_by_biased_score_masks_and_ties(i2s, rows):
    rng = np.random.default_rng(5)
    x = rng.normal(0, 1, (rows, 40)).astype(np.float32)
    x[0], x[1], x[2, 3:], x[3] = -np.inf, np.nan, -np.inf, 0.5
    x[4] = np.linspace(-120, 120, 40)
    bias = rng.normal(0, 0.2, 40).astype(np.float32)
    bias[5], bias[6] = -np.inf, np.nan
    for sigmoid in (False, True):
        for norm in (False, True):
            check_scored(i2s, dev(x), 4, bias, sigmoid=sigmoid, norm=norm)
            zero = i2s.route_topk(dev(x), 4, bias=torch.zeros(40, device="cuda"), bias_on="score", sigmoid=sigmoid, norm=norm)
            assert zero[0][3].tolist() == [0, 1, 2, 3]   # equal scores, by index
            none = i2s.route_topk(dev(x), 4, bias_on="score", sigmoid=sigmoid, norm=norm)   # no bias: by the logits
            assert torch.equal(none[0], i2s.route_topk(dev(x), 4, sigmoid=sigmoid, norm=norm)[0])
    x[5, 7] = np.inf
    e, w, _ = i2s.route_topk(dev(x), 4, bias=dev(bias), bias_on="score")
    assert e[5].tolist() == [-1] * 4 and (w[5] == 0).all() and torch.isfinite(w).all()
    e, w, _ = i2s.route_topk(dev(x), 4, bias=torch.zeros(40, device="cuda"), bias_on="score", sigmoid=True)
    assert e[5, 0].item() == 7 and w[5, 0].item() == 1


@pytest.mark.parametrize("bias_on", ["logit", "score"])
def test_route_sigmoids_far_below_zero(i2s, bias_on):
    """Normed sigmoids of logits from which exp(-l) is beyond binary32: their quotients are ordinary numbers. By hand: chosen
    -88 and -89.5 weigh 1 / (1 + exp(-1.5)) = 0.818 and 0.182; below -104 all are zero."""
    x = torch.tensor([[-88.0, -89.5, -95.0], [-95.0, -95.0, -200.0], [-103.0, -102.0, -1000.0], [-60.0, -89.0, -120.0],
                      [3.0, -89.0, -1.0], [-79.0, -81.0, -83.0], [0.0, -90.0, -90.0], [-200.0, -300.0, -float("inf")]], device="cuda")
    for dtype, k, n in ((torch.float32, 2, 1), (torch.float32, 3, 40), (torch.bfloat16, 3, 1)):
        rows = x.repeat(n, 1).to(dtype)
        e, w, _ = i2s.route_topk(rows, k, sigmoid=True, norm=True, factor=2.0, bias=torch.zeros(3, device="cuda"), bias_on=bias_on)
        v = rows.double().cpu().gather(1, e.long().clamp(min=0).cpu())
        s = torch.where(e.cpu() >= 0, 1 / (1 + torch.exp(-v)), 0)
        best = torch.where(e.cpu() >= 0, v, -1e30).max(1, keepdim=True).values.clamp(max=0)
        zero = torch.exp(best).float() == 0   # in binary32
        want = torch.where(zero, 0, 2 * s / s.sum(1, keepdim=True))
        # the difference of two logits is rounded once, two exponentials within 2 units, three sums, two quotients
        err = (w.double().cpu() - want).abs()
        assert (err <= want * ((v - best).abs() * EPS + 2.0 ** -20) * 2 + 2.0 ** -126).all(), (err, want)
    a, b = i2s.route_topk(x[:1], 2, sigmoid=True, norm=True)[1][0].tolist()
    assert abs(a - 0.8175745) < 1e-6 and abs(b - 0.1824255) < 1e-6


def test_router_sees_the_bias_and_the_weights_of_the_launch_before(i2s):
    """A bias, owners and a sum's weights that are rewritten right before each call, many times without a wait between."""
    n, rows, E, N, K = 60, 300, 24, 64, 64
    rng = np.random.default_rng(1)
    x, biases = torch.zeros((rows, E), device="cuda"), dev(rng.permuted(np.tile(np.arange(E, dtype=np.float32), (n, 1)), axis=1))
    owners, gates = dev(rng.integers(0, E, (n, 5000)).astype(np.int32)), dev(rng.integers(1, 9, (n, rows, 1)).astype(np.float32))
    bias, owner, gate = torch.empty(E, device="cuda"), torch.empty(5000, dtype=torch.int32, device="cuda"), torch.empty((rows, 1), device="cuda")
    wq, bscale = torch.full((E, N, K), 1, dtype=torch.int8, device="cuda"), torch.ones((E, N), device="cuda")
    ones = torch.ones((rows, K), device="cuda")
    route, build = i2s.RouteTopk(x, 1, bias=bias), i2s.RouteBuild(owner, E)
    total = i2s.W8A8Experts(wq, bscale, route.plan, ones, weight=gate)
    unit = i2s.w8a8_mul_mat_experts(wq, bscale, i2s.route_plan(torch.zeros(rows, dtype=torch.int32, device="cuda"), E), ones)[0, 0]
    seen = []
    for i in range(n):
        bias.copy_(biases[i])
        owner.copy_(owners[i])
        gate.copy_(gates[i])
        route()
        total()
        build()
        seen.append((route.expert.clone(), total.out.clone(), build.plan.start.clone()))
    for i, (e, y, start) in enumerate(seen):
        assert (e == biases[i].argmax()).all()
        assert torch.equal(y, (gates[i] * unit).expand(rows, N))
        assert start.diff().tolist() == torch.bincount(owners[i].long(), minlength=E).tolist()


# -- guard bands around outputs and workspaces ---------------------------------------------------------

@pytest.mark.parametrize("rows,experts,k", [(1, 8, 2), (48, 33, 4), (131, 60, 3), (700, 1000, 5), (2049, 128, 8)])
def test_router_and_plans_stay_in_their_buffers(i2s, rows, experts, k):
    rng = np.random.default_rng(rows)
    logits = dev(rng.normal(0, 1, (rows, experts)).astype(np.float32))
    logits[rows // 2, 1:] = -np.inf
    items = rows * k
    g = {"expert": Guarded(4 * items), "weight": Guarded(4 * items), "start": Guarded(4 * (experts + 1)), "list": Guarded(4 * items),
         "ws": Guarded(i2s.lib.route_plan_workspace(items, experts))}
    i32 = lambda n: g[n].buf.view(torch.int32)
    plan = i2s.RoutePlan(items, experts, start=i32("start"), list=i32("list"))
    for bias, bias_on in ((None, "logit"), (torch.zeros(experts, device="cuda"), "score")):
        i2s.route_topk(logits, k, bias=bias, bias_on=bias_on, plan=plan, ws=g["ws"].buf, expert=i32("expert"), weight=g["weight"].f32(items))
        owner = i32("expert").clone()
        want = ref.plan(owner.cpu().numpy(), experts)
        for _ in range(2):   # the router's plan, then that of its experts
            assert plan.start.cpu().tolist() == want[0].tolist()
            assert plan.list.cpu().tolist()[:len(want[1])] == want[1].tolist()
            i2s.route_plan(owner, experts, plan=plan, ws=g["ws"].buf)
        for name, buf in g.items():
            buf.check(f"{name}, {rows} rows of {experts} experts")


@pytest.mark.parametrize("rows,k,E,N,K", [(1, 2, 8, 64, 48), (70, 3, 5, 160, 1040), (9, 1, 3, 96, 16), (600, 4, 7, 288, 208),
                                          (520, 8, 16, 64, 2064)])
@pytest.mark.parametrize("form", ["plain", "up", "down", "rows"])
def test_expert_products_stay_in_their_buffers(i2s, rows, k, E, N, K, form):
    """up: gate and up; down: weighted sums of rows of their own; rows: weighted sums of shared rows. The workspace is as large as
    the query says and no larger."""
    rng = np.random.default_rng(N + K)
    wq, bscale = rng.integers(-127, 128, (E, N, K)).astype(np.int8), np.exp(rng.normal(0, 0.3, (E, N))).astype(np.float32) * np.float32(1e-3)
    owner = rng.integers(-1, E, rows * k).astype(np.int32)
    x_group = 1 if form == "down" else k
    x = rng.normal(0, 1, (rows * k // x_group, K)).astype(np.float32)
    gate = rng.normal(0, 1, (rows, k)).astype(np.float32)
    weighted = form in ("down", "rows")
    plan = i2s.route_plan(dev(owner), E)
    w, d = dev(wq), ref.dots(wq, bscale, owner, x, x_group)
    struct = i2s.w8a8_experts(w.data_ptr(), w.data_ptr(), N, K, E)
    ws = Guarded(i2s.lib.w8a8_mul_mat_experts_workspace(struct, plan.struct, x_group, k if weighted else 1, 1 if form == "up" else 0))
    shape = (rows if weighted else rows * k, N // 2 if form == "up" else N)
    y = Guarded(4 * shape[0] * shape[1])
    y.buf.zero_()
    ws.buf.fill_(0xff)   # whatever it holds before
    out = i2s.w8a8_mul_mat_experts(w, dev(bscale), plan, dev(x), out=y.f32(*shape), x_group=x_group, swiglu=form == "up",
                                   weight=dev(gate) if weighted else None, ws=ws.buf)
    y.check("y")
    ws.check("workspace")
    got = out.cpu().numpy()
    if form == "up":
        want = np.where((owner >= 0)[:, None], ref.swiglu(d), 0)
        assert (np.abs(got - want) <= 2.0 ** -20 * np.abs(want) + ref.swiglu_floor(d)).all()
    else:
        want = ref.weighted(d, owner, E, gate) if weighted else d
        assert np.array_equal(got, want)


@pytest.mark.parametrize("rows,adapters,rank,N,K", [(1, 1, 8, 33, 72), (64, 40, 32, 300, 520), (131, 3, 128, 511, 2056), (700, 5, 64, 264, 136)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_adapters_stay_in_their_buffers(i2s, rows, adapters, rank, N, K, dtype):
    rng = np.random.default_rng(rank)
    half = torch.float16 if dtype == torch.float16 else torch.bfloat16
    A, B = dev(rng.integers(-1, 2, (adapters, rank, K)), half), dev(rng.integers(-1, 2, (adapters, N, rank)), half)
    x, base = dev(rng.integers(-1, 2, (rows, K)), dtype), dev(rng.integers(-8, 9, (rows, N)), dtype)
    owner = dev(rng.integers(-1, adapters, rows).astype(np.int32))
    plan = i2s.route_plan(owner, adapters)
    struct = i2s.lora_adapters(A.data_ptr(), B.data_ptr(), None, K, N, rank, adapters, 1 if half == torch.float16 else 2)
    ws, out = Guarded(i2s.lib.lora_add_workspace(struct, plan.struct)), Guarded(x.element_size() * rows * N)
    y = out.buf.view(dtype).view(rows, N)
    y.fill_(3)
    ws.buf.fill_(0xff)
    i2s.lora_add(A, B, plan, x, base, out=y, ws=ws.buf)
    out.check("out")
    ws.check("workspace")
    for a in range(-1, adapters):
        at = owner == a
        # whole numbers: every sum is exact in 32 bits, and rounded once
        want = base[at].double() + (x[at].double() @ A[a].double().T) @ B[a].double().T if a >= 0 else torch.full_like(y[at], 3).double()
        assert torch.equal(y[at], want.float().to(dtype))


# -- what the parts of an adapter's F32 rows carry -----------------------------------------------------

def full_values(rows, K, seed):
    """F32 values with 24 bits each, of many sizes."""
    rng = np.random.default_rng(seed)
    m = rng.integers(1 << 23, 1 << 24, (rows, K)) | 1
    return (m * np.exp2(rng.integers(-60, 30, (rows, K))) * rng.choice([-1, 1], (rows, K))).astype(np.float32)


def three_bytes(rows, seed):
    """Rows of three whole numbers of 8 bits each, 2^16 a + 2^8 b + c, whose sum has 24."""
    rng = np.random.default_rng(seed)
    v = rng.integers(128, 256, (rows, 3)) | 1
    return (v * np.array([1 << 16, 1 << 8, 1]) * rng.choice([-1, 1], (rows, 1))).astype(np.float32)


def in_parts(x, parts):
    """The sum of a value's bf16 parts, high bits first, each cut off."""
    left, total = x.astype(np.float32), np.zeros_like(x, np.float64)
    for _ in range(parts):
        part = (left.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
        total, left = total + part, (left - part).astype(np.float32)
    return total


@pytest.mark.parametrize("rank", [8, 32, 64, 128])
@pytest.mark.parametrize("rows", [1, 50, 3000])
def test_lora_rows_and_inner_vector_keep_24_bits(i2s, rank, rows):
    """A and B pick one value each (a power of two): out is x's value bit for bit, through the parts of x and of the inner vector;
    then a sum of three positions of 8 bits, which only the inner vector holds in 24."""
    K, N, adapters = 520, 264, 3
    rng = np.random.default_rng(rank + rows)
    own = rng.integers(0, adapters, rows).astype(np.int32)
    plan = i2s.route_plan(dev(own), adapters)
    at = rng.integers(0, K, (adapters, rank))
    A, B = np.zeros((adapters, rank, K), np.float32), np.zeros((adapters, N, rank), np.float32)
    for a in range(adapters):
        A[a, np.arange(rank), at[a]] = 4
        B[a, np.arange(N), np.arange(N) % rank] = 0.5
    x = full_values(rows, K, rank)
    zero = torch.zeros((rows, N), device="cuda")
    out = i2s.lora_add(dev(A).bfloat16(), dev(B).bfloat16(), plan, dev(x), zero, out=torch.empty_like(zero)).cpu().numpy()
    want = 2 * x[np.arange(rows)[:, None], at[own][:, np.arange(N) % rank]]
    assert np.array_equal(out, want)
    for a in range(adapters):
        A[a] = 0
        A[a, :, 100:103] = 1
    x = np.zeros((rows, K), np.float32)
    x[:, 100:103] = three_bytes(rows, rank)
    out = i2s.lora_add(dev(A).bfloat16(), dev(B).bfloat16(), plan, dev(x), zero, out=torch.empty_like(zero)).cpu().numpy()
    assert np.array_equal(out, np.repeat(x.sum(1, keepdims=True) * np.float32(0.5), N, 1))


@pytest.mark.parametrize("rows,K,steps", [(3000, 2048, 8), (3000, 8960, 35), (64, 65536, 32)])
@pytest.mark.parametrize("rank", [16, 64])
def test_lora_long_sums_of_one_sign(i2s, rows, K, steps, rank):
    """t over long K, all products positive, B picking one of t. Of 32 positions six MMAs cut off up to 5 units of 2^-24 each;
    a warp then adds `steps` such sums, a CTA eight warps', up to eight CTAs theirs, each rounded: (30 + steps + 16) * 2^-24 of t.
    One chain over all of K lost 1.2e-5 of the two longer ones."""
    adapters, N = 4, 264
    g = torch.Generator(device="cuda").manual_seed(K)
    A = torch.rand(adapters, rank, K, device="cuda", generator=g).bfloat16()
    x = torch.rand(rows, K, device="cuda", generator=g)
    own = torch.randint(0, adapters, (rows,), device="cuda", generator=g, dtype=torch.int32)
    B = torch.zeros(adapters, N, rank, device="cuda")
    B[:, torch.arange(N), torch.arange(N) % rank] = 1
    zero = torch.zeros(rows, N, device="cuda")
    out = i2s.lora_add(A, B.bfloat16(), i2s.route_plan(own, adapters), x, zero, out=torch.empty_like(zero))
    for a in range(adapters):
        at = own == a
        t = (x[at].double() @ A[a].double().T)[:, torch.arange(N) % rank]
        err = (out[at].double() - t).abs() / t
        assert err.max() <= (30 + steps + 16) * 2.0 ** -24, err.max().item() * 2 ** 24


def test_lora_rows_that_are_not_finite_stay_alone(i2s):
    """An infinity or NaN in a row of x, or an inner product beyond binary32, makes that row NaN, and no other."""
    rows, K, N = 40, 64, 96
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        half = torch.float16 if dtype == torch.float16 else torch.bfloat16
        A, B = torch.ones(2, 16, K, device="cuda").to(half), torch.ones(2, N, 16, device="cuda").to(half)
        x = torch.ones(rows, K, device="cuda", dtype=dtype)
        x[3, 5], x[20, 60], x[21, 0] = float("nan"), float("inf"), -float("inf")
        bad = [3, 20, 21]
        if dtype != torch.float16:
            x[33] = torch.finfo(dtype).max
            bad.append(33)
        own = torch.arange(rows, device="cuda", dtype=torch.int32) % 2
        out = i2s.lora_add(A, B, i2s.route_plan(own, 2), x, torch.zeros(rows, N, device="cuda", dtype=dtype))
        fine = torch.ones(rows, dtype=torch.bool)
        fine[bad] = False
        assert (out.cpu()[fine] == 16 * K).all() and torch.isnan(out.cpu()[~fine]).all()


def test_experts_status_on_another_device_is_refused(i2s):
    """A check while another device is current would wait for that device's stream and read too early."""
    wq, bscale = torch.ones((2, 32, 16), dtype=torch.int8, device="cuda"), torch.ones((2, 32), device="cuda")
    plan = i2s.route_plan(torch.zeros(3, dtype=torch.int32, device="cuda"), 2)
    call = i2s.W8A8Experts(wq, bscale, plan, torch.ones((3, 16), device="cuda"))
    call()
    call.check()
    call._index += 1   # as if its tensors were on the next device
    for use in (call, call.check):
        with pytest.raises(ValueError, match="not on the current device"):
            use()


# -- rows whose places pass 32 bits --------------------------------------------------------------------

def test_rows_far_apart(i2s):
    """Row tensors that reach over more than 2^31 elements: slices of rows 32768 apart, the last of 70001 as right as the first."""
    rows, far, E, N, K = 70001, 32768, 4, 32, 32
    frames = [torch.empty((rows, far), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(3)
    whole = lambda *shape, low, high: torch.randint(low, high, shape, device="cuda", generator=g).float()
    logits, x, out = frames[0][:, 1024:1024 + E], frames[0][:, :K], frames[1][:, 64:64 + N]
    logits.copy_(torch.rand((rows, E), device="cuda", generator=g).argsort(1))   # no two alike
    expert, weight, plan = i2s.route_topk(logits, 2, norm=True)
    own = logits.float().argmax(1)
    assert torch.equal(expert[:, 0].long(), own) and (weight[:, 0] - 1 / (1 + np.exp(-1.0))).abs().max() < 1e-6
    assert plan.start[-1] == 2 * rows
    one = i2s.route_plan(expert[:, 0].contiguous(), E)
    # experts: codes are the values where the largest of a row is 127
    x.copy_(whole(rows, K, low=-100, high=101))
    x[:, 0] = 127
    wq, ones = whole(E, N, K, low=-2, high=3).to(torch.int8), torch.ones((E, N), device="cuda")
    out.fill_(0)
    i2s.w8a8_mul_mat_experts(wq, ones, one, x, out=out)
    want = torch.einsum("rk,rnk->rn", x.float(), wq.float()[own])
    assert torch.equal(out, want.bfloat16())
    # adapters, in place
    A, B = whole(E, 8, K, low=-1, high=2).bfloat16(), whole(E, N, 8, low=-1, high=2).bfloat16()
    x.copy_(whole(rows, K, low=-2, high=3))
    base = whole(rows, N, low=-9, high=10)
    out.copy_(base)
    i2s.lora_add(A, B, one, x, out)
    t = torch.einsum("rk,rak->ra", x.float(), A.float()[own])
    want = base + torch.einsum("ra,rna->rn", t, B.float()[own])
    assert torch.equal(out, want.bfloat16())
