"""Router, expert products and adapters on the GPU against their definitions.

route_topk, route_plan_build: experts, starts and lists are equal. Weights: the softmax's
argument is rounded once (2^-24 of its size A, which its exponential has as a relative error),
the exponential is within 2 units of its last place (2^-22), a sum over E values in 32 lanes takes
E/32 + 5 roundings of 2^-24 each, the quotient and factor two more: relative (A + E/32 + 16) * 2^-24, and
twice the sum's for the quotient. A sigmoid's: 2^-22, two roundings, with ROUTE_NORM k + 8 more.

w8a8_mul_mat_experts: every step is one of binary32, the dot exact, so outputs are compared
bit for bit, rounded once to their dtype. With SWIGLU the exponential is within 2 units, then a sum, a
quotient and a product: relative 2^-20, and half a step of the dtype.

lora_add: the tensor core cuts sums off, at most 5 units of 2^-24 of the absolute sum for each MMA: 3 K/16
of them for t and 3 rank/16 for the outer product, fewer where the warps share them; 2^-22 of the absolute sums
for each, and 16 roundings more. Parts of t: exact with F32 rows, 2^-17 with bf16 (8 bits and their sign twice), 2^-21 with f16.
Then the product with the scale and the sum with base, two roundings of 2^-24 of base and the absolute sum, and half a step.
"""

import numpy as np
import pytest

from tests import owned_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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


def f64(t):
    return t.double().cpu().numpy()


def check_plan(plan, owner, owners):
    start, items = ref.plan(owner, owners)
    assert plan.start.cpu().tolist() == start.tolist()
    assert plan.list.cpu().tolist()[:len(items)] == items.tolist()


# -- plans and the router ---------------------------------------------------------------------------

@pytest.mark.parametrize("items,owners", [(1, 1), (2, 1024), (31, 3), (33, 7), (1000, 60), (4096, 128), (4097, 128),
                                          (5000, 1000), (70001, 257), (65536, 1), (100003, 1024)])
def test_plan(i2s, items, owners):
    rng = np.random.default_rng(items)
    owner = rng.integers(-2, owners + 1, items).astype(np.int32)   # some of none
    if items > 100:
        owner[10:60] = 0   # a run
    plan = i2s.RoutePlan(items, owners)
    plan.list.fill_(-7)
    i2s.route_plan(dev(owner), owners, plan=plan)
    check_plan(plan, owner, owners)
    here = int(((owner >= 0) & (owner < owners)).sum())
    assert (plan.list[here:] == -7).all()   # places behind the last are left as they were


def test_plan_of_nobody_and_of_one(i2s):
    for value, n in ((-1, 50), (-2 ** 31, 5000), (9, 5000), (3, 5000)):
        owner = np.full(n, value, np.int32)
        check_plan(i2s.route_plan(dev(owner), 9), owner, 9)


MODES = [dict(), dict(norm=True), dict(sigmoid=True), dict(sigmoid=True, norm=True)]


def check_route(i2s, logits, k, bias=None, factor=1.0, **mode):
    call = i2s.RouteTopk(logits, k, bias=None if bias is None else dev(bias), factor=factor, **mode)
    call.expert.fill_(77)
    call()
    rows, experts = logits.shape
    values = f64(logits)
    expert, weight = ref.topk(values, k, bias, factor, **mode)
    assert np.array_equal(call.expert.cpu().numpy(), expert)
    top = np.where(np.isfinite(values), values, -1e30).max(1, keepdims=True)
    at = np.where(expert >= 0, np.take_along_axis(values, np.maximum(expert, 0), 1), 0)
    size = np.abs(at - (at.max(1, keepdims=True) if mode.get("norm") else top))
    bound = 2 * ((0 if mode.get("sigmoid") else size) + experts / 32 + k + 24) * 2.0 ** -24 * np.abs(weight) + 2.0 ** -126
    got = f64(call.weight)
    same = np.isnan(weight) & np.isnan(got)
    assert (same | (np.abs(got - weight) <= bound)).all(), np.nanmax(np.abs(got - weight) - bound)
    check_plan(call.plan, expert.reshape(-1), experts)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,experts,k", [(1, 8, 2), (1, 1, 1), (7, 33, 4), (32, 128, 8), (128, 60, 16), (129, 60, 6),
                                            (300, 256, 8), (65, 1000, 16), (1003, 1024, 3), (4000, 129, 8)])
def test_route(i2s, dtype, rows, experts, k):
    rng = np.random.default_rng(rows + experts)
    logits = dev(rng.normal(0, 2, (rows, experts)), DTYPES[dtype])   # 16 bits: many equal ones
    bias = rng.normal(0, 0.5, experts).astype(np.float32)
    for i, mode in enumerate(MODES):
        check_route(i2s, logits, k, bias if i % 2 == rows % 2 else None, 1.0 if i < 2 else 2.5, **mode)


@pytest.mark.parametrize("rows", [5, 200])
def test_route_masks_ties_and_infinities(i2s, rows):
    rng = np.random.default_rng(3)
    x = rng.normal(0, 1, (rows, 40)).astype(np.float32)
    x[0] = -np.inf                      # nothing left
    x[1] = np.nan
    x[2, 3:] = -np.inf                  # fewer than k
    x[3] = 0.5                          # all equal
    x[3, ::2] = -0.0
    x[3, 1::4] = 0.0                    # equal to -0.0
    x[4] = np.finfo(np.float32).min     # the lowest value is a value
    bias = np.zeros(40, np.float32)
    bias[5] = -np.inf                   # an expert taken out of service
    bias[6] = np.nan
    for mode in MODES:
        check_route(i2s, dev(x), 4, **mode)
        check_route(i2s, dev(x), 4, bias, **mode)
    x[0, 7] = x[0, 9] = np.inf
    call = i2s.RouteTopk(dev(x), 4)
    call()
    assert call.expert[0].tolist() == [7, 9, -1, -1]   # the rest of the row is -infinity
    assert torch.isnan(call.weight[0, :2]).all() and (call.weight[0, 2:] == 0).all()
    assert torch.isfinite(call.weight[1:]).all()


def test_route_strided_logits_and_no_plan(i2s):
    wide = torch.randn(500, 100, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).half()
    part = wide[:, 3:64]
    check_route(i2s, part, 5, norm=True)
    for rows in (1, 100, 500):
        e, w, plan = i2s.route_topk(part[:rows], 5, norm=True, plan=False)
        want, _ = ref.topk(f64(part[:rows]), 5, norm=True)
        assert plan is None and np.array_equal(e.cpu().numpy(), want)


# -- expert products --------------------------------------------------------------------------------

class Experts:
    def __init__(self, E, N, K, rows, k, seed=0, none=0.0, skew=None, extreme=False):
        rng = np.random.default_rng(seed)
        self.E, self.N, self.K, self.rows, self.k = E, N, K, rows, k
        self.wq = np.clip(np.rint(rng.normal(0, 40, (E, N, K))), -127, 127).astype(np.int8)
        self.bscale = np.exp(rng.normal(0, 0.3, (E, N))).astype(np.float32) * np.float32(0.001)
        self.x = rng.normal(0, 1, (rows, K)).astype(np.float32)
        if extreme:   # the largest sums there are, of one sign
            self.wq[:] = -128
            self.x = np.full((rows, K), 3.0, np.float32)
        p = np.full(E, 1.0 / E) if skew is None else np.asarray(skew) / np.sum(skew)
        self.owner = rng.choice(E, rows * k, p=p).astype(np.int32)
        self.owner[rng.random(rows * k) < none] = -1
        self.weight = rng.normal(0, 1, (rows, k)).astype(np.float32)

    def device(self, i2s):
        self.plan = i2s.route_plan(dev(self.owner), self.E)
        return dev(self.wq), dev(self.bscale), self.plan


def same_bits(got, want32, dtype):
    want = torch.from_numpy(want32).to(dtype)
    assert torch.equal(got.cpu().nan_to_num(123.0), want.nan_to_num(123.0)), (got.cpu().double() - want.double()).abs().max()


def check_experts(i2s, c, dtype="f32", forms=("plain", "up", "down")):
    dt = DTYPES[dtype]
    w, b, plan = c.device(i2s)
    x = dev(c.x, dt)
    x32 = x.float().cpu().numpy()
    d = ref.dots(c.wq, c.bscale, c.owner, x32, c.k)
    here = c.owner >= 0
    if "plain" in forms:
        out = torch.full((c.rows * c.k, c.N), 5.0, dtype=dt, device="cuda")
        call = i2s.W8A8Experts(w, b, plan, x, out=out, x_group=c.k)
        call()
        call.check()
        same_bits(out, np.where(here[:, None], d, np.float32(5)), dt)   # rows of nobody are left as they were
    if "up" in forms and c.N % 32 == 0:
        out = torch.full((c.rows * c.k, c.N // 2), 5.0, dtype=dt, device="cuda")
        i2s.w8a8_mul_mat_experts(w, b, plan, x, out=out, x_group=c.k, swiglu=True)
        want = ref.swiglu(d)
        err = np.abs(f64(out) - want)
        bound = (2.0 ** -20 + torch.finfo(dt).eps / 2) * np.abs(want) + ref.swiglu_floor(d) + float(torch.finfo(dt).tiny) * torch.finfo(dt).eps
        assert (err <= bound)[here].all(), (err - bound)[here].max()
        assert (f64(out)[~here] == 5).all()
    if "down" in forms:
        # one row of x per item, summed per token
        xi = dev(np.repeat(x32, c.k, 0) * np.linspace(0.5, 2, c.rows * c.k, dtype=np.float32)[:, None], dt)
        d2 = ref.dots(c.wq, c.bscale, c.owner, xi.float().cpu().numpy(), 1)
        call = i2s.W8A8Experts(w, b, plan, xi, weight=dev(c.weight))
        call.out.fill_(9)
        call()
        same_bits(call.out, ref.weighted(d2, c.owner, c.E, c.weight), dt)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,N,K,rows,k", [(1, 1, 16, 1, 1), (8, 64, 48, 1, 2), (3, 130, 144, 5, 2), (16, 96, 1024, 40, 4),
                                          (5, 200, 1040, 9, 1), (4, 37, 2064, 33, 3)])
def test_experts_few_rows(i2s, dtype, E, N, K, rows, k):
    check_experts(i2s, Experts(E, N, K, rows, k, seed=E + K, none=0.1), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,N,K,rows,k", [(2, 160, 80, 50, 2), (3, 129, 1040, 300, 1), (7, 256, 208, 900, 4), (1, 32, 32, 257, 1),
                                          (4, 320, 3104, 130, 2), (6, 64, 2080, 700, 6), (9, 32, 1024, 1000, 9)])
def test_experts_many_rows(i2s, dtype, E, N, K, rows, k):
    check_experts(i2s, Experts(E, N, K, rows, k, seed=N + K, none=0.05), dtype)


@pytest.mark.parametrize("rows", [150, 500])
def test_experts_weights_come_late(i2s, rows):
    """Few rows for each of many weights, over many stages: the rings wait for weights that arrive in no order, and
    two groups of warps take their stages by turns."""
    c = Experts(24, 576, 4832, 1, 1, seed=rows)
    rng = np.random.default_rng(rows)
    c.rows, c.x, c.owner = rows, rng.normal(0, 1, (rows, 4832)).astype(np.float32), rng.integers(0, 24, rows).astype(np.int32)
    w, b, plan = c.device(i2s)
    calls = [i2s.W8A8Experts(w, b, plan, dev(c.x)) for _ in range(2)]
    want = torch.from_numpy(ref.dots(c.wq, c.bscale, c.owner, c.x, 1)).cuda()
    scratch = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(20):
        scratch.fill_(i)   # the weights leave the cache
        calls[i % 2].out.fill_(0)
        calls[i % 2]()
        assert torch.equal(calls[i % 2].out, want)
    calls[0].check()


def test_experts_ragged(i2s):
    """One expert has nearly all, some have one item, some none; more tiles than CTAs."""
    check_experts(i2s, Experts(40, 640, 272, 700, 2, seed=5, skew=[1000, 0, 0, 1, 30] + [0, 1, 2, 0, 5] * 7))
    check_experts(i2s, Experts(40, 640, 272, 100, 2, seed=6, skew=[1000, 0, 0, 1, 30] + [0, 1, 2, 0, 5] * 7))
    check_experts(i2s, Experts(300, 96, 64, 64, 8, seed=7))
    c = Experts(4, 64, 64, 10, 2, seed=8)
    c.owner[:] = -1
    check_experts(i2s, c)


@pytest.mark.parametrize("K", [1024, 1040, 2048, 2064, 5120, 65536])
@pytest.mark.parametrize("rows", [3, 40])
def test_experts_largest_sums(i2s, K, rows):
    check_experts(i2s, Experts(1, 40, K, rows, 1, extreme=True), forms=("plain", "down"))


def test_experts_rows_that_are_not_finite(i2s):
    c = Experts(3, 96, 160, 30, 2, seed=9)
    c.x[3, 5], c.x[4, 0], c.x[5, 159], c.x[7] = np.nan, np.inf, -np.inf, 0.0
    c.x[8] *= np.float32(1e-30)    # below the floor
    c.x[9, 0] = np.finfo(np.float32).max
    for dtype in ("f32", "bf16"):
        check_experts(i2s, c, dtype, forms=("plain", "down"))
    w, b, plan = c.device(i2s)
    out = i2s.w8a8_mul_mat_experts(w, b, plan, dev(c.x), x_group=2, swiglu=True)
    bad = torch.isnan(out).all(1).cpu().numpy().reshape(-1, 2).all(1)
    assert np.flatnonzero(bad).tolist() == [3, 4, 5] and not torch.isnan(out[~dev(np.repeat(bad, 2))]).any()
    bad[9] = True   # gate times up of the largest value is about 1e74 by the formula: infinite in 32 bits
    assert torch.isfinite(out[~dev(np.repeat(bad, 2))]).all()


def test_experts_strided_rows(i2s):
    c = Experts(4, 70, 96, 20, 2, seed=10)
    w, b, plan = c.device(i2s)
    for dt in (torch.float32, torch.float16):
        wide = torch.zeros(20, 200, dtype=dt, device="cuda")
        x = wide[:, 8:104]
        x.copy_(dev(c.x, dt))
        frame = torch.full((40, 91), 3.0, dtype=dt, device="cuda")
        out = frame[:, 7:77]
        i2s.w8a8_mul_mat_experts(w, b, plan, x, out=out, x_group=2)
        d = ref.dots(c.wq, c.bscale, c.owner, x.float().cpu().numpy(), 2)
        same_bits(out, d, dt)
        assert (frame[:, :7] == 3).all() and (frame[:, 77:] == 3).all()
        one = torch.full((20, 91), 3.0, dtype=dt, device="cuda")
        i2s.w8a8_mul_mat_experts(w, b, i2s.route_plan(dev(c.owner), 4), x.repeat_interleave(2, 0), out=one[:, 7:77],
                                 weight=dev(c.weight))
        same_bits(one[:, 7:77], ref.weighted(d, c.owner, 4, c.weight), dt)
        assert (one[:, :7] == 3).all() and (one[:, 77:] == 3).all()


def test_plans_that_are_not_in_order(i2s):
    """Starts and entries out of range: what is valid is computed, nothing else is touched."""
    c = Experts(4, 64, 64, 30, 1, seed=11)
    w, b, plan = c.device(i2s)
    x = dev(c.x)
    for start, entries in (([-5, 10, 3, 50, 2 ** 31 - 1], None), ([0, 0, 0, 0, 0], None), ([2 ** 31 - 1] * 5, None),
                           ([0, 10, 20, 25, 30], [-1, 30, 2 ** 31 - 1, -2 ** 31] + list(range(26)))):
        plan.start.copy_(torch.tensor(start, dtype=torch.int32))
        lst = list(range(30)) if entries is None else entries
        plan.list.copy_(torch.tensor(lst, dtype=torch.int32))
        begin = np.maximum.accumulate(np.clip(start, 0, 30))
        owner = np.full(30, -1)
        for e in range(4):
            for i in lst[begin[e]:begin[e + 1]]:
                if 0 <= i < 30:
                    owner[i] = e
        frame = torch.full((34, 64), 2.0, device="cuda")
        i2s.w8a8_mul_mat_experts(w, b, plan, x, out=frame[2:32])
        d = ref.dots(c.wq, c.bscale, owner, c.x, 1)
        same_bits(frame[2:32], np.where(owner[:, None] >= 0, d, np.float32(2)), torch.float32)
        assert (frame[:2] == 2).all() and (frame[32:] == 2).all()
        A, B = torch.ones(4, 8, 64, device="cuda").bfloat16(), torch.ones(4, 64, 8, device="cuda").bfloat16()
        frame.fill_(2)
        i2s.lora_add(A, B, plan, torch.ones_like(x), torch.zeros_like(frame[2:32]), out=frame[2:32])
        assert torch.equal(frame[2:32].cpu(), torch.from_numpy(np.where(owner[:, None] >= 0, 512.0, 2.0)).float().expand(30, 64))
        assert (frame[:2] == 2).all() and (frame[32:] == 2).all()


def test_experts_give_up(i2s):
    c = Experts(4, 64, 2064, 30, 2, seed=12)
    w, b, plan = c.device(i2s)
    call = i2s.W8A8Experts(w, b, plan, dev(c.x), x_group=2, test_stall=True)
    call()
    with pytest.raises(i2s.I2SError) as e:
        call.check()
    assert e.value.status == -6
    again = i2s.W8A8Experts(w, b, plan, dev(c.x), x_group=2, ws=call.ws)
    again()
    again.check()
    same_bits(again.out, ref.dots(c.wq, c.bscale, c.owner, c.x, 2), torch.float32)


# -- adapters -----------------------------------------------------------------------------------------

class Lora:
    def __init__(self, adapters, rank, N, K, rows, dtype, seed=0, none=0.2, size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.dt = DTYPES[dtype]
        half = torch.float16 if dtype == "f16" else torch.bfloat16
        self.A = (torch.randn(adapters, rank, K, generator=g) * size).to(half)
        self.B = torch.randn(adapters, N, rank, generator=g).to(half)
        self.scale = torch.randn(adapters, generator=g)
        self.x = torch.randn(rows, K, generator=g).to(self.dt)
        self.base = (torch.randn(rows, N, generator=g) * 3).to(self.dt)
        self.owner = torch.randint(0, adapters, (rows,), generator=g, dtype=torch.int32)
        self.owner[torch.rand(rows, generator=g) < none] = -1
        self.adapters, self.rank, self.N, self.K, self.rows = adapters, rank, N, K, rows

    def check(self, out, untouched, scale=None):
        owner = self.owner.numpy()
        want, inner, outer = ref.lora(self.A, self.B, self.scale if scale is None else scale, owner, self.x, self.base)
        here = owner >= 0
        parts = {torch.float32: 0.0, torch.float16: 2.0 ** -21, torch.bfloat16: 2.0 ** -17}[self.dt]
        bound = (inner * (3 * (self.K // 16 + 1) + 16) * 2.0 ** -22 + outer * ((3 * (self.rank // 16 + 1) + 16) * 2.0 ** -22 + parts)
                 + (self.base.double().abs() + outer) * 2.0 ** -23)
        bound = bound + (want.abs() + bound) * (torch.finfo(self.dt).eps / 2) + 2.0 ** -25
        err = (out.cpu().double() - want).abs()
        assert (err <= bound)[here].all(), (err / bound)[here].max()
        assert torch.equal(out.cpu()[~here], untouched.cpu()[~here])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("adapters,rank,N,K,rows", [(1, 8, 1, 8, 1), (1, 16, 100, 72, 1), (5, 24, 257, 520, 7), (3, 64, 64, 2048, 40),
                                                    (40, 32, 300, 1000, 64), (2, 128, 511, 264, 131), (4, 40, 33, 4104, 600),
                                                    (300, 8, 40, 64, 500), (1, 104, 1000, 16, 65), (3, 16, 264, 72, 6500), (2, 64, 500, 136, 7001),
                                                    (1, 128, 33, 520, 6407), (90, 8, 64, 2056, 6450)])
def test_lora(i2s, dtype, adapters, rank, N, K, rows):
    c = Lora(adapters, rank, N, K, rows, dtype, seed=rank + K)
    plan = i2s.route_plan(c.owner.cuda(), adapters)
    out = torch.full((rows, N), 7.0, dtype=c.dt, device="cuda")
    x, base = c.x.cuda(), c.base.cuda()
    i2s.lora_add(c.A.cuda(), c.B.cuda(), plan, x, base, out=out, scale=c.scale.cuda())
    c.check(out, torch.full((rows, N), 7.0, dtype=c.dt))
    assert torch.equal(base.cpu(), c.base) and torch.equal(x.cpu(), c.x)
    got = i2s.lora_add(c.A.cuda(), c.B.cuda(), plan, x, base)   # in place, no scales
    assert got is base
    c.check(base, c.base, torch.ones(adapters))


@pytest.mark.parametrize("dtype", DTYPES)
def test_lora_strided(i2s, dtype):
    """x a slice, base and out a slice of a fused projection, at odd and at aligned places."""
    c = Lora(3, 16, 96, 64, 50, dtype, seed=4)
    plan = i2s.route_plan(c.owner.cuda(), 3)
    wide = torch.zeros(50, 160, dtype=c.dt, device="cuda")
    wide[:, 16:80] = c.x.cuda()
    for first in (0, 16, 3):
        y = torch.full((50, 240), 3.0, dtype=c.dt, device="cuda")
        y[:, first:first + 96] = c.base.cuda()
        i2s.lora_add(c.A.cuda(), c.B.cuda(), plan, wide[:, 16:80], y[:, first:first + 96], scale=c.scale.cuda())
        c.check(y[:, first:first + 96], c.base)
        assert (y[:, :first] == 3).all() and (y[:, first + 96:] == 3).all()


def test_lora_ranges(i2s):
    """Values whose inner products leave 16-bit ranges, and rows that are not finite."""
    c = Lora(2, 16, 64, 128, 40, "f16", seed=5, none=0.0, size=300.0)
    c.x *= 100
    c.B *= 2.0 ** -10
    c.scale *= 2.0 ** -6
    c.x[7] *= 2.0 ** -10
    plan = i2s.route_plan(c.owner.cuda(), 2)
    out = i2s.lora_add(c.A.cuda(), c.B.cuda(), plan, c.x.cuda(), c.base.cuda(), scale=c.scale.cuda())
    c.check(out, c.base)
    for dtype in DTYPES:
        c = Lora(2, 16, 64, 128, 40, dtype, seed=6, none=0.0)
        c.x[3, 5], c.x[20, 100] = float("nan"), float("inf")
        out = i2s.lora_add(c.A.cuda(), c.B.cuda(), plan, c.x.cuda(), c.base.cuda())
        fine = torch.ones(40, dtype=torch.bool)
        fine[[3, 20]] = False
        assert torch.isfinite(out.cpu()[fine]).all() and not torch.isfinite(out.cpu()[~fine]).any()
    c = Lora(2, 16, 64, 128, 40, "f32", seed=7, none=0.0)
    c.x *= 1e30   # F32 rows keep their range
    c.base *= 1e30
    out = i2s.lora_add(c.A.cuda(), c.B.cuda(), i2s.route_plan(c.owner.cuda(), 2), c.x.cuda(), c.base.cuda(), scale=c.scale.cuda())
    c.check(out, c.base)


# -- together -------------------------------------------------------------------------------------------

def layer(i2s, logits, x, w1, b1, w2, b2, A, B, owner):
    """A sparse MLP with the requests' adapters on its output: the calls, to be made again."""
    rows, k = x.shape[0], 3
    route = i2s.RouteTopk(logits, k, norm=True)
    up = i2s.W8A8Experts(w1, b1, route.plan, x, x_group=k, swiglu=True)
    down = i2s.W8A8Experts(w2, b2, route.plan, up.out, weight=route.weight)
    mine = i2s.RouteBuild(owner, A.shape[0])
    add = i2s.LoraAdd(A, B, mine.plan, x, down.out)
    return [route, up, down, mine, add], (route, up, down, add)


@pytest.mark.parametrize("rows", [1, 37, 400])
def test_sparse_layer_eager_graph_and_streams(i2s, rows):
    rng = np.random.default_rng(rows)
    E, K, F, adapters, k = 12, 160, 96, 5, 3
    w1 = Experts(E, 2 * F, K, 1, 1, seed=1)
    w2 = Experts(E, K, F, 1, 1, seed=2)
    lora = Lora(adapters, 16, K, K, rows, "f32", seed=3)
    logits, x, owner = (torch.empty(rows, E, device="cuda"), torch.empty(rows, K, device="cuda"),
                        torch.empty(rows, dtype=torch.int32, device="cuda"))

    def fill(seed):
        r = np.random.default_rng(seed)
        logits.copy_(dev(r.normal(0, 1, (rows, E)).astype(np.float32)))
        x.copy_(dev(r.normal(0, 30, (rows, K)).astype(np.float32)))
        owner.copy_(dev(r.integers(-1, adapters, rows).astype(np.int32)))

    def verify(parts):
        route, up, down, add = parts
        expert, weight = ref.topk(f64(logits), k, norm=True)
        assert np.array_equal(route.expert.cpu().numpy(), expert)
        flat = expert.reshape(-1)
        d = ref.dots(w1.wq, w1.bscale, flat, x.cpu().numpy(), k)
        want = ref.swiglu(d)
        assert (np.abs(f64(up.out) - want) <= 2.0 ** -20 * np.abs(want) + ref.swiglu_floor(d)).all()
        # the next operator's definition on what it was given
        d2 = ref.dots(w2.wq, w2.bscale, flat, up.out.cpu().numpy(), 1)
        lora.base = torch.from_numpy(ref.weighted(d2, flat, E, route.weight.cpu().numpy()))
        lora.x, lora.owner = x.cpu(), owner.cpu()
        lora.check(add.out, lora.base, torch.ones(adapters))

    args = (logits, x, dev(w1.wq), dev(w1.bscale), dev(w2.wq), dev(w2.bscale), lora.A.cuda(), lora.B.cuda(), owner)
    fill(0)
    calls, parts = layer(i2s, *args)
    for call in calls:
        call()
    verify(parts)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        for call in calls:
            call()
    for seed in (1, 2):   # the graph routes what it finds
        fill(seed)
        graph.replay()
        verify(parts)
    # two layers at once on two streams, each with its own buffers
    other, other_parts = layer(i2s, *args)
    torch.cuda.synchronize()
    second = torch.cuda.Stream()
    for _ in range(3):
        for a, b in zip(calls, other):
            a()
            with torch.cuda.stream(second):
                b()
    torch.cuda.synchronize()
    verify(parts)
    verify(other_parts)
    first = [t.out.clone() for t in parts[1:]]
    for call in calls:
        call()
    assert all(torch.equal(a, t.out) for a, t in zip(first, parts[1:]))   # the same bits again
