"""The 8-bit KV cache operators on the GPU against their definitions.

kv8_write and kv8_read are defined step by step in binary32, so pools and values
are compared bit for bit. kv8_norm_rope and kv8_attention are compared with 64
bits, within bounds from the number of roundings:

norm and rotation: the square sum of up to 128 terms (8 sequential additions of
  one lane's terms and of the 5 exchanges: relative 10 * 2^-24), the mean, eps,
  root, reciprocal and two products (7 more roundings), cosine and sine (their
  argument and the function: within 2^-22), two products and one sum: together
  below 2^-19 of the larger of a pair's values; plus half a step of the dtype.
attention: with A the largest sum |q||k| * scale that the row sees, a logit is
  within A * 2^-18 (two f16 parts of q and up to 16 tensor-core steps of 2^-22
  each, then the scales), its exponential within 2^-18 * (A + 1) of itself, the
  sums over n tokens within (n/16 + 16) * 2^-22; twice that for the quotient.
  The low f16 part of a weight is rounded to steps of 2^-24 at the finest, an
  error of 2^-25 where the row's largest weight is at least 2^8: with n tokens
  seen, n * 2^-33 of the largest value that a block seen can hold.
  Probabilities of 16-bit rows are rounded to f16, 2^-12 relative, or absolutely
  2^-25 of the largest of the row's running tile, both below 2^-11 of
  sum p|v| with the largest |v|; plus half a step of the dtype.
"""

import ctypes

import numpy as np
import pytest

from tests import kv8_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ALL = ["f32", "f16", "bf16"]


@pytest.fixture(scope="module")
def i2s():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_quantized_matmul_gb300 import build as libbuild
    libbuild.build()
    from int8_quantized_matmul_gb300 import i2s as mod
    assert mod.device_supported() == 1
    return mod


class Setup:
    """A pool in use, with garbage wherever no token lies, and a batch over it."""

    def __init__(self, i2s, kv, dim, page, lens, news, seed=0, pad_rows=0, max_rows=None, extra_width=0, first_page=0):
        rng = np.random.default_rng(seed)
        self.kv, self.dim, self.page, self.lens, self.news = kv, dim, page, lens, news
        used = [-(-n // page) for n in lens]
        n_pages = sum(used) + 2
        width = max(1, max(used)) + extra_width
        raw = rng.integers(0, 256, n_pages * kv * ref.slab_bytes(dim, page), dtype=np.uint8)
        pool = ref.Pool(raw, kv, dim, page)
        pool.codes = np.clip(np.rint(rng.normal(0, 40, pool.codes.shape)), -127, 127).astype(np.int8)
        # blocks that no token lies in hold NaN and infinite scales
        pool.scales = rng.choice(np.array([np.nan, np.inf, -np.inf, 3e38], np.float32), pool.scales.shape)
        order = rng.permutation(n_pages)
        table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for s, n in enumerate(used):
            table[s, :n] = order[at:at + n]
            for i in range(-(-lens[s] // 16)):
                p = order[at + i * 16 // page]
                pool.scales[p, :, :, i * 16 % page // 16] = np.exp(rng.normal(0, 0.7, (kv, 2))) * 0.02
            at += n
        self.pool, self.table = ref.Pool(pool.bytes(), kv, dim, page), table
        self.row_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.rows = int(self.row_start[-1]) + pad_rows
        self.first_page = first_page
        if first_page:   # the pages lie far into a larger pool
            self.data = torch.empty((first_page + n_pages, kv * ref.slab_bytes(dim, page)), dtype=torch.uint8, device="cuda")
            self.data[first_page:].view(-1).copy_(torch.from_numpy(self.pool.bytes()))
        else:
            self.data = torch.from_numpy(self.pool.bytes()).cuda().view(n_pages, -1)
        self.cache = i2s.Kv8Cache(first_page + n_pages, kv, dim, page, data=self.data)
        dev = np.where(table >= 0, table + first_page, table).astype(np.int32)
        self.batch = i2s.Kv8Batch(torch.from_numpy(self.row_start).cuda(),
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(dev).cuda(),
                                  rows=self.rows, max_rows=max_rows or max(1, max(news)))

    def pool_now(self):
        return self.data[self.first_page:].cpu().numpy().reshape(-1)


def rows_tensor(rng, rows, heads, dim, dtype, layout="packed", std=1.0):
    """(tensor, its values as float32)."""
    x = torch.from_numpy((rng.standard_normal((rows, heads, dim)) * std).astype(np.float32)).to(DTYPES[dtype]).cuda()
    if layout == "heads first":
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    elif layout == "slice":
        big = torch.full((rows, heads + 3, dim), float("nan"), dtype=x.dtype, device="cuda")
        big[:, 1:1 + heads] = x
        x = big[:, 1:1 + heads]
    return x, x.float().cpu().numpy()


def same_bits(a, b):
    a, b = np.ascontiguousarray(a), np.ascontiguousarray(b)
    np.testing.assert_array_equal(a.view(np.uint8), b.view(np.uint8))


# -- write and read -------------------------------------------------------------------------------

WRITES = [
    # kv, dim, page, lens, news
    (1, 128, 16, [1], [1]),
    (2, 128, 64, [17, 16, 15, 33], [1, 1, 1, 1]),
    (8, 128, 64, [100, 0, 64, 65, 2], [1, 0, 64, 2, 2]),
    (3, 64, 32, [50, 31, 32, 129], [37, 31, 1, 100]),
    (1, 64, 256, [300, 700], [299, 45]),
    (2, 128, 128, [130, 1000], [5, 1000]),
]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("layout", ["packed", "heads first", "slice"])
@pytest.mark.parametrize("case", WRITES)
def test_write_is_bit_exact(i2s, case, layout, dtype):
    kv, dim, page, lens, news = case
    st = Setup(i2s, kv, dim, page, lens, news, seed=len(lens) + dim, pad_rows=5)
    rng = np.random.default_rng(7)
    # a spread of sizes: some blocks' scales grow, some keep the one they have
    k, kf = rows_tensor(rng, st.rows, kv, dim, dtype, layout, std=3.0)
    v, vf = rows_tensor(rng, st.rows, kv, dim, dtype, layout, std=0.2)
    i2s.kv8_write(st.cache, st.batch, k, v)
    ref.write(st.pool, st.table, lens, st.row_start, kf, vf)
    assert st.batch.status() == 0
    same_bits(st.pool_now(), st.pool.bytes())
    i2s.kv8_write(st.cache, st.batch, k, v)   # the same tokens again change nothing
    same_bits(st.pool_now(), st.pool.bytes())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("layout", ["packed", "heads first", "slice"])
@pytest.mark.parametrize("case", WRITES)
def test_read_is_the_codes_times_the_scales(i2s, case, layout, dtype):
    kv, dim, page, lens, news = case
    st = Setup(i2s, kv, dim, page, lens, news, seed=3, pad_rows=4)
    rng = np.random.default_rng(8)
    k, kf = rows_tensor(rng, st.rows, kv, dim, dtype, layout)
    v, vf = rows_tensor(rng, st.rows, kv, dim, dtype, layout)
    i2s.kv8_read(st.cache, st.batch, k, v)
    for which, (got, before) in enumerate(((k, kf), (v, vf))):
        want = before.copy()   # rows behind the last sequence stay as they were
        for s, n in enumerate(news):
            x, _ = ref.cached(st.pool, st.table, s, lens[s], which)
            want[st.row_start[s]:st.row_start[s + 1]] = x[lens[s] - n:].astype(np.float32)
        want = torch.from_numpy(want).to(DTYPES[dtype])
        assert torch.equal(got.cpu(), want)
    assert st.batch.status() == 0


def test_many_sequences_in_the_rows_of_one_block(i2s):
    """More sequence starts than a CTA looks at at once, empty sequences among them, beside long ones."""
    news = [1] * 50 + [0] * 40 + [1, 0, 2] * 20 + [70] + [0, 1] * 30 + [16, 33]
    lens = [n + (7 * i) % 41 for i, n in enumerate(news)]
    st = Setup(i2s, 2, 64, 16, lens, news, seed=8, pad_rows=7)
    rng = np.random.default_rng(9)
    k, kf = rows_tensor(rng, st.rows, 2, 64, "f32", std=2.0)
    v, vf = rows_tensor(rng, st.rows, 2, 64, "f32", std=2.0)
    i2s.kv8_write(st.cache, st.batch, k, v)
    ref.write(st.pool, st.table, lens, st.row_start, kf, vf)
    same_bits(st.pool_now(), st.pool.bytes())
    kv = torch.full((st.rows, 4, 64), 3.0, device="cuda")   # read back into slices of one row
    i2s.kv8_read(st.cache, st.batch, kv[:, :2], kv[:, 2:])
    for which in (0, 1):
        want = np.full((st.rows, 2, 64), 3.0, np.float32)
        for s, n in enumerate(news):
            x, _ = ref.cached(st.pool, st.table, s, lens[s], which)
            want[st.row_start[s]:st.row_start[s + 1]] = x[lens[s] - n:].astype(np.float32)
        same_bits(kv[:, 2 * which:2 * which + 2].cpu().numpy(), want)
    assert st.batch.status() == 0


def test_tokens_appended_one_by_one_match_the_definition(i2s):
    """40 single-token appends: every block grows through all its fill levels."""
    kv, dim, page, total = 2, 128, 32, 40
    st = Setup(i2s, kv, dim, page, [total], [1], seed=11)
    rng = np.random.default_rng(12)
    for n in range(1, total + 1):
        st.batch.kv_len.fill_(n)
        k, kf = rows_tensor(rng, 1, kv, dim, "f32", std=float(np.exp(rng.normal(0, 1))))
        v, vf = rows_tensor(rng, 1, kv, dim, "f32", std=0.01 * n)
        i2s.kv8_write(st.cache, st.batch, k, v)
        ref.write(st.pool, st.table, [n], st.row_start, kf, vf)
    same_bits(st.pool_now(), st.pool.bytes())


def test_a_block_with_nan_or_infinity_reads_as_nan_until_rewritten(i2s):
    st = Setup(i2s, 1, 64, 16, [20, 20, 20], [6, 6, 6], seed=2)
    rng = np.random.default_rng(1)
    k, kf = rows_tensor(rng, 18, 1, 64, "f32")
    v, vf = rows_tensor(rng, 18, 1, 64, "f32")
    k[3, 0, 5], kf[3, 0, 5] = float("nan"), np.nan        # position 17 of sequence 0
    v[7, 0, 0], vf[7, 0, 0] = float("-inf"), -np.inf      # position 15 of sequence 1
    i2s.kv8_write(st.cache, st.batch, k, v)
    ref.write(st.pool, st.table, st.lens, st.row_start, kf, vf)
    same_bits(st.pool_now(), st.pool.bytes())
    back_k, back_v = i2s.kv8_read(st.cache, st.batch)
    bad_k, bad_v = back_k.isnan().any(-1)[:, 0].tolist(), back_v.isnan().any(-1)[:, 0].tolist()
    assert bad_k == [False, False, True, True, True, True] + 12 * [False]     # block 16.. of sequence 0
    assert bad_v == 6 * [False] + [True, True, False, False, False, False] + 6 * [False]
    st.batch.kv_len[0] = 21                                # a finite token more: the block stays NaN
    k2, v2 = torch.ones_like(k), torch.ones_like(v)
    i2s.kv8_write(st.cache, st.batch, k2, v2)              # positions 15..20: block 1 from its first token
    assert not i2s.kv8_read(st.cache, st.batch)[0].isnan().any()


def test_write_and_read_beyond_four_gigabytes(i2s):
    """Pages whose byte offset passes 32 bits."""
    page_bytes = 8 * ref.slab_bytes(128, 64)
    first = (1 << 32) // page_bytes + 5
    st = Setup(i2s, 8, 128, 64, [70, 200], [70, 3], seed=4, first_page=first)
    rng = np.random.default_rng(5)
    k, kf = rows_tensor(rng, st.rows, 8, 128, "f32")
    v, vf = rows_tensor(rng, st.rows, 8, 128, "f32")
    i2s.kv8_write(st.cache, st.batch, k, v)
    ref.write(st.pool, st.table, st.lens, st.row_start, kf, vf)
    same_bits(st.pool_now(), st.pool.bytes())
    q, qf = rows_tensor(rng, st.rows, 16, 128, "f32")
    check_attention(i2s, st, q, qf, "f32")


# -- norm and rotation ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("dim,rot,interleaved,norm", [
    (128, 128, False, True), (128, 128, True, True), (128, 32, False, False), (128, 8, False, True),
    (128, 40, True, False), (64, 64, False, True), (64, 64, True, False), (64, 24, False, True), (64, 0, False, True),
    (128, 104, False, True)])
@pytest.mark.parametrize("rows,qh,kh", [(1, 1, 1), (7, 12, 2), (33, 5, 0), (130, 0, 3)])
def test_norm_rope(i2s, dtype, dim, rot, interleaved, norm, rows, qh, kh):
    rng = np.random.default_rng(rows + dim + rot)
    base = 1000000.0
    turns = i2s.kv8_rope_turns(base, rot) if rot else None
    pos = rng.integers(-5, 1 << 31, rows).astype(np.int32)
    pos[0] = (1 << 31) - 1
    dpos = torch.from_numpy(pos).cuda()
    q, qf = rows_tensor(rng, rows, qh, dim, dtype, "slice", std=2.0) if qh else (None, None)
    k, kf = rows_tensor(rng, rows, kh, dim, dtype, "heads first", std=0.01) if kh else (None, None)
    gq, gk = (torch.from_numpy((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)).cuda() for _ in range(2))
    got = i2s.kv8_norm_rope(q, k, dpos, turns, gamma_q=gq if norm else None, gamma_k=gk if norm else None, eps=1e-6,
                            interleaved=interleaved)
    integers = [int(t) % (1 << 64) for t in turns.tolist()] if rot else []
    for x, y, g in ((qf, got[0], gq), (kf, got[1], gk)):
        if x is None:
            assert y is None
            continue
        want = ref.norm_rope(x, g.cpu().numpy() if norm else None, 1e-6, pos, integers, interleaved)
        y = y.float().cpu().numpy().astype(np.float64)
        # the larger of a pair bounds the rounding of both
        size = np.abs(ref.norm_rope(x, g.cpu().numpy() if norm else None, 1e-6, pos, [], interleaved))
        if rot:
            a, b = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved else
                    (slice(0, rot // 2), slice(rot // 2, rot)))
            both = size[..., a] + size[..., b]
            size[..., a], size[..., b] = both, both
        eps = torch.finfo(DTYPES[dtype]).eps / 2 if dtype != "f32" else 0.0
        tiny = 2.0 ** -25 if dtype == "f16" else 0.0   # half a step of f16's subnormals
        assert (np.abs(y - want) <= size * 2.0 ** -19 + np.abs(want) * eps * (1 + 2.0 ** -9) + tiny).all()


def test_norm_rope_in_place_in_a_fused_row(i2s):
    rng = np.random.default_rng(3)
    rows, qh, kh, dim = 9, 4, 2, 128
    fused, f = rows_tensor(rng, rows, qh + 2 * kh, dim, "f32")
    turns = i2s.kv8_rope_turns(10000.0, dim)
    pos = torch.arange(100, 100 + rows, dtype=torch.int32, device="cuda")
    q, k = fused[:, :qh], fused[:, qh:qh + kh]
    want = i2s.kv8_norm_rope(q, k, pos, turns)
    values = fused[:, qh + kh:].clone()
    i2s.kv8_norm_rope(q, k, pos, turns, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(fused[:, qh + kh:], values)


def test_norm_rope_zero_head_and_zero_position(i2s):
    x = torch.zeros((2, 1, 64), device="cuda")
    x[1] = torch.randn((1, 64), device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, _ = i2s.kv8_norm_rope(x, None, pos, i2s.kv8_rope_turns(10000.0, 64))
    assert torch.equal(out, x)   # position 0 turns nothing
    out, _ = i2s.kv8_norm_rope(x, None, pos, None, gamma_q=torch.ones(64, device="cuda"), eps=1e-6)
    assert torch.equal(out[0], torch.zeros_like(out[0]))


# -- attention ----------------------------------------------------------------------------------------

def check_attention(i2s, st, q, qf, dtype, causal=True, window=0, scale=None, out=None, with_lse=True, ws=None):
    heads = qf.shape[1]
    scale = st.dim ** -0.5 if scale is None else scale
    lse = torch.full((st.rows, heads), 99.0, device="cuda") if with_lse else None
    if out is None:
        out = torch.full((st.rows, heads, st.dim), 7.0, dtype=DTYPES[dtype], device="cuda")
    before = out.float().cpu().numpy().copy()
    i2s.kv8_attention(st.cache, st.batch, q, out=out, scale=scale, causal=causal, window=window, lse=lse, ws=ws)
    torch.cuda.synchronize()
    compare_attention(st, qf, dtype, causal, window, scale, out, lse, before)


def compare_attention(st, qf, dtype, causal, window, scale, out, lse, before):
    want, want_lse, weight, size, reach = ref.attention(st.pool, st.table, st.lens, st.row_start, qf, float(np.float32(scale)),
                                                 causal, window)
    got = out.float().cpu().numpy().astype(np.float64)
    last = st.row_start[-1]
    np.testing.assert_array_equal(got[last:], before[last:])   # rows behind the last sequence
    got, want, weight, size, want_lse, reach = (x[:last] for x in (got, want, weight, size, want_lse, reach))
    n = max(st.lens + [1])
    rel = 2 * (2.0 ** -18 * (size + 1) * 2 + (n / 16 + 16) * 2.0 ** -22)
    tol = weight * rel[..., None] + reach[..., None] * 2.0 ** -33
    if dtype != "f32":
        tol += weight.max(-1, keepdims=True) * 2.0 ** -11 + np.abs(want) * torch.finfo(DTYPES[dtype]).eps / 2 * 1.01 + 2.0 ** -24
    worst = np.abs(got - want) - tol
    assert (worst <= 0).all(), (float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))
    if lse is not None:
        got_lse = lse.cpu().numpy().astype(np.float64)
        assert (got_lse[last:] == 99.0).all()
        got_lse = got_lse[:last]
        np.testing.assert_array_equal(np.isneginf(got_lse), np.isneginf(want_lse))
        fine = ~np.isneginf(want_lse)
        assert (np.abs(got_lse - want_lse)[fine] <= (rel + 2.0 ** -22 * np.abs(np.where(fine, want_lse, 0)))[fine]).all()


ATTENTION = [
    # kv, group, dim, page, lens, news, causal, window
    (1, 1, 128, 16, [1], [1], True, 0),
    (2, 6, 128, 64, [75], [1], True, 0),
    (2, 6, 128, 16, [15, 16, 17, 1, 400], [1, 1, 1, 1, 1], True, 0),
    (8, 2, 128, 64, [300, 0, 64, 1037], [1, 0, 1, 1], True, 0),
    (1, 8, 64, 32, [513, 31], [1, 1], True, 0),
    (3, 5, 64, 128, [129, 255, 2000], [1, 1, 1], True, 100),
    (2, 7, 128, 256, [4096], [1], True, 0),
    (1, 16, 128, 64, [777, 20], [1, 1], True, 0),
    (2, 6, 128, 16, [90, 33, 5, 700], [3, 6, 5, 1], True, 0),         # drafts
    (2, 6, 128, 16, [90, 33, 5, 700], [3, 6, 5, 1], True, 20),
    (4, 4, 64, 64, [100, 64, 1], [8, 64, 1], True, 0),
    (1, 2, 128, 32, [333], [333], True, 0),                           # a prompt
    (2, 3, 128, 64, [500, 130, 129], [257, 130, 64], True, 0),        # chunks
    (2, 3, 128, 64, [500, 130, 129], [257, 130, 64], True, 33),
    (2, 2, 64, 32, [400, 65], [128, 65], True, 1),                    # each row sees itself alone
    (1, 4, 128, 64, [10, 100], [20, 100], True, 0),                   # rows before position 0 see nothing
    (2, 4, 128, 64, [0, 40], [3, 3], True, 0),                        # an empty cache
    (2, 4, 128, 64, [200, 40], [70, 3], False, 0),                    # every row sees all tokens
    (2, 1, 64, 16, [40, 3], [1, 2], False, 0),
    (1, 64, 128, 64, [200], [5], True, 0),
    (1, 13, 64, 64, [200, 100, 47], [9, 21, 2], True, 0),
]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention(i2s, case, dtype):
    kv, group, dim, page, lens, news, causal, window = ATTENTION[case]
    st = Setup(i2s, kv, dim, page, lens, news, seed=case, pad_rows=3, extra_width=2)
    rng = np.random.default_rng(case + 100)
    q, qf = rows_tensor(rng, st.rows, kv * group, dim, dtype, std=1.5)
    check_attention(i2s, st, q, qf, dtype, causal, window)
    assert st.batch.status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new", [1, 4, 70])
def test_attention_strides(i2s, dtype, new):
    st = Setup(i2s, 2, 128, 32, [150, 90], [new, new], seed=1)
    rng = np.random.default_rng(2)
    q, qf = rows_tensor(rng, st.rows, 6, 128, dtype, "slice")
    out = torch.full((6, st.rows, 128), 5.0, dtype=DTYPES[dtype], device="cuda").transpose(0, 1)
    check_attention(i2s, st, q, qf, dtype, out=out, with_lse=False)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("size", [1e-30, 1e-5, 300.0, 1e20])
def test_attention_of_small_and_large_queries(i2s, size, new):
    """Queries outside f16's range, with a scale that brings the logits back."""
    st = Setup(i2s, 1, 128, 64, [200], [new], seed=6)
    rng = np.random.default_rng(9)
    q, qf = rows_tensor(rng, st.rows, 4, 128, "f32", std=size)
    check_attention(i2s, st, q, qf, "f32", scale=128 ** -0.5 / size)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_with_scales_far_apart(i2s, new):
    """Value scales from 1e-7 to 1e4 from block to block, and sharp logits."""
    st = Setup(i2s, 2, 128, 64, [350], [new], seed=21)
    rng = np.random.default_rng(22)
    for p in st.table[0][st.table[0] >= 0]:
        st.pool.scales[p, :, 1] = np.exp(rng.uniform(np.log(1e-7), np.log(1e4), st.pool.scales[p, :, 1].shape))
        st.pool.scales[p, :, 0] = np.where(np.isfinite(st.pool.scales[p, :, 0]), 0.05, np.nan)
    st.data.view(-1).copy_(torch.from_numpy(st.pool.bytes()))
    st.pool = ref.Pool(st.pool.bytes(), 2, 128, 64)
    q, qf = rows_tensor(rng, st.rows, 4, 128, "f32", std=3.0)
    check_attention(i2s, st, q, qf, "f32")


@pytest.mark.parametrize("new", [1, 40])
def test_a_nan_block_is_nan_where_it_is_seen_and_nowhere_else(i2s, new):
    st = Setup(i2s, 1, 128, 64, [100, 100], [new, new], seed=5)
    p = st.table[0][0]
    st.pool.scales[p, 0, 0, 1] = np.nan   # tokens 16..31 of sequence 0
    st.data.view(-1).copy_(torch.from_numpy(st.pool.bytes()))
    q, _ = rows_tensor(np.random.default_rng(1), st.rows, 2, 128, "f32")
    out = i2s.kv8_attention(st.cache, st.batch, q)
    assert out[:new].isnan().all() and not out[new:].isnan().any()
    out = i2s.kv8_attention(st.cache, st.batch, q, window=20)   # behind every row's window
    assert not out.isnan().any()


@pytest.mark.parametrize("new", [2, 40])
def test_a_nan_block_that_one_row_sees_does_not_reach_the_others(i2s, new):
    st = Setup(i2s, 1, 128, 64, [100], [new], seed=5)
    first = 100 - new   # row 0 sees tokens 31..first, row 1 32..first + 1
    for which in (0, 1):
        page = st.pool.raw.copy()
        st.pool.scales[st.table[0][0], 0, which, 1] = np.nan   # tokens 16..31
        st.data.view(-1).copy_(torch.from_numpy(st.pool.bytes()))
        q, _ = rows_tensor(np.random.default_rng(1), st.rows, 2, 128, "f32")
        out = i2s.kv8_attention(st.cache, st.batch, q, window=first - 31 + 1)
        assert out[0].isnan().all() and not out[1:].isnan().any()
        st.pool = ref.Pool(page.reshape(-1), 1, 128, 64)


@pytest.mark.parametrize("new", [1, 3, 50])
def test_bad_pages_lengths_and_rows_are_cut_and_reported(i2s, new):
    st = Setup(i2s, 2, 128, 32, [130, 64, 80], [new] * 3, seed=13)
    rng = np.random.default_rng(3)
    q, qf = rows_tensor(rng, st.rows, 4, 128, "f32")
    k, kf = rows_tensor(rng, st.rows, 2, 128, "f32")
    for bad in (-1, st.cache.n_pages, 1 << 30):
        st.batch.page_table[0, 1] = bad        # tokens 32..63 of sequence 0
        st.table[0, 1] = -1
        check_attention(i2s, st, q, qf, "f32")
        assert st.batch.status() == i2s.KV8_BAD_PAGE
        assert st.batch.status() == 0
    # a page that a write and a read need: nothing else changes
    st.batch.page_table[0, 4] = -3
    st.table[0, 4] = -1
    i2s.kv8_write(st.cache, st.batch, k, k)
    assert st.batch.status() == i2s.KV8_BAD_PAGE
    ref.write(st.pool, st.table, st.lens, st.row_start, kf, kf)
    same_bits(st.pool_now(), st.pool.bytes())
    i2s.kv8_read(st.cache, st.batch)
    with pytest.raises(i2s.I2SError):
        st.batch.check()
    # a length past the table, and one below zero
    st.batch.kv_len[1] = 1 << 30
    st.batch.kv_len[2] = -5
    out = i2s.kv8_attention(st.cache, st.batch, q)
    assert st.batch.status() & i2s.KV8_BAD_LENGTH
    assert torch.equal(out[2 * new:], torch.zeros_like(out[2 * new:]))
    # row starts that go backwards or leave the tensor
    st.batch.kv_len.copy_(torch.tensor(st.lens, dtype=torch.int32))
    for starts in ([0, 2 * new, new, 3 * new], [0, new, 2 * new, 1 << 30], [-4, new, 2 * new, 3 * new]):
        st.batch.row_start.copy_(torch.tensor(starts, dtype=torch.int32))
        i2s.kv8_attention(st.cache, st.batch, q)
        i2s.kv8_write(st.cache, st.batch, k, k)
        i2s.kv8_read(st.cache, st.batch)
        assert st.batch.status() & i2s.KV8_BAD_ROWS


@pytest.mark.parametrize("new", [1, 30])
def test_attention_replayed_from_a_graph_after_the_lengths_change(i2s, new):
    st = Setup(i2s, 2, 128, 64, [300, 150], [new, new], seed=17)
    rng = np.random.default_rng(4)
    q, qf = rows_tensor(rng, st.rows, 6, 128, "f32")
    lse = torch.empty((st.rows, 6), device="cuda")
    one = i2s.Kv8Attention(st.cache, st.batch, q, lse=lse)
    two = i2s.Kv8Attention(st.cache, st.batch, q, ws=one.ws)   # another graph with the same workspace
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        one()
        two()
        for call in (one, two):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call()
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for lens in ([300, 150], [77, 149], [new, new]):
        st.lens = lens
        st.batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        one.out.zero_()
        for g in graphs + graphs[:1]:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(one.out, two.out)
        compare_attention(st, qf, "f32", True, 0, 128 ** -0.5, one.out, lse, one.out.cpu().numpy())


@pytest.mark.parametrize("news", [1, 3, 9])
def test_attention_of_thousands_of_sequences(i2s, news):
    """More sequences than a CTA has threads, in every kernel's own count of them."""
    seqs = 1500
    lens = [news + (13 * i) % 60 for i in range(seqs)]
    lens[700], lens[1499] = 900, 2000
    st = Setup(i2s, 1, 64, 16, lens, [news if i % 7 else 0 for i in range(seqs)], seed=news)
    q, qf = rows_tensor(np.random.default_rng(1), st.rows, 2, 64, "f32")
    check_attention(i2s, st, q, qf, "f32")
    assert st.batch.status() == 0


@pytest.mark.parametrize("new", [1, 130])
def test_attention_over_many_tokens_stays_exact(i2s, new):
    """Long sums: of 20000 tokens, within the bound that does not grow as fast as they do."""
    st = Setup(i2s, 1, 128, 64, [20000], [new], seed=3)
    q, qf = rows_tensor(np.random.default_rng(1), st.rows, 1 if new > 1 else 2, 128, "f32")
    out = i2s.kv8_attention(st.cache, st.batch, q).cpu().numpy().astype(np.float64)
    want = ref.attention(st.pool, st.table, st.lens, st.row_start, qf, float(np.float32(128 ** -0.5)), True, 0)[0]
    # 22-bit operands; a chain of at most 512 tokens (64 tensor-core steps, each cut below 2^-23 of the sum): 2^-17
    assert np.linalg.norm(out - want) <= 2.0 ** -17 * np.linalg.norm(want)


def test_attention_of_shares_longer_than_one_accumulation(i2s):
    """So many tokens that a CTA's share of an item exceeds the 256 blocks it sums at once: sequences that read the same
    32768 tokens, 8 x 8 x 2048 blocks over 456 CTAs. Against 64 bits for the first and the last sequence."""
    heads, dim, seqs, n = 8, 64, 8, 32768
    st = Setup(i2s, heads, dim, 256, [n], [1], seed=77)
    table = st.batch.page_table.expand(seqs, -1).contiguous()
    starts = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    lens = [n - 3 * i for i in range(seqs)]
    batch = i2s.Kv8Batch(starts, torch.tensor(lens, dtype=torch.int32, device="cuda"), table, rows=seqs, max_rows=1)
    q, qf = rows_tensor(np.random.default_rng(5), seqs, heads, dim, "f32")
    out = i2s.kv8_attention(st.cache, batch, q).cpu().numpy().astype(np.float64)
    assert batch.status() == 0
    for s in (0, seqs - 1):
        want = ref.attention(st.pool, st.table, [lens[s]], [0, 1], qf[s:s + 1], float(np.float32(dim ** -0.5)), True, 0)[0]
        assert np.linalg.norm(out[s] - want[0]) <= 2.0 ** -17 * np.linalg.norm(want)


def test_attention_on_two_streams_at_once(i2s):
    calls, wants = [], []
    for new, seed in ((1, 41), (40, 42)):
        st = Setup(i2s, 2, 128, 32, [3000, 500], [new, new], seed=seed)
        q, qf = rows_tensor(np.random.default_rng(seed), st.rows, 4, 128, "f32")
        call = i2s.Kv8Attention(st.cache, st.batch, q)
        call()
        calls.append(call)
        wants.append(call.out.clone())
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for call, stream in zip(calls, streams):
            with torch.cuda.stream(stream):
                call.out.fill_(-1.0)
                call()
    torch.cuda.synchronize()
    for call, want in zip(calls, wants):
        assert torch.equal(call.out, want)


def test_attention_is_the_same_every_time(i2s):
    for news in ([1, 1, 1], [40, 3, 99]):
        st = Setup(i2s, 2, 128, 64, [3000, 150, 700], news, seed=23)
        q, _ = rows_tensor(np.random.default_rng(4), st.rows, 8, 128, "f32")
        call = i2s.Kv8Attention(st.cache, st.batch, q)
        call()
        first = call.out.clone()
        for _ in range(5):
            call.ws.fill_(255)
            call()
            assert torch.equal(first, call.out)


# -- a decoder layer's run of them ----------------------------------------------------------------------

@pytest.mark.parametrize("new", [1, 24])
def test_projections_norm_rope_write_attention_together(i2s, new):
    """W8A8 q, k, v -> kv8_norm_rope -> kv8_write -> kv8_attention -> W8A8 o on one stream, in a captured graph: the
    attention equals the definition on what the cache then holds."""
    hidden, qh, kv, dim, page = 256, 4, 2, 64, 32
    lens, seqs = [40 + new, new], 2
    st = Setup(i2s, kv, dim, page, lens, [new] * seqs, seed=31)
    M = st.rows
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((M, hidden), generator=g, device="cuda")
    qkv = torch.empty((M, (qh + 2 * kv) * dim), device="cuda")

    def packed(n, k):
        wq, bs = i2s.w8a8_quantize_weights(torch.randn((n, k), generator=g, device="cuda") * k ** -0.5)
        return i2s.w8a8_pack_weights(wq), bs
    w, bs = packed(qkv.shape[1], hidden)
    wo, bo = packed(hidden, qh * dim)
    q, k, v = qkv.view(M, -1, dim).split([qh, kv, kv], 1)
    out = torch.empty((M, qh, dim), device="cuda")
    y = torch.empty((M, hidden), device="cuda")
    pos = torch.cat([torch.arange(n - new, n) for n in lens]).to(torch.int32).cuda()
    gamma = torch.full((dim,), 1.5, device="cuda")
    steps = [i2s.W8A8Group([(w, bs, qkv.shape[1], hidden, x, qkv)], M),
             i2s.Kv8NormRope(q, k, pos, i2s.kv8_rope_turns(1e6, dim), gamma_q=gamma, gamma_k=gamma, q_out=q, k_out=k),
             i2s.Kv8Write(st.cache, st.batch, k, v), i2s.Kv8Attention(st.cache, st.batch, q, out=out),
             i2s.W8A8Group([(wo, bo, hidden, qh * dim, out.view(M, -1), y)], M)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for step in steps:
            step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for step in steps:
                step()
    side.synchronize()
    x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert st.batch.status() == 0
    st.pool = ref.Pool(st.pool_now(), kv, dim, page)
    qf = q.float().cpu().numpy()
    compare_attention(st, qf, "f32", True, 0, dim ** -0.5, out, None, out.cpu().numpy())
    # what the cache holds is the normed, rotated keys within half a step of the block's scale
    kept, _ = i2s.kv8_read(st.cache, st.batch)
    step = k.abs().amax().item() / 127
    assert (kept - k).abs().max().item() <= 1.01 * step
    want = i2s.w8a8_mul_mat_packed(wo, bo, hidden, qh * dim, out.view(M, -1))[0]
    assert torch.equal(y, want)


def test_window_that_a_c_integer_does_not_hold_is_refused(i2s):
    st = Setup(i2s, 2, 64, 16, [20], [1], seed=23)
    q = torch.zeros((1, 4, 64), device="cuda")
    for window in (1 << 32, -(1 << 32)):
        with pytest.raises(ValueError, match="out of range"):
            i2s.Kv8Attention(st.cache, st.batch, q, window=window)
    i2s.Kv8Attention(st.cache, st.batch, q, window=(1 << 31) - 1)()
    assert st.batch.status() == 0


def test_status_is_read_and_cleared_in_the_order_of_its_stream(i2s):
    st = Setup(i2s, 2, 64, 16, [40], [1], seed=24)
    q = torch.zeros((1, 4, 64), device="cuda")
    call = i2s.Kv8Attention(st.cache, st.batch, q)
    st.batch.page_table[0, 1] = -1
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):   # each call's bit is there, none of an earlier one's, none cleared late
            call()
            assert st.batch.status() == i2s.KV8_BAD_PAGE
            call()
            assert st.batch.status() == i2s.KV8_BAD_PAGE
            assert st.batch.status() == 0


@pytest.mark.parametrize("dim,group", [(64, 8), (128, 7), (128, 1)])
def test_f32_sums_of_one_sign_lose_little(i2s, dim, group):
    """Values of one sign, weights nearly alike: what a tensor core cuts off is always of that sign too, on average
    2^-24 of the sum (a unit in the last place is between 2^-24 and 2^-23 of it, and half of one is lost) at each of the
    32 steps (16 of two parts) of the 256 tokens summed at a time, when the sum is on average half of what it will be:
    32 * 2^-24 / 2 = 9.5e-7. Logits below 0.1 * 4, weights and the other sums add less than 2^-23 by their norm."""
    lens, news = [700, 990, 512], [60, 75, 47]
    st = Setup(i2s, 2, dim, 64, lens, news, seed=41)
    st.pool.codes[:, :, 1] = np.maximum(np.abs(st.pool.codes[:, :, 1]), 1)
    st.data.view(-1).copy_(torch.from_numpy(st.pool.bytes()))
    rng = np.random.default_rng(5)
    q, qf = rows_tensor(rng, st.rows, 2 * group, dim, "f32", std=0.1)
    got = i2s.kv8_attention(st.cache, st.batch, q).cpu().numpy()
    assert st.batch.status() == 0
    want = ref.attention(st.pool, st.table, lens, st.row_start, qf, dim ** -0.5, True, 0)[0]
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert off <= 32 * 2.0 ** -25 + 2.0 ** -23, off


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_sums_moved_while_the_maxima_grow(i2s, dim, dtype):
    """Logits that grow along the cache at another rate in each row, so O is scaled and moved at nearly every one of 16
    tiles: right, and the same bits every time. Two warpgroups share a query tile here (F32 rows always do, 16-bit rows
    where there are fewer than 152 pairs of tiles: 4 heads x 16)."""
    kv, group, n = 4, 2, 2048
    st = Setup(i2s, kv, dim, 64, [n], [n], seed=dim)
    rng = np.random.default_rng(8)
    sign = np.where(rng.random(dim) < 0.5, -1, 1)
    for b in range(n // 16):   # keys along one direction, longer and longer
        p, sub = st.table[0][b * 16 // 64], b * 16 % 64 // 16
        at = slice(sub * 16, sub * 16 + 16)
        st.pool.codes[p, :, 0, at] = np.clip(100 * sign + rng.normal(0, 10, (kv, 16, dim)), -127, 127).astype(np.int8)
        st.pool.scales[p, :, 0, sub] = 1e-4 * (b + 1)
    st.data.view(-1).copy_(torch.from_numpy(st.pool.bytes()))
    st.pool = ref.Pool(st.pool.bytes(), kv, dim, 64)
    # a row's logits reach 0 to 80 (115 in powers of two): up to 7 a tile, past the slack of 6
    x = rng.random((n, kv * group, 1)) * sign * (80 / (dim * 100 * 1e-4 * 128) * dim ** 0.5) + rng.normal(0, 0.05, (n, kv * group, dim))
    q = torch.from_numpy(x.astype(np.float32)).to(DTYPES[dtype]).cuda()
    check_attention(i2s, st, q, q.float().cpu().numpy(), dtype)
    assert st.batch.status() == 0
    call = i2s.Kv8Attention(st.cache, st.batch, q)
    call()
    first = call.out.clone()
    for _ in range(30):
        call()
        assert torch.equal(first, call.out)


@pytest.mark.parametrize("news", [[3, 1, 15], [40, 0, 100], [1] * 40])
@pytest.mark.parametrize("lead", [1, 5, 17, 70])
def test_a_batch_whose_first_row_is_not_row_0(i2s, lead, news):
    """row_start[0] > 0, as a slice of a larger batch's row starts has it: the rows before belong to no sequence, those
    behind are written, read and attended with as if they began at 0. Batches of few rows per sequence and of many."""
    kv, dim = 2, 64
    lens = [n + (11 * i) % 37 for i, n in enumerate(news)]
    st = Setup(i2s, kv, dim, 32, lens, news, seed=lead, pad_rows=3)
    rng = np.random.default_rng(lead)
    starts, rows = st.row_start + np.int32(lead), st.rows + lead
    batch = i2s.Kv8Batch(torch.from_numpy(starts).cuda(), st.batch.kv_len, st.batch.page_table, rows=rows,
                         max_rows=max(news))
    k, kf = rows_tensor(rng, rows, kv, dim, "f32", std=2.0)
    v, vf = rows_tensor(rng, rows, kv, dim, "f32", std=2.0)
    i2s.kv8_write(st.cache, batch, k, v)
    ref.write(st.pool, st.table, lens, starts, kf, vf)
    same_bits(st.pool_now(), st.pool.bytes())
    back = [torch.full((rows, kv, dim), 3.0, device="cuda") for _ in range(2)]
    i2s.kv8_read(st.cache, batch, *back)
    for which in (0, 1):
        want = np.full((rows, kv, dim), 3.0, np.float32)
        for s, n in enumerate(news):
            x, _ = ref.cached(st.pool, st.table, s, lens[s], which)
            want[starts[s]:starts[s + 1]] = x[lens[s] - n:].astype(np.float32)
        same_bits(back[which].cpu().numpy(), want)
    q, qf = rows_tensor(rng, rows, 4, dim, "f32")
    out, lse = torch.full((rows, 4, dim), 7.0, device="cuda"), torch.full((rows, 4), 99.0, device="cuda")
    i2s.kv8_attention(st.cache, batch, q, out=out, lse=lse)
    assert (out[:lead] == 7.0).all() and (lse[:lead] == 99.0).all()
    compare_attention(st, qf[lead:], "f32", True, 0, dim ** -0.5, out[lead:], lse[lead:],
                      np.full((st.rows, 4, dim), 7.0, np.float32))
    assert batch.status() == 0


@pytest.mark.parametrize("n,new,group,kv", [(32768, 320, 4, 8), (16000, 512, 5, 16), (8192, 512, 5, 16)])
def test_f16_sums_behind_a_heavy_first_token_lose_little(i2s, n, new, group, kv):
    """Values of one sign, and a first token with 2^16 times the weight of each of the others: the sum has most of its
    size from the start, so whatever the tensor core cuts off later, always towards zero, is cut from all of it. A step
    of 16 tokens aligns 16 products with the sum and cuts each at a quarter of the sum's unit, and the new sum at one:
    on average 16 / 8 + 1 / 2 = 2.5 units, of at most 2^-23 of the sum. With one query tile in a CTA (the first case has
    too few for two, the second too many tokens for f16) the sums are moved every 1024 tokens, and of the later chains
    each is small: 64 steps. The third has two (16 heads x 10 pairs, 8192 tokens), whose sums are not moved: 512 steps.
    The mean of the relative errors shows it below the rounding of the outputs, at most 2^-11 each, 5 standard deviations
    of whose mean over 655360 and more outputs are below 2e-6; the weights' rounding (f16) averages out over the tokens
    likewise, the first one's weight is a power of two. What is left is rounding in F32: together below 2^-17."""
    dim = 64
    st = Setup(i2s, kv, dim, 64, [n], [new], seed=n)
    rng = np.random.default_rng(6)
    pages = st.table[0][st.table[0] >= 0]
    st.pool.codes[:, :, 1] = rng.integers(40, 128, st.pool.codes[:, :, 1].shape)
    st.pool.codes[:, :, 0] = rng.integers(-3, 4, st.pool.codes[:, :, 0].shape)
    st.pool.scales[pages] = 0.01
    first = st.pool.codes[pages[0], :, 0]
    first[:, 0] = 110
    st.pool.codes[pages[0], :, 0] = first
    st.data.view(-1).copy_(torch.from_numpy(st.pool.bytes()))
    x = 16 * np.log(2.0) * dim ** 0.5 / (dim * 110 * 0.01) + rng.normal(0, 0.02, (new, kv * group, dim))
    q = torch.from_numpy(x).to(torch.float16).cuda()
    got = i2s.kv8_attention(st.cache, st.batch, q).double()
    assert st.batch.status() == 0
    off = 0.0
    pos = torch.arange(n - new, n, device="cuda")[:, None]
    for h in range(kv):
        k, v = (torch.from_numpy(np.ascontiguousarray(
            st.pool.codes[pages, h, which].reshape(-1, dim)[:n])).cuda().double() * np.float64(np.float32(0.01)) for which in (0, 1))
        for g in range(h * group, h * group + group):
            score = q[:, g].double() @ k.T * np.float64(np.float32(dim ** -0.5))
            score = score.masked_fill_(torch.arange(n, device="cuda") > pos, float("-inf"))
            want = torch.softmax(score, -1) @ v
            off += ((got[:, g] - want) / want).mean().item() / (kv * group)
    steps = 512 if n == 8192 else 64
    assert abs(off) <= steps * 2.5 * 2.0 ** -23 + 2.0 ** -17, off


@pytest.mark.parametrize("new", [2, 40])
def test_value_scales_up_to_2_87_are_used_and_larger_ones_are_nan(i2s, new):
    """Scales just below 2^87 give right rows in both kernels; from 2^87 on (values from 127 * 2^87, which kv8_write stores) the
    rows that see the block are NaN, and no others."""
    st = Setup(i2s, 1, 128, 64, [100], [new], seed=5)
    first = 100 - new   # row 0 sees tokens 31..first, row 1 32..first + 1
    page = st.table[0][0]
    q, qf = rows_tensor(np.random.default_rng(1), st.rows, 2, 128, "f32")
    st.pool.scales[page, 0, 1, 1] = np.float32(1.99 * 2.0 ** 86)   # tokens 16..31
    st.data.view(-1).copy_(torch.from_numpy(st.pool.bytes()))
    check_attention(i2s, st, q, qf, "f32", window=first - 31 + 1)
    for size in (2.0 ** 87, 1.5 * 2.0 ** 100, 2.0 ** 121):
        st.pool.scales[page, 0, 1, 1] = np.float32(size)
        st.data.view(-1).copy_(torch.from_numpy(st.pool.bytes()))
        out = i2s.kv8_attention(st.cache, st.batch, q, window=first - 31 + 1)
        assert out[0].isnan().all() and out[1:].isfinite().all()


@pytest.mark.parametrize("kv,group,lens,new,dtype", [
    (1, 2, [3000], 40, "f32"),        # split along the cache, joined
    (2, 6, [300, 130], 100, "f32"),   # a CTA for each query tile
    (2, 6, [300, 130], 100, "bf16"),
    (8, 8, [1000], 620, "bf16"),      # two query tiles in a CTA
])
def test_rows_of_a_kernel_that_gave_up_are_nan(i2s, kv, group, lens, new, dtype):
    """Waits that nothing ends run out after about a second, with copies and products under way: the call ends, the status
    says so, its rows are NaN whatever an earlier call left in the workspace, and the next call is right."""
    st = Setup(i2s, kv, 64, 64, lens, [new] * len(lens), seed=19, pad_rows=2)
    q, qf = rows_tensor(np.random.default_rng(3), st.rows, kv * group, 64, dtype)
    lse = torch.zeros((st.rows, kv * group), device="cuda")
    call = i2s.Kv8Attention(st.cache, st.batch, q, lse=lse)
    call.out.fill_(7.0)
    call()
    assert st.batch.status() == 0
    want, want_lse = call.out.clone(), lse.clone()
    args = call._args
    call._args = args[:6] + (ctypes.c_uint(i2s.KV8_CAUSAL | i2s.KV8_TEST_STALL),) + args[7:]
    call()
    with pytest.raises(i2s.I2SError) as e:
        st.batch.check()
    assert e.value.status == -6   # I2S_E_DEVICE_TIMEOUT
    last = st.rows - 2
    assert call.out[:last].isnan().all() and lse[:last].isnan().all()
    assert torch.equal(call.out[last:], want[last:])
    call._args = args
    for _ in range(2):
        call()
        assert torch.equal(call.out, want) and torch.equal(lse, want_lse)
        assert st.batch.status() == 0
    compare_attention(st, qf, dtype, True, 0, 64 ** -0.5, call.out, None, call.out.float().cpu().numpy())


def test_f32_sums_of_one_sign_over_many_tokens_lose_little(i2s):
    """20000 tokens in one CTA (8 heads x 10 query tiles: no split), values of one sign: 78 sums of 256 tokens, each of
    which loses on average 2.5 units, at most 2^-23 of it, at each of its 16 steps of high parts (the low parts have
    either sign), when it is on average half of what it will be: 16 * 2.5 * 2^-24; the 78 additions to the running sum
    round by at most 2^-24 of it, when it is on average half: 78 * 2^-25; operands of 22 bits and F32: 2^-22. In one
    accumulator 1250 steps would lose 1.9e-4."""
    kv, group, dim, n, new = 8, 4, 64, 20000, 320
    st = Setup(i2s, kv, dim, 64, [n], [new], seed=12)
    st.pool.codes[:, :, 1] = np.maximum(np.abs(st.pool.codes[:, :, 1]), 1)
    st.data.view(-1).copy_(torch.from_numpy(st.pool.bytes()))
    q, _ = rows_tensor(np.random.default_rng(5), new, kv * group, dim, "f32", std=0.1)
    got = i2s.kv8_attention(st.cache, st.batch, q).double()
    assert st.batch.status() == 0
    pos = torch.arange(n - new, n, device="cuda")[:, None]
    hidden = torch.arange(n, device="cuda") > pos
    k, v = (torch.from_numpy(ref.cached(st.pool, st.table, 0, n, which)[0]).cuda() for which in (0, 1))
    off = size = 0.0
    for h in range(kv * group):
        score = (q[:, h].double() @ k[:, h // group].T * np.float64(np.float32(dim ** -0.5))).masked_fill_(hidden, float("-inf"))
        want = torch.softmax(score, -1) @ v[:, h // group]
        off, size = off + (got[:, h] - want).square().sum().item(), size + want.square().sum().item()
    assert (off / size) ** 0.5 <= 16 * 2.5 * 2.0 ** -24 + 78 * 2.0 ** -25 + 2.0 ** -22


@pytest.mark.parametrize("dtype,dim", [("f16", 64), ("bf16", 128)])
def test_attention_of_16_bit_rows_split_along_a_long_cache(i2s, dtype, dim):
    """10 query tiles in all: 15 CTAs share the cache of each, 10 tiles of it or more, so each moves its sums once before
    its part is joined with the others'."""
    st = Setup(i2s, 2, dim, 64, [20000], [320], seed=27)
    q, qf = rows_tensor(np.random.default_rng(28), st.rows, 4, dim, dtype, std=1.5)
    check_attention(i2s, st, q, qf, dtype)
    assert st.batch.status() == 0


def test_two_query_tiles_in_a_cta_give_the_same_bits_every_time(i2s):
    st = Setup(i2s, 8, 128, 64, [1500, 900, 700], [800, 650, 700], seed=29)
    q, _ = rows_tensor(np.random.default_rng(30), st.rows, 24, 128, "bf16", std=1.5)
    call = i2s.Kv8Attention(st.cache, st.batch, q)
    call()
    first = call.out.clone()
    for _ in range(20):
        call.out.zero_()
        call()
        assert torch.equal(first, call.out)
