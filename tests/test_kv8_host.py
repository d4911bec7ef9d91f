"""The kv8_* calls on the host (no GPU): sizes, and every refusal before any CUDA call."""

import ctypes
import math

import numpy as np
import pytest

from int8_quantized_matmul_gb300 import build as libbuild
from tests import kv8_reference as ref

A = 1 << 40   # dummy addresses, never dereferenced


@pytest.fixture(scope="module")
def i2s():
    libbuild.build()
    from int8_quantized_matmul_gb300 import i2s as mod
    return mod


class Call:
    """Valid arguments of the kv8 calls, to be spoiled one at a time."""

    def __init__(self, i2s):
        self.L = i2s.lib
        self.E = {v: k for k, v in i2s.STATUS.items()}
        self.cache = i2s.kv8_cache(A, 100, 2, 128, 64)
        self.batch = i2s.kv8_batch(2 * A, 3 * A, 4 * A, 5 * A, 10, 20, 3, 10)
        self.q = i2s.kv8_rows(6 * A, 6 * 128, 128, 0)
        self.out = i2s.kv8_rows(7 * A, 6 * 128, 128, 0)
        self.k = i2s.kv8_rows(8 * A, 256, 128, 0)
        self.v = i2s.kv8_rows(9 * A, 256, 128, 0)
        self.q_heads, self.scale, self.flags, self.window, self.lse, self.ws, self.ws_bytes = 6, 0.1, 1, 0, None, 10 * A, 1 << 40

    def write(self):
        return self.L.kv8_write(self.cache, self.batch, self.k, self.v, None)

    def read(self):
        return self.L.kv8_read(self.cache, self.batch, self.k, self.v, None)

    def attend(self):
        return self.L.kv8_attention(self.cache, self.batch, self.q, self.q_heads, self.out, self.scale, self.flags,
                                    self.window, self.lse, self.ws, self.ws_bytes, None)

    def need(self):
        return self.L.kv8_attention_workspace(self.cache, self.batch, self.q_heads)


def test_page_bytes(i2s):
    for heads in (1, 8):
        for dim in (64, 128):
            for page in (16, 32, 64, 128, 256):
                assert i2s.kv8_page_bytes(heads, dim, page) == heads * ref.slab_bytes(dim, page)
    for bad in ((0, 128, 64), (1025, 128, 64), (1, 96, 64), (1, 0, 64), (1, 128, 48), (1, 128, 8), (1, 128, 512)):
        assert i2s.kv8_page_bytes(*bad) == 0


BAD = [
    ("I2S_E_NULL_PTR", "cache", "pages", None), ("I2S_E_BAD_SHAPE", "cache", "n_pages", 0),
    ("I2S_E_BAD_SHAPE", "cache", "n_pages", 1 << 31), ("I2S_E_BAD_SHAPE", "cache", "heads", 0),
    ("I2S_E_BAD_SHAPE", "cache", "head_dim", 96), ("I2S_E_BAD_SHAPE", "cache", "page_tokens", 24),
    ("I2S_E_MISALIGNED", "cache", "pages", A + 8), ("I2S_E_NULL_PTR", "batch", "row_start", None),
    ("I2S_E_NULL_PTR", "batch", "kv_len", None), ("I2S_E_NULL_PTR", "batch", "page_table", None),
    ("I2S_E_NULL_PTR", "batch", "status", None), ("I2S_E_BAD_SHAPE", "batch", "rows", 0),
    ("I2S_E_BAD_SHAPE", "batch", "seqs", 0), ("I2S_E_BAD_SHAPE", "batch", "seqs", 4097),
    ("I2S_E_BAD_SHAPE", "batch", "table_width", 0), ("I2S_E_BAD_SHAPE", "batch", "table_width", 1 << 25),
    ("I2S_E_BAD_SHAPE", "batch", "max_rows", 0), ("I2S_E_BAD_SHAPE", "batch", "max_rows", 11),
    ("I2S_E_MISALIGNED", "batch", "status", 5 * A + 2), ("I2S_E_MISALIGNED", "batch", "kv_len", 3 * A + 1),
]


@pytest.mark.parametrize("name", ["write", "read", "attend"])
def test_cache_and_batch_refusals(i2s, name):
    for want, part, field, value in BAD:
        c = Call(i2s)
        setattr(getattr(c, part), field, value)
        assert getattr(c, name)() == c.E[want], (part, field, value)


@pytest.mark.parametrize("name", ["write", "read", "attend"])
def test_blocks_are_counted_in_32_bits(i2s, name):
    c = Call(i2s)
    c.batch.seqs, c.batch.table_width = 1000, (1 << 34) // (1000 * 2 * 64) + 1
    assert getattr(c, name)() == c.E["I2S_E_BAD_SHAPE"]


@pytest.mark.parametrize("name,inputs,outputs", [("write", "kv", ""), ("read", "", "kv"), ("attend", ["q"], ["out"])])
def test_row_tensor_refusals(i2s, name, inputs, outputs):
    for t in list(inputs) + list(outputs):
        for want, field, value in (("I2S_E_NULL_PTR", "data", None), ("I2S_E_MISALIGNED", "data", 20 * A + 8),
                                   ("I2S_E_BAD_SHAPE", "row_stride", -256), ("I2S_E_BAD_SHAPE", "row_stride", 1 << 38),
                                   ("I2S_E_MISALIGNED", "head_stride", 130),
                                   ("I2S_E_BAD_ARG", "dtype", 3), ("I2S_E_BAD_ARG", "dtype", -1)):
            c = Call(i2s)
            setattr(getattr(c, t), field, value)
            assert getattr(c, name)() == c.E[want], (t, field, value)
        c = Call(i2s)   # two dtypes
        getattr(c, t).dtype = 2
        assert getattr(c, name)() == c.E["I2S_E_BAD_ARG"]
    for t in outputs:   # elements that coincide
        for rs, hs in ((0, 128), (256, 0), (128, 128), (768, 64)):
            c = Call(i2s)
            getattr(c, t).row_stride, getattr(c, t).head_stride = rs, hs
            assert getattr(c, name)() == c.E["I2S_E_BAD_ARG"], (t, rs, hs)


def test_overlaps_are_refused(i2s):
    size = 100 * i2s.kv8_page_bytes(2, 128, 64)
    for name, t, at in (("write", "k", A), ("write", "v", A + size - 16), ("read", "k", A), ("read", "v", 8 * A + 16),
                        ("read", "k", 4 * A), ("attend", "out", 6 * A), ("attend", "out", A + 16), ("attend", "out", 10 * A),
                        ("attend", "out", 2 * A)):
        c = Call(i2s)
        getattr(c, t).data = at
        assert getattr(c, name)() == c.E["I2S_E_BAD_ARG"], (name, t, at)
    for at in (6 * A, 7 * A, A, 10 * A):
        c = Call(i2s)
        c.lse = at
        assert c.attend() == c.E["I2S_E_BAD_ARG"]
    for at in (6 * A, A, 3 * A):
        c = Call(i2s)
        c.ws = at
        assert c.attend() == c.E["I2S_E_BAD_ARG"]
    c = Call(i2s)
    c.cache.pages = 5 * A - 1024   # the pool over the status word
    assert c.write() == c.E["I2S_E_BAD_ARG"]


def test_read_outputs_may_be_slices_of_one_row(i2s):
    for off, ok in ((256, True), (128, False), (384, False), (-256, True)):
        c = Call(i2s)
        c.k = i2s.kv8_rows(8 * A, 512, 128, 0)
        c.v = i2s.kv8_rows(8 * A + 4 * off, 512, 128, 0)
        assert (c.read() == c.E["I2S_E_BAD_ARG"]) == (not ok), off


def test_attention_refusals(i2s):
    for want, field, value in (("I2S_E_BAD_SHAPE", "q_heads", 0), ("I2S_E_BAD_SHAPE", "q_heads", 5),
                               ("I2S_E_BAD_SHAPE", "q_heads", 130), ("I2S_E_BAD_ARG", "flags", 2),
                               ("I2S_E_BAD_ARG", "window", -1), ("I2S_E_BAD_ARG", "scale", math.nan),
                               ("I2S_E_BAD_ARG", "scale", math.inf), ("I2S_E_NULL_PTR", "ws", None),
                               ("I2S_E_MISALIGNED", "ws", 10 * A + 16), ("I2S_E_MISALIGNED", "lse", 11 * A + 2)):
        c = Call(i2s)
        setattr(c, field, value)
        assert c.attend() == c.E[want], (field, value)
    c = Call(i2s)
    c.flags, c.window = 0, 8
    assert c.attend() == c.E["I2S_E_BAD_ARG"]   # a window needs KV8_CAUSAL
    c = Call(i2s)
    c.ws_bytes = c.need() - 1
    assert c.need() > 0 and c.attend() == c.E["I2S_E_WORKSPACE_TOO_SMALL"]
    for field, value in (("seqs", 0), ("rows", 0), ("max_rows", 11)):
        c = Call(i2s)
        setattr(c.batch, field, value)
        assert c.need() == 0
    c = Call(i2s)
    c.q_heads = 5
    assert c.need() == 0


def test_norm_rope_refusals(i2s):
    L, E = i2s.lib, {v: k for k, v in i2s.STATUS.items()}
    rows = i2s.kv8_rows

    def call(q=None, q_out=None, qh=6, gq=None, k=None, k_out=None, kh=2, gk=None, n=10, dim=128, eps=1e-6, pos=20 * A,
             turns=21 * A, rot=128, flags=0):
        return L.kv8_norm_rope(q or rows(A, 768, 128, 0), q_out or rows(2 * A, 768, 128, 0), qh, gq,
                               k or rows(3 * A, 256, 128, 0), k_out or rows(4 * A, 256, 128, 0), kh, gk, n, dim, eps, pos,
                               turns, rot, flags, None)
    for want, kw in (("I2S_E_BAD_SHAPE", {"qh": -1}), ("I2S_E_BAD_SHAPE", {"qh": 0, "kh": 0}), ("I2S_E_BAD_SHAPE", {"n": 0}),
                     ("I2S_E_BAD_SHAPE", {"dim": 80}), ("I2S_E_BAD_SHAPE", {"rot": 12}), ("I2S_E_BAD_SHAPE", {"rot": 136}),
                     ("I2S_E_BAD_SHAPE", {"rot": -8}), ("I2S_E_NULL_PTR", {"pos": None}), ("I2S_E_NULL_PTR", {"turns": None}),
                     ("I2S_E_BAD_ARG", {"eps": -1.0}), ("I2S_E_BAD_ARG", {"eps": math.nan}), ("I2S_E_BAD_ARG", {"flags": 2}),
                     ("I2S_E_MISALIGNED", {"gq": 5 * A + 4}), ("I2S_E_MISALIGNED", {"turns": 21 * A + 4}),
                     ("I2S_E_NULL_PTR", {"q": rows(None, 768, 128, 0)}), ("I2S_E_BAD_ARG", {"q": rows(A, 768, 128, 1)}),
                     ("I2S_E_BAD_ARG", {"k": rows(3 * A, 256, 128, 1), "k_out": rows(4 * A, 256, 128, 1)}),
                     ("I2S_E_BAD_ARG", {"q_out": rows(A + 64, 768, 128, 0)}),          # over its input, not in place
                     ("I2S_E_BAD_ARG", {"q_out": rows(3 * A, 768, 128, 0)}),           # over the other input
                     ("I2S_E_BAD_ARG", {"q_out": rows(4 * A, 768, 128, 0)}),           # over the other output
                     ("I2S_E_BAD_ARG", {"q_out": rows(2 * A, 128, 128, 0)}),           # onto itself
                     ("I2S_E_BAD_ARG", {"gq": 2 * A + 16}), ("I2S_E_BAD_ARG", {"pos": 4 * A + 64}),
                     ("I2S_E_BAD_ARG", {"turns": 2 * A})):                             # over a small operand
        assert call(**kw) == E[want], kw
    # in place in fused rows: slices of one row, but not the same or crossing ones
    fused = rows(A, 1280, 128, 0)
    for off, ok in ((768, True), (640, False), (0, False), (1152, False)):
        k = rows(A + 4 * off, 1280, 128, 0)
        got = call(q=fused, q_out=fused, k=k, k_out=k)
        assert (got == E["I2S_E_BAD_ARG"]) == (not ok), off


def test_rope_turns(i2s):
    turns = np.zeros(64, np.uint64)
    assert i2s.lib.kv8_rope_turns_host(10000.0, 128, turns.ctypes.data) == 0
    want = [10000.0 ** (-2 * i / 128) / (2 * math.pi) for i in range(64)]
    got = turns.astype(np.float64) / 2.0 ** 64
    # a power and a quotient in binary64, cut to whole 2^-64 turns
    np.testing.assert_allclose(got, want, rtol=2.0 ** -50, atol=2.0 ** -64)
    for base, rot in ((10000.0, 4), (10000.0, 12), (10000.0, 136)):
        assert i2s.lib.kv8_rope_turns_host(base, rot, turns.ctypes.data) == -1
    for base in (0.5, math.inf, math.nan):
        assert i2s.lib.kv8_rope_turns_host(base, 128, turns.ctypes.data) == -8
    assert i2s.lib.kv8_rope_turns_host(10000.0, 128, None) == -2


def test_read_status_needs_a_word(i2s):
    assert i2s.lib.kv8_read_status(None, ctypes.byref(ctypes.c_int32()), None) == -2


def test_reference_quantizer_and_round_trip():
    """The numpy definition itself: halves away from zero, the floor, and one-by-one appends that only ever grow a scale."""
    assert ref.quantize(np.array([0.5, -0.5, 1.5, 0.49999997, 200.0], np.float32), 1.0).tolist() == [1, -1, 2, 0, 127]
    rng = np.random.default_rng(0)
    pool = ref.Pool(np.zeros(2 * ref.slab_bytes(64, 16), np.uint8), 1, 64, 16)
    x = rng.standard_normal((20, 1, 64)).astype(np.float32)
    last = 0.0
    for n in range(1, 21):
        ref.write(pool, [[0, 1]], [n], [0, 1], x[n - 1:n], x[n - 1:n])
        if n <= 16:
            assert pool.scales[0, 0, 0, 0] >= last
            last = pool.scales[0, 0, 0, 0]
    back, there = ref.cached(pool, [[0, 1]], 0, 20, 0)
    assert there.all()
    # each growth requantizes once: at most 16 half steps of the final scale
    assert np.abs(back[:16] - x[:16]).max() <= 8 * last
    ref.write(pool, [[0, 1]], [20], [0, 20], x, x)   # at once: half a step
    back, _ = ref.cached(pool, [[0, 1]], 0, 20, 0)
    assert np.abs(back[:16] - x[:16]).max() <= 0.5001 * np.abs(x[:16]).max() / 127


def test_query_rows_of_a_head_are_counted_in_32_bits(i2s):
    c = Call(i2s)
    c.batch.rows, c.q_heads = 1 << 25, 128
    c.batch.max_rows = (1 << 24) - 1
    assert c.need() > 0
    c.batch.max_rows = 1 << 24   # times 64 query heads: 2^30
    assert c.need() == 0 and c.attend() == c.E["I2S_E_BAD_SHAPE"]


def test_sizes_that_a_c_integer_does_not_hold_are_refused(i2s):
    torch = pytest.importorskip("torch")
    starts, lens, table = (torch.zeros(n, dtype=torch.int32) for n in (3, 2, 8))
    for kw in ({"rows": 10, "max_rows": (1 << 32) + 4}, {"rows": (1 << 64) + 10, "max_rows": 4}):
        with pytest.raises(ValueError, match="out of range"):
            i2s.Kv8Batch(starts, lens, table.view(2, 4), **kw)


def test_a_batch_or_workspace_on_another_device_is_refused(i2s):
    """Before any pointer is taken: the kernels would follow those of another device."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace as Some
    here, there = torch.device("cuda:0"), torch.device("cuda:1")
    cache = Some(device=here, heads=2, head_dim=64)
    for call in (i2s.Kv8Write, i2s.Kv8Read):
        with pytest.raises(ValueError, match="batch: on cuda:1, the cache is on cuda:0"):
            call(cache, Some(device=there, rows=1), None, None)
    with pytest.raises(ValueError, match="batch: on cuda:1, the cache is on cuda:0"):
        i2s.Kv8Attention(cache, Some(device=there, rows=1), None)
    for ws in (there, torch.device("cpu")):
        with pytest.raises(ValueError, match="ws: on "):
            i2s.Kv8Attention(cache, Some(device=here, rows=1), None, ws=Some(device=ws))


def test_status_of_a_batch_on_another_device_is_refused(i2s, monkeypatch):
    """The current stream is the current device's: the word would be read before the calls that set it."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    batch = i2s.Kv8Batch.__new__(i2s.Kv8Batch)
    batch.device = torch.device("cuda:1")
    for read in (batch.status, batch.check):
        with pytest.raises(ValueError, match="not on the current device"):
            read()


def test_norm_rope_does_not_look_at_arguments_it_ignores(i2s):
    """The gamma of a tensor without heads, and positions and turns where nothing turns: any pointer will do."""
    E = {v: k for k, v in i2s.STATUS.items()}
    q, out = i2s.kv8_rows(A, 768, 128, 0), i2s.kv8_rows(2 * A, 768, 128, 0)

    def call(gk=None, pos=20 * A, turns=21 * A, rot=128):
        return i2s.lib.kv8_norm_rope(q, out, 6, None, None, None, 0, gk, 10, 128, 1e-6, pos, turns, rot, 0, None)
    want = call()   # valid: ends at the device check where there is no GPU
    assert want not in (E["I2S_E_MISALIGNED"], E["I2S_E_BAD_ARG"], E["I2S_E_NULL_PTR"])
    for kw in ({"gk": 5 * A + 4}, {"gk": 2 * A}, {"rot": 0, "pos": 20 * A + 2}, {"rot": 0, "turns": 21 * A + 4},
               {"rot": 0, "pos": 2 * A}):
        assert call(**kw) == want, kw
