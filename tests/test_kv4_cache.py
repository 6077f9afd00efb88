"""The paged 4-bit cache: writing and reading back bit for bit against the rule
and the layout, at every part of a block of 16 tokens, strides, non-finite rows,
far pages, bad indices, and the refusals."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_ref as ref
from kv_ref import ints, offsets

FAKE = 0x7F0000000000
gpu = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


class Twin:
    """A cache and what it has to hold: codes and scales on the CPU."""

    def __init__(self, batch, width, heads, dim, page, seed=0):
        from accelerator_gb300 import lowbit
        rng = np.random.default_rng(seed)
        pages = batch * width + 3
        self.table = rng.permutation(pages)[:batch * width].reshape(batch, width).astype(np.int32)
        self.codes = [torch.from_numpy(rng.integers(-7, 8, (pages, heads, page, dim))) for _ in range(2)]
        self.scales = [torch.from_numpy(rng.random((pages, heads, page), dtype=np.float32)).to(torch.bfloat16) for _ in range(2)]
        self.cache = lowbit.Kv4Cache(ref.pack(self.codes, self.scales, page, dim).cuda(), page, dim)
        self.page, self.dim, self.heads, self.rng = page, dim, heads, rng

    def rows(self, n, kind, spread=1.0):
        x = self.rng.standard_normal((n, self.heads, self.dim)).astype(np.float32) * np.float32(spread)
        return torch.from_numpy(x).to(DTYPES[kind])

    def put(self, both, starts, first):
        for x, codes, scales in zip(both, self.codes, self.scales):
            c, s = ref.quantise(x)
            for b in range(len(first)):
                for i in range(starts[b + 1] - starts[b]):
                    pos = first[b] + i
                    where = (self.table[b, pos // self.page], slice(None), pos % self.page)
                    codes[where], scales[where] = c[starts[b] + i], s[starts[b] + i]

    def same(self):
        got, want = self.cache.data.cpu(), ref.pack(self.codes, self.scales, self.page, self.dim)
        half = self.page * self.dim
        assert torch.equal(got[..., :half], want[..., :half])
        a, b = (x[..., half:].contiguous().view(torch.bfloat16).float() for x in (got, want))
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))

    def tokens(self, starts, first):
        """(K, V) in float32 of the rows of a batch."""
        found = []
        for codes, scales in zip(self.codes, self.scales):
            rows = []
            for b in range(len(first)):
                for pos in range(first[b], first[b] + starts[b + 1] - starts[b]):
                    where = (self.table[b, pos // self.page], slice(None), pos % self.page)
                    rows.append(codes[where].float() * scales[where].float()[:, None])
            found.append(torch.stack(rows))
        return found


def test_the_layout_has_a_place_for_each_element():
    for page in (16, 32, 64, 128):
        for dim in (64, 128):
            (keys, values), nibble = ref.places(page, dim)
            every = torch.cat([2 * at + nibble for at in (keys, values)]).flatten().sort().values
            assert torch.equal(every, torch.arange(2 * page * dim))


def test_the_rule_against_64_bits():
    """c is the nearest integer to x / s, and s within half a step of bfloat16 of max / 7."""
    g = torch.Generator().manual_seed(0)
    for kind in DTYPES.values():
        x = (torch.randn(500, 128, generator=g) * torch.exp(torch.randn(500, 1, generator=g) * 2)).to(kind)
        c, s = ref.quantise(x)
        top = x.double().abs().amax(-1) / 7
        assert ((s.double() - top).abs() <= top * (2.0 ** -8 + 2.0 ** -23)).all()
        assert ((c - x.double() / s.double()[:, None]).abs() <= 0.5 + 7.1 * 2.0 ** -24 + 0.04 * (c.abs() == 7)).all()


@gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_append_and_read(libgemm, page, dim, kind):
    from accelerator_gb300 import lowbit
    heads = 3
    p = Twin(7, 4, heads, dim, page, seed=page + dim)
    at = np.array([0, page - 1, page, 5, 0, 2 * page + 3, 1])
    for counts, spread in (([1, 1, 1, 1, 1, 1, 1], 0.3), ([page, 2, 0, page + 1, 3 * page // 2, 1, 2], 1.0),
                           ([1, 0, 1, 2, 1, page // 2, 1], 4.0), ([1, 1, 1, 1, 1, 1, 1], 1e-3)):
        starts = offsets(counts)
        both = [p.rows(int(starts[-1]), kind, spread) for _ in range(2)]
        lowbit.kv_append(p.cache, both[0].cuda(), both[1].cuda(), ints(p.table), ints(starts), ints(at))
        assert libgemm.debug_status() == libgemm.OK
        p.put(both, starts, at)
        p.same()
        at = at + counts
    for first in (at * 0, np.maximum(at - 3, 0)):
        starts = offsets(at - first)
        want = p.tokens(starts, first)
        for back in DTYPES.values():
            got = lowbit.kv_read(p.cache, ints(p.table), ints(starts), ints(first), int(starts[-1]), dtype=back)
            for x, y in zip(got, want):
                assert torch.equal(x.cpu(), y.to(back))
    assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("heads", [1, 4, 5])
@pytest.mark.parametrize("dim", [64, 128])
def test_every_part_of_a_block(libgemm, dim, heads):
    """Each first token and count of a block of 16, and the rest left as it was."""
    from accelerator_gb300 import lowbit
    p = Twin(16, 3, heads, dim, 16, seed=heads)
    for n in (1, 2, 3, 15, 16, 17, 20):
        starts, first = offsets([n] * 16), np.arange(16)
        both = [p.rows(16 * n, "bf16") for _ in range(2)]
        lowbit.kv_append(p.cache, both[0].cuda(), both[1].cuda(), ints(p.table), ints(starts), ints(first))
        p.put(both, starts, first)
        p.same()
    assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_append_strided(libgemm, kind, shift):
    """Slices of one joint projection, with rows that are not 16-byte aligned too."""
    from accelerator_gb300 import lowbit
    p = Twin(2, 3, 2, 64, 16, seed=3)
    joint = torch.randn(40, 5 * 2 * 64 + 1 + shift, device="cuda").to(DTYPES[kind])
    K = joint[:, 128 + shift:256 + shift].unflatten(1, (2, 64))
    V = joint[:, 256 + shift:512 + shift].unflatten(1, (2, 128))[:, :, 3:67]
    starts, first = np.array([0, 25, 40]), np.array([9, 30])
    lowbit.kv_append(p.cache, K, V, ints(p.table), ints(starts), ints(first))
    p.put([K.cpu(), V.cpu()], starts, first)
    p.same()
    assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_append_non_finite(libgemm, bad):
    """The token and head that was given one reads as NaN, the others as they would."""
    from accelerator_gb300 import lowbit
    p = Twin(1, 2, 2, 128, 16, seed=4)
    both = [p.rows(12, "fp32"), p.rows(12, "fp32")]
    both[0][7, 1, 5] = both[1][3, 0, 127] = bad
    starts, first = np.array([0, 12]), np.array([10])
    lowbit.kv_append(p.cache, both[0].cuda(), both[1].cuda(), ints(p.table), ints(starts), ints(first))
    p.put(both, starts, first)
    p.same()
    K, V = lowbit.kv_read(p.cache, ints(p.table), ints([0, 12]), ints([10]), 12, dtype=torch.float32)
    for x, (row, head) in ((K, (7, 1)), (V, (3, 0))):
        nan = torch.isnan(x)
        assert nan[row, head].all() and nan.sum() == 128


@gpu
@pytest.mark.parametrize("value", [0.0, 1e-38, 2.0 ** -126 * 7, 2.0 ** -110, 1e-30, 3e38])
def test_append_zeros_and_tiny_and_huge(libgemm, value):
    from accelerator_gb300 import lowbit
    p = Twin(1, 1, 1, 64, 16, seed=5)
    x = torch.clamp(p.rows(5, "fp32"), -1, 1) * value
    x[1] = value * 0.5       # halves of a step, and a row of one value
    x[2, :, 1:] = x[2, :, :1] * 0.5 / 7
    lowbit.kv_append(p.cache, x.cuda(), x.cuda(), ints(p.table), ints([0, 5]), ints([0]))
    p.put([x, x], np.array([0, 5]), np.array([0]))
    p.same()


@gpu
def test_one_page_in_two_sequences(libgemm):
    """A shared first page, whose other tokens two sequences write in one call."""
    from accelerator_gb300 import lowbit
    p = Twin(2, 2, 2, 64, 16, seed=6)
    p.table[1, 0] = p.table[0, 0]
    both = [p.rows(9, "fp16") for _ in range(2)]
    starts, first = np.array([0, 5, 9]), np.array([2, 7])
    lowbit.kv_append(p.cache, both[0].cuda(), both[1].cuda(), ints(p.table), ints(starts), ints(first))
    p.put(both, starts, first)
    p.same()


@gpu
def test_pages_past_32_bit_offsets(libgemm):
    """A pool of more than 2^32 bytes, written, read and attended to at its far end."""
    from accelerator_gb300 import lowbit
    pages, heads, page, dim = 70000, 4, 128, 128
    cache = lowbit.Kv4Cache.empty(pages, heads, dim, page)
    table = ints([[pages - 1, 3, pages - 2]])
    K, V = (torch.randn(300, heads, dim, device="cuda") for _ in range(2))
    lowbit.kv_append(cache, K, V, table, ints([0, 300]), ints([0]))
    k, v = lowbit.kv_read(cache, table, ints([0, 300]), ints([0]), 300, dtype=torch.float32)
    for x, y in ((k, K), (v, V)):
        assert ((x - y).abs() <= y.abs().amax(-1, keepdim=True) / 7 * 0.55).all()
    for rows in (2, 100):
        Q = torch.randn(rows, 8, dim, device="cuda").to(torch.bfloat16)
        O = lowbit.kv_attention(Q, cache, table, ints([0, rows]), ints([300])).double()
        a = torch.einsum("thgd,nhd->thgn", Q.double().view(rows, heads, 2, dim), k.double()) / dim ** 0.5
        hide = torch.arange(300, device="cuda") > torch.arange(300 - rows, 300, device="cuda")[:, None]
        want = torch.einsum("thgn,nhd->thgd", a.masked_fill(hide[:, None, None], -float("inf")).softmax(-1), v.double())
        assert (O - want.reshape(rows, 8, dim)).abs().max() <= 0.01 * want.abs().max()
    assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("rows", [2, 60])
def test_bad_indices_are_reported(libgemm, rows):
    """Page numbers, positions and offsets out of range: nothing outside the
    cache is touched, and the next status says so."""
    from accelerator_gb300 import lowbit
    p = Twin(2, 8, 1, 64, 16, seed=16)
    Q, K = (torch.randn(2 * rows, h, 64, device="cuda").to(torch.bfloat16) for h in (2, 1))
    good = dict(table=p.table, starts=[0, rows, 2 * rows], at=[65, 66])
    pages = p.cache.data.shape[0]
    high, low = p.table.copy(), p.table.copy()
    high[0, 4], low[1, 4] = pages, -1
    for change in (dict(table=high), dict(table=low), dict(at=[20, 129]), dict(at=[-1, 30]), dict(starts=[0, 2 * rows + 1, 2 * rows]),
                   dict(starts=[0, rows, 2000]), dict(starts=[0, -3, 2 * rows]), dict(starts=[1, rows, 2 * rows])):
        a = {**good, **change}
        table, starts, at = ints(a["table"]), ints(a["starts"]), ints(a["at"])
        for call in (lambda: lowbit.kv_append(p.cache, K, K, table, starts, at),
                     lambda: lowbit.kv_read(p.cache, table, starts, at, 2 * rows),
                     lambda: lowbit.kv_attention(Q, p.cache, table, starts, at)):
            assert libgemm.debug_status() == libgemm.OK
            call()
            assert libgemm.debug_status() == libgemm.ERR_INDEX, change
            assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("width", [40, 200])     # the long one takes scratch and a second launch
def test_capture_and_other_stream(libgemm, width):
    from accelerator_gb300 import lowbit
    p = Twin(2, width, 2, 128, 64, seed=17)
    n = 50 * width
    table, starts, first, lengths = ints(p.table), ints([0, 1, 2]), ints([n, 55]), ints([n + 1, 56])
    K, V, Q = p.rows(2, "bf16").cuda(), p.rows(2, "bf16").cuda(), torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)

    def step(stream=None):
        lowbit.kv_append(p.cache, K, V, table, starts, first, stream=stream)
        return (lowbit.kv_attention(Q, p.cache, table, starts, lengths, stream=stream),
                *lowbit.kv_read(p.cache, table, starts, first, 2, stream=stream))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert libgemm.debug_status() == libgemm.OK


@gpu
def test_handles_and_refusals_of_the_binding(libgemm, monkeypatch):
    import copy
    from accelerator_gb300 import lowbit
    p = Twin(2, 3, 2, 64, 16)
    table, starts, at = ints(p.table), ints([0, 1, 2]), ints([3, 4])
    Q, K = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16), p.rows(2, "bf16").cuda()
    c = p.cache
    with pytest.raises(AttributeError):
        c.heads = 3
    other = copy.deepcopy(c)
    assert other.data.data_ptr() != c.data.data_ptr() and torch.equal(other.data, c.data)
    assert torch.equal(lowbit.kv_attention(Q, other, table, starts, at), lowbit.kv_attention(Q, c, table, starts, at))
    for bad in ((c.data[:, :, :-1], 16, 64), (c.data, 24, 64), (c.data, 16, 96), (c.data, 16, 128), (c.data.float(), 16, 64),
                (c.data.cpu(), 16, 64), (c.data[::2], 16, 64), (c.data[0], 16, 64)):
        with pytest.raises(TypeError):
            lowbit.Kv4Cache(*bad)
    with pytest.raises(TypeError):
        lowbit.kv_attention(Q.float(), c, table, starts, at)
    with pytest.raises(TypeError):
        lowbit.kv_attention(Q[:, :, :32], c, table, starts, at)
    with pytest.raises(libgemm.GemmError, match="gemm_kv4_attention"):
        lowbit.kv_attention(Q[:, :3], c, table, starts, at)          # 3 heads over 2
    with pytest.raises(libgemm.GemmError):
        lowbit.kv_attention(Q, c, table, starts, at, out=Q)
    with pytest.raises(libgemm.GemmError):
        lowbit.kv_attention(Q, c, table, starts, at, causal=False, window=5)
    with pytest.raises(TypeError):
        lowbit.kv_append(c, K, K.float(), table, starts, at)
    with pytest.raises(ValueError):
        lowbit.kv_append(c, K, K[:1], table, starts, at)
    count = libgemm.launch_count()
    monkeypatch.setattr(lowbit, "_current_device", lambda: 1)
    for call in (lambda: lowbit.kv_append(c, K, K, table, starts, at), lambda: lowbit.kv_read(c, table, starts, at, 2),
                 lambda: lowbit.kv_attention(Q, c, table, starts, at)):
        with pytest.raises(TypeError):
            call()
    assert libgemm.launch_count() == count


# ---- without a GPU ---------------------------------------------------------------

G = 1 << 24


class CKv4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int32), ("page", ctypes.c_int32),
                ("dim", ctypes.c_int32)]


def _call(libgemm, what, **change):
    a = dict(data=FAKE, pages=10, heads=2, page=16, dim=64, X=FAKE + 4 * G, Y=FAKE + 5 * G, row=128, head=64, kind=1, q_heads=2,
             scale=0.125, causal=1, window=0, table=FAKE + 6 * G, width=5, starts=FAKE + 7 * G, at=FAKE + 8 * G, tokens=4,
             sequences=2)
    a.update(change)
    p = lambda n: a[n] or None      # noqa: E731
    c = CKv4(p("data"), a["pages"], a["heads"], a["page"], a["dim"])
    tail = (p("table"), a["width"], p("starts"), p("at"), a["tokens"], a["sequences"], None)
    lib = libgemm.lib()
    ref_c = None if a.get("null") else ctypes.byref(c)
    if what == "append":
        return lib.gemm_kv4_append(ref_c, p("X"), a["row"], a["head"], p("Y"), a["row"], a["head"], a["kind"], *tail)
    if what == "read":
        return lib.gemm_kv4_read(ref_c, p("X"), p("Y"), a["kind"], *tail)
    return lib.gemm_kv4_attention(ref_c, p("X"), a["row"], a["head"], p("Y"), a["row"], a["head"], a["kind"], a["q_heads"],
                                  a["scale"], a["causal"], a["window"], *tail)


@pytest.mark.parametrize("what", ["append", "read", "attention"])
@pytest.mark.parametrize("change,want", [
    ({"null": 1}, 1), ({"dim": 96}, 1), ({"page": 24}, 1), ({"page": 8}, 1), ({"heads": 0}, 1), ({"pages": -1}, 1),
    ({"tokens": -1}, 1), ({"tokens": 1 << 31}, 1), ({"sequences": 0}, 1), ({"width": -1}, 1), ({"width": 1 << 27}, 1), ({"kind": 3}, 1),
    ({"data": 0}, 1), ({"table": 0}, 1), ({"starts": 0}, 1), ({"at": 0}, 1), ({"X": 0}, 1), ({"Y": 0}, 1),
    ({"data": FAKE + 8}, 2), ({"table": FAKE + 6 * G + 1}, 2), ({"X": FAKE + 4 * G + 1}, 2),
    ({"Y": FAKE + 10 * 2 * 16 * 68 - 16}, 1), ({"tokens": 0, "sequences": 0, "X": 0, "Y": 0}, 0)])
def test_shared_checks(libgemm, what, change, want):
    assert _call(libgemm, what, **change) == want


@pytest.mark.parametrize("change", [{"kind": 0}, {"q_heads": 3}, {"q_heads": 0}, {"window": -1}, {"window": 4, "causal": 0},
                                    {"scale": float("nan")}, {"row": -1}, {"head": -64}, {"Y": FAKE + 4 * G}])
def test_attention_checks(libgemm, change):
    assert _call(libgemm, "attention", **change) == libgemm.ERR_INVALID_ARG


def test_no_device_is_an_error(libgemm):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for what in ("append", "read", "attention"):
        assert _call(libgemm, what) in (libgemm.ERR_CUDA, libgemm.ERR_UNSUPPORTED_DEVICE)
