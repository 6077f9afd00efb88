"""The paged 8-bit cache: writing and reading back bit for bit against the
rule, attention over it against 64 bits, at lengths around every page and tile
edge, head layouts, masks that leave rows empty, strides, poisoned memory that
must not be read, and the refusals."""
import ctypes

import numpy as np
import pytest

import lowbit_ref as ref

FAKE = 0x7F0000000000
gpu = pytest.mark.gpu


def dtypes():
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def ints(x):
    import torch
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def as_numpy(t):
    return t.float().cpu().numpy()


class Pool:
    """A cache of random contents, its twin in numpy, and page tables that
    hand out its pages in a shuffled order."""

    def __init__(self, batch, width, heads, dim, page, seed=0, spare=3):
        import torch
        from accelerator_gb300 import lowbit
        self.rng = np.random.default_rng(seed)
        pages = batch * width + spare
        shape = (pages, heads, page, dim)
        k, v = (np.clip(np.rint(self.rng.standard_normal(shape) * 32), -127, 127).astype(np.int64) for _ in range(2))
        ks, vs = (np.exp(self.rng.standard_normal(shape[:2])).astype(np.float32) * np.float32(0.02) for _ in range(2))
        self.k, self.v = (ref.Cache((c + 128).astype(np.uint8), s, page) for c, s in ((k, ks), (v, vs)))
        self.table = self.rng.permutation(pages)[:batch * width].reshape(batch, width).astype(np.int32)
        self.gpu = lowbit.KvCache(*(torch.from_numpy((c + 128).astype(np.uint8)).cuda() for c in (k, v)),
                                  *(torch.from_numpy(s).cuda() for s in (ks, vs)))
        self.page, self.heads, self.dim = page, heads, dim

    def rows(self, n, heads, kind, spread=1.0):
        import torch
        x = self.rng.standard_normal((n, heads, self.dim)).astype(np.float32) * np.float32(spread)
        return torch.from_numpy(x).cuda().to(dtypes()[kind])

    def same(self):
        """The GPU's cache holds what its twin does, every byte of it."""
        for twin, codes, scales in ((self.k, self.gpu.k_codes, self.gpu.k_scales), (self.v, self.gpu.v_codes, self.gpu.v_scales)):
            np.testing.assert_array_equal(scales.cpu().numpy(), twin.s)
            np.testing.assert_array_equal(codes.cpu().numpy().astype(np.int64) - 128, twin.c)


@gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_append_and_read(libgemm, page, dim, kind):
    import torch
    from accelerator_gb300 import lowbit
    heads = 3
    pool = Pool(7, 4, heads, dim, page, seed=page + dim)
    at = np.array([0, page - 1, page, 5, 0, 2 * page + 3, 1])
    for step, (counts, spread) in enumerate([([1, 1, 1, 1, 1, 1, 1], 0.3), ([page, 2, 0, page + 1, 3 * page // 2, 1, 2], 1.0),
                                             ([1, 0, 1, 2, 1, page // 2, 1], 4.0), ([1, 1, 1, 1, 1, 1, 1], 1.0)]):
        starts = offsets(counts)
        K, V = (pool.rows(int(starts[-1]), heads, kind, spread) for _ in range(2))
        lowbit.kv_append(pool.gpu, K, V, ints(pool.table), ints(starts), ints(at))
        assert libgemm.debug_status() == libgemm.OK
        pool.k.append(as_numpy(K), pool.table, starts, at)
        pool.v.append(as_numpy(V), pool.table, starts, at)
        pool.same()
        at = at + counts
    starts = offsets(at)
    for back in ("fp32", "bf16", "fp16"):
        got = lowbit.kv_read(pool.gpu, ints(pool.table), ints(starts), ints(at * 0), int(starts[-1]), dtype=dtypes()[back])
        for twin, x in zip((pool.k, pool.v), got):
            want = np.concatenate([twin.tokens(pool.table[b], at[b]).transpose(1, 0, 2) for b in range(7)])
            assert torch.equal(x.cpu(), torch.from_numpy(want.astype(np.float32)).to(dtypes()[back]))
    some = np.maximum(at - 3, 0)      # a range that starts inside a page
    starts = offsets(at - some)
    K, _ = lowbit.kv_read(pool.gpu, ints(pool.table), ints(starts), ints(some), int(starts[-1]), dtype=torch.float32)
    want = np.concatenate([pool.k.tokens(pool.table[b], at[b]).transpose(1, 0, 2)[some[b]:] for b in range(7)])
    np.testing.assert_array_equal(K.cpu().numpy(), want.astype(np.float32))
    assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_append_strided(libgemm, kind, shift):
    """Slices of one joint projection, with rows that are not 16-byte aligned too."""
    import torch
    from accelerator_gb300 import lowbit
    pool = Pool(2, 3, 2, 64, 16, seed=3)
    joint = torch.randn(40, 5 * 2 * 64 + 1 + shift, device="cuda").to(dtypes()[kind])
    K = joint[:, 128 + shift:256 + shift].unflatten(1, (2, 64))
    V = joint[:, 256 + shift:512 + shift].unflatten(1, (2, 128))[:, :, 3:67]
    starts, first = np.array([0, 25, 40]), np.array([9, 30])
    lowbit.kv_append(pool.gpu, K, V, ints(pool.table), ints(starts), ints(first))
    pool.k.append(as_numpy(K), pool.table, starts, first)
    pool.v.append(as_numpy(V), pool.table, starts, first)
    pool.same()
    assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_append_non_finite(libgemm, bad):
    """A page and head that was given a NaN or an infinity reads as NaN until
    it is begun anew; the others are as they would be."""
    import torch
    from accelerator_gb300 import lowbit
    pool = Pool(1, 3, 2, 64, 16, seed=4)
    table, first = ints(pool.table), np.array([10])
    for n, poison in ((12, True), (3, False)):
        K, V = pool.rows(n, 2, "fp32"), pool.rows(n, 2, "fp32")
        if poison:
            K[7, 1, 5] = bad
        lowbit.kv_append(pool.gpu, K, V, table, ints([0, n]), ints(first))
        pool.k.append(as_numpy(K), pool.table, [0, n], first)
        pool.v.append(as_numpy(V), pool.table, [0, n], first)
        pool.same()
        first = first + n
    K, _ = lowbit.kv_read(pool.gpu, table, ints([0, 25]), ints([0]), 25, dtype=torch.float32)
    nan = torch.isnan(K).cpu().numpy()
    assert nan[16:, 1].all() and nan.sum() == 9 * 64
    K = pool.rows(2, 2, "fp32")
    lowbit.kv_append(pool.gpu, K, K, table, ints([0, 2]), ints([16]))
    K, _ = lowbit.kv_read(pool.gpu, table, ints([0, 2]), ints([16]), 2, dtype=torch.float32)
    assert torch.isfinite(K).all()


@gpu
def test_append_zeros_and_tiny_and_huge(libgemm):
    from accelerator_gb300 import lowbit
    for value in (0.0, 1e-38, 2.0 ** -126 * 127, 3e38):
        pool = Pool(1, 1, 1, 64, 16, seed=5)
        K = pool.rows(4, 1, "fp32") * 0 + value
        K[1] *= -0.3
        lowbit.kv_append(pool.gpu, K, K, ints(pool.table), ints([0, 4]), ints([0]))
        pool.k.append(as_numpy(K), pool.table, [0, 4], [0])
        pool.v.append(as_numpy(K), pool.table, [0, 4], [0])
        pool.same()


def check_attention(libgemm, pool, counts, lengths, q_heads, kind, causal=True, window=0, scale=None, Q=None, out=None):
    from accelerator_gb300 import lowbit
    starts = offsets(counts)
    if Q is None:
        Q = pool.rows(int(starts[-1]), q_heads, kind, 1.5)
    O = lowbit.kv_attention(Q, pool.gpu, ints(pool.table), ints(starts), ints(lengths), causal=causal, window=window,
                            scale=scale, out=out)
    assert libgemm.debug_status() == libgemm.OK
    want, spread, reach = ref.attention(as_numpy(Q), pool.k, pool.v, pool.table, starts, lengths,
                                        pool.dim ** -0.5 if scale is None else scale, causal, window)
    got = as_numpy(O).astype(np.float64)
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - want) / ref.attention_limit(want, spread, reach, pool.dim, kind), initial=0)
    assert worst <= 1, worst
    return O


@gpu
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_at_every_edge(libgemm, page, dim, kind):
    lengths = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 0, 511]
    pool = Pool(len(lengths), -(-512 // page), 2, dim, page, seed=page + dim)
    for share in (1, 4):
        check_attention(libgemm, pool, [1] * len(lengths), lengths, 2 * share, kind)


@gpu
@pytest.mark.parametrize("heads,share", [(1, 1), (1, 16), (1, 17), (2, 8), (3, 5), (5, 3), (8, 1), (1, 40)])
def test_head_layouts(libgemm, heads, share):
    pool = Pool(3, 5, heads, 64, 64, seed=heads + share)
    check_attention(libgemm, pool, [1, 2, 3], [200, 77, 300], heads * share, "fp16")


@gpu
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 33), (True, 100), (False, 0)])
@pytest.mark.parametrize("dim,share", [(64, 1), (128, 4), (128, 3)])
def test_prompts(libgemm, dim, share, causal, window):
    counts, lengths = [1, 40, 0, 129, 64, 200, 5], [1, 40, 10, 150, 300, 200, 129]
    pool = Pool(7, 10, 2, dim, 32, seed=dim + share)
    check_attention(libgemm, pool, counts, lengths, 2 * share, "bf16", causal=causal, window=window)


@gpu
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing_are_zero(libgemm, causal):
    """More queries than tokens, and empty caches."""
    import torch
    pool = Pool(4, 2, 2, 64, 32, seed=8)
    counts, lengths = [5, 3, 40, 1], [2, 0, 30, 0]
    O = check_attention(libgemm, pool, counts, lengths, 6, "bf16", causal=causal)
    assert (O[:3] == 0).all() and (O[5:18] == 0).all() and (O[-1] == 0).all() and (O[4] != 0).any()
    assert torch.isfinite(O).all()


@gpu
@pytest.mark.parametrize("dim,kind", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("window", [0, 700])
def test_long(libgemm, dim, kind, window):
    """Long enough to be split, with sequences of very different lengths."""
    pool = Pool(3, 300, 2, dim, 16, seed=dim, spare=1)
    check_attention(libgemm, pool, [1, 2, 1], [4800, 17, 2049], 8, kind, window=window)


@gpu
def test_scales_that_differ_by_orders(libgemm):
    """Value scales of pages from 2^-10 to 2^10 and scores of large magnitude."""
    import torch
    pool = Pool(2, 8, 1, 64, 16, seed=11)
    for twin, t in ((pool.v, pool.gpu.v_scales), (pool.k, pool.gpu.k_scales)):
        twin.s[:] = np.exp2(pool.rng.uniform(-10, 10 if twin is pool.v else -3, twin.s.shape)).astype(np.float32)
        t.copy_(torch.from_numpy(twin.s))
    check_attention(libgemm, pool, [1, 3], [128, 100], 4, "fp16")
    check_attention(libgemm, pool, [1, 3], [128, 100], 4, "bf16", scale=-0.5)
    pool.v.s[:] = 0
    pool.gpu.v_scales.zero_()
    check_attention(libgemm, pool, [1, 3], [128, 100], 4, "bf16")


@gpu
@pytest.mark.parametrize("magnitude", [2.0 ** -60, 1.0, 2.0 ** 60])
def test_queries_of_any_magnitude(libgemm, magnitude):
    """bfloat16 has float's range; the scores are brought back by the scale."""
    pool = Pool(2, 4, 2, 128, 16, seed=12)
    Q = pool.rows(5, 4, "fp32") * magnitude
    Q[:, :, ::7] *= 2.0 ** -20
    check_attention(libgemm, pool, [2, 3], [64, 30], 4, "bf16", scale=float(0.1 / magnitude), Q=Q.to(dtypes()["bf16"]))


@gpu
def test_strided_queries_and_results(libgemm):
    import torch
    pool = Pool(2, 4, 2, 64, 16, seed=13)
    joint = torch.randn(9, 8 * 64 + 3, device="cuda").to(torch.bfloat16)
    for shift in (0, 3):
        Q = joint[:, shift:shift + 256].unflatten(1, (4, 64))
        store = torch.full((9, 4, 100), float("nan"), dtype=torch.bfloat16, device="cuda")
        check_attention(libgemm, pool, [4, 5], [60, 33], 4, "bf16", Q=Q, out=store[:, :, shift:shift + 64])
        assert torch.isnan(store[:, :, shift + 64:]).all() and torch.isnan(store[:, :, :shift]).all()


@gpu
@pytest.mark.parametrize("new", [1, 70])
def test_nothing_beyond_the_mask_is_used(libgemm, new):
    """Poison in every page that no query sees, and in pages that some do not see."""
    pool = Pool(2, 12, 2, 64, 16, seed=14)
    lengths = [100, 81]
    O = check_attention(libgemm, pool, [new, new], lengths, 4, "fp16", Q=(Q := pool.rows(2 * new, 4, "fp16")))
    used = {int(p) for b, n in enumerate(lengths) for p in pool.table[b, :-(-n // 16)]}
    for p in set(range(pool.gpu.k_codes.shape[0])) - used:
        for t in (pool.gpu.k_scales, pool.gpu.v_scales):
            t[p] = float("nan")
    import torch
    from accelerator_gb300 import lowbit
    starts = ints([0, new, 2 * new])
    again = lowbit.kv_attention(Q, pool.gpu, ints(pool.table), starts, ints(lengths))
    assert torch.equal(O, again)
    # tokens 96 .. 99 of sequence 0: only its last four queries see them
    for scales in (pool.gpu.v_scales, pool.gpu.k_scales):
        kept = scales.clone()
        scales[int(pool.table[0, 6])] = float("nan")
        again = lowbit.kv_attention(Q, pool.gpu, ints(pool.table), starts, ints(lengths))
        nan = torch.isnan(again).flatten(1)
        hit = torch.zeros(2 * new, dtype=torch.bool, device="cuda")
        hit[max(0, new - 4):new] = True
        assert torch.equal(nan.all(1), hit) and torch.equal(nan.any(1), hit)
        assert torch.equal(again[~hit], O[~hit])
        scales.copy_(kept)


@gpu
def test_nan_queries_stay_in_their_rows(libgemm):
    import torch
    from accelerator_gb300 import lowbit
    pool = Pool(1, 4, 1, 128, 16, seed=15)
    for kind in ("bf16", "fp16"):
        Q = pool.rows(3, 4, kind)
        O = lowbit.kv_attention(Q, pool.gpu, ints(pool.table), ints([0, 3]), ints([50]))
        Q[1, 2, 77] = float("nan")
        again = lowbit.kv_attention(Q, pool.gpu, ints(pool.table), ints([0, 3]), ints([50]))
        assert torch.isnan(again[1, 2]).all()
        O[1, 2] = again[1, 2] = 0
        assert torch.equal(O, again)


@gpu
def test_pages_past_32_bit_offsets(libgemm):
    """A pool of more than 2^32 code bytes, read and written at its far end."""
    import torch
    from accelerator_gb300 import lowbit
    pages, heads, page, dim = 70000, 4, 128, 128
    codes = [torch.empty((pages, heads, page, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((pages, heads), device="cuda") for _ in range(2)]
    cache = lowbit.KvCache(*codes, *scales)
    table = ints([[pages - 1, 3, pages - 2]])
    K, V = (torch.randn(300, heads, dim, device="cuda") for _ in range(2))
    lowbit.kv_append(cache, K, V, table, ints([0, 300]), ints([0]))
    k, v = lowbit.kv_read(cache, table, ints([0, 300]), ints([0]), 300, dtype=torch.float32)
    for x, y in ((k, K), (v, V)):
        assert (x - y).abs().max() <= y.abs().max() / 127 * 0.5001
    Q = torch.randn(2, 8, dim, device="cuda").to(torch.bfloat16)
    O = lowbit.kv_attention(Q, cache, table, ints([0, 2]), ints([300])).double()
    x = Q.double().view(2, heads, 2, dim)
    a = torch.einsum("thgd,nhd->thgn", x, k.double()) / dim ** 0.5
    a[0, :, :, 299] = -float("inf")
    want = torch.einsum("thgn,nhd->thgd", a.softmax(-1), v.double()).reshape(2, 8, dim)
    assert (O - want).abs().max() <= 0.01 * want.abs().max()
    assert libgemm.debug_status() == libgemm.OK


@gpu
def test_bad_indices_are_reported(libgemm):
    """Page numbers, positions and offsets out of range: nothing outside the
    cache is touched, and the next status says so."""
    import torch
    from accelerator_gb300 import lowbit
    pool = Pool(2, 3, 1, 64, 16, seed=16)
    Q, K = pool.rows(4, 2, "bf16"), pool.rows(4, 1, "bf16")
    good = dict(table=pool.table, starts=[0, 2, 4], at=[20, 30])
    pages = pool.gpu.k_codes.shape[0]
    high, low = pool.table.copy(), pool.table.copy()
    high[0, 1], low[1, 1] = pages, -1
    for change in (dict(table=high), dict(table=low), dict(at=[20, 49]), dict(at=[-1, 30]), dict(starts=[0, 5, 4]),
                   dict(starts=[0, 2, 2000]), dict(starts=[0, -3, 4])):
        a = {**good, **change}
        table, starts, at = ints(a["table"]), ints(a["starts"]), ints(a["at"])
        for call in (lambda: lowbit.kv_append(pool.gpu, K, K, table, starts, at),
                     lambda: lowbit.kv_read(pool.gpu, table, starts, at, 4),
                     lambda: lowbit.kv_attention(Q, pool.gpu, table, starts, at)):
            assert libgemm.debug_status() == libgemm.OK
            call()
            assert libgemm.debug_status() == libgemm.ERR_INDEX, change
            assert libgemm.debug_status() == libgemm.OK
    assert torch.isfinite(lowbit.kv_attention(Q, pool.gpu, *(ints(good[n]) for n in ("table", "starts", "at")))).all()
    assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("width", [40, 200])     # the long one takes scratch and a second launch
def test_capture_and_other_stream(libgemm, width):
    import torch
    from accelerator_gb300 import lowbit
    pool = Pool(2, width, 2, 128, 64, seed=17)
    n = 50 * width
    table, starts, first, lengths = ints(pool.table), ints([0, 1, 2]), ints([n, 55]), ints([n + 1, 56])
    K, V, Q = pool.rows(2, 2, "bf16"), pool.rows(2, 2, "bf16"), pool.rows(2, 8, "bf16")

    def step(stream=None):
        lowbit.kv_append(pool.gpu, K, V, table, starts, first, stream=stream)
        return (lowbit.kv_attention(Q, pool.gpu, table, starts, lengths, stream=stream),
                *lowbit.kv_read(pool.gpu, table, starts, first, 2, stream=stream))

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
def test_refusals_of_the_binding(libgemm):
    import torch
    from accelerator_gb300 import lowbit
    pool = Pool(2, 3, 2, 64, 16)
    table, starts, at = ints(pool.table), ints([0, 1, 2]), ints([3, 4])
    Q, K = pool.rows(2, 4, "bf16"), pool.rows(2, 2, "bf16")
    c = pool.gpu
    with pytest.raises(TypeError):
        lowbit.KvCache(c.k_codes[:, :, :15], c.v_codes, c.k_scales, c.v_scales)
    with pytest.raises(TypeError):
        lowbit.KvCache(c.k_codes, c.v_codes, c.k_scales.double(), c.v_scales)
    for bad in ((table.long(), starts, at), (table, starts.cpu(), at), (table, starts, at[None])):
        with pytest.raises(TypeError):
            lowbit.kv_attention(Q, c, *bad)
    with pytest.raises(ValueError):
        lowbit.kv_attention(Q, c, table, starts[:2], at)
    with pytest.raises(TypeError):
        lowbit.kv_attention(Q.float(), c, table, starts, at)
    with pytest.raises(TypeError):
        lowbit.kv_attention(Q[:, :, :32], c, table, starts, at)
    with pytest.raises(libgemm.GemmError):
        lowbit.kv_attention(Q[:, :3], c, table, starts, at)          # 3 heads over 2
    with pytest.raises(libgemm.GemmError):
        lowbit.kv_attention(Q, c, table, starts, at, causal=False, window=5)
    with pytest.raises(libgemm.GemmError):
        lowbit.kv_attention(Q, c, table, starts, at, window=-1)
    with pytest.raises(libgemm.GemmError):
        lowbit.kv_attention(Q, c, table, starts, at, out=Q)
    with pytest.raises(TypeError):
        lowbit.kv_append(c, K, K[:, :1], table, starts, at)
    with pytest.raises(ValueError):
        lowbit.kv_append(c, K, K[:1], table, starts, at)
    with pytest.raises(TypeError):
        lowbit.kv_append(c, K, K.float(), table, starts, at)
    with pytest.raises(TypeError):
        lowbit.kv_read(c, table, starts, at, 2, dtype=torch.float64)


# ---- without a GPU ---------------------------------------------------------------

G = 1 << 24


class CKv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_void_p), ("vs", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("heads", ctypes.c_int32), ("page", ctypes.c_int32), ("dim", ctypes.c_int32)]


def _call(libgemm, what, **change):
    a = dict(k=FAKE, v=FAKE + G, ks=FAKE + 2 * G, vs=FAKE + 3 * G, pages=10, heads=2, page=16, dim=64, X=FAKE + 4 * G,
             Y=FAKE + 5 * G, row=128, head=64, kind=1, q_heads=2, scale=0.125, causal=1, window=0, table=FAKE + 6 * G,
             width=5, starts=FAKE + 7 * G, at=FAKE + 8 * G, tokens=4, sequences=2)
    a.update(change)
    p = lambda n: a[n] or None      # noqa: E731
    c = CKv(p("k"), p("v"), p("ks"), p("vs"), a["pages"], a["heads"], a["page"], a["dim"])
    tail = (p("table"), a["width"], p("starts"), p("at"), a["tokens"], a["sequences"], None)
    lib = libgemm.lib()
    ref_c = None if a.get("null") else ctypes.byref(c)
    if what == "append":
        return lib.gemm_kv_append(ref_c, p("X"), a["row"], a["head"], p("Y"), a["row"], a["head"], a["kind"], *tail)
    if what == "read":
        return lib.gemm_kv_read(ref_c, p("X"), p("Y"), a["kind"], *tail)
    return lib.gemm_kv_attention(ref_c, p("X"), a["row"], a["head"], p("Y"), a["row"], a["head"], a["kind"], a["q_heads"],
                                 a["scale"], a["causal"], a["window"], *tail)


@pytest.mark.parametrize("what", ["append", "read", "attention"])
@pytest.mark.parametrize("change,want", [
    ({"null": 1}, 1), ({"dim": 96}, 1), ({"page": 24}, 1), ({"page": 8}, 1), ({"heads": 0}, 1), ({"pages": -1}, 1),
    ({"tokens": -1}, 1), ({"tokens": 1 << 31}, 1), ({"sequences": 0}, 1), ({"width": -1}, 1), ({"width": 1 << 27}, 1), ({"kind": 3}, 1),
    ({"k": 0}, 1), ({"vs": 0}, 1), ({"table": 0}, 1), ({"starts": 0}, 1), ({"at": 0}, 1), ({"X": 0}, 1), ({"Y": 0}, 1),
    ({"k": FAKE + 8}, 2), ({"ks": FAKE + 2 * G + 2}, 2), ({"table": FAKE + 6 * G + 1}, 2), ({"X": FAKE + 4 * G + 1}, 2),
    ({"Y": FAKE + G}, 1), ({"tokens": 0, "sequences": 0, "X": 0, "Y": 0}, 0)])
def test_shared_checks(libgemm, what, change, want):
    assert _call(libgemm, what, **change) == want


@pytest.mark.parametrize("change", [{"kind": 0}, {"q_heads": 3}, {"q_heads": 0}, {"window": -1}, {"window": 4, "causal": 0},
                                    {"scale": float("nan")}, {"row": -1}, {"head": -64}, {"Y": FAKE + 4 * G}])
def test_attention_checks(libgemm, change):
    assert _call(libgemm, "attention", **change) == libgemm.ERR_INVALID_ARG


def test_no_device_is_an_error(libgemm):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for what in ("append", "read", "attention"):
        assert _call(libgemm, what) in (libgemm.ERR_CUDA, libgemm.ERR_UNSUPPORTED_DEVICE)
