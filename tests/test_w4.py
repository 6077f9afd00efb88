"""4-bit weights: the quantiser and its inverse bit for bit against the rule,
the product against a 64-bit one of the same values, at sizes around every
tile edge, types, groups, strides and alignments, and the refusals."""
import ctypes

import numpy as np
import pytest

import lowbit_ref as ref

FAKE = 0x7F0000000000


def torch_types():
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def on_gpu(x, kind):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(torch_types()[kind])


def as_numpy(t):
    return t.float().cpu().numpy()


def matrix(K, N, kind, seed=0):
    """Values of the type, as float32: normal, with a column of zeros, one of
    tiny and one of large magnitude, and ties of b / s."""
    rng = np.random.default_rng(seed + 31 * K + N)
    B = rng.standard_normal((K, N)).astype(np.float32) * 0.05
    B[:, 0] = 0
    if N > 3:
        B[:, 1] *= np.float32(2.0 ** -12)
        B[:, 2] *= 512
        B[:, 3] = np.float32(2.0 ** -7) * (np.arange(K) % 15 - 7)    # multiples of half a step
        B[0, 3] = np.float32(7 * 2.0 ** -6)
    return as_numpy(on_gpu(B, kind)) if kind != "fp32" else B


SIZES = [(1, 1), (1, 17), (31, 15), (32, 16), (33, 64), (64, 65), (65, 63), (127, 129), (128, 128), (300, 77),
         (1000, 333)]


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("K,N", SIZES)
def test_quantize_and_back(libgemm, K, N, kind, group):
    import torch
    from accelerator_gb300 import lowbit
    B = matrix(K, N, kind)
    W = lowbit.w4_quantize(on_gpu(B, kind), group)
    q, s = ref.w4_quantize(B, group)
    words, scales = ref.w4_pack(q, s, group)
    np.testing.assert_array_equal(W.codes.cpu().numpy().view(np.uint32), words)
    np.testing.assert_array_equal(as_numpy(W.scales), scales)
    for back in ("fp32", "bf16", "fp16"):
        got = lowbit.w4_dequantize(W, dtype=torch_types()[back])
        want = torch.from_numpy(ref.w4_values(q, s, group).astype(np.float32)).to(torch_types()[back])
        assert torch.equal(got.cpu(), want)
    assert libgemm.debug_status() == libgemm.OK


@pytest.mark.gpu
def test_quantize_strided_and_unaligned(libgemm):
    import torch
    from accelerator_gb300 import lowbit
    B = matrix(150, 90, "bf16")
    store = torch.full((150, 131), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = store[:, 3:93]
    view.copy_(on_gpu(B, "bf16"))
    W = lowbit.w4_quantize(view, 64)
    q, s = ref.w4_quantize(B, 64)
    np.testing.assert_array_equal(W.codes.cpu().numpy().view(np.uint32), ref.w4_pack(q, s, 64)[0])
    out = torch.full((150, 131), float("nan"), dtype=torch.float32, device="cuda")
    lowbit.w4_dequantize(W, out=out[:, 5:95])
    np.testing.assert_array_equal(as_numpy(out[:, 5:95]), ref.w4_values(q, s, 64).astype(np.float32))
    assert torch.isnan(out[:, :5]).all() and torch.isnan(out[:, 95:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_non_finite_group_reads_as_nan(libgemm, bad):
    from accelerator_gb300 import lowbit
    B = matrix(130, 20, "fp32")
    B[40, 7] = bad
    W = lowbit.w4_quantize(on_gpu(B, "fp32"), 32)
    got = as_numpy(lowbit.w4_dequantize(W, dtype=torch_types()["fp32"]))
    nan = np.isnan(got)
    assert nan[32:64, 7].all() and nan.sum() == 32
    C = as_numpy(lowbit.gemm_w4(on_gpu(np.ones((2, 130), np.float32), "bf16"), W))
    assert np.isnan(C[:, 7]).all() and np.isnan(C).sum() == 2


@pytest.mark.gpu
def test_magnitudes_at_the_ends_of_the_range(libgemm):
    from accelerator_gb300 import lowbit
    B = np.zeros((64, 4), np.float32)
    B[:, 0] = np.float32(3.4e38) * np.linspace(-1, 1, 64, dtype=np.float32)
    B[:, 1] = np.float32(2.0 ** -126)           # s under 2^-126: zeros
    B[:, 2] = np.float32(2.0 ** -123) * 1.75    # s = 2^-125 * 2 / 2 ...: kept
    W = lowbit.w4_quantize(on_gpu(B, "fp32"), 64)
    q, s = ref.w4_quantize(B, 64)
    np.testing.assert_array_equal(W.codes.cpu().numpy().view(np.uint32), ref.w4_pack(q, s, 64)[0])
    got = as_numpy(lowbit.w4_dequantize(W, dtype=torch_types()["fp32"]))
    np.testing.assert_array_equal(got, ref.w4_values(q, s, 64).astype(np.float32))
    assert (got[:, 1] == 0).all() and (got[:, 2] != 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_small_magnitudes_round_alike(libgemm, kind):
    """Steps down to 2^-126, where a quotient's remainder would underflow: ties
    and values beside them as at any other magnitude."""
    from accelerator_gb300 import lowbit
    steps = np.array([-126, -125, -118, -110, -101, -100, -99, -60, 0, 40])
    B = np.empty((128, len(steps)), np.float32)
    for c, e in enumerate(steps):
        B[:, c] = np.ldexp(np.float32(1), e) * (np.arange(128) % 29 - 14) / 2        # multiples of half a step
        B[::3, c] *= np.float32(1 + 2.0 ** -7)
        B[0, c] = np.ldexp(np.float32(7), e)
    B = as_numpy(on_gpu(B, kind)) if kind != "fp32" else B
    W = lowbit.w4_quantize(on_gpu(B, kind), 64)
    q, s = ref.w4_quantize(B, 64)
    assert (s != 0).all()
    np.testing.assert_array_equal(W.codes.cpu().numpy().view(np.uint32), ref.w4_pack(q, s, 64)[0])


def product_limit(X, V, Y, out_kind):
    """Sums of K exact products in binary32, at most K / 8 + 64 roundings of
    2^-23 of S deep, and the result's own rounding."""
    S = np.abs(X.astype(np.float64)) @ np.abs(V)
    return S * (X.shape[1] / 8 + 64) * 2.0 ** -23 + ref.rounding(Y, out_kind) + 1e-30


def check_product(M, K, N, kind, out_kind, group, x=None, pad=0, offset=0):
    import torch
    from accelerator_gb300 import binding, lowbit
    rng = np.random.default_rng(M + 7 * K + 13 * N)
    q = rng.integers(-7, 8, (K, N)).astype(np.int8)
    s = ref.bf16_round(np.exp(rng.standard_normal((-(-K // group), N)) * 0.5).astype(np.float32) * 0.01)
    words, scales = ref.w4_pack(q, s, group)
    W = lowbit.W4Matrix(torch.from_numpy(words.view(np.uint8)).cuda(),
                        torch.from_numpy(scales).cuda().to(torch.bfloat16), K, N, group)
    store = torch.full((M * (K + pad) + offset + 8,), float("nan"), dtype=torch_types()[kind], device="cuda")
    X = store[offset: offset + M * (K + pad)].view(M, K + pad)[:, :K]
    X.copy_(on_gpu(rng.standard_normal((M, K)).astype(np.float32), kind))
    out = torch.full((M, N + 3), float("nan"), dtype=torch_types()[out_kind], device="cuda")
    lowbit.gemm_w4(X, W, C=out[:, :N])
    assert binding.debug_status() == binding.OK
    Xn, V = as_numpy(X).astype(np.float64), ref.w4_values(q, s, group)
    Y = Xn @ V
    got = as_numpy(out)[:, :N].astype(np.float64)
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - Y) / product_limit(Xn, V, Y, out_kind))
    assert worst <= 1, worst
    assert torch.isnan(out[:, N:]).all()
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 63, 16), (1, 64, 17), (2, 65, 33), (3, 31, 40), (1, 1024, 1024),
                                   (8, 333, 100), (9, 500, 65), (16, 129, 48), (17, 1000, 31), (33, 257, 129),
                                   (70, 200, 50), (1, 8192, 33), (5, 4100, 1001), (2, 130, 4096)])
def test_product(libgemm, M, K, N, group):
    for kind, out_kind in (("bf16", "bf16"), ("fp16", "fp32")):
        check_product(M, K, N, kind, out_kind, group)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("out_same", [True, False])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 0), (0, 1), (5, 3)])
def test_product_strides_and_alignment(libgemm, kind, out_same, pad, offset):
    check_product(6, 330, 70, kind, kind if out_same else "fp32", 64, pad=pad, offset=offset)


@pytest.mark.gpu
def test_product_is_the_same_on_every_run_and_for_every_row(libgemm):
    import torch
    from accelerator_gb300 import lowbit
    W = lowbit.w4_quantize(on_gpu(matrix(2000, 555, "bf16"), "bf16"), 128)
    X = torch.randn(7, 2000, device="cuda", dtype=torch.bfloat16)
    a = lowbit.gemm_w4(X, W, dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(a, lowbit.gemm_w4(X, W, dtype=torch.float32))


@pytest.mark.gpu
def test_empty_sizes(libgemm):
    import torch
    from accelerator_gb300 import lowbit
    W = lowbit.w4_quantize(torch.empty((0, 20), device="cuda"), 32)
    assert lowbit.w4_dequantize(W).shape == (0, 20)
    C = torch.full((3, 20), float("nan"), device="cuda")
    lowbit.gemm_w4(torch.empty((3, 0), dtype=torch.float16, device="cuda"), W, C=C)
    assert (C == 0).all()
    V = lowbit.w4_quantize(torch.empty((20, 0), device="cuda"), 32)
    assert lowbit.gemm_w4(torch.empty((3, 20), dtype=torch.float16, device="cuda"), V).shape == (3, 0)
    assert lowbit.gemm_w4(torch.empty((0, 0), dtype=torch.float16, device="cuda"), W).shape == (0, 20)


@pytest.mark.gpu
def test_capture_and_other_stream(libgemm):
    import torch
    from accelerator_gb300 import lowbit
    B = torch.randn(700, 300, device="cuda")
    X = torch.randn(2, 700, device="cuda", dtype=torch.float16)
    want = lowbit.gemm_w4(X, lowbit.w4_quantize(B, 64))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = lowbit.gemm_w4(X, lowbit.w4_quantize(B, 64, stream=side), stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = lowbit.gemm_w4(X, lowbit.w4_quantize(B, 64))
    again.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, want)


@pytest.mark.gpu
def test_refusals_of_the_binding(libgemm):
    import torch
    from accelerator_gb300 import lowbit
    B = torch.randn(64, 32, device="cuda")
    with pytest.raises(libgemm.GemmError):
        lowbit.w4_quantize(B, 48)
    with pytest.raises(TypeError):
        lowbit.w4_quantize(B.double())
    with pytest.raises(TypeError):
        lowbit.w4_quantize(B.cpu())
    with pytest.raises(TypeError):
        lowbit.w4_quantize(B.t())
    W = lowbit.w4_quantize(B, 32)
    X = torch.randn(2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lowbit.gemm_w4(X[:, :60], W)
    with pytest.raises(TypeError):
        lowbit.gemm_w4(X.float(), W)
    with pytest.raises(TypeError):
        lowbit.gemm_w4(X, W, dtype=torch.float16)
    with pytest.raises(ValueError):
        lowbit.gemm_w4(X, W, C=torch.empty((2, 31), device="cuda"))
    with pytest.raises(TypeError):
        lowbit.W4Matrix(W.codes[:-16], W.scales, 64, 32, 32)
    with pytest.raises(ValueError):
        lowbit.w4_dequantize(W, out=torch.empty((64, 33), device="cuda"))


# ---- without a GPU: the C entry points check before they touch a device ---------

def test_sizes(libgemm):
    a, b = ctypes.c_int64(), ctypes.c_int64()
    f = libgemm.lib().gemm_w4_sizes
    assert f(65, 17, 64, ctypes.byref(a), ctypes.byref(b)) == libgemm.OK
    assert (a.value, b.value) == (2 * 2 * 512, 2 * 2 * 32)
    assert f(0, 17, 64, ctypes.byref(a), ctypes.byref(b)) == libgemm.OK and (a.value, b.value) == (0, 0)
    from accelerator_gb300 import lowbit
    for K, N, group in ((0, 5, 32), (5, 0, 64), (1, 1, 128), (64, 16, 32), (1000, 333, 64), (8192, 8191, 128), (129, 17, 128)):
        assert f(K, N, group, ctypes.byref(a), ctypes.byref(b)) == libgemm.OK
        assert lowbit.w4_sizes(K, N, group) == (a.value, b.value)
    for args in ((-1, 4, 32), (4, -1, 32), (4, 4, 16), (1 << 31, 4, 32), (1 << 30, 1 << 30, 32)):
        assert f(*args, ctypes.byref(a), ctypes.byref(b)) == libgemm.ERR_INVALID_ARG
    assert f(4, 4, 32, None, ctypes.byref(b)) == libgemm.ERR_INVALID_ARG


G = 1 << 20


@pytest.mark.parametrize("call,want", [
    # B, ldb, type, K, N, group, codes, scales
    ((FAKE, 32, 0, 64, 32, 48, FAKE + G, FAKE + 2 * G), 1), ((FAKE, 31, 0, 64, 32, 32, FAKE + G, FAKE + 2 * G), 1),
    ((FAKE, 32, 3, 64, 32, 32, FAKE + G, FAKE + 2 * G), 1), ((FAKE, 32, 0, -1, 32, 32, FAKE + G, FAKE + 2 * G), 1),
    ((0, 32, 0, 64, 32, 32, FAKE + G, FAKE + 2 * G), 1), ((FAKE, 32, 0, 64, 32, 32, 0, FAKE + 2 * G), 1),
    ((FAKE, 32, 0, 64, 32, 32, FAKE + G, 0), 1), ((FAKE + 2, 32, 0, 64, 32, 32, FAKE + G, FAKE + 2 * G), 2),
    ((FAKE, 32, 0, 64, 32, 32, FAKE + G + 8, FAKE + 2 * G), 2), ((FAKE, 32, 0, 64, 32, 32, FAKE + G, FAKE + 2 * G + 4), 2), ((FAKE, 32, 0, 64, 32, 32, FAKE + G, FAKE + 2 * G + 2), 2),
    ((FAKE, 32, 0, 64, 32, 32, FAKE + 16, FAKE + 2 * G), 1), ((FAKE, 32, 0, 64, 32, 32, FAKE + G, FAKE + G + 16), 1),
    ((0, 32, 0, 0, 32, 32, 0, 0), 0)])
def test_quantize_checks(libgemm, call, want):
    assert libgemm.lib().gemm_w4_quantize(*[c or None if i in (0, 6, 7) else c for i, c in enumerate(call)], None) == want
    B, ldb, kind, K, N, group, codes, scales = call
    assert libgemm.lib().gemm_w4_dequantize(codes or None, scales or None, K, N, group, B or None, ldb, kind, None) == want


@pytest.mark.parametrize("change,want", [
    ({}, None), ({"group": 0}, 1), ({"xt": 0}, 1), ({"ct": 2}, 1), ({"ct": 3}, 1), ({"M": -1}, 1), ({"ldx": 63}, 1),
    ({"ldc": 31}, 1), ({"X": 0}, 1), ({"C": 0}, 1), ({"codes": 0}, 1), ({"X": FAKE + 1}, 2), ({"C": FAKE + 3 * G + 1}, 2),
    ({"codes": FAKE + G + 4}, 2), ({"C": FAKE}, 1), ({"C": FAKE + G + 32}, 1), ({"C": FAKE + 2 * G}, 1), ({"M": 0, "X": 0}, 0),
    ({"M": 1 << 31}, 1), ({"M": 1 << 30, "ldx": 1 << 60}, 1)])
def test_product_checks(libgemm, change, want):
    a = dict(X=FAKE, ldx=64, xt=1, codes=FAKE + G, scales=FAKE + 2 * G, C=FAKE + 3 * G, ldc=32, ct=1, M=2, K=64, N=32, group=32)
    a.update(change)
    if want is None:
        import torch
        if torch.cuda.is_available():
            pytest.skip("would run on the GPU")
    rc = libgemm.lib().gemm_w4(a["X"] or None, a["ldx"], a["xt"], a["codes"] or None, a["scales"], a["C"] or None,
                               a["ldc"], a["ct"], a["M"], a["K"], a["N"], a["group"], None)
    assert rc == want if want is not None else rc in (libgemm.ERR_CUDA, libgemm.ERR_UNSUPPORTED_DEVICE)
