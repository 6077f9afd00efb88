"""The plan of a step and rotary positions, against plain Python and 64 bits:
lengths and counts around page edges, pages that run out, padded rows, both
layouts, parts of heads, strides, in place, far positions, the way back, bad
numbers and refusals; and a few steps of everything together."""
import copy
import math
import random

import pytest
import torch

from kv_ref import ints

FAKE = 0x7F0000000000
G = 1 << 24
gpu = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


# ---- the plan --------------------------------------------------------------------

def plan(table, lengths, counts, free, available, page, tokens):
    """The rule in plain Python; `table` is written."""
    pages = lambda n: min(-(-n // page), len(table[0]))      # noqa: E731
    starts, heights, positions, slots, height = [0], [available], [], [], available
    for b, (n, t) in enumerate(zip(lengths, counts)):
        for column in range(pages(n), pages(n + t)):
            height -= 1
            table[b][column] = free[height] if height >= 0 else -1
        heights.append(height)
        starts.append(starts[-1] + t)
        for at in range(n, n + t):
            page_of = table[b][at // page] if at // page < len(table[0]) else -1
            positions.append(at)
            slots.append(page_of * page + at % page if page_of >= 0 else -1)
    pad = [-1] * (tokens - len(positions))
    return dict(starts=starts, first=list(lengths), lengths=[n + t for n, t in zip(lengths, counts)], positions=positions + pad,
                slots=slots + pad, available=[max(0, height)], heights=heights)


def run_plan(libgemm, table, lengths, counts, free, available, page, tokens, width=None, **kw):
    from accelerator_gb300 import sequences
    width = len(table[0]) if table else width
    t = ints(table).view(len(lengths), width)
    got = sequences.kv_plan(t, ints(lengths), ints(counts), ints(free), ints([available]), page, tokens, **kw)
    return t, got


def check_plan(libgemm, table, lengths, counts, free, available, page, tokens, status=None):
    t, got = run_plan(libgemm, table, lengths, counts, free, available, page, tokens)
    assert libgemm.debug_status() == (libgemm.OK if status is None else status)
    table = copy.deepcopy(table)
    want = plan(table, lengths, counts, free, available, page, tokens)
    assert t.tolist() == table
    for name, x in want.items():
        assert getattr(got, name).tolist() == x, name
    assert got.slots.dtype == torch.int64 and got.positions.dtype == torch.int32


@gpu
@pytest.mark.parametrize("page", [1, 16, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 256, 257, 1023, 1025, 2100])
def test_plan(libgemm, n, page):
    rng = random.Random(n + page)
    for kind in ("decode", "prompts", "rests"):
        lengths = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, 300)]) for _ in range(n)]
        most = {"decode": 1, "prompts": 40 if n > 256 else 600, "rests": 3}[kind]
        counts = [1 if kind == "decode" else rng.choice([0, 1, page, rng.randint(0, most)]) for _ in range(n)]
        width = max(-(-(a + b) // page) for a, b in zip(lengths, counts)) + rng.randint(0, 2)
        table = [[rng.randint(0, 5000) if i < -(-a // page) else -7 for i in range(width)] for a in lengths]
        need = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lengths, counts))
        free = rng.sample(range(10000, 30000 + need), need + 9)
        check_plan(libgemm, table, lengths, counts, free, need + rng.randint(0, 9), page, sum(counts) + rng.choice([0, 0, 1, 300]))


@gpu
def test_plan_of_nothing(libgemm):
    _, got = run_plan(libgemm, [], [], [], [3], 1, 16, 5, width=4)
    assert got.starts.tolist() == [0] and got.positions.tolist() == [-1] * 5 and got.slots.tolist() == [-1] * 5
    check_plan(libgemm, [[1], [2]], [3, 0], [0, 0], [], 0, 16, 0)
    check_plan(libgemm, [[1], [2]], [3, 16], [0, 0], [], 0, 16, 7)
    assert libgemm.debug_status() == libgemm.OK


@gpu
def test_long_sequences(libgemm):
    """One of more rows than a round of the fill has, far into the cache."""
    rng = random.Random(1)
    lengths, counts, page = [2 ** 30 - 5, 3, 100000], [700, 5000, 1], 64
    width = -(-(2 ** 30 + 700) // page)
    from accelerator_gb300 import sequences
    table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    held = [2 ** 24 - 1, 0, 1562]                 # the column of the last token's page
    for b in range(3):
        table[b, held[b]] = 77 + b
    free = rng.sample(range(10 ** 9, 2 ** 31 - 1), 200)
    got = sequences.kv_plan(table, ints(lengths), ints(counts), ints(free), ints([150]), page, sum(counts))
    assert libgemm.debug_status() == libgemm.OK
    at, height = 0, 150
    slots, positions = got.slots.tolist(), got.positions.tolist()
    for b, (n, t) in enumerate(zip(lengths, counts)):
        for pos in range(n, n + t):
            column, last = pos // page, (n - 1) // page
            number = 77 + b if column == last else free[height - (column - last)]
            assert positions[at] == pos and slots[at] == number * page + pos % page
            assert int(table[b, column]) == number if pos % (7 * page) == 0 else True
            at += 1
        height -= -(-(n + t) // page) - -(-n // page)
    assert got.available.tolist() == [height]


@gpu
def test_plan_reports_what_does_not_fit(libgemm):
    bad = libgemm.ERR_INDEX
    # pages run out within the second sequence, the last has its own
    check_plan(libgemm, [[1, -1, -1], [2, -1, -1], [3, -1, -1]], [10, 16, 3], [16, 20, 2], [50, 51, 52], 2, 16, 38, status=bad)
    # a sequence longer than its row of the table
    check_plan(libgemm, [[1, -1], [2, -1]], [10, 30], [16, 9], [50, 51, 52], 3, 16, 25, status=bad)
    # counts past the room of the rows: starts ends there, and later sequences have none
    t, got = run_plan(libgemm, [[-1, -1]] * 3, [0, 0, 0], [5, 10, 4], [7, 8, 9], 3, 16, 9)
    assert libgemm.debug_status() == bad
    assert got.starts.tolist() == [0, 5, 9, 9] and got.positions.tolist() == [0, 1, 2, 3, 4, 0, 1, 2, 3]
    # negative numbers count as 0; a height past the stack is held to it
    t, got = run_plan(libgemm, [[-1, -1]] * 3, [-4, 2, 0], [3, -1, 2], [7, 8, 9], 3, 16, 5)
    assert libgemm.debug_status() == bad
    assert got.starts.tolist() == [0, 3, 3, 5] and got.first.tolist() == [0, 2, 0]
    t, got = run_plan(libgemm, [[-1, -1]], [0], [3], [7, 8, 9], 99, 16, 3)
    assert libgemm.debug_status() == bad and t.tolist()[0][0] == 9
    t, got = run_plan(libgemm, [[-1, -1]], [2 ** 31 - 2], [2 ** 31 - 1], [7, 8, 9], 3, 16, 8)
    assert libgemm.debug_status() == bad and got.slots.tolist() == [-1] * 8
    assert libgemm.debug_status() == libgemm.OK


@gpu
def test_plan_in_place_and_recorded(libgemm):
    """Steps that go on where the last ended, in a graph and on another stream."""
    from accelerator_gb300 import sequences
    page, steps, n = 16, 40, 5
    lengths, counts = [0, 3, 15, 16, 31], [1, 2, 1, 0, 1]
    want_table = [[-1] * 10 for _ in range(n)]
    for b, a in enumerate(lengths):
        for i in range(-(-a // page)):
            want_table[b][i] = 100 + 10 * b + i
    free = list(range(30))
    table, L, C, F, A = ints(want_table), ints(lengths), ints(counts), ints(free), ints([30])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = sequences.kv_plan(table, L, C, F, A, page, 5, update=True, stream=side)
    side.synchronize()
    assert p.lengths is L and p.available is A
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = sequences.kv_plan(table, L, C, F, A, page, 5, update=True)
    now, height = lengths, 30
    for step in range(steps):
        if step:
            graph.replay()
        want = plan(want_table, now, counts, free, height, page, 5)
        now, height = want["lengths"], want["available"][0]
        if step:
            for name, x in want.items():
                assert getattr(p, name).tolist() == x, (name, step)
        assert table.tolist() == want_table and L.tolist() == now and A.tolist() == [height]
    assert libgemm.debug_status() == libgemm.OK


@gpu
def test_plan_refusals_of_the_binding(libgemm, monkeypatch):
    from accelerator_gb300 import lowbit, sequences
    table, L, C, F, A = ints([[1, 2], [3, 4]]), ints([3, 4]), ints([1, 1]), ints([5, 6]), ints([2])
    for bad in ((table.long(), L, C, F, A), (table, L.cpu(), C, F, A), (table, L, C.float(), F, A), (table, L, C, F, ints([1, 2])),
                (table.t(), L, C, F, A), (table[0], L, C, F, A), (table, L[None], C, F, A),
                (table, L, C, F.view(2, 1), A), (table, L, C, F.repeat(2)[::2], A)):
        with pytest.raises(TypeError):
            sequences.kv_plan(*bad, 16, 2)
    with pytest.raises(ValueError):
        sequences.kv_plan(table, L[:1], C, F, A, 16, 2)
    with pytest.raises(ValueError):
        sequences.kv_plan(table, L, C, F, A, 16, -1)
    for page in (0, 3, -16, 1 << 21, (1 << 32) + 16, 16 - (1 << 32)):
        with pytest.raises(libgemm.GemmError):
            sequences.kv_plan(table, L, C, F, A, page, 2)
    with pytest.raises(libgemm.GemmError):
        sequences.kv_plan(table, L, L, F, A, 16, 2, update=True)        # lengths in place, and counts
    with pytest.raises(libgemm.GemmError):
        sequences.kv_plan(table, L, C, F, F[:1], 16, 2, update=True)    # the stack's height on the stack
    count = libgemm.launch_count()
    monkeypatch.setattr(lowbit, "_current_device", lambda: 1)
    with pytest.raises(TypeError):
        sequences.kv_plan(table, L, C, F, A, 16, 2)
    assert libgemm.launch_count() == count


# ---- rotary positions --------------------------------------------------------------

def turned(x, positions, table, inverse=False):
    """In 64 bits: pairs as complex numbers."""
    part, x = table.rotary_dim, x.double()
    f = torch.tensor(table.frequencies, dtype=torch.float64, device=x.device)
    a = positions.double()[:, None, None] * (-f if inverse else f)
    by = torch.polar(torch.full_like(a, table.magnitude), a)
    y = x.clone()
    if table.layout == "half":
        z = torch.complex(x[..., : part // 2].contiguous(), x[..., part // 2: part].contiguous()) * by
        y[..., : part // 2], y[..., part // 2: part] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :part].reshape(*x.shape[:2], -1, 2).contiguous()) * by
        y[..., :part] = torch.view_as_real(z).flatten(-2)
    return y


def check_turned(got, x, positions, table, inverse=False):
    """Off by one rounding to the type, and by what binary32 makes of a pair (a, b)
    before it: the angle as a binary32 count of half turns (pi * 2^-25 radians), sine
    and cosine by 2 units in the last place, their product with the magnitude, and a
    product and a sum of each half -- under 10 roundings of 2^-24 of |a| + |b|
    times the magnitude, plus frequencies of 53 bits (2^-52 of the angle)."""
    want, part = turned(x, positions, table, inverse), table.rotary_dim
    size = x.double().abs()
    limit = torch.zeros_like(want)
    other = torch.empty(part, dtype=torch.long, device=x.device)
    i = torch.arange(part // 2, device=x.device)
    lo, hi = (i, i + part // 2) if table.layout == "half" else (2 * i, 2 * i + 1)
    other[lo], other[hi] = hi, lo
    angle = positions.double()[:, None, None] * max(abs(f) for f in table.frequencies) * 2.0 ** -51
    limit[..., :part] = (size[..., :part] + size[..., other]) * abs(table.magnitude) * (10 * 2.0 ** -24 + angle)
    limit = limit + torch.clamp(HALF_STEP[x.dtype] * want.abs(), min=LEAST[x.dtype])
    off = (got.double() - want).abs()
    assert (off <= limit).all(), (off / limit).max().item()
    assert torch.equal(got[..., part:], x[..., part:])


@gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dim,part", [(64, 64), (128, 128), (128, 32), (80, 80), (96, 48), (256, 256), (72, 70), (6, 2), (33, 32), (1024, 1024), (2, 2)])
def test_rotary(libgemm, dim, part, kind, layout):
    from accelerator_gb300 import sequences
    g = torch.Generator(device="cuda").manual_seed(dim + part)
    for rows, q_heads, k_heads in ((1, 1, 1), (1, 32, 8), (5, 3, 0), (77, 7, 2), (1300, 4, 1)):
        if rows * q_heads * dim > 2000000:
            continue
        table = sequences.Rotary(part, layout=layout)
        Q, K = (torch.randn(rows, max(h, 1), dim, device="cuda", generator=g).to(DTYPES[kind]) for h in (q_heads, k_heads))
        K = K if k_heads else None
        positions = torch.randint(0, 5000, (rows,), device="cuda", generator=g).to(torch.int32)
        for inverse in (False, True):
            q, k = sequences.rotary(Q, K, positions, table, inverse=inverse)
            check_turned(q, Q, positions, table, inverse)
            assert (k is None) == (K is None)
            if K is not None:
                check_turned(k, K, positions, table, inverse)
    assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0), dict(base=500000.0),
                                dict(scaling="yarn", factor=16.0, original=4096), dict(scaling="yarn", factor=1.5, original=64, base=1e6),
                                dict(frequencies=[0.0, -1.0, math.pi, 1e-9] * 16, magnitude=-0.5), dict(frequencies=[7.5 * math.pi] * 64)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_frequencies_and_far_positions(libgemm, kw, layout):
    from accelerator_gb300 import sequences
    part = 2 * len(kw["frequencies"]) if "frequencies" in kw else 128
    table = sequences.Rotary(part, layout=layout, **kw)
    positions = ints([0, 1, 2, 1000, 65537, 1 << 20, 10 ** 7, 2 ** 31 - 1])
    Q = torch.randn(8, 3, 128, device="cuda")
    q, _ = sequences.rotary(Q, None, positions, table)
    check_turned(q, Q, positions, table)
    again, _ = sequences.rotary(q, None, positions, table, inverse=True)      # back, times the magnitude twice
    limit = 30 * 2.0 ** -24 * (Q.abs() + 1).max() * max(1.0, table.magnitude ** 2)
    assert (again[..., :part] - Q[..., :part] * table.magnitude ** 2).abs().max() <= limit


def test_tables_that_are_refused():
    from accelerator_gb300 import sequences
    with pytest.raises(TypeError):
        sequences.Rotary(64, device="cpu")
    for part in (63, 0, -2):
        with pytest.raises(ValueError):
            sequences.Rotary(part, device="cpu")
    for kw in (dict(layout="other"), dict(scaling="other"), dict(base=0.0), dict(factor=-1.0), dict(scaling="yarn"), dict(frequencies=[1.0]),
               dict(frequencies=[1.0] * 31 + [float("nan")]), dict(magnitude=float("inf")), dict(magnitude=1e39),
               dict(frequencies=[1.0] * 32, scaling="linear")):
        with pytest.raises(ValueError):
            sequences.Rotary(64, device="cpu", **kw)


@gpu
def test_scalings(libgemm):
    from accelerator_gb300 import sequences
    plain = sequences.Rotary(128).frequencies
    assert plain[0] == 1.0 and math.isclose(plain[32], 0.01) and math.isclose(plain[63], 10000.0 ** (-126 / 128))
    assert all(math.isclose(a, b / 4) for a, b in zip(sequences.Rotary(128, scaling="linear", factor=4.0).frequencies, plain))
    ntk = sequences.Rotary(128, scaling="ntk", factor=4.0).frequencies
    assert ntk[0] == 1.0 and math.isclose(ntk[63], plain[63] / 4)             # the slowest pair is stretched by the factor
    yarn = sequences.Rotary(128, scaling="yarn", factor=4.0, original=4096)
    for f, p in zip(yarn.frequencies, plain):
        turns = 4096 * p / (2 * math.pi)
        assert math.isclose(f, p) if turns >= 32 else math.isclose(f, p / 4) if turns <= 1 else p / 4 < f < p
    assert math.isclose(yarn.magnitude, 1 + 0.1 * math.log(4))
    again = copy.deepcopy(yarn)
    assert torch.equal(again.turns, yarn.turns) and again.turns.data_ptr() != yarn.turns.data_ptr()
    assert (again.layout, again.magnitude, again.frequencies) == (yarn.layout, yarn.magnitude, yarn.frequencies)
    with pytest.raises(AttributeError):
        yarn.magnitude = 1.0


@gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_rotary_in_place_of_a_joint_projection(libgemm, layout, kind, shift):
    """Slices of one array, in place; what lies between them stays as it was.
    Rows with a negative position stay, too."""
    from accelerator_gb300 import sequences
    table = sequences.Rotary(48, layout=layout)
    joint = torch.randn(50, 7 * 64 + 5, device="cuda").to(DTYPES[kind])
    before = joint.clone()

    def slices(x):
        return x[:, shift:shift + 256].unflatten(1, (4, 64)), x[:, 256 + shift:384 + shift].unflatten(1, (2, 64))

    positions = torch.arange(50, device="cuda", dtype=torch.int32) * 31
    positions[7] = -1
    positions[49] = -2 ** 31
    Q, K = slices(joint)
    got = sequences.rotary(Q, K, positions, table, out=(Q, K))
    assert got[0] is Q and got[1] is K
    kept = positions >= 0
    for x, y in zip(slices(joint), slices(before)):
        check_turned(x[kept], y[kept], positions[kept], table)
        assert torch.equal(x[~kept], y[~kept])
        y.copy_(x)
    assert torch.equal(joint, before)
    # heads of queries and keys that take turns
    mixed = torch.randn(9, 3, 2, 64, device="cuda").to(DTYPES[kind])
    before = mixed.clone()
    sequences.rotary(mixed[:, :, 0], mixed[:, :, 1], positions[:9].abs(), table, out=(mixed[:, :, 0], mixed[:, :, 1]))
    for i in (0, 1):
        check_turned(mixed[:, :, i], before[:, :, i], positions[:9].abs(), table)
    # one key for all rows and heads: a broadcast input
    one = torch.randn(1, 1, 64, device="cuda").to(DTYPES[kind]).expand(9, 2, 64)
    q, k = sequences.rotary(mixed[:, :, 0], one, positions[:9].abs(), table)
    check_turned(k, one, positions[:9].abs(), table)
    assert libgemm.debug_status() == libgemm.OK


@gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_the_way_back_is_the_gradient(libgemm, layout):
    """Of sum(w * rotary(x)): against the formula's, and against differences."""
    from accelerator_gb300 import sequences
    table = sequences.Rotary(32, layout=layout, scaling="yarn", factor=2.0, original=128)
    x = torch.randn(6, 2, 40, device="cuda", dtype=torch.float64)
    w, positions = torch.randn(6, 2, 40, device="cuda"), ints([0, 1, 5, 77, 1000, 123456])
    leaf = x.clone().requires_grad_()
    (turned(leaf, positions, table) * w).sum().backward()
    got, _ = sequences.rotary(w, None, positions, table, inverse=True)
    assert (got.double() - leaf.grad).abs().max() <= 20 * 2.0 ** -24 * w.abs().max() * table.magnitude
    for _ in range(20):      # the map is linear: a difference is exact but for binary32's roundings
        d = torch.randn_like(w)
        up, down = (sequences.rotary((x.float() + s * d), None, positions, table)[0].double() for s in (1, -1))
        slope = ((up - down) * w).sum() / 2
        assert (slope - (got.double() * d).sum()).abs() <= 480 * 40 * 2.0 ** -24 * 16


@gpu
def test_rotary_recorded_and_on_another_stream(libgemm):
    from accelerator_gb300 import sequences
    table = sequences.Rotary(64)
    Q, K, positions = torch.randn(40, 4, 64, device="cuda"), torch.randn(40, 2, 64, device="cuda"), ints(range(40))
    want = sequences.rotary(Q, K, positions, table)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sequences.rotary(Q, K, positions, table, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sequences.rotary(Q, K, positions, table)
    positions.add_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, sequences.rotary(Q, K, positions, table)))


@gpu
def test_rotary_refusals_of_the_binding(libgemm, monkeypatch):
    from accelerator_gb300 import lowbit, sequences
    table = sequences.Rotary(64)
    Q, K, positions = torch.randn(4, 4, 64, device="cuda"), torch.randn(4, 2, 64, device="cuda"), ints(range(4))
    for bad in ((Q.double(), K, positions), (Q, K.half(), positions), (Q, K.cpu(), positions), (Q[0], K, positions), (Q, K, positions.long()),
                (Q, K, positions[None]), (Q.transpose(1, 2), K, positions), (Q, K, ints(range(8))[::2])):
        with pytest.raises(TypeError):
            sequences.rotary(*bad, table)
    for bad in ((Q, K[:3], positions), (Q, K, positions[:3]), (Q[..., :32], K[..., :32], positions)):
        with pytest.raises(ValueError):
            sequences.rotary(*bad, table)
    with pytest.raises(ValueError):
        sequences.rotary(Q, K, positions, table, out=(K, K))
    both = torch.randn(4, 6, 64, device="cuda")
    for out in ((Q, Q[:, :2]), (both[:, :4], both[:, 3:5]), (K.new_empty(64).expand(4, 4, 64), K)):
        with pytest.raises((libgemm.GemmError, TypeError)):
            sequences.rotary(Q, K, positions, table, out=out)
    wide = torch.randn(5, 4, 64, device="cuda")
    with pytest.raises(libgemm.GemmError):
        sequences.rotary(wide[:4], None, positions, table, out=(wide[1:], None))      # a row further
    count = libgemm.launch_count()
    monkeypatch.setattr(lowbit, "_current_device", lambda: 1)
    with pytest.raises(TypeError):
        sequences.rotary(Q, K, positions, table)
    assert libgemm.launch_count() == count


# ---- together ------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_steps_of_everything_together(libgemm, bits):
    """Prompts, then steps in which sequences rest or get some tokens: plan,
    positions, cache and attention, against 64 bits over what the cache holds, whose
    keys are the turned ones."""
    from accelerator_gb300 import lowbit, sequences
    page, heads, dim, n = 16, 2, 64, 4
    cache = (lowbit.Kv4Cache if bits == 4 else lowbit.KvCache).empty(40, heads, dim, page)
    table = torch.full((n, 9), -1, dtype=torch.int32, device="cuda")
    free, available = torch.randperm(40, device="cuda").to(torch.int32), ints([40])
    lengths, turn = ints([0] * n), sequences.Rotary(dim, scaling="yarn", factor=4.0, original=64)
    keys, total = [torch.zeros(0, heads, dim, device="cuda", dtype=torch.bfloat16) for _ in range(n)], [0] * n
    for counts in ([50, 1, 0, 33], [1, 1, 1, 1], [1, 0, 20, 1], [1, 1, 1, 0], [17, 1, 1, 40]):
        tokens = sum(counts)
        joint = torch.randn(tokens, 8 + 2 * heads, dim, device="cuda").to(torch.bfloat16)
        Q, K, V = joint.split((8, heads, heads), 1)
        p = sequences.kv_plan(table, lengths, ints(counts), free, available, page, tokens, update=True)
        Q, K = sequences.rotary(Q, K, p.positions, turn)
        lowbit.kv_append(cache, K, V, table, p.starts, p.first)
        O = lowbit.kv_attention(Q, cache, table, p.starts, p.lengths).double()
        assert libgemm.debug_status() == libgemm.OK
        total = [a + b for a, b in zip(total, counts)]
        assert p.lengths.tolist() == total
        # slots name the same places as the table
        row = torch.arange(tokens, device="cuda")
        seq = torch.searchsorted(p.starts[1:].long(), row, right=True)
        assert torch.equal(p.slots, table[seq, (p.positions // page).long()].long() * page + p.positions % page)
        starts = ints([0, *torch.tensor(total).cumsum(0).tolist()])
        k, v = lowbit.kv_read(cache, table, starts, ints([0] * n), sum(total), dtype=torch.float32)
        at = 0
        for b in range(n):
            rows = slice(at, at + counts[b])
            keys[b], at = torch.cat([keys[b], K[rows]]), at + counts[b]
            mine = slice(int(starts[b]), int(starts[b + 1]))
            if total[b] == 0:
                continue
            step = keys[b].float().abs().amax(-1, keepdim=True) / 7 if bits == 4 else keys[b].float().abs().max() / 127
            assert ((k[mine] - keys[b].float()).abs() <= 0.56 * step if bits == 4 else (k[mine] - keys[b].float()).abs() <= 4 * step).all()
            q = Q[rows].double().view(-1, heads, 4, dim)
            a = torch.einsum("thgd,nhd->thgn", q, k[mine].double()) / 8
            hide = torch.arange(total[b], device="cuda") > torch.arange(total[b] - counts[b], total[b], device="cuda")[:, None]
            want = torch.einsum("thgn,nhd->thgd", a.masked_fill(hide[:, None, None], -float("inf")).softmax(-1), v[mine].double())
            assert ((O[rows] - want.reshape(-1, 8, dim)).abs() <= 0.01 * v[mine].abs().max()).all() if counts[b] else True
    assert available.item() == 40 - sum(-(-t // page) for t in total)


@gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("counts", [[1, 0, 1], [300, 0, 41]])
def test_rows_behind_the_last_sequence(libgemm, bits, counts):
    """A step with room for more rows than it has: the calls on a cache leave the
    rows behind as they were (and report the offsets that end before them), and the
    others get what they get alone."""
    from accelerator_gb300 import lowbit, sequences
    page, heads, dim, rows, spare = 16, 2, 64, sum(counts), 3
    turn = sequences.Rotary(dim)
    Q, K, V = [torch.randn(rows + spare, n, dim, device="cuda").to(torch.bfloat16) for n in (8, heads, heads)]
    Q[rows:] = K[rows:] = V[rows:] = float("nan")
    got = []
    for room in (0, spare):
        cache = (lowbit.Kv4Cache if bits == 4 else lowbit.KvCache).empty(40, heads, dim, page)
        for x in ([cache.data] if bits == 4 else [cache.k_codes, cache.v_codes]):
            x.zero_()
        table = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
        p = sequences.kv_plan(table, ints([0, 0, 0]), ints(counts), ints(range(40)), ints([40]), page, rows + room)
        assert p.positions[rows:].tolist() == p.slots[rows:].tolist() == [-1] * room
        q, k = [torch.full_like(x[:rows + room], 7.0) for x in (Q, K)]
        sequences.rotary(Q[:rows + room], K[:rows + room], p.positions, turn, out=(q, k))
        assert (q[rows:] == 7).all() and (k[rows:] == 7).all()
        assert libgemm.debug_status() == libgemm.OK
        status = libgemm.ERR_INDEX if room else libgemm.OK
        lowbit.kv_append(cache, k, V[:rows + room], table, p.starts, p.first)
        assert libgemm.debug_status() == status
        O = torch.full_like(q, 7.0)
        lowbit.kv_attention(q, cache, table, p.starts, p.lengths, out=O)
        assert libgemm.debug_status() == status
        assert (O[rows:] == 7).all()
        got.append((q[:rows], k[:rows], O[:rows], *([cache.data] if bits == 4 else [cache.k_codes, cache.v_codes, cache.k_scales])))
    assert got[0][2].isfinite().all()
    for x, y in zip(*got):
        assert torch.equal(x, y)


# ---- without a GPU ---------------------------------------------------------------

def _plan(libgemm, **change):
    at = {name: FAKE + i * G for i, name in enumerate(("table", "lengths", "counts", "free", "available", "starts", "first", "after",
                                                       "heights", "left", "positions", "slots"))}
    a = dict(at, width=5, capacity=9, page=16, tokens=4, sequences=2)
    a.update(change)
    p = lambda n: a[n] or None      # noqa: E731
    return libgemm.lib().gemm_kv_plan(p("table"), a["width"], p("lengths"), p("counts"), p("free"), a["capacity"], p("available"), a["page"],
                                      a["tokens"], a["sequences"], p("starts"), p("first"), p("after"), p("heights"), p("left"),
                                      p("positions"), p("slots"), None)


@pytest.mark.parametrize("change,want", [
    *(({name: 0}, 1) for name in ("table", "lengths", "counts", "free", "available", "starts", "first", "after", "heights", "left",
                                  "positions", "slots")),
    ({"tokens": -1}, 1), ({"tokens": 1 << 31}, 1), ({"sequences": -1}, 1), ({"sequences": 2 ** 31 - 1}, 1), ({"width": -1}, 1),
    ({"capacity": -1}, 1), ({"page": 0}, 1), ({"page": 24}, 1), ({"page": 1 << 21}, 1), ({"width": 1 << 31}, 1),
    ({"table": FAKE + 2}, 2), ({"slots": FAKE + 11 * G + 4}, 2), ({"left": FAKE + 9 * G + 1}, 2),
    ({"after": FAKE + 2 * G}, 1), ({"after": FAKE + G + 4}, 1), ({"starts": FAKE + 6 * G}, 1), ({"left": FAKE + 3 * G}, 1),
    ({"positions": FAKE + 11 * G}, 1), ({"table": FAKE + 3 * G - 8}, 1)])
def test_plan_checks(libgemm, change, want):
    assert _plan(libgemm, **change) == want


def _rotary(libgemm, **change):
    a = dict(Q=FAKE, qr=256, qh=64, Qo=FAKE + G, qor=256, qoh=64, heads=4, K=FAKE + 2 * G, kr=128, kh=64, Ko=FAKE + 3 * G, kor=128, koh=64,
             k_heads=2, kind=1, rows=9, dim=64, part=64, layout=0, positions=FAKE + 4 * G, turns=FAKE + 5 * G, magnitude=1.0)
    a.update(change)
    p = lambda n: a[n] or None      # noqa: E731
    return libgemm.lib().gemm_rotary(p("Q"), a["qr"], a["qh"], p("Qo"), a["qor"], a["qoh"], a["heads"], p("K"), a["kr"], a["kh"], p("Ko"),
                                     a["kor"], a["koh"], a["k_heads"], a["kind"], a["rows"], a["dim"], a["part"], a["layout"],
                                     p("positions"), p("turns"), a["magnitude"], 0, None)


JOINT = dict(Q=FAKE, qr=512, K=FAKE + 512, kr=512, Qo=FAKE, qor=512, Ko=FAKE + 512, kor=512)      # bytes: 4 heads of 64 are 512


@pytest.mark.parametrize("change,want", [
    ({"Q": 0}, 1), ({"Qo": 0}, 1), ({"K": 0}, 1), ({"Ko": 0}, 1), ({"positions": 0}, 1), ({"turns": 0}, 1), ({"kind": 3}, 1), ({"kind": -1}, 1),
    ({"rows": -1}, 1), ({"rows": 1 << 31}, 1), ({"heads": 0}, 1), ({"k_heads": -1}, 1), ({"heads": 1 << 15}, 1), ({"dim": 1026, "part": 64}, 1),
    ({"part": 63}, 1), ({"part": 66}, 1), ({"part": 0}, 1), ({"layout": 2}, 1), ({"magnitude": float("nan")}, 1), ({"qr": -1}, 1), ({"koh": -64}, 1),
    ({"qoh": 63}, 1), ({"qor": 255}, 1), ({"Q": FAKE + 1}, 2), ({"Ko": FAKE + 3 * G + 1}, 2), ({"positions": FAKE + 4 * G + 2}, 2),
    ({"turns": FAKE + 5 * G + 4}, 2), ({"kind": 0, "Q": FAKE + 2}, 2), ({"Qo": FAKE + 16}, 1), ({"Qo": FAKE, "qor": 260}, 1), ({"Qo": FAKE + 2 * G}, 1),
    ({"Qo": FAKE + 3 * G}, 1), ({"Ko": FAKE}, 1), ({"Qo": FAKE + 4 * G}, 1), ({"Ko": FAKE + 5 * G}, 1), ({"rows": 0, "Q": 0, "positions": 0}, 0),
    (dict(JOINT, K=FAKE + 510, Ko=FAKE + 510), 1), (dict(JOINT, k_heads=5, kh=64), 1)])
def test_rotary_checks(libgemm, change, want):
    assert _rotary(libgemm, **change) == want


def test_no_device_is_an_error(libgemm):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    closed = (libgemm.ERR_CUDA, libgemm.ERR_UNSUPPORTED_DEVICE)
    assert _plan(libgemm) in closed and _plan(libgemm, after=FAKE + G, left=FAKE + 4 * G) in closed
    assert _rotary(libgemm) in closed and _rotary(libgemm, K=0, Ko=0, k_heads=0) in closed
    assert _rotary(libgemm, Qo=FAKE) in closed and _rotary(libgemm, **JOINT) in closed
    assert _rotary(libgemm, Q=FAKE, Qo=FAKE, qr=384, qor=384, qh=128, qoh=128, heads=3, K=FAKE + 128, Ko=FAKE + 128, kr=384, kor=384, kh=128,
                   koh=128, k_heads=3) in closed
