"""Adapters of many requests on the GPU against a plain 64-bit form (tests/plain_around.py)."""
import pytest
import torch

import plain_around as pa
import sparse_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def make(lengths, ids, K, N, R, A, dtype=BF16, out=F32, seed=0, before=0, after=0, whole=False):
    """Segments of the given lengths, `before` and `after` rows outside; whole: small whole numbers, whose
    sums are exact."""
    g = torch.Generator(device="cuda").manual_seed(seed + K + N + R)
    off = [before]
    for n in lengths:
        off.append(off[-1] + n)
    T = off[-1] + after
    if whole:
        draw = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(dtype)  # noqa: E731
        scale = 2.0 ** torch.randint(-1, 3, (A,), generator=g, device="cuda").float()
    else:
        draw = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5).to(dtype)  # noqa: E731
        scale = torch.randn(A, generator=g, device="cuda")
    base = torch.randint(-9, 10, (T, N), generator=g, device="cuda").to(out) if whole else torch.randn(T, N, generator=g, device="cuda").to(out)
    return {"x": draw(T, K), "down": draw(A, R, K), "up": draw(A, N, R), "scale": scale, "offsets": off, "ids": list(ids), "base": base}


def run(o, base="base", scale=True, x=None):
    """base: "base", "none", or "y" (in place)."""
    T, N = o["base"].shape
    y = o["base"].clone() if base == "y" else torch.full((T, N), 7.0, dtype=o["base"].dtype, device="cuda")
    ws = moe.alloc_adapter_workspace()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    moe.moe_adapter_matmul(o["x"] if x is None else x, o["down"], o["up"], o["scale"] if scale else None, i32(o["offsets"]), i32(o["ids"]), y, ws,
                           base={"base": o["base"], "none": None, "y": y}[base])
    moe.moe_check_errors(ws)
    return y


def check(o, base="base", scale=True, exact=False, x=None):
    got = run(o, base, scale, x)
    start = o["base"].double() if base == "y" else torch.full_like(got, 7.0, dtype=torch.float64)
    want, bound = pa.adapter(o["x"].double(), o["down"].double(), o["up"].double(), o["scale"] if scale else None, o["offsets"],
                             o["ids"], start, None if base == "none" else o["base"].double())
    if exact:
        assert torch.equal(got.double(), want)
        return
    limit = bound + pa.HALF_STEP[got.dtype] * (want.abs() + bound) + pa.TINY[got.dtype]
    err = (got.double() - want).abs()
    assert bool((err <= limit).all()), "off by %.3g of the bound" % float((err / limit).max())


SHAPES = [  # lengths, ids, K, N, R, adapters
    ([1], [0], 8, 8, 8, 1),
    ([1], [2], 2048, 6144, 16, 4),
    ([1, 1, 1, 1], [3, 0, 3, 1], 1000, 520, 24, 4),
    ([2, 3, 4, 5, 7, 8, 9], [0, 1, 2, 0, 1, 2, 0], 264, 136, 40, 3),
    ([0, 5, 0, 0, 1, 0], [0, 1, 2, 0, 1, 2], 72, 80, 8, 3),
    ([17, 0, 130, 1], [1, 0, 0, 1], 520, 264, 16, 2),
    ([300], [0], 256, 512, 64, 1),
    ([127, 129, 256], [1, 2, 0], 712, 328, 48, 3),
    ([1000, 3], [0, 1], 640, 1032, 128, 2),
    ([128], [0], 64, 64, 8, 1),
    ([513], [0], 6144, 264, 32, 1),
]


@pytest.mark.parametrize("lengths,ids,K,N,R,A", SHAPES)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32)])
def test_sizes(lengths, ids, K, N, R, A, dtype, out):
    check(make(lengths, ids, K, N, R, A, dtype, out))


@pytest.mark.parametrize("lengths,ids,K,N,R,A", SHAPES)
def test_exact_in_whole_numbers(lengths, ids, K, N, R, A):
    """Numbers of few bits, whose products and sums are exact in fp32 and between the products in 16 bits twice."""
    o = make(lengths, ids, K, N, R, A, BF16, F32, whole=True)
    check(o, exact=True)
    check(o, base="y", exact=True)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("out", [BF16, F16, F32])
def test_types(dtype, out):
    check(make([5, 200, 1, 33], [1, 0, 1, -1], 200, 136, 16, 2, dtype, out))


@pytest.mark.parametrize("base", ["base", "none", "y"])
@pytest.mark.parametrize("lengths,ids", [([1, 4, 2], [0, -1, 1]), ([150, 140, 10], [-1, 1, 0])])
def test_bases_and_rows_outside(base, lengths, ids):
    o = make(lengths, ids, 136, 264, 16, 2, before=3, after=5, out=BF16)
    check(o, base=base)
    check(o, base=base, scale=False)


def test_many_single_tokens():
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(-1, 9, (150,), generator=g).tolist()
    check(make([1] * 150, ids, 1024, 384, 16, 9))


def test_many_segments_of_all_lengths():
    g = torch.Generator().manual_seed(2)
    lengths = (torch.rand(400, generator=g) ** 6 * 300).long().tolist()
    ids = torch.randint(-1, 5, (400,), generator=g).tolist()
    check(make(lengths, ids, 128, 72, 8, 5))
    check(make([0] * 1200 + [3, 1], [0] * 1200 + [1, 0], 128, 72, 8, 2))


def test_strided_rows():
    o = make([40, 200], [1, 0], 328, 128, 32, 2)
    wide = torch.full((240, 400), float("nan"), dtype=BF16, device="cuda")
    wide[:, 8:336] = o["x"]
    check(o, x=wide[:, 8:336])


def test_rows_without_an_adapter_and_outside_are_not_read():
    for n in (3, 150):
        o = make([n, n, n], [0, -1, 1], 128, 64, 8, 2, before=2, after=2)
        clean = run(o)
        o["x"][:2] = o["x"][-2:] = float("nan")
        o["x"][2 + n:2 + 2 * n] = float("nan")
        assert torch.equal(clean, run(o))


def test_what_is_not_finite_stays_in_its_row():
    for n in (4, 200):
        o = make([n, n], [0, 1], 256, 128, 16, 2)
        clean = run(o)
        o["x"][n + 1, 100] = float("nan")
        o["x"][2, 5] = float("inf")
        got = run(o)
        rows = [r for r in range(2 * n) if r not in (2, n + 1)]
        assert torch.equal(got[rows], clean[rows]) and got[n + 1].isnan().all() and not got[2].isfinite().any()


def test_an_adapter_that_is_not_finite_stays_with_its_rows():
    for n in (4, 200):
        o = make([n, n, n], [0, 1, 2], 256, 128, 8, 3)
        clean = run(o)
        o["down"][1], o["up"][1] = float("nan"), float("nan")
        got = run(o)
        assert torch.equal(got[:n], clean[:n]) and torch.equal(got[2 * n:], clean[2 * n:]) and got[n:2 * n].isnan().all()


@pytest.mark.parametrize("n", [3, 200])
def test_bad_lists_are_recorded(n):
    o = make([n, n, n], [0, 1, 0], 64, 64, 8, 2)
    T = 3 * n
    good = run(o)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(off, ids):
        y, ws = torch.full((T, 64), 7.0, device="cuda"), moe.alloc_adapter_workspace()
        moe.moe_adapter_matmul(o["x"], o["down"], o["up"], o["scale"], i32(off), i32(ids), y, ws, base=o["base"])
        with pytest.raises(moe.MoeError):
            moe.moe_check_errors(ws)
        moe.moe_check_errors(ws)
        return y
    for bad in (2, -2, 1 << 30):
        y = call(o["offsets"], [0, bad, 0])
        assert y[n:2 * n].isnan().all() and torch.equal(y[:n], good[:n]) and torch.equal(y[2 * n:], good[2 * n:])
    y = call([0, n, 2 * n, T + 1], [0, 1, 0])
    assert torch.equal(y[:2 * n], good[:2 * n]) and (y[2 * n:] == 7).all()
    y = call([-1, n, 2 * n, T], [0, 1, 0])
    assert (y[:n] == 7).all() and torch.equal(y[2 * n:], good[2 * n:])
    call([0, 2 * n, n, T], [0, 1, 0])


def test_more_than_two_to_the_31_elements():
    """Outputs and rows past 2^31 elements, with tiles and with few rows a segment."""
    T, K, N = 360000, 64, 6144
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    down, up = torch.randn(2, 8, K, generator=g, device="cuda").to(BF16), torch.randn(2, N, 8, generator=g, device="cuda").to(BF16)
    y, ws = torch.empty(T, N, dtype=BF16, device="cuda"), moe.alloc_adapter_workspace()
    for lengths in ([T - 500, 500], [2, 3] * (T // 5)):
        off = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
        ids = (torch.arange(len(lengths), device="cuda") % 2).to(torch.int32)
        y.fill_(7)
        moe.moe_adapter_matmul(x, down, up, None, off, ids, y, ws)
        moe.moe_check_errors(ws)
        rows = torch.tensor([0, 4, (1 << 31) // N - 1, (1 << 31) // N + 1, T - 501, T - 500, T - 1], device="cuda")
        of = ids[torch.searchsorted(off, rows.to(torch.int32), right=True) - 1].long()
        u = torch.einsum("tk,trk->tr", x[rows].double(), down[of].double())
        want = torch.einsum("tr,tnr->tn", u, up[of].double())
        mag = torch.einsum("tr,tnr->tn", torch.einsum("tk,trk->tr", x[rows].double().abs(), down[of].double().abs()), up[of].double().abs())
        assert bool(((y[rows].double() - want).abs() <= 2.0 ** -8 * want.abs() + (K * 2 * pa.U + 2.0 ** -17) * 1.01 * mag).all())


def test_a_small_workspace_takes_several_passes():
    o = make([100, 400, 3, 260], [1, 0, -1, 1], 264, 136, 24, 2, before=7, after=4)
    want = run(o)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for rows in (128, 300):
        for in_place in (False, True):
            ws = moe.alloc_adapter_workspace(rows, 24)
            y = o["base"].clone() if in_place else torch.full_like(o["base"], 7.0)
            moe.moe_adapter_matmul(o["x"], o["down"], o["up"], o["scale"], i32(o["offsets"]), i32(o["ids"]), y, ws,
                                   base=y if in_place else o["base"])
            moe.moe_check_errors(ws)
            assert torch.equal(y[7:-4], want[7:-4])
    with pytest.raises(moe.MoeError):
        moe.moe_adapter_matmul(o["x"], o["down"], o["up"], o["scale"], i32(o["offsets"]), i32(o["ids"]), y, ws[:256])


def test_in_a_graph():
    o = make([1, 1, 70, 1], [0, 1, 2, 0], 512, 512, 16, 3, out=BF16)
    want = run(o)
    ws, y = moe.alloc_adapter_workspace(), torch.empty_like(o["base"])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    off, ids = i32(o["offsets"]), i32(o["ids"])
    call = lambda: moe.moe_adapter_matmul(o["x"], o["down"], o["up"], o["scale"], off, ids, y, ws, base=o["base"])  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        y.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("R", [72, 128])
@pytest.mark.parametrize("n", [5, 9, 15, 17, 33, 63, 65, 100, 127, 129, 137, 250])
def test_short_tiles_of_a_cluster(n, R):
    """The CTAs that share a tile's inputs have rows of their own to add up, some an odd number and some none."""
    o = make([n], [0], 2048, 264, R, 1, out=F32)
    check(o)
    first = run(o)
    for _ in range(5):
        assert torch.equal(run(o), first)


@pytest.mark.parametrize("n", [3, 200])
@pytest.mark.parametrize("many", [False, True])
def test_a_bad_offset_inside_a_list(n, many):
    """What stands in no well-ordered segment stays as it was, and every other row has its result or what it held;
    with runs of empty segments the search takes more than one step."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x, down, up = (torch.randn(*s, generator=g, device="cuda").to(BF16) for s in ((4 * n, 64), (2, 8, 64), (2, 64, 8)))
    base = torch.randn(4 * n, 64, generator=g, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(off):
        y, ws = torch.full((4 * n, 64), 7.0, device="cuda"), moe.alloc_adapter_workspace(4 * n, 8)
        moe.moe_adapter_matmul(x, down, up, None, i32(off), i32([i % 2 for i in range(len(off) - 1)]), y, ws, base=base)
        return y, ws
    for wrong in (5000000, -7, -2**31, 2**31 - 1, 4 * n + 1, 3 * n, 0):
        off = [0, n, wrong, 2 * n, 3 * n]
        if many:
            off = [0] * 41 + off[:3] + [2 * n] * 50 + off[4:] + [3 * n] * 41
        y, ws = call(off)
        with pytest.raises(moe.MoeError):
            moe.moe_check_errors(ws)
        claims = [0] * (4 * n)
        for a, b in zip(off, off[1:]):
            if 0 <= a <= b <= 4 * n:
                for r in range(a, b):
                    claims[r] += 1
        held = (y == 7).all(1).tolist()
        assert all(h for h, c in zip(held, claims) if c == 0)
        for i, (a, b) in enumerate(zip(off, off[1:])):
            rows = [r for r in range(a, b) if claims[r] == 1 and not held[r]] if 0 <= a <= b <= 4 * n else []
            if rows:
                u = x[rows].double() @ down[i % 2].double().T
                want = base[rows].double() + u @ up[i % 2].double().T
                mag = (x[rows].double().abs() @ down[i % 2].double().abs().T) @ up[i % 2].double().abs().T
                # sums of 64 and 8 terms, u as two 16-bit parts, the output's rounding
                assert bool(((y[rows].double() - want).abs() <= (160 * pa.U + 2.0 ** -17) * mag + 4 * pa.U * want.abs()).all())
    y, ws = call([0, n, n, 2 * n, 3 * n])      # the next call is right
    moe.moe_check_errors(ws)
    assert not (y[:3 * n] == 7).all(1).any() and (y[3 * n:] == 7).all()


@pytest.mark.parametrize("n", [2, 200])
def test_errors_say_what_became_of_the_rows(n):
    o = make([n, n], [0, 5], 64, 64, 8, 2)
    with pytest.raises(moe.MoeError, match="rows are NaN"):
        run(o)
    with pytest.raises(moe.MoeError, match="skipped"):
        run(dict(o, offsets=[0, n, 2 * n + 1], ids=[0, 1]))


@pytest.mark.parametrize("rows", [1, 128, 256])
def test_the_least_workspace(rows):
    """One or two tiles' rows a pass."""
    o = make([100, 400, 3, 260], [1, 0, -1, 1], 264, 136, 24, 2, before=7, after=4)
    want = run(o)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(moe.moe_adapter_workspace_size(rows, 24), dtype=torch.uint8, device="cuda")
    for in_place in (False, True):
        y = o["base"].clone() if in_place else torch.full_like(o["base"], 7.0)
        moe.moe_adapter_matmul(o["x"], o["down"], o["up"], o["scale"], i32(o["offsets"]), i32(o["ids"]), y, ws,
                               base=y if in_place else o["base"])
        moe.moe_check_errors(ws)
        assert torch.equal(y[7:-4], want[7:-4])
    with pytest.raises(moe.MoeError):
        moe.moe_adapter_matmul(o["x"], o["down"], o["up"], o["scale"], i32(o["offsets"]), i32(o["ids"]), y,
                               ws[:moe.moe_adapter_workspace_size(128, 24) - 1])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lengths,R", [([300, 140], 24), ([500], 128), ([2, 1], 24)])
def test_what_stands_between_the_products_keeps_its_digits(dtype, lengths, R):
    """Sums of more digits than one or two 16-bit numbers of bf16 hold, each handed on to an fp32 output as it is.
    All of them are whole numbers below 2^24, whatever order they are added in: exact."""
    g = torch.Generator(device="cuda").manual_seed(R)
    T, S, K, N = sum(lengths), len(lengths), 1024, 264
    draw = lambda *s: torch.randint(-100, 101, s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, down, base = draw(T, K), draw(S, R, K), draw(T, N).float()
    up = torch.zeros(S, N, R, dtype=dtype, device="cuda")
    n = torch.arange(N, device="cuda")
    up[:, n, n % R] = (1 - 2 * (n // R % 2)).to(dtype)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    off = [sum(lengths[:i]) for i in range(S + 1)]
    y, ws = torch.empty(T, N, device="cuda"), moe.alloc_adapter_workspace(T, R)
    moe.moe_adapter_matmul(x, down, up, None, i32(off), i32(list(range(S))), y, ws, base=base)
    moe.moe_check_errors(ws)
    want, _ = pa.adapter(x.double(), down.double(), up.double(), None, off, range(S), torch.zeros_like(base, dtype=torch.float64), base.double())
    assert float(want.abs().max()) > 2 ** 17 and torch.equal(y.double(), want)


@pytest.mark.parametrize("n", [2, 300])
@pytest.mark.parametrize("dtype,x,up,scale", [(BF16, 1e-20, 1e35, 1.0), (BF16, 1e25, 1e-25, 1e10), (BF16, 1e-25, 1e25, 1e-15),
                                              (BF16, 1e30, 1e-30, 1e7), (F16, 1e3, 1e-3, 1e36), (F16, 1e-3, 1e3, 1e-36),
                                              (F16, 1e5, 1e-6, 1e38)])
def test_factors_far_from_one(n, dtype, x, up, scale):
    """Sums, factors and results within fp32's range, the products of some of them beyond it."""
    o = make([n, n], [0, 1], 256, 136, 16, 2, dtype, F32)
    o["x"], o["up"] = (o["x"].double().abs() * x).to(dtype), (o["up"].double() * up).to(dtype)
    o["down"].abs_()
    o["scale"] = torch.full((2,), scale, device="cuda")
    o["base"] *= 0
    check(o)
    check(o, base="none")
