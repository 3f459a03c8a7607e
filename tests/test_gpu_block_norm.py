"""Norms around a block on the GPU against plain 64-bit forms (tests/plain_around.py)."""
import itertools

import pytest
import torch

import plain_around as pa
import sparse_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def operands(T, H, stream, dt, gate, post=True, pre=True, seed=0, pad=0):
    """Operands of both directions; rows of x and y `pad` elements apart beyond H."""
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * T + H)
    x = (randn(g, T, H + pad) * torch.exp(randn(g, T, 1))).to(stream)[:, :H]
    y = (0.5 * randn(g, T, H + pad)).to(dt)[:, :H]
    shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    return {"x": x, "y": y, "gate": None if shape is None else randn(g, *shape).to(dt),
            "post_w": 1 + 0.3 * randn(g, H) if post else None, "pre_w": 1 + 0.3 * randn(g, H) if pre else None,
            "dout": randn(g, T, H).to(stream), "dn": randn(g, T, H).to(dt) if pre else None}


def close(got, want, bound, dtype, what):
    err = (got.double() - want).abs()
    limit = bound + pa.HALF_STEP[dtype] * (want.abs() + bound) + pa.TINY[dtype]
    assert got.dtype is dtype and bool((err <= limit).all()), "%s: off by %.3g of the bound" % (what, float((err / limit).max()))


def run(o, eps=1e-5, a=1.0, b=1.0, want=("dx", "dy", "dgate", "dpost", "dpre"), alias=False):
    """All outputs of both directions: what is not asked for or does not apply is absent."""
    x, y, gate, dt = o["x"], o.get("y"), o.get("gate"), (o["y"] if o.get("y") is not None else o["dn"]).dtype
    T, H = x.shape
    fill = lambda like, t: torch.full(tuple(like), 77.0, dtype=t, device="cuda")  # noqa: E731
    kept = fill((T, 2), F32)
    f = {"out": fill((T, H), x.dtype)} | ({"n": fill((T, H), dt)} if o["pre_w"] is not None else {})
    ops = {k: o.get(k) for k in ("y", "post_w", "gate", "pre_w")}
    moe.moe_block_norm_forward(x, eps, **ops, **f, residual_scale=a, branch_scale=b, kept=kept)
    full = gate is not None and gate.shape == x.shape
    r = {"dx": fill((T, H), x.dtype), "dy": fill((T, H), dt) if y is not None else None,
         "dgate": None if gate is None else fill(gate.shape, dt if full else F32),
         "dpost": fill((H,), F32) if o.get("post_w") is not None else None, "dpre": fill((H,), F32) if "n" in f else None}
    r = {k: v for k, v in r.items() if v is not None and k in want}
    dout, dn = o.get("dout"), o.get("dn")
    if alias:
        dout, dn = dout.clone(), dn.clone()
        r["dx"], r["dy"] = dout, dn
    ws = moe.alloc_block_norm_workspace(T, H)
    moe.moe_block_norm_backward(x, kept, ws, **ops, dout=dout, dn=dn, **r, residual_scale=a, branch_scale=b)
    moe.moe_check_errors(ws)
    return f | r


def check(o, got, eps=1e-5, a=1.0, b=1.0):
    d = {k: None if v is None else v.double() for k, v in o.items()}
    T, H = o["x"].shape
    gate = d.get("gate")
    if gate is not None and gate.dim() == 1:
        gate = gate.view(1, H)
    ops = dict(y=d.get("y"), post=d.get("post_w"), gate=gate, pre=d["pre_w"], a=a, b=b)
    f = pa.norm_forward(d["x"], eps, **ops)
    r = pa.norm_backward(d["x"], eps, **ops, dout=d.get("dout"), dn=d.get("dn"))
    for k, v in got.items():
        want, bound = (f if k in ("out", "n") else r)[k]
        close(v, want.reshape(v.shape), bound.reshape(v.shape), v.dtype, k)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("T,H", [(1, 8), (1, 6144), (3, 64), (5, 264), (33, 1000), (130, 512), (700, 2048), (9, 7168), (2, 8192)])
def test_sizes(T, H, gate):
    o = operands(T, H, BF16, BF16, gate)
    check(o, run(o, a=0.9, b=0.75), a=0.9, b=0.75)


@pytest.mark.parametrize("stream,dt", list(itertools.product([F32, BF16, F16], [F32, BF16, F16])))
def test_types(stream, dt):
    for gate in ("full", "token"):
        o = operands(37, 1096, stream, dt, gate, seed=5)
        check(o, run(o))


def test_largest_rows_in_fp32():
    """A row of every operand fills the kernel's shared memory: one row at a time."""
    o = operands(700, 8192, F32, F32, "full")
    check(o, run(o))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("T,H,stream,dt", [(1300, 128, F32, BF16), (9, 256, BF16, F16), (21, 6400, BF16, BF16), (13, 8192, F32, F32)])
def test_no_norm_of_the_sum(T, H, stream, dt, gate, post):
    """A block without a next one's norm, on one warp a row and on the widest."""
    o = operands(T, H, stream, dt, gate, post, False)
    check(o, run(o, a=0.5), a=0.5)


@pytest.mark.parametrize("post,pre,gate", [(False, False, "none"), (True, False, "channel"), (False, True, "full"),
                                           (False, True, "token"), (True, False, "token")])
def test_parts_left_out(post, pre, gate):
    o = operands(41, 328, BF16, F16, gate, post, pre)
    check(o, run(o))


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("T,H,stream,dt", [(2000, 1024, F32, BF16), (1001, 6144, BF16, BF16), (15000, 64, F16, F32), (1500, 7168, BF16, F16),
                                           (3000, 2056, F32, F32)])
def test_many_rows(T, H, stream, dt, gate):
    """Several rows a CTA, forward too; with everything there and with parts left out."""
    o = operands(T, H, stream, dt, gate)
    check(o, run(o, a=1.1, b=0.5), a=1.1, b=0.5)
    o = operands(T, H, stream, dt, gate, post=False)
    check(o, run(o))
    if gate == "none":
        o = {k: v for k, v in o.items() if k in ("x", "pre_w", "dout", "dn")}
        check(o, run(o))


@pytest.mark.parametrize("post,pre", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("T,H", [(4000, 512), (2000, 4104)])
def test_many_rows_are_the_same_every_time(T, H, post, pre):
    """One exchange between a row's warps or two; the rows of a CTA follow one another without a pause."""
    o = operands(T, H, BF16, BF16, "channel", post, pre)
    first = run(o)
    check(o, first)
    for _ in range(10):
        for k, v in run(o).items():
            assert torch.equal(v, first[k]), k


def test_many_rows_in_place():
    o = operands(2500, 1032, BF16, BF16, "full", pad=24)
    got = run(o)
    check(o, got)
    dense = {k: None if v is None else v.contiguous() for k, v in o.items()}
    for k, v in run(dense, alias=True).items():
        assert torch.equal(v, got[k])
    x, y = dense["x"].clone(), dense["y"].clone()
    moe.moe_block_norm_forward(x, 1e-5, y=y, post_w=o["post_w"], gate=o["gate"], pre_w=o["pre_w"], out=x, n=y)
    assert torch.equal(x, got["out"]) and torch.equal(y, got["n"])


def test_more_than_two_to_the_31_elements():
    T, H = 540000, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(T, H, dtype=BF16, device="cuda").normal_(generator=g)
    w = 1 + 0.3 * randn(g, H)
    n, kept = torch.empty_like(x), torch.empty(T, 2, device="cuda")
    moe.moe_block_norm_forward(x, 1e-5, pre_w=w, n=n, kept=kept)
    ws = moe.alloc_block_norm_workspace(T, H)
    dx = torch.empty_like(x)
    moe.moe_block_norm_backward(x, kept, ws, pre_w=w, dn=n, dx=dx)
    moe.moe_check_errors(ws)
    for at in (0, (1 << 31) // H - 1, (1 << 31) // H, T - 3):
        p = slice(at, at + 3)
        o = {"x": x[p], "pre_w": w, "dn": n[p], "dout": None}
        check(o, {"n": n[p], "dx": dx[p]})


def test_a_first_norm():
    """Without y: the norm ahead of a block alone, with and without a scale."""
    o = operands(50, 768, F32, BF16, "none")
    o = {k: v for k, v in o.items() if k in ("x", "pre_w", "dout", "dn")}
    check(o, run(o))
    check(o, run(o, a=0.5), a=0.5)
    o["dout"] = None
    check(o, run(o))


def test_gradient_along_one_way_only():
    o = operands(50, 768, F32, BF16, "channel")
    o["dout"] = None
    check(o, run(o))
    o = operands(50, 768, F32, BF16, "channel", pre=False)
    o["dn"] = None
    check(o, run(o))


@pytest.mark.parametrize("name", ["dx", "dy", "dgate", "dpost", "dpre"])
def test_one_gradient_alone(name):
    for gate in ("channel", "token", "full"):
        o = operands(20, 200, BF16, BF16, gate)
        every, one = run(o), run(o, want=(name,))
        assert torch.equal(every[name], one[name])


def test_strided_rows_and_results_in_place():
    o = operands(300, 1032, BF16, BF16, "full", pad=24)
    assert not o["x"].is_contiguous()
    got = run(o)
    check(o, got)
    dense = {k: None if v is None else v.contiguous() for k, v in o.items()}
    for k, v in run(dense).items():
        assert torch.equal(v, got[k])
    for k, v in run(o, alias=True).items():
        assert torch.equal(v, got[k])
    x, y = dense["x"].clone(), dense["y"].clone()
    moe.moe_block_norm_forward(x, 1e-5, y=y, post_w=o["post_w"], gate=o["gate"], pre_w=o["pre_w"], out=x, n=y)
    assert torch.equal(x, got["out"]) and torch.equal(y, got["n"])


def test_rows_of_zeros():
    o = operands(6, 128, F32, F32, "none")
    o["x"][2] = 0
    o["y"][2] = 0
    got = run(o, eps=0.0)
    assert (got["out"][2] == 0).all() and (got["n"][2] == 0).all() and (got["dy"][2] == 0).all()
    assert torch.equal(got["dx"][2], o["dout"][2])
    keep = [0, 1, 3, 4, 5]
    rest = {k: v[keep] if v is not None and v.dim() == 2 else v for k, v in o.items()}
    check(rest, {k: v[keep] if v.dim() == 2 else v for k, v in got.items() if k[:2] in ("ou", "n", "dx", "dy")}, eps=0.0)


def test_what_is_not_finite_stays_in_its_row():
    o = operands(5, 256, BF16, BF16, "token")
    clean = run(o)
    o["y"][1, 7], o["x"][3, 200] = float("nan"), float("inf")
    got = run(o, want=("dx", "dy", "dgate"))
    for k, v in got.items():
        for row in (0, 2, 4):
            assert torch.equal(v[row], clean[k][row]), k
    assert got["n"][1].isnan().all() and not got["n"][3].isfinite().all()


def test_large_and_small_rows():
    """Rows whose squares are near fp32's largest and smallest numbers' square roots."""
    o = operands(4, 512, F32, F32, "none")
    o["x"][0] *= 1e15
    o["y"][1] *= 1e16
    o["y"][2] *= 1e-15
    check(o, run(o, eps=0.0), eps=0.0)


def test_no_rows():
    o = {"x": torch.empty(0, 64, device="cuda"), "y": torch.empty(0, 64, device="cuda"), "post_w": torch.ones(64, device="cuda"),
         "pre_w": torch.ones(64, device="cuda"), "gate": torch.ones(64, device="cuda"), "dout": torch.empty(0, 64, device="cuda"),
         "dn": torch.empty(0, 64, device="cuda")}
    got = run(o)
    assert (got["dpre"] == 0).all() and (got["dpost"] == 0).all() and (got["dgate"] == 0).all()


def test_the_same_again_and_in_a_graph():
    o = operands(1000, 1536, BF16, BF16, "channel")
    first = run(o)
    again = run(o)
    T, H = o["x"].shape
    ws, kept = moe.alloc_block_norm_workspace(T, H), torch.empty(T, 2, device="cuda")
    r = {k: torch.empty_like(v) for k, v in first.items()}
    ops = {k: o[k] for k in ("y", "post_w", "gate", "pre_w")}

    def step():
        moe.moe_block_norm_forward(o["x"], 1e-5, **ops, out=r["out"], n=r["n"], kept=kept)
        moe.moe_block_norm_backward(o["x"], kept, ws, **ops, dout=o["dout"], dn=o["dn"],
                                    **{k: v for k, v in r.items() if k[0] == "d"})
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in r.values():
        v.fill_(5)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    moe.moe_check_errors(ws)
    for k, v in first.items():
        assert torch.equal(v, again[k]) and torch.equal(v, r[k]), k
