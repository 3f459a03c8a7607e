"""Balance loss, counts and the gradient of the router's logits on the GPU against a plain 64-bit form."""
import pytest
import torch

import plain_around as pa
import sparse_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def make(T, E, K, S, dtype=F32, seed=0, varied=False, masked=False, spread=1.5, before=0, after=0):
    """A routing of T tokens in S sequences, `before` and `after` tokens outside all of them."""
    g = torch.Generator().manual_seed(seed + T * 7 + E)
    l = (spread * torch.randn(T, E, generator=g)).to(dtype)
    ids = (l.float() + torch.randn(E, generator=g)).topk(K, dim=1)[1].to(torch.int32)
    keff = torch.randint(0, K + 1, (T,), generator=g, dtype=torch.int32) if varied else torch.full((T,), K, dtype=torch.int32)
    ids[torch.arange(K)[None] >= keff[:, None]] = -1
    cut = torch.sort(torch.randint(before, T - after + 1, (S - 1,), generator=g))[0].tolist()
    valid = (torch.rand(T, generator=g) < 0.7).to(torch.uint8) if masked else None
    return {"logits": l, "ids": ids, "keff": keff, "offsets": [before] + cut + [T - after], "valid": valid, "E": E, "K": K,
            "dw": torch.randn(T, K, generator=g)}


def config(o, norm=True, scale=2.5):
    return moe.MoeConfig.make(64, o["E"], o["K"], 64, norm_topk_prob=int(norm), routed_scaling_factor=scale)


def run(o, dloss=None, dw=False, norm=True, scale=2.5, gdtype=None, logits=None):
    S = len(o["offsets"]) - 1
    cfg = config(o, norm, scale)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    l = o["logits"].cuda() if logits is None else logits
    T = l.shape[0]
    loss, tokens = torch.full((1,), 9.0, device="cuda"), torch.full((S,), 9, dtype=torch.int32, device="cuda")
    counts = torch.full((S, o["E"]), 9, dtype=torch.int32, device="cuda")
    ws = moe.alloc_balance_workspace(cfg, T, S)
    off = torch.tensor(o["offsets"], dtype=torch.int32, device="cuda")
    args = (cfg, l, o["ids"].cuda(), o["keff"].cuda(), off)
    moe.moe_balance_forward(*args, loss, counts, tokens, ws, valid=dev(o["valid"]))
    d = None
    if dloss is not None or dw:
        d = torch.full(l.shape, 9.0, dtype=gdtype or l.dtype, device="cuda")
        moe.moe_balance_backward(*args, counts, tokens, d, ws, dloss=None if dloss is None else torch.tensor([dloss], device="cuda"),
                                 dw=o["dw"].cuda() if dw else None, valid=dev(o["valid"]))
    moe.moe_check_errors(ws)
    return loss.cpu(), counts.cpu(), tokens.cpu(), None if d is None else d.cpu()


def check(o, dloss=None, dw=False, norm=True, scale=2.5, gdtype=None, logits=None):
    loss, counts, tokens, d = run(o, dloss, dw, norm, scale, gdtype, logits)
    want = pa.balance(o["logits"], o["ids"], o["keff"], o["offsets"], o["K"], o["valid"], dloss, o["dw"] if dw else None, norm, scale)
    assert torch.equal(counts.long(), want[0]) and torch.equal(tokens.long(), want[1])
    assert abs(float(loss) - float(want[2])) <= want[3]
    if d is not None:
        limit = want[5] + pa.HALF_STEP[d.dtype] * (want[4].abs() + want[5]) + pa.TINY[d.dtype]
        err = (d.double() - want[4]).abs()
        assert bool((err <= limit).all()), "off by %.3g of the bound" % float((err / limit).max())


@pytest.mark.parametrize("T,E,K,S", [(1, 8, 1, 1), (1, 1, 1, 1), (7, 33, 3, 2), (64, 64, 4, 3), (100, 256, 8, 1), (257, 384, 8, 40),
                                     (300, 333, 7, 5), (90, 512, 16, 90), (50, 511, 2, 3), (1300, 16, 2, 4), (700, 129, 5, 2)])
@pytest.mark.parametrize("varied,masked", [(False, False), (True, True)])
def test_sizes(T, E, K, S, varied, masked):
    o = make(T, E, K, S, varied=varied, masked=masked)
    check(o, dloss=0.3)
    check(o, dloss=-2.0, dw=True)


@pytest.mark.parametrize("E,K", [(8, 8), (13, 2), (32, 8), (32, 9), (31, 16), (64, 16), (61, 3), (48, 1)])
@pytest.mark.parametrize("T,S", [(3, 3), (45, 4), (2777, 60)])
def test_narrow_rows(E, K, T, S):
    """Several rows of a warp at once: cut by sequences, some of them padding, low or without an end beside others."""
    o = make(T, E, K, S, varied=True, masked=True, seed=E * K)
    o["logits"][1::5] -= 90
    o["logits"][2::7, ::2] = -float("inf")
    o["logits"][o["valid"] == 0] = float("nan")
    check(o, dloss=0.7, dw=True)
    check(o, dw=True, norm=False)
    o["ids"][::3] = o["ids"][::3, :1]
    check(o, dloss=0.7, dw=True)


@pytest.mark.parametrize("dtype,gdtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
def test_types(dtype, gdtype):
    for E in (60, 61):
        check(make(80, E, 5, 3, dtype=dtype, varied=True), dloss=100.0, dw=True, gdtype=gdtype)


@pytest.mark.parametrize("norm", [True, False])
def test_weights_alone(norm):
    check(make(65, 48, 6, 2, varied=True), dw=True, norm=norm, scale=1.7)


def test_many_tokens_in_one_sequence_and_across_chunks():
    """More tokens than one chunk a CTA, cut at every kind of place."""
    o = make(12000, 12, 3, 9, seed=3)
    check(o, dloss=1.0, dw=True)


def test_many_short_sequences():
    """One token each, and lengths from none to many side by side in a chunk."""
    o = make(70, 100, 4, 70, varied=True, masked=True)
    o["offsets"] = list(range(71))
    check(o, dloss=1.0, dw=True)
    for E in (40, 41):
        o = make(2000, E, 3, 2, dtype=BF16, varied=True, masked=True)
        g = torch.Generator().manual_seed(6)
        lengths = (torch.rand(300, generator=g) ** 5 * 60).long().tolist()
        off = [5]
        for n in lengths:
            off.append(min(1990, off[-1] + n))
        o["offsets"] = off
        check(o, dloss=1.0, dw=True)


def test_tokens_outside_sequences_and_empty_ones():
    o = make(60, 24, 3, 4, before=9, after=11)
    check(o, dloss=1.0, dw=True)
    o["offsets"] = [5, 5, 20, 20, 20, 41, 41]
    check(o, dloss=1.0, dw=True)
    o["offsets"] = [60, 60]
    loss, counts, tokens, d = run(o, dloss=1.0, dw=True)
    assert float(loss) == 0 and not counts.any() and not tokens.any() and not d.any()


@pytest.mark.parametrize("T", [40, 400])
def test_long_runs_of_empty_sequences(T):
    """Between, ahead of and behind the few that have tokens."""
    o = make(T, 24, 3, 4, varied=True)
    runs = ((0, 700), (3, 1), (17, 333), (18, 256), (19, 1500), (T - 2, 30), (T, 90))
    o["offsets"] = [at for at, n in runs for _ in range(n)]
    check(o, dloss=1.0, dw=True)


def test_padding_is_not_read():
    o = make(40, 24, 3, 2, masked=True)
    clean = run(o, dloss=1.0, dw=True)
    o["logits"][o["valid"] == 0] = float("nan")
    o["dw"][o["valid"] == 0] = float("nan")
    o["ids"][o["valid"] == 0] = 99999
    for a, b in zip(clean, run(o, dloss=1.0, dw=True)):
        assert torch.equal(a, b)
    o["valid"][:] = 0
    loss, counts, _, d = run(o, dloss=1.0, dw=True)
    assert float(loss) == 0 and not counts.any() and not d.any()


def test_slots_behind_keff_are_not_read():
    o = make(40, 24, 3, 2, varied=True)
    clean = run(o, dloss=1.0, dw=True)
    behind = torch.arange(3)[None] >= o["keff"][:, None]
    o["ids"][behind] = 12345
    o["dw"][behind] = float("nan")
    for a, b in zip(clean, run(o, dloss=1.0, dw=True)):
        assert torch.equal(a, b)


def test_scores_far_from_zero():
    """Rows whose scores are all denormal or zero in fp32, saturated rows, and experts closed by -inf or the
    type's lowest value."""
    o = make(12, 40, 4, 2, spread=2.0)
    o["logits"][0] -= 95
    o["logits"][1] -= 500
    o["logits"][2] += 300
    o["logits"][3, ::2] = -float("inf")
    o["logits"][4, :20] = torch.finfo(F32).min
    o["logits"][5, 3] = float("inf")
    o["logits"][6] = -float("inf")           # nothing is left
    o["logits"][7] = torch.finfo(F32).min
    o["logits"][8, 1:] -= 200
    o["ids"] = o["logits"].topk(4, dim=1)[1].to(torch.int32)
    check(o, dloss=1.0, dw=True)
    check(o, dloss=1.0, dw=True, norm=False)


def test_an_expert_kept_twice():
    o = make(30, 16, 4, 1)
    o["ids"][:, 2] = o["ids"][:, 0]
    check(o, dloss=1.0, dw=True)
    check(o, dw=True, norm=False)


def test_rows_of_a_wider_tensor():
    for E, wide, at in ((32, 48, 4), (32, 47, 3), (30, 64, 0)):
        o = make(50, E, 4, 3, dtype=BF16)
        big = torch.full((50, wide), float("nan"), dtype=BF16, device="cuda")
        big[:, at:at + E] = o["logits"].cuda()
        check(o, dloss=1.0, dw=True, logits=big[:, at:at + E])


def test_even_and_uneven_loads():
    T, E = 64, 16
    o = make(T, E, 1, 1)
    o["logits"][:] = 0.25
    o["ids"] = (torch.arange(T) % E).view(T, 1).to(torch.int32)
    assert abs(float(run(o)[0]) - 1) < 1e-6
    o["logits"][:] = -40.0
    o["logits"][:, 3] = 40.0
    o["ids"][:] = 3
    assert abs(float(run(o)[0]) - E) < 1e-4


def test_bad_lists_are_recorded():
    o = make(40, 24, 3, 2)
    want = run(o)
    bad = dict(o, ids=o["ids"].clone())
    bad["ids"][5, 1], bad["ids"][6, 0] = 24, -7
    with pytest.raises(moe.MoeError):
        run(bad, dloss=1.0, dw=True)
    bad = dict(o, keff=o["keff"].clone())
    bad["keff"][3], bad["keff"][4] = 4, 1 << 30
    with pytest.raises(moe.MoeError):
        run(bad, dloss=1.0, dw=True)
    for off in ([0, 30, 20], [-5, 10, 40], [0, 10, 41], [41, 50, 60]):
        with pytest.raises(moe.MoeError):
            run(dict(o, offsets=off), dloss=1.0, dw=True)
    assert torch.equal(run(o)[1], want[1])


def test_the_same_again_and_in_a_graph():
    o = make(5000, 96, 6, 7)
    first = run(o, dloss=1.0, dw=True)
    cfg, S = config(o), 7
    ws = moe.alloc_balance_workspace(cfg, 6000, 20)      # of more tokens
    loss, counts = torch.empty(1, device="cuda"), torch.empty(S, 96, dtype=torch.int32, device="cuda")
    tokens, d = torch.empty(S, dtype=torch.int32, device="cuda"), torch.empty(5000, 96, device="cuda")
    off = torch.tensor(o["offsets"], dtype=torch.int32, device="cuda")
    args = (cfg, o["logits"].cuda(), o["ids"].cuda(), o["keff"].cuda(), off)
    one, dw = torch.ones(1, device="cuda"), o["dw"].cuda()

    def step():
        moe.moe_balance_forward(*args, loss, counts, tokens, ws)
        moe.moe_balance_backward(*args, counts, tokens, d, ws, dloss=one, dw=dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for v in (loss, counts, tokens, d):
            v.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, (loss, counts, tokens, d)):
            assert torch.equal(a, b.cpu())
    moe.moe_check_errors(ws)


def test_the_error_of_wrong_offsets_names_the_loss():
    o = make(40, 24, 3, 2)
    with pytest.raises(moe.MoeError, match="loss is NaN"):
        run(dict(o, offsets=[0, 30, 20]))


def test_sequences_over_one_another_end_soon():
    """Every other one of 200000 sequences has all tokens: a wrong list, which costs no more than a walk over it."""
    T, S, E = 100000, 200000, 64
    cfg = moe.MoeConfig.make(64, E, 2, 64)
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randn(T, E, generator=g, device="cuda")
    ids, keff = l.topk(2, dim=1)[1].to(torch.int32), torch.full((T,), 2, dtype=torch.int32, device="cuda")
    loss, tokens = torch.zeros(1, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda")
    counts, ws = torch.empty(S, E, dtype=torch.int32, device="cuda"), moe.alloc_balance_workspace(cfg, T, S)
    at = torch.arange(S + 1, device="cuda")

    def time(off):
        best = float("inf")
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            moe.moe_balance_forward(cfg, l, ids, keff, off, loss, counts, tokens, ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    good = time((at // 2).to(torch.int32))
    moe.moe_check_errors(ws)
    assert int(tokens.sum()) == T and float(loss) > 0
    wrong = time((at % 2 * T).to(torch.int32))
    assert loss.isnan().all()
    with pytest.raises(moe.MoeError):
        moe.moe_check_errors(ws)
    # looking at all of its tokens for each sequence would be T / 2 times a row's work more
    assert wrong <= 50 * good, (wrong, good)
