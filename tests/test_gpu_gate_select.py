"""The gated choice of experts on the GPU (moe_select_experts, moe_route_gated,
moe_forward_gated) against the fp64 oracle.

Choices have to be equal: the kernel orders the same fp64 formula, and the
inputs hold no two experts within 1e-12 of each other that are not equal. Gates
are fp64 values rounded once to fp32: off by at most 2^-24 of the value, with
2^-40 left for the fp64 steps (expected below 1e-13)."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from parity import DevLayer, check_output, log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import block_fp8_routed_amd as moe
    moe.load()
    yield
    torch.cuda.synchronize()


def check_gates(got, want, what):
    got = got.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), what
    bound = np.abs(want) * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -149
    bad = np.abs(got - want) > bound
    assert not bad.any(), f"{what}: {bad.sum()} gates off, first {got[bad][0]} vs {want[bad][0]}"


def check(logits, k, balance=None, ld_pad=0, **rule):
    import block_fp8_routed_amd as moe
    T, E = logits.shape
    dev = logits.cuda()
    if ld_pad:
        wide = torch.full((T, E + ld_pad), 1e30, dtype=logits.dtype, device="cuda")
        wide[:, :E] = dev
        dev = wide[:, :E]
    b = None if balance is None else torch.from_numpy(balance).float().cuda()
    idx, gates = moe.moe_select_experts(dev, k, moe.Gating(**rule), balance_bias=b)
    torch.cuda.synchronize()
    ref_idx, ref_g = oracle.gated_choice(logits.double().numpy(), k,
                                         balance=None if b is None else b.cpu().numpy(), **rule)
    what = f"T={T} E={E} k={k} {rule}"
    assert idx.dtype == torch.int32 and gates.dtype == torch.float32
    got = idx.cpu().numpy()
    bad = np.nonzero((got != ref_idx).any(axis=1))[0]
    assert not len(bad), f"{what}: token {bad[0]}: {got[bad[0]]} vs {ref_idx[bad[0]]}"
    check_gates(gates, ref_g, what)
    log(f"gated choice {what}: ok")


def draw(T, E, seed=0, std=1.2, dtype=torch.float32):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.normal(0, std, (T, E)) + g.normal(0, 0.5, E)).to(dtype)


def bias(E, seed=0, std=0.1):
    return np.random.default_rng(100 + seed).normal(0, std, E).astype(np.float32)


SIGMOID8 = dict(score="sigmoid", groups=8, top_groups=4, group_rank=2, renormalise=True, scale=2.5)
SOFTMAX1 = dict(score="softmax", groups=1, top_groups=1, group_rank=1, renormalise=False, scale=1.0)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 64, 257])
@pytest.mark.parametrize("E,k", [(512, 10), (256, 8), (128, 8), (64, 16)])
def test_grouped_sigmoid(T, E, k):
    check(draw(T, E, T), k, bias(E), **SIGMOID8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (5, 5), (63, 7), (65, 16), (128, 8), (200, 3),
                                 (511, 10), (513, 10), (1000, 16), (1024, 16)])
def test_ungrouped_softmax(E, k, dtype):
    check(draw(9, E, E, dtype=dtype), k, **SOFTMAX1)


@pytest.mark.parametrize("groups,per,top,rank,k", [
    (2, 64, 1, 1, 8), (3, 7, 2, 2, 4), (4, 5, 4, 2, 16), (5, 13, 1, 1, 13), (16, 2, 7, 2, 14),
    (64, 16, 9, 2, 16), (64, 1, 5, 1, 5), (33, 31, 2, 1, 16), (2, 512, 1, 2, 16), (7, 100, 3, 2, 6),
    (60, 3, 60, 2, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_shapes(groups, per, top, rank, k, score):
    E = groups * per
    for renorm in (False, True):
        check(draw(11, E, groups), k, bias(E, groups, 0.02), score=score, groups=groups,
              top_groups=top, group_rank=rank, renormalise=renorm, scale=0.75)


def test_rows_apart():
    for dtype in (torch.float32, torch.bfloat16):
        check(draw(33, 160, 2, dtype=dtype), 6, ld_pad=3, score="softmax", groups=8, top_groups=3,
              group_rank=1, renormalise=False, scale=16.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lower_index(score, dtype):
    check(torch.zeros(3, 96, dtype=dtype), 7, score=score, groups=6, top_groups=2, group_rank=2)
    # few distinct values: most experts and groups tie
    l = torch.from_numpy(np.random.default_rng(5).integers(0, 3, (40, 128)).astype(np.float32))
    check(l.to(dtype), 9, score=score, groups=16, top_groups=5, group_rank=2)
    check(l.to(dtype), 16, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 8])
def test_masks(score, groups):
    rule = dict(score=score, groups=groups, top_groups=max(1, groups // 2), group_rank=2,
                renormalise=True, scale=2.0)
    E, k = 64, 10
    l = draw(12, E, 9)
    l[0] = float("-inf")                            # nothing left
    l[1] = float("nan")
    l[2] = torch.finfo(torch.float32).min
    l[3, 3:] = float("-inf")                        # fewer than k
    l[4, :60] = float("nan")
    l[5, ::2] = float("-inf")
    l[6, :8] = float("-inf")                        # an empty first group
    l[7, 1:8] = float("-inf")                       # a group of one
    l[8, 5] = float("inf")
    l[9, [7, 40]] = float("inf")
    l[10, 8:] = torch.finfo(torch.bfloat16).min
    l[11] = -200.0 + l[11]                          # scores down to e^-200
    check(l, k, bias(E, 3, 0.5), **rule)
    check(l, k, None, **rule)
    check(l.to(torch.bfloat16), k, np.full(E, -3.0, np.float32), **rule)


def test_far_apart_scores_and_biases():
    """Scores far below the bias's fp32 step still order the experts, and
    biases far above the scores decide alone."""
    l = draw(6, 64, 4) - 30.0
    check(l, 8, np.full(64, 0.5, np.float32), score="sigmoid")
    check(l, 8, np.arange(64, dtype=np.float32) * 1e6, score="sigmoid", renormalise=False)
    check(draw(6, 64, 4, std=60.0), 8, score="softmax", renormalise=False)


def test_long_batch():
    check(draw(3001, 512, 1), 10, bias(512), **SIGMOID8)
    check(draw(5000, 160, 2, dtype=torch.bfloat16), 6, score="softmax", groups=8, top_groups=3,
          group_rank=1, renormalise=False, scale=16.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k,groups,top,rank", [
    (1, 1, 1, 1, 1), (7, 7, 1, 1, 1), (40, 3, 1, 1, 1), (64, 16, 16, 5, 2), (100, 6, 4, 2, 2),
    (128, 8, 1, 1, 1), (160, 6, 8, 3, 1), (200, 16, 1, 1, 1), (256, 8, 8, 4, 2), (255, 9, 15, 4, 2),
    (256, 16, 32, 5, 2), (257, 8, 1, 1, 1)])
def test_many_tokens(E, k, groups, top, rank, score, dtype):
    """Batches long enough that tokens share a wavefront, the last one part
    full, with and without a bias."""
    l = draw(4099, E, E + k, dtype=dtype)
    rule = dict(score=score, groups=groups, top_groups=top, group_rank=rank, scale=1.5)
    check(l, k, bias(E, k, 0.05), ld_pad=5, **rule)
    check(l, k, None, renormalise=False, **rule)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_and_ties_among_many_tokens(score):
    """Tokens of one wavefront that need different ways: masked to a few
    experts or none, equal scores, and ordinary ones."""
    E, k = 128, 9
    rng = np.random.default_rng(8)
    l = draw(4500, E, 3)
    l[::7] = torch.from_numpy(rng.integers(0, 3, (len(l[::7]), E)).astype(np.float32))
    l[::11, 4:] = float("-inf")
    l[::13] = float("nan")
    l[1::17, :64] = torch.finfo(torch.float32).min
    l[2::19, 5] = float("inf")
    for groups in (1, 16):
        rule = dict(score=score, groups=groups, top_groups=max(1, groups // 3), group_rank=2)
        check(l, k, bias(E, 3, 0.5), **rule)
        check(l, k, None, **rule)


@pytest.mark.parametrize("E,k,groups,top", [(64, 4, 1, 1), (512, 10, 8, 4), (60, 16, 12, 4),
                                            (160, 6, 8, 3), (9, 9, 1, 1), (128, 8, 64, 5)])
@pytest.mark.parametrize("T", [7, 4200])
def test_padded_batch(E, k, groups, top, T):
    """Rows of padding, masked in every way, between ordinary ones; rows with a
    few experts left."""
    l = draw(T, E, 5)
    l[1::2] = float("-inf")
    l[3::8] = float("nan")
    l[5::16] = torch.finfo(torch.float32).min
    l[2::6, min(2, E - 1):] = float("-inf")
    for score in ("softmax", "sigmoid"):
        for rank in (1, 2):
            rule = dict(score=score, groups=groups, top_groups=top, group_rank=rank)
            check(l, k, bias(E, 3, 0.5), **rule)
            check(l, k, None, renormalise=False, **rule)


def test_no_tokens():
    import block_fp8_routed_amd as moe
    idx, gates = moe.moe_select_experts(torch.empty(0, 64, device="cuda"), 4, moe.Gating())
    assert idx.shape == gates.shape == (0, 4)


# ------------------------------------------------------------- with the layer --
@pytest.mark.parametrize("name,tokens", [("c1", 1), ("c1", 16), ("c1", 37), ("c3", 8), ("c2", 300)])
def test_route_gated(name, tokens):
    """The choice made from the router's own logits, which it also returns."""
    import block_fp8_routed_amd as moe
    layer = DevLayer(W.CONFIGS[name], tokens=tokens)
    s = layer.shape
    bal = torch.from_numpy(bias(s.experts)).cuda()
    rule = dict(SIGMOID8, top_groups=5)
    idx, gates, logits = moe.moe_route_gated(layer.x, layer.router_w, s.top_k, moe.Gating(**rule),
                                             s.inter, s.block, router_bias=layer.bias,
                                             balance_bias=bal, with_logits=True)
    ref_idx, ref_g = oracle.gated_choice(logits.double().cpu().numpy(), s.top_k,
                                         balance=bal.cpu().numpy(), **rule)
    assert (idx.cpu().numpy() == ref_idx).all()
    check_gates(gates, ref_g, name)
    _, _, plain = layer.route(with_logits=True)
    assert torch.equal(plain, logits)
    i2, g2 = moe.moe_select_experts(logits, s.top_k, moe.Gating(**rule), balance_bias=bal)
    assert torch.equal(i2, idx) and torch.equal(g2, gates)


@pytest.mark.parametrize("name,tokens,path", [
    ("c0", 3, "auto"), ("c1", 1, "auto"), ("c1", 4, "auto"), ("c1", 16, "auto"), ("c1", 37, "auto"),
    ("c1", 100, "auto"), ("c1", 5, "mfma"), ("c3", 8, "auto"), ("c3", 60, "auto")])
def test_forward_gated(name, tokens, path):
    import block_fp8_routed_amd as moe
    layer = DevLayer(W.CONFIGS[name], tokens=tokens)
    s = layer.shape
    bal = torch.from_numpy(bias(s.experts)).cuda()
    rule = dict(SIGMOID8, groups=4, top_groups=2) if name != "c0" else dict(SIGMOID8, groups=2,
                                                                            top_groups=1)
    gating = moe.Gating(**rule)
    idx, gates = moe.moe_route_gated(layer.x, layer.router_w, s.top_k, gating, s.inter, s.block,
                                     router_bias=layer.bias, balance_bias=bal)
    out = moe.moe_forward_gated(layer.x, layer.router_w, layer.bank, s.top_k, s.block, gating,
                                shared=layer.shared, router_bias=layer.bias, balance_bias=bal,
                                path=path)
    sh = W.bank_expert(layer.shared_host, 0) if s.shared else None
    ref = oracle.gated_layer(layer.x_host, idx.cpu().numpy(), gates.cpu().numpy().astype(np.float64),
                             layer.expert, s.inter, s.block, shared=sh)
    check_output(out, ref, what=f"forward_gated {name} T={tokens} {path}")


def test_forward_gated_leaves_the_layer_alone():
    """moe_forward before and after gated calls on one workspace: same bits."""
    import block_fp8_routed_amd as moe
    layer = DevLayer(W.CONFIGS["c1"], tokens=4)
    s = layer.shape
    cfg = moe.make_config(4, s.hidden, s.experts, s.inter, s.top_k, s.block, False, layer.x.dtype)
    ws = moe.make_workspace(cfg, layer.x.device)
    a = layer.forward(workspace=ws).clone()
    gating = moe.Gating(**SIGMOID8)
    g1 = moe.moe_forward_gated(layer.x, layer.router_w, layer.bank, s.top_k, s.block, gating,
                               workspace=ws).clone()
    b = layer.forward(workspace=ws).clone()
    g2 = moe.moe_forward_gated(layer.x, layer.router_w, layer.bank, s.top_k, s.block, gating,
                               workspace=ws)
    assert torch.equal(a, b) and torch.equal(g1, g2) and not torch.equal(a, g1)


@pytest.mark.parametrize("name,tokens", [("c1", 4), ("c1", 100)])
def test_forward_gated_in_a_graph(name, tokens):
    import block_fp8_routed_amd as moe
    layer = DevLayer(W.CONFIGS[name], tokens=tokens)
    s = layer.shape
    gating = moe.Gating(**SIGMOID8)
    bal = torch.from_numpy(bias(s.experts)).cuda()
    cfg = moe.make_config(tokens, s.hidden, s.experts, s.inter, s.top_k, s.block, False,
                          layer.x.dtype)
    ws, ws2 = moe.make_workspace(cfg, "cuda"), moe.make_workspace(cfg, "cuda")
    out = torch.empty(tokens, s.hidden, device="cuda")

    def call(o, w):
        return moe.moe_forward_gated(layer.x, layer.router_w, layer.bank, s.top_k, s.block, gating,
                                     balance_bias=bal, out=o, workspace=w)

    call(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    x0 = layer.x.clone()
    for i in range(4):
        layer.x.copy_(x0 * (1.0 + 0.25 * i))
        out.zero_()
        graph.replay()
        want = call(torch.empty_like(out), ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"


def test_another_stream():
    import block_fp8_routed_amd as moe
    l = draw(2000, 256, 3)
    want = moe.moe_select_experts(l.cuda(), 8, moe.Gating(**SIGMOID8))
    side = torch.cuda.Stream()
    dev = l.cuda()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_select_experts(dev, 8, moe.Gating(**SIGMOID8), stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 300, 4500])
def test_choice_in_a_graph_and_on_two_streams(T):
    import block_fp8_routed_amd as moe
    gating = moe.Gating(score="sigmoid", groups=8, top_groups=4, group_rank=2, scale=2.5)
    b = torch.from_numpy(bias(128)).cuda()
    l = draw(T, 128, T).cuda()
    moe.moe_select_experts(l, 8, gating, balance_bias=b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx, gates = moe.moe_select_experts(l, 8, gating, balance_bias=b)
    l0 = l.clone()
    for i in range(4):
        l.copy_(l0.roll(i, 1))
        graph.replay()
        want = moe.moe_select_experts(l, 8, gating, balance_bias=b)
        torch.cuda.synchronize()
        assert torch.equal(idx, want[0]) and torch.equal(gates, want[1]), f"replay {i}"
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [moe.moe_select_experts(l, 8, gating, balance_bias=b, stream=s)
           for _ in range(6) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
