"""The gated choice where scores stop telling logits apart: the fp64 score of
two different logits is then one number, and the lower index wins."""
import numpy as np
import pytest
import torch

from test_gpu_gate_select import bias, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import block_fp8_routed_amd as moe
    moe.load()
    yield
    torch.cuda.synchronize()


def group_rows(maxima, per, T, rest=-5.0):
    """Rows whose groups hold one expert of the given logit (at a place that
    moves from group to group) and the rest far below it, repeated to T rows."""
    maxima = np.asarray(maxima, np.float32)
    n, groups = maxima.shape
    l = np.full((n, groups, per), np.float32(rest))
    for g in range(groups):
        l[:, g] = np.minimum(l[:, g], maxima[:, g:g + 1])
        l[:, g, (3 * g + 1) % per] = maxima[:, g]
    l = np.tile(l.reshape(n, groups * per), (-(-T // n), 1))[:T]
    return torch.from_numpy(l)


INF = float("inf")
# equal best logits on both sides of the cut, and a group of another logit with
# the same score: a smaller logit of a lower index, or a larger one of a higher
EQUAL_SCORES = {
    "sigmoid": [[39.5, -1.0, 40.0, 40.0], [40.0, 40.0, -1.0, 41.0], [50.0, -1.0, INF, INF],
                [0.0, -3.0, 1e-18, 1e-18], [-2.0, 38.0, 60.0, 60.0], [1e-18, 1e-18, -3.0, 2e-18],
                [-900.0, -2000.0, -800.0, -800.0], [40.0, 40.0, 40.0, 40.0],
                [-1e-18, 0.0, 0.0, 0.0], [2.0, 3.0, 3.0, 1.0], [90.0, 40.0, 39.5, 90.0]],
    "softmax": [[0.0, -5.0, 1e-18, 1e-18], [1e-18, 1e-18, -3.0, 2e-18],
                [-900.0, 0.0, -800.0, -800.0], [-800.0, -800.0, 0.0, -790.0],
                [5.0, 5.0, 5.0, 1.0], [2.0, 3.0, 3.0, 1.0], [50.0, -1.0, INF, INF]],
}


@pytest.mark.parametrize("T", [1, 3, 11, 4200])
@pytest.mark.parametrize("per", [4, 8, 13])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_groups_of_equal_scores(score, per, T, dtype):
    rows = EQUAL_SCORES[score]
    for first in range(len(rows) if T == 1 else 1):
        l = group_rows(rows[first:] + rows[:first], per, T, rest=-1e4).to(dtype)
        for top in (1, 2, 3):
            check(l, min(3, top * per), None, score=score, groups=4, top_groups=top, group_rank=1,
                  renormalise=False)


@pytest.mark.parametrize("T", [1, 6, 4200])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("renormalise", [False, True])
def test_sigmoid_of_logits_far_below_zero(groups, renormalise, T):
    """1 / (1 + e^-l) leaves fp64's range below l = -709.8 and is 0 there: such
    experts, finite masks of -1e4 or -1e9 among them, get no share of the gates."""
    E = 32
    rng = np.random.default_rng(4)
    l = np.full((12, E), np.float32(-1e9))
    l[1] = -1e4
    l[2] = -720.0
    l[3] = -705.0
    l[4] = -5000.0
    l[4, 9] = -705.0
    l[5] = rng.choice(np.float32([-705, -720, -1e4, -1e9]), E)
    l[6] = rng.choice(np.float32([-709.0, -709.5, -708.25]), E)
    l[7, 3] = 1.5
    l[8] = -800.0 - np.arange(E)
    l[9] = -700.0 - 0.125 * np.arange(E)
    l[10, ::5] = -3.0e38
    l[11] = -3.0e38
    for first in range(12 if T == 1 else 1):
        rows = torch.from_numpy(np.tile(np.roll(l, -first, 0), (-(-T // 12), 1))[:T])
        rule = dict(score="sigmoid", groups=groups, top_groups=max(1, groups // 2),
                    group_rank=1, renormalise=renormalise, scale=2.5)
        check(rows, 6, None, **rule)
        check(rows, 6, bias(E, 2, 0.5), **rule)


@pytest.mark.parametrize("tokens", [4096, 4099])
def test_route_gated_with_tokens_that_share_a_wavefront(tokens):
    """Long batches on the 128-expert layer: four tokens a wavefront read the
    router's partial logits, and the finished ones are handed back."""
    import block_fp8_routed_amd as moe
    import oracle
    import workloads as W
    from parity import DevLayer
    from test_gpu_gate_select import SIGMOID8, check_gates
    layer = DevLayer(W.CONFIGS["c1"], tokens=tokens)
    s = layer.shape
    bal = torch.from_numpy(bias(s.experts)).cuda()
    idx, gates, logits = moe.moe_route_gated(layer.x, layer.router_w, s.top_k,
                                             moe.Gating(**SIGMOID8), s.inter, s.block,
                                             router_bias=layer.bias, balance_bias=bal,
                                             with_logits=True)
    ref_idx, ref_g = oracle.gated_choice(logits.double().cpu().numpy(), s.top_k,
                                         balance=bal.cpu().numpy(), **SIGMOID8)
    assert (idx.cpu().numpy() == ref_idx).all()
    check_gates(gates, ref_g, f"T={tokens}")
    _, _, plain = layer.route(with_logits=True)
    assert torch.equal(plain, logits)


@pytest.mark.parametrize("name,tokens", [("c1", 40), ("c3", 64)])
def test_forward_gated_in_fp8(name, tokens):
    """The FP8 expert passes behind the gated choice: each token's result is that
    of the plain bf16 passes on the same choice, but for the quantisation of x and
    h (2^-4 a value at most, of random sign: a few percent in norm)."""
    import block_fp8_routed_amd as moe
    import workloads as W
    from parity import DevLayer
    from test_gpu_gate_select import SIGMOID8
    layer = DevLayer(W.CONFIGS[name], tokens=tokens)
    s = layer.shape
    gating = moe.Gating(**dict(SIGMOID8, groups=4, top_groups=2))
    bal = torch.from_numpy(bias(s.experts)).cuda()

    def call(path):
        return moe.moe_forward_gated(layer.x, layer.router_w, layer.bank, s.top_k, s.block, gating,
                                     shared=layer.shared, router_bias=layer.bias,
                                     balance_bias=bal, path=path).double()

    a, b, again = call("mfma_fp8"), call("mfma"), call("mfma_fp8")
    assert torch.equal(a, again)
    err = float((a - b).norm() / b.norm())
    print(f"gated layer {name} in FP8: {err:.4f} of the bf16 passes in norm")
    assert err < 0.1
