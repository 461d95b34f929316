"""Pins of the oracle of the operators beside the layer (CPU): each function
against an independent evaluation, and constructed cases whose answer is known."""
import itertools

import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_against_torch(score):
    l = np.random.default_rng(1).normal(0, 3, (5, 17))
    want = torch.softmax(torch.from_numpy(l), 1) if score == "softmax" else \
        torch.sigmoid(torch.from_numpy(l))
    assert np.allclose(oracle.expert_scores(l, score), want.numpy(), rtol=1e-13, atol=0)


def test_scores_of_masked_and_infinite_logits():
    l = np.array([[0.0, -np.inf, np.nan, float(np.finfo(np.float32).min), 0.0],
                  [-np.inf] * 5, [np.inf, 1.0, np.inf, -np.inf, 0.0]])
    soft = oracle.expert_scores(l, "softmax")
    assert soft[0].tolist() == [0.5, 0, 0, 0, 0.5]
    assert soft[1].tolist() == [0] * 5
    assert soft[2].tolist() == [0.5, 0, 0.5, 0, 0]
    sig = oracle.expert_scores(l, "sigmoid")
    assert sig[0].tolist() == [0.5, 0, 0, 0, 0.5] and sig[2, 0] == 1.0


@pytest.mark.parametrize("groups,top_groups,rank", [(1, 1, 1), (2, 1, 1), (4, 2, 2), (3, 2, 1)])
def test_choice_against_every_subset(groups, top_groups, rank):
    """The chosen set has the largest sum of c among the k-subsets of the best
    groups, which are found by trying every combination of groups."""
    rng = np.random.default_rng(groups)
    E, k = 12, 3
    per = E // groups
    for _ in range(20):
        l, b = rng.normal(size=(1, E)), rng.normal(0, 0.3, E)
        idx, gates = oracle.gated_choice(l, k, "sigmoid", b, groups, top_groups, rank, False, 2.0)
        s = 1 / (1 + np.exp(-l[0]))
        c = s + b
        gs = [max(sum(q) for q in itertools.combinations(c[g * per:(g + 1) * per], rank))
              for g in range(groups)]
        kept = max(itertools.combinations(range(groups), top_groups),
                   key=lambda q: sum(gs[g] for g in q))
        pool = [e for e in range(E) if e // per in kept]
        best = max(itertools.combinations(pool, k), key=lambda q: sum(c[list(q)]))
        assert set(idx[0]) == set(best)
        assert all(c[idx[0, j]] >= c[idx[0, j + 1]] for j in range(k - 1))
        assert np.allclose(gates[0], 2.0 * s[idx[0]])


def test_choice_ties_masks_and_renormalisation():
    idx, gates = oracle.gated_choice(np.zeros((1, 8)), 3, "softmax", groups=4, top_groups=2)
    assert idx[0].tolist() == [0, 1, 2] and np.allclose(gates, 1 / 3)
    # a fully masked row: lowest indices, gates 0
    idx, gates = oracle.gated_choice(np.full((1, 8), -np.inf), 3, "sigmoid", groups=4,
                                     top_groups=2)
    assert idx[0].tolist() == [0, 1, 2] and not gates.any()
    # a masked expert with a large bias is not chosen before the others
    l = np.array([[1.0, -np.inf, 0.5, 0.0]])
    idx, _ = oracle.gated_choice(l, 3, "sigmoid", np.array([0, 9.0, 0, 0]))
    assert idx[0].tolist() == [0, 2, 3]
    # an empty group does not beat one whose biased scores are negative
    l = np.array([[-np.inf, -np.inf, 0.0, 0.0]])
    idx, _ = oracle.gated_choice(l, 1, "sigmoid", np.full(4, -5.0), 2, 1, 2)
    assert idx[0].tolist() == [2]


def test_linear_against_scalar_loops():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(3, 256))
    codes, exps = oracle.quantise_activations(x, 128)
    w = rng.integers(0, 127, (130, 256)).astype(np.uint8)
    s = rng.uniform(0.1, 2, (2, 2)).astype(np.float32)
    bias = rng.normal(size=130)
    y, mag = oracle.linear_e4m3(codes, exps, w, s, bias)
    dec = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    for t, n in [(0, 0), (1, 127), (2, 128), (0, 129)]:
        terms = [dec[codes[t, k]] * 2.0 ** exps[t, k // 128] * dec[w[n, k]]
                 * float(s[n // 128, k // 128]) for k in range(256)]
        assert np.isclose(y[t, n], sum(terms) + bias[n], rtol=1e-12)
        assert np.isclose(mag[t, n], sum(map(abs, terms)) + abs(bias[n]), rtol=1e-12)


def test_swiglu_against_torch():
    gu = np.random.default_rng(4).normal(0, 4, (3, 20))
    t = torch.from_numpy(gu)
    want = torch.nn.functional.silu(t[:, :10]) * t[:, 10:]
    assert np.allclose(oracle.swiglu(gu), want.numpy(), rtol=1e-13)
    assert oracle.swiglu(np.array([[-1e4, 3.0]]))[0, 0] == 0.0


def test_gated_layer_with_the_layers_own_gates_is_the_layer():
    import workloads as W
    shape = W.CONFIGS["c0"]
    d = W.gen_layer(shape)
    ref = oracle.moe_layer(d["x"], d["router_w"], None, lambda e: W.bank_expert(d["bank"], e),
                           shape.top_k, shape.inter, shape.block)
    l = oracle.router_logits(d["x"], d["router_w"])
    idx = oracle.select_topk(l, shape.top_k)
    out = oracle.gated_layer(d["x"], idx, oracle.gate_weights(l, idx),
                             lambda e: W.bank_expert(d["bank"], e), shape.inter, shape.block)
    assert np.allclose(out, ref["out"], rtol=1e-12, atol=1e-14)
    # softmax scores renormalised over the k largest are the layer's own gates
    i2, g2 = oracle.gated_choice(l, shape.top_k, "softmax")
    assert (i2 == idx).all() and np.allclose(g2, oracle.gate_weights(l, idx), rtol=1e-12)
