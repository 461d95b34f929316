"""Rows sorted by expert and back (moe_dispatch, moe_combine) and their gradients,
against a plain evaluation in 64 bits. Indexes and copied rows are exact; sums of n
fp32 terms are within n 2^-24 of the sum of their magnitudes (one rounding each), and
half a step of the output type (2^-8 of the value for bf16) comes on top."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def choices(T, k, E, seed, kind="any"):
    """[T][k] expert ids: "any" in range (with repeats), "distinct", "share" (half of
    them outside), "one" expert for all, "none" valid, "holes" (some tokens without)."""
    r = np.random.default_rng(seed)
    idx = r.integers(0, E, (T, k))
    if kind == "distinct":
        idx = np.argsort(r.random((T, E)), axis=1)[:, :k]
    elif kind == "share":
        idx = r.integers(-E // 2 - 1, E + E // 2 + 1, (T, k))
    elif kind == "one":
        idx[:] = E - 1
    elif kind == "none":
        idx = np.where(r.random((T, k)) < 0.5, -1, E + 5)
    elif kind == "holes":
        idx[r.random(T) < 0.4] = -1
    return idx.astype(np.int32)


def permutation(idx, E):
    flat = idx.reshape(-1).astype(np.int64)
    valid = (flat >= 0) & (flat < E)
    slots = np.nonzero(valid)[0]
    order = slots[np.argsort(flat[slots], kind="stable")]
    inv = np.full(flat.size, -1, np.int32)
    inv[order] = np.arange(order.size)
    pair = np.full(flat.size, -1, np.int32)
    pair[:order.size] = order
    offsets = np.searchsorted(flat[order], np.arange(E + 1)).astype(np.int32)
    return offsets, pair, inv.reshape(idx.shape)


def matrix(rows, cols, dtype, seed, pad=0, lead=0):
    """Random rows on the GPU, `pad` elements apart and `lead` behind an aligned start."""
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(rows * (cols + pad) + lead, generator=g).to(dtype).cuda()
    return wide[lead:].view(rows, cols + pad)[:, :cols] if rows else wide[lead:].view(0, cols)


SIZES = [  # tokens, k, experts, hidden
    (1, 1, 1, 1), (1, 10, 512, 4096), (3, 2, 7, 24), (17, 8, 128, 2048), (5, 16, 1024, 100),
    (130, 3, 64, 514), (511, 8, 128, 16), (512, 8, 128, 40), (513, 8, 128, 40),
    (4097, 1, 1024, 8), (1500, 16, 33, 72), (9000, 10, 512, 36), (40000, 8, 60, 7),
]


@pytest.mark.parametrize("T,k,E,H", SIZES)
@pytest.mark.parametrize("kind", ["any", "share"])
def test_dispatch(T, k, E, H, kind):
    import block_fp8_routed_amd as moe
    idx = choices(T, k, E, T + k, kind)
    x = matrix(T, H, torch.bfloat16 if T % 2 else torch.float32, 3)
    buf = torch.full((T * k, H), 7.0, dtype=x.dtype, device="cuda")
    rows, offsets, pair, inv = moe.moe_dispatch(x, torch.from_numpy(idx).cuda(), E, out=buf)
    o, p, i = permutation(idx, E)
    assert np.array_equal(offsets.cpu().numpy(), o)
    assert np.array_equal(inv.cpu().numpy(), i)
    assert np.array_equal(pair.cpu().numpy(), p)
    n = int(o[-1])
    assert torch.equal(rows[:n], x[torch.from_numpy(p[:n].astype(np.int64) // k).cuda()])
    assert bool((rows[n:] == 7).all())


@pytest.mark.parametrize("T", [12, 3000])
@pytest.mark.parametrize("kind", ["distinct", "one", "none", "holes"])
def test_dispatch_of_uneven_choices(T, kind):
    import block_fp8_routed_amd as moe
    idx = choices(T, 4, 9, 5, kind)
    x = matrix(T, 32, torch.float32, 4)
    rows, offsets, pair, inv = moe.moe_dispatch(x, torch.from_numpy(idx).cuda(), 9)
    o, p, i = permutation(idx, 9)
    assert np.array_equal(offsets.cpu().numpy(), o) and np.array_equal(inv.cpu().numpy(), i)
    assert np.array_equal(pair.cpu().numpy(), p)
    n = int(o[-1])
    assert torch.equal(rows[:n], x[torch.from_numpy(p[:n].astype(np.int64) // 4).cuda()])


def test_dispatch_of_no_tokens_writes_offsets():
    import block_fp8_routed_amd as moe
    for E in (1, 300, 1024):
        x = torch.empty(0, 16, device="cuda")
        rows, offsets, pair, inv = moe.moe_dispatch(x, torch.empty(0, 4, dtype=torch.int32, device="cuda"), E)
        assert rows.shape == (0, 16) and pair.shape == (0,) and inv.shape == (0, 4)
        assert offsets.tolist() == [0] * (E + 1)
        assert moe.moe_dispatch_backward(rows, inv).shape == (0, 16)
        gates = torch.empty(0, 4, device="cuda")
        assert moe.moe_combine(rows, gates, inv).shape == (0, 16)
        assert moe.moe_combine_backward(x, rows, gates, inv)[0].shape == (0, 16)


@pytest.mark.parametrize("pad,lead", [(8, 0), (3, 0), (0, 1), (4, 4), (2, 2), (16, 8)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_addresses(pad, lead, dtype):
    """Rows apart and starts off every alignment; what lies between rows stays."""
    import block_fp8_routed_amd as moe
    T, k, E, H = 37, 3, 11, 72
    kind = TYPES[dtype]
    idx = choices(T, k, E, 1, "share")
    o, p, i = permutation(idx, E)
    n, d_idx = int(o[-1]), torch.from_numpy(idx).cuda()
    x = matrix(T, H, kind, 2, pad, lead)
    whole = torch.full((T * k * (H + pad) + lead,), 5.0, dtype=kind, device="cuda")
    buf = whole[lead:].view(T * k, H + pad)[:, :H]
    rows, _, _, inv = moe.moe_dispatch(x, d_idx, E, out=buf)
    assert rows is buf
    token = torch.from_numpy(p[:n].astype(np.int64) // k).cuda()
    assert torch.equal(rows[:n], x[token])
    rest = whole.clone()
    rest[lead:].view(T * k, H + pad)[:n, :H] = 5.0
    assert bool((rest == 5.0).all())
    y = matrix(T * k, H, kind, 6, pad, lead)
    gates = torch.rand(T, k, device="cuda")
    shared = matrix(T, H, kind, 7, pad, lead)
    out = torch.full((T * (H + pad) + lead,), 9.0, dtype=torch.float32, device="cuda")
    got = moe.moe_combine(y, gates, inv, shared=shared, out=out[lead:].view(T, H + pad)[:, :H])
    ref, mag = combined(y, gates, i, shared)
    assert within(got, ref, (k + 1) * 2.0 ** -24 * mag)
    rest = out.clone()
    rest[lead:].view(T, H + pad)[:, :H] = 9.0
    assert bool((rest == 9.0).all())
    d_out = matrix(T, H, torch.float32, 8, pad, lead)
    d_whole = torch.full_like(whole, 3.0)
    d_y, d_gates = moe.moe_combine_backward(d_out, y, gates, inv,
                                            out=d_whole[lead:].view(T * k, H + pad)[:, :H])
    check_gradients(d_out, y, gates, i, d_y, d_gates, 3.0)
    rest = d_whole.clone()
    rest[lead:].view(T * k, H + pad)[:n, :H] = 3.0
    assert bool((rest == 3.0).all())


def within(got, ref, bound):
    """got against ref in 64 bits: bound (of fp32 sums) and the output's own rounding."""
    got64 = got.double().cpu().numpy()
    err = np.abs(got64 - ref)
    lim = bound + HALF[got.dtype] * (np.abs(ref) + bound) + 1e-45
    assert np.isfinite(got64).all()
    assert (err <= lim).all(), f"error {err.max():.3e}, {np.max(err / lim):.2f} of the bound"
    return True


def combined(y, gates, inv, shared=None):
    y, g = y.double().cpu().numpy(), gates.double().cpu().numpy()
    v = np.where((inv >= 0)[:, :, None], y[np.maximum(inv, 0)], 0.0) * g[:, :, None]
    s = 0.0 if shared is None else shared.double().cpu().numpy()
    return v.sum(axis=1) + s, np.abs(v).sum(axis=1) + np.abs(s)


def check_gradients(d_out, y, gates, inv, d_y, d_gates, untouched):
    d, v, g = (t.double().cpu().numpy() for t in (d_out, y, gates))
    k, H = inv.shape[1], v.shape[1]
    ok = inv >= 0
    rows = inv[ok]
    ref = (g[:, :, None] * d[:, None, :])[ok]
    assert within(d_y[torch.from_numpy(rows.astype(np.int64)).cuda()], ref, 2.0 ** -24 * np.abs(ref))
    left = np.setdiff1d(np.arange(v.shape[0]), rows)
    assert bool((d_y[torch.from_numpy(left).cuda()] == untouched).all())
    t = np.where(ok[:, :, None], v[np.maximum(inv, 0)], 0.0) * d[:, None, :]
    assert within(d_gates, t.sum(axis=2), H * 2.0 ** -24 * np.abs(t).sum(axis=2))
    assert bool((d_gates.cpu()[torch.from_numpy(~ok)] == 0).all())


@pytest.mark.parametrize("T,k,E,H", SIZES)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_combine_and_gradients(T, k, E, H, dtype, out):
    import block_fp8_routed_amd as moe
    if T * k * H > 6_000_000:
        H = max(1, 6_000_000 // (T * k))
    _, _, i = permutation(choices(T, k, E, T, "share" if T % 3 else "any"), E)
    inv = torch.from_numpy(i).cuda()
    y = matrix(T * k, H, TYPES[dtype], T)
    gates = torch.rand(T, k, generator=torch.Generator().manual_seed(T)).cuda()
    shared = matrix(T, H, TYPES[dtype], 9) if k % 2 else None
    ref, mag = combined(y, gates, i, shared)
    got = moe.moe_combine(y, gates, inv, shared=shared, out_dtype=TYPES[out])
    assert within(got, ref, (k + 1) * 2.0 ** -24 * mag)
    ref, mag = combined(y, torch.ones_like(gates), i)
    assert within(moe.moe_dispatch_backward(y, inv, out_dtype=TYPES[out]), ref,
                  k * 2.0 ** -24 * mag)
    d_out = matrix(T, H, TYPES[out], 10)
    buf = torch.full_like(y, 2.0)
    d_y, d_gates = moe.moe_combine_backward(d_out, y, gates, inv, out=buf)
    check_gradients(d_out, y, gates, i, d_y, d_gates, 2.0)


def test_rows_that_no_slot_may_name():
    """inv outside [0, rows) counts as no row, whatever it holds; NaN in rows without
    a slot, and infinities beside a gate of an absent one, stay out."""
    import block_fp8_routed_amd as moe
    inv = torch.tensor([[0, -1, 5], [-7, 2 ** 31 - 1, 6], [1, 3, -2 ** 31]], dtype=torch.int32).cuda()
    y = matrix(6, 40, torch.float32, 1)
    y[2] = float("nan")
    y[4] = float("inf")
    gates = torch.tensor([[1., float("nan"), 2.], [float("inf"), 1., 1.], [.5, .25, float("nan")]]).cuda()
    out = moe.moe_combine(y, gates, inv)
    want = torch.stack((y[0] + 2 * y[5], torch.zeros(40).cuda(), .5 * y[1] + .25 * y[3]))
    assert torch.allclose(out, want, rtol=2.0 ** -22, atol=1e-6)
    assert torch.isfinite(moe.moe_dispatch_backward(y, inv)).all()
    d_y, d_gates = moe.moe_combine_backward(torch.ones(3, 40).cuda(), y, gates, inv,
                                            out=torch.zeros_like(y))
    assert torch.equal(d_y[2], torch.zeros(40).cuda()) and torch.equal(d_y[4], torch.zeros(40).cuda())
    assert d_gates[1].tolist() == [0, 0, 0] and d_gates[0, 1] == 0 and d_gates[2, 2] == 0


def test_nan_and_infinities_follow_their_rows():
    import block_fp8_routed_amd as moe
    T, k, E, H = 20, 2, 4, 64
    idx = choices(T, k, E, 2, "distinct")
    for kind in TYPES.values():
        x = matrix(T, H, kind, 1)
        x[3, 5], x[4, 6] = float("nan"), float("inf")
        rows, _, _, inv = moe.moe_dispatch(x, torch.from_numpy(idx).cuda(), E)
        out = moe.moe_combine(rows, torch.ones(T, k, device="cuda"), inv)
        bad = ~torch.isfinite(out)
        assert bad.sum() == 2 and torch.isnan(out[3, 5]) and out[4, 6] == float("inf")


def test_gradients_against_differences():
    """<d_out, combine(y, g)> is linear in y and in g: its differences along a random
    direction are the gradients' products with it."""
    import block_fp8_routed_amd as moe
    T, k, E, H = 33, 4, 8, 48
    idx = torch.from_numpy(choices(T, k, E, 3, "share")).cuda()
    x, dx = matrix(T, H, torch.float32, 1), matrix(T, H, torch.float32, 2)
    gates, dg = torch.rand(T, k, device="cuda"), torch.randn(T, k, device="cuda")
    d_out = matrix(T, H, torch.float32, 5)

    def loss(x, gates):
        rows, _, _, inv = moe.moe_dispatch(x, idx, E, out=torch.zeros(T * k, H, device="cuda"))
        out = moe.moe_combine(rows * rows, gates, inv)
        return float((out.double() * d_out.double()).sum()), rows, inv

    _, rows, inv = loss(x, gates)
    d_y, d_gates = moe.moe_combine_backward(d_out, rows * rows, gates, inv,
                                            out=torch.zeros_like(rows))
    d_x = moe.moe_dispatch_backward(2 * rows * d_y, inv)
    along = float((d_gates.double() * dg.double()).sum() + (d_x.double() * dx.double()).sum())
    # a central difference of step h of a cubic: h^2 of the third derivative is exact to
    # h^2 |d3|; h = 2^-8 leaves 1e-5 of it, fp32 sums 2^-22 / h = 6e-5 of the terms
    h = 2.0 ** -8
    diff = (loss(x + h * dx, gates + h * dg)[0] - loss(x - h * dx, gates - h * dg)[0]) / (2 * h)
    size = float((d_gates.abs() * dg.abs()).sum() + (d_x.abs() * dx.abs()).sum())
    assert abs(diff - along) <= 2e-4 * size


def test_results_repeat_and_do_not_depend_on_the_batch():
    import block_fp8_routed_amd as moe
    T, k, E, H = 700, 8, 64, 264
    idx = torch.from_numpy(choices(T, k, E, 3)).cuda()
    x = matrix(T, H, torch.bfloat16, 1)
    gates = torch.rand(T, k, device="cuda")

    def run(sel):
        rows, _, _, inv = moe.moe_dispatch(x[sel], idx[sel], E)
        out = moe.moe_combine(rows, gates[sel].contiguous(), inv)
        _, dg = moe.moe_combine_backward(out, rows, gates[sel].contiguous(), inv)
        return out, dg

    whole, again, part = run(slice(0, T)), run(slice(0, T)), run(slice(100, 150))
    for a, b, c in zip(whole, again, part):
        assert torch.equal(a, b) and torch.equal(a[100:150], c)


def test_streams_and_graphs():
    """On a side stream, and captured: replays with other inputs in place give the
    eager results, with eager work between them."""
    import block_fp8_routed_amd as moe
    for T in (40, 3000):
        k, E, H = 4, 16, 80
        x = matrix(T, H, torch.bfloat16, 1)
        idx = torch.from_numpy(choices(T, k, E, 1, "share")).cuda()
        gates = torch.rand(T, k, device="cuda")

        def step():
            rows, offsets, pair, inv = moe.moe_dispatch(x, idx, E)
            out = moe.moe_combine(rows, gates, inv)
            d_y, d_g = moe.moe_combine_backward(out, rows, gates, inv)
            return offsets, pair, inv, out, d_g, moe.moe_dispatch_backward(d_y, inv)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for seed in range(4):
            x.copy_(matrix(T, H, torch.bfloat16, 20 + seed))
            idx.copy_(torch.from_numpy(choices(T, k, E, 30 + seed, "share")))
            gates.copy_(torch.rand(T, k))
            want = step()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(held, want):
                assert torch.equal(a, b), seed
