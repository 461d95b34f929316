"""Dispatch, combine and the 4-bit products past 32-bit byte offsets, on a stream of
the caller's, with a workspace of the caller's, and two at once. Large results are
checked where they lie furthest, against plain torch operations or the formula in 64
bits (bounds as in test_gpu_dispatch.py and test_gpu_linear_w4.py)."""
import numpy as np
import pytest
import torch

from test_gpu_dispatch import choices, matrix, permutation, within
from test_gpu_linear_w4 import activations, check, reference, takes_tiles, weights

pytestmark = pytest.mark.gpu


def test_rows_past_4_gib():
    import block_fp8_routed_amd as moe
    T, k, E, H = 40000, 8, 96, 8192  # 5.2 GB of rows
    idx = choices(T, k, E, 1, "distinct")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    rows, offsets, pair, inv = moe.moe_dispatch(x, torch.from_numpy(idx).cuda(), E)
    o, p, i = permutation(idx, E)
    assert np.array_equal(offsets.cpu().numpy(), o) and np.array_equal(inv.cpu().numpy(), i)
    token = torch.from_numpy(p.astype(np.int64) // k).cuda()
    for at in range(0, T * k, 32000):
        assert torch.equal(rows[at:at + 32000], x[token[at:at + 32000]])
    gates = torch.rand(T, k, generator=g, device="cuda")
    out = moe.moe_combine(rows, gates, inv)
    some = np.r_[0:40, T - 40:T]
    y = rows[torch.from_numpy(i[some].reshape(-1).astype(np.int64)).cuda()].double().cpu().numpy()
    v = y.reshape(len(some), k, H) * gates.double().cpu().numpy()[some][:, :, None]
    at = torch.from_numpy(some).cuda()
    assert within(out[at], v.sum(axis=1), k * 2.0 ** -24 * np.abs(v).sum(axis=1))
    d_y, d_gates = moe.moe_combine_backward(out, rows, gates, inv)
    d = out.double().cpu().numpy()[some]
    ref = gates.double().cpu().numpy()[some][:, :, None] * d[:, None, :]
    got = d_y[torch.from_numpy(i[some].reshape(-1).astype(np.int64)).cuda()]
    assert within(got, ref.reshape(-1, H), 2.0 ** -24 * np.abs(ref.reshape(-1, H)))
    t = y.reshape(len(some), k, H) * d[:, None, :]
    assert within(d_gates[at], t.sum(axis=2), H * 2.0 ** -24 * np.abs(t).sum(axis=2))
    dx = moe.moe_dispatch_backward(d_y, inv)
    u = got.double().cpu().numpy().reshape(len(some), k, H)
    assert within(dx[at], u.sum(axis=1), k * 2.0 ** -24 * np.abs(u).sum(axis=1))


@pytest.mark.parametrize("rows", [1, 120])
def test_experts_past_4_gib(rows):
    """A bank of 5.4 GB; the first and the last experts have the rows, few (stream) or
    many (tiles)."""
    import block_fp8_routed_amd as moe
    E, N, K, G = 640, 4096, 4096, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(E, N, K // G, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    counts = np.zeros(E, np.int64)
    counts[[0, 320, 638, 639]] = rows
    offsets = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    M = int(offsets[-1])
    x = activations(M, K, 3)
    for out in (torch.float32, torch.bfloat16):
        got = moe.moe_grouped_linear_w4(x, torch.from_numpy(offsets).cuda(), w, s, out_dtype=out)
        for e in (0, 320, 638, 639):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            some = slice(0, 200)  # of the features
            ref, err = reference(x[lo:hi], w[e][some], s[e][some], None, None, False, out == torch.bfloat16)
            check(got[lo:hi, some], ref, err, f"expert {e}")


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_products_of_rows_past_4_gib(out):
    import block_fp8_routed_amd as moe
    M, N, K, G = 600_000, 128, 4096, 128  # x and its fp16 rows: 4.9 GB each
    assert takes_tiles(M, N, K, out)
    w, s, z, _ = weights((), N, K, G, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    got = moe.moe_linear_w4(x, w, s, z, out_dtype=out)
    at = torch.tensor([0, 1, 262143, 262144, 524287, 524288, 524289, 599_998, 599_999]).cuda()
    check(got[at], *reference(x[at], w, s, z, None, False, out == torch.bfloat16))
    # a stride that passes 32 bits within 16 rows
    wide = torch.randn(16, 1 << 28, generator=g, device="cuda", dtype=torch.bfloat16)
    few = wide[:, 5 * 8:5 * 8 + K]
    check(moe.moe_linear_w4(few, w, s, z, out_dtype=out),
          *reference(few, w, s, z, None, False, out == torch.bfloat16))


def test_caller_streams_and_workspaces():
    """Two streams at once, each with its own workspace, behind work that is still under
    way on them; too small or misaligned workspaces are refused."""
    import block_fp8_routed_amd as moe
    T, k, E, H, N = 3000, 4, 16, 512, 1024
    idx = torch.from_numpy(choices(T, k, E, 6, "share")).cuda()
    x0 = matrix(T, H, torch.bfloat16, 7)
    w, s, z, _ = weights((E,), N, H, 64, 8)
    rows, offsets, _, inv = moe.moe_dispatch(x0, idx, E, out=torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda"))
    want = moe.moe_grouped_linear_w4(rows, offsets, w, s, z, out=torch.zeros(T * k, N, dtype=torch.bfloat16, device="cuda"))
    need = moe.linear_w4_workspace_bytes(T * k, E, N, H, moe.MOE_BF16)
    need_d = moe.dispatch_workspace_bytes(T, k, E)
    assert need > 0 and need_d > 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for st in streams:
        x = torch.zeros_like(x0)
        buf = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros(T * k, N, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        ws_d = torch.empty(need_d, dtype=torch.uint8, device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(20):
                x.zero_()
            x.copy_(x0)
        r, o, _, i = moe.moe_dispatch(x, idx, E, out=buf, workspace=ws_d, stream=st)
        y = moe.moe_grouped_linear_w4(r, o, w, s, z, out=out, workspace=ws, stream=st)
        gates = torch.ones(T, k, device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        got.append((y, moe.moe_combine(y, gates, i, stream=st), x, ws, ws_d, gates))
    torch.cuda.synchronize()
    ref = moe.moe_combine(want, torch.ones(T, k, device="cuda"), inv)
    for y, c, *_ in got:
        assert torch.equal(y, want) and torch.equal(c, ref)
    for call in (lambda ws: moe.moe_grouped_linear_w4(rows, offsets, w, s, z, workspace=ws),
                 lambda ws: moe.moe_dispatch(x0, idx, E, workspace=ws)):
        for ws in (torch.empty(64, dtype=torch.uint8, device="cuda"),
                   torch.empty(need + need_d + 16, dtype=torch.uint8, device="cuda")[16:]):
            with pytest.raises(moe.MoeError) as e:
                call(ws)
            assert e.value.status == moe.MOE_ERR_WORKSPACE


def test_two_captured_graphs_at_once():
    """Graphs of the same calls hold workspaces of their own: replayed on two streams
    together they give the eager results."""
    import block_fp8_routed_amd as moe
    T, k, E, H = 2500, 2, 8, 512
    w, s, _, _ = weights((E,), 1024, H, 128, 9, zeros=False)
    cases = []
    for seed in range(2):
        x = matrix(T, H, torch.bfloat16, 10 + seed)
        idx = torch.from_numpy(choices(T, k, E, 20 + seed)).cuda()

        def layer(x=x, idx=idx):
            rows, offsets, _, inv = moe.moe_dispatch(x, idx, E)
            y = moe.moe_grouped_linear_w4(rows, offsets, w, s)
            return moe.moe_combine(y, torch.ones(T, k, device="cuda"), inv)

        want = layer()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = layer()
        # (with the layer the inputs, whose addresses the graph holds, stay alive)
        cases.append((graph, held, want, torch.cuda.Stream(), layer))
    for _ in range(3):
        for graph, held, _, st, _ in cases:
            held.zero_()
        torch.cuda.synchronize()
        for graph, _, _, st, _ in cases:
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for _, held, want, _, _ in cases:
            assert torch.equal(held, want)
