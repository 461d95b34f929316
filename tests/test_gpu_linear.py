"""The dense block-FP8 operators on the GPU (moe_linear, moe_linear_e4m3,
moe_swiglu_quantize_e4m3) against the fp64 oracle.

Tolerance of a product, per element, with `mag` the sum of its terms'
magnitudes (which bounds every running sum):
  * fp32 output: per 128 columns four matrix instructions of 32 products (two
    internal steps of at most 24 bits below the largest of eight products
    each, then a sum) and one multiply-add; then at most a few joins of partial
    sums and the bias. Counting eight roundings of 2^-24 per 32 columns for
    the instruction and two per 128 for the rest, K columns err by at most
    (K/4 + K/64 + 8) 2^-24 mag; the sums seen stay below a tenth of it.
  * bf16 output: the FP8 matrix instruction cuts each of eight products at
    2^-13 of the largest of them (measured on 2^16 + 2^s), so eight products
    lose at most 8 * 2^-13 of their largest: 2^-10 mag in all, on top of the
    fp32 steps.
plus half a step of the output type. In norm, bf16 results are also within
2^-8: half a step at worst for every element, and the cuts, which go either
way, some 2^-15.

Tolerance of SwiGLU: h in fp32 takes an exponential (argument exact, result
within 2 ulps), a sum, a quotient and a product; with every step's half ulp
that is below 8 * 2^-24 of |h|. The codes must be admissible for h within that
band (the oracle's h_admissible_codes)."""
import numpy as np
import pytest
import torch

import oracle
from parity import log

pytestmark = pytest.mark.gpu

F32_MIN = 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import block_fp8_routed_amd as moe
    moe.load()
    yield
    torch.cuda.synchronize()


def weights(N, K, seed=0, scales=None):
    """E4M3 bytes and block scales with sizes 2^-4 .. 2^4 apart."""
    g = np.random.default_rng(seed + 17)
    w = g.integers(0, 256, (N, K)).astype(np.uint8)
    w[(w & 0x7F) == 0x7F] = 0x35
    s = scales if scales is not None else \
        (np.exp2(g.uniform(-4, 4, (-(-N // 128), K // 128))) * 1e-3).astype(np.float32)
    return w, s


def rows(M, K, seed=0, big=True):
    g = np.random.default_rng(seed)
    x = g.standard_normal((M, K)).astype(np.float32)
    if big:
        x *= np.exp2(g.integers(-6, 7, (M, 1))).astype(np.float32)
        x[:, ::61] *= 20
    return torch.from_numpy(x).to(torch.bfloat16)


def compare(got, codes, exps, w, s, bias, K, what):
    want, mag = oracle.linear_e4m3(codes, exps, w, s, bias)
    g = got.double().cpu().numpy()
    assert g.shape == want.shape and np.isfinite(g).all(), what
    tol = (K / 4 + K / 64 + 8) * 2.0 ** -24 * mag + F32_MIN
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -10 * mag
    tol = tol + (np.abs(want) + tol) * torch.finfo(got.dtype).eps / 2
    bad = np.abs(g - want) > tol
    ratio = float((np.abs(g - want) / tol).max())
    norm = float(np.linalg.norm(g - want) / max(np.linalg.norm(want), 1e-300))
    log(f"linear {what}: worst error {ratio:.3f} of its bound, {norm:.2e} in norm")
    if got.dtype == torch.bfloat16:
        assert norm <= 2.0 ** -8, f"{what}: {norm} in norm"
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def run(M, N, K, out_dtype=torch.float32, bias=False, seed=0, scales=None, ld_x=0, ld_out=0, x=None):
    import block_fp8_routed_amd as moe
    x = rows(M, K, seed) if x is None else x
    w, s = weights(N, K, seed, scales)
    b = np.random.default_rng(seed).normal(size=N).astype(np.float32) if bias else None
    codes, exps = oracle.quantise_activations(x.float().numpy(), 128)
    xd = x.cuda()
    if ld_x:
        wide = torch.full((M, K + ld_x), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :K] = xd
        xd = wide[:, :K]
    wd, sd = torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda()
    bd = None if b is None else torch.from_numpy(b).cuda()
    out = None
    if ld_out:
        buf = torch.full((M + 1, N + ld_out), -7.0, dtype=out_dtype, device="cuda")
        out = buf[:M, :N]
    got = moe.moe_linear(xd, wd, sd, bias=bd, out_dtype=out_dtype, out=out)
    what = f"M={M} N={N} K={K} {out_dtype} bias={bias} ld +{ld_x}/+{ld_out}"
    compare(got, codes, exps, w, s, b, K, what)
    if ld_out:
        assert bool((buf[:M, N:] == -7.0).all()) and bool((buf[M:] == -7.0).all()), what
    # the two entry points give the same bits
    if M * K:
        cd, ed = moe.moe_quantize_act_e4m3(x.cuda())
        assert np.array_equal(ed.cpu().numpy().astype(np.int64) - 127, exps)
        two = moe.moe_linear_e4m3(cd, ed, wd, sd, bias=bd, out_dtype=out_dtype)
        assert torch.equal(two, got), what
    return got


# rows around the switches between kernels and the tile edges
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127,
                               128, 129, 200, 255, 256, 257, 300, 513])
def test_rows(M):
    run(M, 300, 384, seed=M)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 7, 8, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 130,
                               191, 255, 256, 257, 320, 511, 576, 1000])
@pytest.mark.parametrize("M", [1, 16, 70, 260])
def test_output_features(M, N):
    run(M, N, 256, out_dtype=torch.bfloat16, bias=N % 2 == 1, seed=N)


@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 896, 1024, 1152, 2048, 4096, 8192])
@pytest.mark.parametrize("M", [1, 7, 33, 130])
def test_input_features(M, K):
    run(M, 200, K, seed=K)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 2048), (16, 8192, 512), (40, 4096, 1024),
                                   (77, 2112, 4096), (1000, 1024, 512), (515, 2500, 768),
                                   (2049, 640, 256)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_larger(M, N, K, out_dtype):
    run(M, N, K, out_dtype=out_dtype, bias=True, seed=M)


@pytest.mark.parametrize("M", [1, 9, 50, 300])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_rows_apart(M, out_dtype):
    run(M, 200, 256, out_dtype=out_dtype, ld_x=8, ld_out=5, seed=3)
    run(M, 132, 256, out_dtype=out_dtype, ld_x=264, ld_out=4, bias=True, seed=4)
    run(M, 131, 128, out_dtype=out_dtype, ld_out=1, seed=5)


@pytest.mark.parametrize("M", [2, 30, 140])
def test_scales(M):
    """Zero, negative, tiny and huge block scales, next to one another."""
    s = np.array([[0.0, 1e-3, 2.0 ** -140, -0.5], [1e20, 0.0, 1e-20, 3.0],
                  [0.0, 0.0, 0.0, 0.0]], np.float32)
    run(M, 300, 512, scales=s, seed=1)


@pytest.mark.parametrize("M", [1, 20, 150])
def test_activation_range(M):
    """Rows of zeros, of the smallest and of the largest bf16 values."""
    K = 384
    x = rows(M, K, 8)
    x[0] = 0
    if M > 4:
        x[1, :128] = 0
        x[2] = x[2] * 2.0 ** -100
        x[3] = torch.where(x[3] > 0, 3.0e38, -3.0e38).to(torch.bfloat16)
        x[4, 128:] = 2.0 ** -133
    s = np.full((2, 3), 1e-30, np.float32)
    run(M, 160, K, x=x, scales=s)


# products of more than 256 tiles of 64 x 64: one of every kind of tile for each
# output type, with part-full tiles on both edges
TILES = [(300, 4000), (700, 5000), (17300, 300), (2000, 4000), (2200, 5000)]


@pytest.mark.parametrize("M,N", TILES)
@pytest.mark.parametrize("K", [128, 384])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_tiles(M, N, K, out_dtype):
    run(M, N, K, out_dtype, bias=True, seed=M + K, ld_x=8, ld_out=8 if K == 128 else 1)


@pytest.mark.parametrize("M,N,K", [(300, 4000, 1152), (300, 4000, 4224), (700, 5000, 1280),
                                   (2000, 4000, 640), (2200, 5000, 512)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_tiles_of_more_blocks(M, N, K, out_dtype):
    run(M, N, K, out_dtype, seed=M + K)


@pytest.mark.parametrize("M,N", [(300, 4000), (700, 5000), (2200, 5000)])
def test_tiles_repeat_and_replay(M, N):
    import block_fp8_routed_amd as moe
    K = 768
    w, s = (torch.from_numpy(a).cuda() for a in weights(N, K, 6))
    x = rows(M, K, 6).cuda()
    codes, exps = moe.moe_quantize_act_e4m3(x)
    buf = torch.empty(exps.numel() + 4, dtype=torch.uint8, device="cuda")
    for out_dtype in (torch.bfloat16, torch.float32):
        want = moe.moe_linear(x, w, s, out_dtype=out_dtype)
        for skip in (0, 1, 2):  # exponents at any address
            moved = buf[skip:skip + exps.numel()].view(exps.shape)
            moved.copy_(exps)
            assert torch.equal(moe.moe_linear_e4m3(codes, moved, w, s, out_dtype=out_dtype), want)
        out = torch.empty_like(want)
        ws = torch.empty(moe.linear_workspace_bytes(M, N, K, False), dtype=torch.uint8,
                         device="cuda")
        moe.moe_linear(x, w, s, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_linear(x, w, s, out=out, workspace=ws)
        x0 = x.clone()
        for i in range(4):
            x.copy_(x0 * (i + 1))
            out.zero_()
            graph.replay()
            eager = moe.moe_linear(x, w, s, out_dtype=out_dtype)
            torch.cuda.synchronize()
            assert torch.equal(out, eager), f"replay {i}"
        x.copy_(x0)


# the stream's forms: one round of 32 x 16, 32 x 32, 48 x 32, 64 x 32, 48 x 64, 64 x 64
@pytest.mark.parametrize("M,N", [(31, 4090), (33, 2000), (90, 2600), (96, 3900), (130, 3300),
                                 (140, 5300), (255, 4090), (300, 3200), (20, 8100), (17, 9000),
                                 (120, 4090), (60, 8000)])
@pytest.mark.parametrize("K", [128, 1024, 2176, 4224])
def test_stream_forms(M, N, K):
    out_dtype = torch.float32 if (M + K // 128) % 2 else torch.bfloat16
    run(M, N, K, out_dtype, bias=True, seed=M + K, ld_out=3)


@pytest.mark.parametrize("M", [5, 70, 300])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_exponents_at_any_address(M, out_dtype):
    """Exponents that start at an odd byte; out that starts at an odd element."""
    import block_fp8_routed_amd as moe
    N, K = 200, 1024
    x = rows(M, K, M)
    w, s = (torch.from_numpy(a).cuda() for a in weights(N, K, M))
    codes, exps = moe.moe_quantize_act_e4m3(x.cuda())
    want = moe.moe_linear_e4m3(codes, exps, w, s, out_dtype=out_dtype)
    for skip in (1, 2, 3):
        buf = torch.empty(exps.numel() + 4, dtype=torch.uint8, device="cuda")
        moved = buf[skip:skip + exps.numel()].view(exps.shape)
        moved.copy_(exps)
        flat = torch.zeros(M * N + 4, dtype=out_dtype, device="cuda")
        out = flat[skip:skip + M * N].view(M, N)
        moe.moe_linear_e4m3(codes, moved, w, s, out=out)
        assert torch.equal(out, want), skip
        assert not flat[:skip].any() and not flat[skip + M * N:].any(), skip


def test_a_row_does_not_depend_on_the_others():
    """Each row of a batch has the bits it has in another batch of the same
    size, whatever the other rows hold."""
    import block_fp8_routed_amd as moe
    w, s = (torch.from_numpy(a).cuda() for a in weights(520, 512, 2))
    for M in (3, 16, 40, 150, 400):
        x = rows(M, 512, M).cuda()
        y = x * 64
        y[M // 2] = x[M // 2]
        a, b = moe.moe_linear(x, w, s), moe.moe_linear(y, w, s)
        assert torch.equal(a[M // 2], b[M // 2])


def test_no_rows():
    import block_fp8_routed_amd as moe
    w, s = (torch.from_numpy(a).cuda() for a in weights(200, 256))
    assert moe.moe_linear(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), w, s).shape == (0, 200)
    c, e = moe.moe_swiglu_quantize_e4m3(torch.empty(0, 512, dtype=torch.bfloat16, device="cuda"))
    assert c.shape == (0, 256) and e.shape == (0, 2)
    assert moe.moe_linear_e4m3(c, e, w, s).shape == (0, 200)


@pytest.mark.parametrize("M,N,K", [(1, 1000, 1024), (16, 2000, 2048), (33, 500, 4096),
                                   (300, 600, 512), (900, 1024, 1024)])
def test_runs_repeat_and_replay(M, N, K):
    """The same bits on every run, on another stream, and from a captured
    graph replayed between eager calls on other inputs."""
    import block_fp8_routed_amd as moe
    w, s = (torch.from_numpy(a).cuda() for a in weights(N, K, 5))
    x = rows(M, K, 5).cuda()
    want = moe.moe_linear(x, w, s)
    for _ in range(3):
        assert torch.equal(moe.moe_linear(x, w, s), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_linear(x, w, s, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    n = moe.linear_workspace_bytes(M, N, K, False)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    moe.moe_linear(x, w, s, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_linear(x, w, s, out=out, workspace=ws)
    x0 = x.clone()
    for i in range(4):
        x.copy_(x0 * (i + 1))
        out.zero_()
        graph.replay()
        eager = moe.moe_linear(x, w, s)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), f"replay {i}"


def test_two_calls_at_once():
    """Products on two streams, each with its own workspace, many in flight."""
    import block_fp8_routed_amd as moe
    sets = []
    for i, (M, N, K) in enumerate([(16, 1024, 2048), (200, 768, 1024)]):
        w, s = (torch.from_numpy(a).cuda() for a in weights(N, K, i))
        x = rows(M, K, i).cuda()
        sets.append((x, w, s, moe.moe_linear(x, w, s), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (x, w, s, _, st) in enumerate(sets):
            got[i].append(moe.moe_linear(x, w, s, stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, sets[i][3]) for g in got[i])


# ------------------------------------------------------------------- SwiGLU --
BAND = 8 * 2.0 ** -24


def check_swiglu(gu, what):
    import block_fp8_routed_amd as moe
    codes, exps = (a.cpu().numpy() for a in moe.moe_swiglu_quantize_e4m3(gu))
    h = oracle.swiglu(gu.double().cpu().numpy())
    e = exps.astype(np.int64) - 127
    # below fp32's normal range h is rounded to its subnormal steps
    ok = oracle.h_admissible_codes(h, BAND * np.abs(h) + 4 * F32_MIN, codes, e, 128)
    want, _ = oracle.quantise_activations(h, 128)
    flips = int((codes != want).sum())
    log(f"swiglu {what}: {flips} of {codes.size} codes the other side of a midpoint")
    assert ok.all(), f"{what}: {(~ok).sum()} inadmissible codes, first {np.argwhere(~ok)[0]}"
    # at most a code in a thousand may sit within 2^-21 of a midpoint
    assert flips <= max(2, codes.size // 1000)
    sign = np.signbit(gu.float().cpu().numpy())
    I = codes.shape[1]
    assert np.array_equal(codes >> 7, (sign[:, :I] ^ sign[:, I:]).astype(np.uint8)), what


@pytest.mark.parametrize("T", [1, 2, 3, 17, 130])
@pytest.mark.parametrize("I", [128, 256, 640, 768, 1024, 4096])
def test_swiglu(T, I):
    g = np.random.default_rng(T * I)
    gu = torch.from_numpy(g.normal(0, 1.5, (T, 2 * I))).to(torch.bfloat16).cuda()
    check_swiglu(gu, f"T={T} I={I}")
    wide = torch.full((T, 2 * I + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :2 * I] = gu
    import block_fp8_routed_amd as moe
    a, b = moe.moe_swiglu_quantize_e4m3(wide[:, :2 * I]), moe.moe_swiglu_quantize_e4m3(gu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_swiglu_ranges():
    """Gates far into both tails, products at both ends of fp32, zero blocks."""
    g = np.random.default_rng(0)
    gu = g.normal(0, 1, (9, 512)).astype(np.float32)
    gu[0] = 0
    gu[1, :256] *= 60
    gu[2, :256] = -np.abs(gu[2, :256]) * 40
    gu[3, :256] = np.abs(gu[3, :256]) * 1e18
    gu[4, 256:] *= 1e-30
    gu[5] *= 1e-18
    gu[6, :128] = 0
    gu[7] *= 2.0 ** np.arange(-32, 32).repeat(8)
    check_swiglu(torch.from_numpy(gu).to(torch.bfloat16).cuda(), "ranges")


def test_swiglu_overflow_and_nan():
    import block_fp8_routed_amd as moe
    gu = torch.ones(4, 256, dtype=torch.bfloat16, device="cuda")
    gu[0, 0], gu[0, 128] = 3e38, 3e38          # beyond fp32: its largest value
    gu[1, 5] = float("nan")
    gu[2, 7] = float("-inf")                   # -inf / inf
    gu[3, 9], gu[3, 137] = float("inf"), -1.0
    codes, exps = (a.cpu().numpy() for a in moe.moe_swiglu_quantize_e4m3(gu))
    dec = oracle.e4m3fn_decode(codes)
    e = exps.astype(np.int64)[:, 0] - 127
    assert dec[0, 0] * 2.0 ** e[0] == 2.0 ** 128 and e[0] == 120
    one = float(oracle.swiglu(np.ones((1, 2)))[0, 0])
    want, we = oracle.quantise_activations(np.full((1, 128), one), 128)
    for r, c in ((1, 5), (2, 7)):
        assert codes[r, c] == 0x7F and e[r] == we[0, 0]
        assert (np.delete(codes[r], c) == want[0, 0]).all()
    assert dec[3, 9] * 2.0 ** e[3] == -2.0 ** 128


# --------------------------------------------------- the operators in a row --
@pytest.mark.parametrize("T,H,I", [(1, 2048, 768), (16, 1024, 512), (50, 512, 384), (300, 1024, 640)])
def test_feed_forward_block(T, H, I):
    """gate/up product, SwiGLU with quantised output, down product: each step
    is held to the oracle on the step before's own values, and the whole to the
    unquantised block: x, the weights' sums and h each carry a quantisation of
    at most 2^-4 per value, independent from value to value, so the result is
    within a few percent in norm (2^-4 / sqrt(3) per operand on average)."""
    import block_fp8_routed_amd as moe
    x = rows(T, H, 3, big=False)
    w1, s1 = weights(2 * I, H, 1, np.full((-(-2 * I // 128), H // 128), 2e-4, np.float32))
    w2, s2 = weights(H, I, 2, np.full((-(-H // 128), I // 128), 2e-4, np.float32))
    d = [torch.from_numpy(a).cuda() for a in (w1, s1, w2, s2)]
    gu = moe.moe_linear(x.cuda(), d[0], d[1])
    codes, exps = moe.moe_swiglu_quantize_e4m3(gu)
    out = moe.moe_linear_e4m3(codes, exps, d[2], d[3], out_dtype=torch.float32)
    c, e = oracle.quantise_activations(x.float().numpy(), 128)
    compare(gu, c, e, w1, s1, None, H, f"gate/up T={T}")
    check_swiglu(gu, f"block T={T}")
    compare(out, codes.cpu().numpy(), exps.cpu().numpy().astype(np.int64) - 127, w2, s2, None, I,
            f"down T={T}")
    plain = oracle.swiglu(x.double().numpy() @ oracle.block_weights(w1, s1).T) \
        @ oracle.block_weights(w2, s2).T
    err = np.linalg.norm(out.double().cpu().numpy() - plain) / np.linalg.norm(plain)
    log(f"feed-forward block T={T}: {err:.4f} of the unquantised block in norm")
    assert err < 0.1


@pytest.mark.parametrize("T", [1, 60, 700])
def test_feed_forward_block_in_a_graph(T):
    """The block captured with its own allocations, replayed on changing inputs
    between eager runs of it; rows of `out` behind the batch stay as they are."""
    import block_fp8_routed_amd as moe
    H, I = 1024, 768
    w1, s1 = (torch.from_numpy(a).cuda() for a in weights(2 * I, H, 31))
    w2, s2 = (torch.from_numpy(a).cuda() for a in weights(H, I, 32))
    x = rows(T, H, T, big=False).cuda()
    buf = torch.full((T + 3, H), 5.0, dtype=torch.bfloat16, device="cuda")

    def block(out=None):
        h = moe.moe_linear(x, w1, s1)
        codes, exps = moe.moe_swiglu_quantize_e4m3(h)
        return moe.moe_linear_e4m3(codes, exps, w2, s2, out=out)

    block(buf[:T])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(buf[:T])
    x0 = x.clone()
    for i in range(4):
        x.copy_(x0 * (0.5 + i))
        buf[:T] = 0
        graph.replay()
        eager = block()
        torch.cuda.synchronize()
        assert torch.equal(buf[:T], eager), f"replay {i}"
        assert bool((buf[T:] == 5.0).all())
