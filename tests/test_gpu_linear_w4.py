"""Products with 4-bit weights (moe_linear_w4, moe_grouped_linear_w4) against the
formula in 64 bits, and the layer that they make with moe_dispatch and moe_combine.

The bound of an element: a term x (q or z) s meets at most 64 + K / 32 fp32 roundings
(32 inside an instruction, four instructions of a group, the group's scale and zero
point, one addition a group or instruction after it), each 2^-24 of the magnitudes
summed so far, which sum |x| (q + z) |s| bounds; half a step of the output type
comes on top. SwiGLU passes the errors of gate and up on with |silu'| <= 1.1 and
|silu|, and adds 2^-20 of its own value (exponential, quotient, two products; the
exponential's argument has 2^-24 |g|, |g| up to 8 here).

bf16 output of larger batches multiplies fp16 weights q S 2^-24 - z s, S = 2^24 s:
half a step of fp16's 11 bits is 2^-11 of a value. S is rounded once, which moves
(q - z) s by 2^-11 of itself; z s once, 2^-11 z s; the result once, 2^-11 of it. Below
fp16's normal numbers z s and the result are off by up to 2^-25 instead, where the
row's largest s is at least 2^-10: 2^-14 of that scale, for every |x|. `half` adds these (and 2^-20 of the first for
their products). Both forms of the larger batches hold a row of x as fp16 times a power
of two that brings its largest magnitude to 2^14 at least: a small value is off by up
to 2^-25, 2^-39 or less of that magnitude, half of it where it rounds to nearest."""
import numpy as np
import pytest
import torch

from test_gpu_dispatch import HALF, TYPES, choices, permutation

pytestmark = pytest.mark.gpu


def weights(lead, N, K, G, seed, scales="f32", zeros=True, bias=False):
    r = np.random.default_rng(seed)
    w = r.integers(0, 256, (*lead, N, K // 2)).astype(np.uint8)
    s = (np.exp2(r.uniform(-2, 2, (*lead, N, K // G))) * 0.02 * r.choice([-1, 1], (*lead, N, K // G)))
    s = torch.from_numpy(s.astype(np.float32)).to(TYPES[scales])
    z = torch.from_numpy(r.integers(0, 20, s.shape).astype(np.uint8)) if zeros else None
    b = torch.from_numpy(r.normal(size=(*lead, N)).astype(np.float32)) if bias else None
    return tuple(None if t is None else t.cuda() for t in (torch.from_numpy(w), s, z, b))


def activations(M, K, seed, pad=0):
    r = np.random.default_rng(seed)
    x = r.normal(size=(M, K + pad)).astype(np.float32)
    x[:, r.random(K + pad) < 0.02] *= 12
    return torch.from_numpy(x).to(torch.bfloat16).cuda()[:, :K]


def values(w, s, z):
    """(W, (q + z) |s|, z |s|) of [n][k/2] codes in 64 bits."""
    w, s = w.cpu().numpy(), s.double().cpu().numpy()
    z = np.full(s.shape, 8.0) if z is None else z.cpu().numpy().astype(np.float64)
    n, half = w.shape
    q = np.empty((n, 2 * half))
    q[:, 0::2], q[:, 1::2] = w & 15, w >> 4
    G = 2 * half // s.shape[1]
    s, z = np.repeat(s, G, axis=1), np.repeat(z, G, axis=1)
    return (q - z) * s, (q + z) * np.abs(s), z * np.abs(s)


def reference(x, w, s, z, b, swiglu, half=True):
    """(out, bound of the errors before its rounding) in 64 bits."""
    x = x.double().cpu().numpy()
    v, mag, zero = values(w, s, z)
    y = x @ v.T
    a = np.abs(x)
    err = ((64 + x.shape[1] / 32) * 2.0 ** -24 * (a @ mag.T)
           + 2.0 ** -40 * a.max(axis=1)[:, None] * np.abs(v).sum(axis=1))
    if half:
        smax = s.double().abs().amax(dim=1).cpu().numpy()
        err = (err + (1 + 2.0 ** -20) * (a @ (2.0 ** -10 * np.abs(v) + 2.0 ** -11 * zero).T)
               + 2.0 ** -14 * a.sum(axis=1)[:, None] * smax)
    if b is not None:
        b = b.double().cpu().numpy()
        y, err = y + b, err + 2.0 ** -24 * (np.abs(y) + np.abs(b))
    if swiglu:
        i = y.shape[1] // 2
        g, u, eg, eu = y[:, :i], y[:, i:], err[:, :i], err[:, i:]
        e = np.exp(-np.abs(g))
        silu = g * np.where(g >= 0, 1 / (1 + e), e / (1 + e))
        y = silu * u
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + 2.0 ** -20 * np.abs(y)
    return y, err


def check(got, ref, err, what=""):
    got64 = got.double().cpu().numpy()
    off = np.abs(got64 - ref)
    lim = err + HALF[got.dtype] * (np.abs(ref) + err) + 1e-45
    assert np.isfinite(got64).all(), what
    assert (off <= lim).all(), f"{what}: {np.max(off / lim):.2f} of the bound"


def takes_tiles(M, N, K, out, E=1):
    """Whether a product runs on the tiles of larger batches (they alone have a workspace)."""
    import block_fp8_routed_amd as moe
    code = moe.MOE_BF16 if out == torch.bfloat16 else moe.MOE_F32
    return moe.linear_w4_workspace_bytes(M, E, N, K, code) > 0


ROWS = [1, 2, 15, 16, 17, 33, 64, 65, 130, 193, 300]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("G,N,K", [(128, 96, 1024), (64, 35, 448), (32, 130, 352), (32, 1, 32),
                                   (64, 200, 64), (128, 64, 128)])
def test_product(M, G, N, K):
    import block_fp8_routed_amd as moe
    for i, (scales, zeros, bias, out) in enumerate([("f32", True, True, "f32"),
                                                    ("bf16", False, False, "bf16")]):
        w, s, z, b = weights((), N, K, G, M + i, scales, zeros, bias)
        x = activations(M, K, M)
        got = moe.moe_linear_w4(x, w, s, z, bias=b, out_dtype=TYPES[out])
        check(got, *reference(x, w, s, z, b, False, out == "bf16"), f"{scales} {out}")


@pytest.mark.parametrize("M,N,K,G", [(4100, 420, 512, 128), (4133, 702, 352, 32), (3000, 1026, 320, 64),
                                     (2049, 1030, 1056, 32), (1500, 4096, 256, 128), (700, 4096, 1024, 64),
                                     (20000, 130, 512, 128), (30001, 66, 1088, 64), (20000, 2048, 32, 32)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_products_of_larger_batches(M, N, K, G, swiglu):
    import block_fp8_routed_amd as moe
    N += swiglu and N % 2
    for i, out in enumerate(TYPES.values()):
        assert takes_tiles(M, N, K, out)
        w, s, z, b = weights((), N, K, G, M + i, "bf16" if i else "f32", i == M % 2, M % 3 > 0)
        x = activations(M, K, M)
        s = s * 0.1 if swiglu else s
        got = moe.moe_linear_w4(x, w, s, z, bias=b, swiglu=swiglu, out_dtype=out)
        check(got, *reference(x, w, s, z, b, swiglu, out == torch.bfloat16), str(out))


@pytest.mark.parametrize("M", [1, 16, 40, 129, 200, 520])
@pytest.mark.parametrize("G,N,K", [(128, 1536, 2048), (64, 258, 320), (32, 2, 96), (32, 130, 128)])
def test_swiglu(M, G, N, K):
    import block_fp8_routed_amd as moe
    w, s, z, b = weights((), N, K, G, M, "bf16", M % 2 == 0, True)
    x = activations(M, K, M)
    for out in TYPES.values():
        got = moe.moe_linear_w4(x, w, s * 0.05, z, bias=b, swiglu=True, out_dtype=out)
        assert got.shape == (M, N // 2)
        check(got, *reference(x, w, s * 0.05, z, b, True, out == torch.bfloat16), str(out))


@pytest.mark.parametrize("M,N,K,G", [(1, 4096, 4096, 128), (16, 512, 8192, 64), (77, 2112, 4096, 32),
                                     (1000, 640, 1024, 128), (2049, 300, 512, 64),
                                     (5, 48, 4128, 32), (11, 40, 12288, 128), (200, 4096, 1056, 32),
                                     (150, 70, 8320, 64), (3000, 2048, 256, 32)])
def test_long_and_wide_products(M, N, K, G):
    import block_fp8_routed_amd as moe
    w, s, z, _ = weights((), N, K, G, 3, "f32", True)
    x = activations(M, K, 4)
    for out in TYPES.values():
        got = moe.moe_linear_w4(x, w, s, z, out_dtype=out)
        check(got, *reference(x, w, s, z, None, False, out == torch.bfloat16), str(out))


def test_every_code_and_zero_point():
    """One column set at a time: out is exactly (q - z) s x for every q and z."""
    import block_fp8_routed_amd as moe
    K, N = 128, 256 * 16
    q, z = np.meshgrid(np.arange(16), np.arange(256))
    codes = (q.reshape(-1) | q.reshape(-1) << 4).astype(np.uint8)
    w = torch.from_numpy(np.repeat(codes[:, None], K // 2, axis=1)).cuda()
    zero = torch.from_numpy(np.repeat(z.reshape(-1, 1), 4, axis=1).astype(np.uint8)).cuda()
    s = torch.full((N, 4), 0.5, device="cuda")
    for M in (1, 128, 1700):
        x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        x[torch.arange(M), torch.arange(M) % K] = 2.0
        want = torch.from_numpy((q - z).reshape(-1).astype(np.float32)).cuda().expand(M, N)
        for out in TYPES.values():
            assert torch.equal(moe.moe_linear_w4(x, w, s, zero, out_dtype=out), want.to(out))


@pytest.mark.parametrize("M", [1, 20, 208, 1100])
def test_columns_meet_their_codes(M):
    """x = a unit vector picks one column of W: exact."""
    import block_fp8_routed_amd as moe
    N, K, G = 48 if M < 1000 else 2100, 416, 32
    w, s, z, _ = weights((), N, K, G, 5)
    v, _, zero = values(w, s, z)
    for k0 in range(0, K, M):
        x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        n = min(M, K - k0)
        x[torch.arange(n), k0 + torch.arange(n)] = 1.0
        got = moe.moe_linear_w4(x, w, s, z, out_dtype=torch.float32)[:n]
        assert np.array_equal(got.cpu().numpy(), v[:, k0:k0 + n].T.astype(np.float32))
        got = moe.moe_linear_w4(x, w, s, z)[:n].double().cpu().numpy()
        want = v[:, k0:k0 + n].T
        # the weight's own error, as above, and its rounding to bf16
        err = ((1 + 2.0 ** -20) * (2.0 ** -10 * np.abs(want) + 2.0 ** -11 * zero[:, k0:k0 + n].T)
               + 2.0 ** -14 * s.double().abs().amax(dim=1).cpu().numpy())
        assert (np.abs(got - want) <= err + 2.0 ** -8 * (np.abs(want) + err)).all()


@pytest.mark.parametrize("M", [4, 100, 4100])
def test_small_values_beside_a_large_one(M):
    """A row's small values, down to 2^-24 of its largest, count where the large
    one's weight is 0."""
    import block_fp8_routed_amd as moe
    N, K, G = 32 if M < 4000 else 900, 256, 64
    w, s, _, _ = weights((), N, K, G, 21, zeros=False)
    w[:, 50] = 0x88  # columns 100 and 101: 8 - 8
    s = torch.full_like(s, 0.25)
    x = activations(M, K, 22)
    x = (torch.sign(x) * (1 + x.abs() % 1)).to(torch.bfloat16) * 2.0 ** -24
    x[:, 100] = 1.0
    for out in TYPES.values():
        got = moe.moe_linear_w4(x, w, s, out_dtype=out).double().cpu().numpy()
        small = x.double().cpu().numpy()
        small[:, 100] = 0
        want = small @ values(w, s, None)[0].T
        # Larger batches: 2^-24 is 2^-10 beside 2^14, a normal number of fp16, and 8 - 8 is 0
        # before it meets x: nothing of the large value is left. Smaller ones sum x q and
        # 8 x apart: there the large column's two terms of 8 * 0.25 are rounded with the
        # rest, 2^-24 of 4 each time, which the bound of the whole row counts.
        seen = torch.from_numpy(small) if takes_tiles(M, N, K, out) else x
        _, err = reference(seen, w, s, None, None, False, out == torch.bfloat16)
        assert (np.abs(got - want) <= err + HALF[out] * (np.abs(want) + err)).all()


@pytest.mark.parametrize("M", [3, 100, 4100])
def test_strided_rows_and_outputs(M):
    import block_fp8_routed_amd as moe
    N, K, G = 70 if M < 4000 else 910, 256, 64
    w, s, z, _ = weights((), N, K, G, 6)
    x = activations(M, K, 7, pad=24)
    for out in TYPES.values():
        for pad in (2, 7, 10):
            whole = torch.full((M, N + pad), 4.0, dtype=out, device="cuda")
            got = moe.moe_linear_w4(x, w, s, z, out=whole[:, 1:N + 1])
            check(got, *reference(x, w, s, z, None, False, out == torch.bfloat16))
            assert bool((whole[:, 0] == 4).all()) and bool((whole[:, N + 1:] == 4).all())


@pytest.mark.parametrize("M", [16, 64, 200, 4100])
def test_a_row_of_nan_stays_in_its_row(M):
    import block_fp8_routed_amd as moe
    w, s, z, _ = weights((), 50 if M < 4000 else 900, 256, 64, 8)
    for out in TYPES.values():
        x = activations(M, 256, 9)
        want = moe.moe_linear_w4(x, w, s, z, out_dtype=out)
        x[5] = float("nan")
        x[7, 3] = float("inf")
        got = moe.moe_linear_w4(x, w, s, z, out_dtype=out)
        rest = torch.ones(M, dtype=torch.bool)
        rest[[5, 7]] = False
        assert torch.equal(got[rest], want[rest]) and bool(torch.isnan(got[5]).all())


@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** -118, 2.0 ** 114])
def test_ends_of_the_range(scale):
    """Large and small rows, their sums and the scales' products within fp32's range."""
    import block_fp8_routed_amd as moe
    for M, N in ((2, 40), (90, 40), (4100, 900)):
        w, s, z, _ = weights((), N, 256, 128, 10)
        x = (activations(M, 256, 11).float() * scale).to(torch.bfloat16)
        ref, err = reference(x, w, s, z, None, False, False)
        # below 2^-126 fp32 keeps steps of 2^-149, one for each of the roundings
        err = err + (64 + 256 / 32) * 2.0 ** -149 * 256 * 512
        check(moe.moe_linear_w4(x, w, s, z, out_dtype=torch.float32), ref, err)


def grouped_reference(x, offsets, w, s, z, b, swiglu, half=True):
    n = w.shape[1] // 2 if swiglu else w.shape[1]
    ref, err = np.zeros((x.shape[0], n)), np.zeros((x.shape[0], n))
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo < hi:
            one = [None if t is None else t[e] for t in (w, s, z, b)]
            ref[lo:hi], err[lo:hi] = reference(x[lo:hi], *one, swiglu, half)
    return ref, err


COUNTS = {
    "one_row": [0, 0, 1, 0], "even": [5, 5, 5, 5], "uneven": [0, 300, 1, 0, 17, 16, 0, 64, 129, 0],
    "single": [140], "none": [0, 0, 0], "last": [0] * 99 + [33], "many": [1, 0, 2] * 230,
    "tiles": [32, 64, 128, 256, 31, 33, 63, 65],
    "large": [700, 1, 0, 90, 1300, 31, 33, 64, 65, 2200, 0, 0],
}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("G", [32, 128])
def test_grouped(name, swiglu, G):
    import block_fp8_routed_amd as moe
    counts = COUNTS[name]
    E, N, K = len(counts), 72 if name != "large" else 1030, 256
    offsets = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    behind = 7  # rows of no expert
    M = int(offsets[-1]) + behind
    w, s, z, b = weights((E,), N, K, G, 12, "bf16" if G == 32 else "f32", swiglu, True)
    s = s * 0.1
    x = activations(M, K, 13)
    n = N // 2 if swiglu else N
    kind = torch.bfloat16 if swiglu else torch.float32
    assert takes_tiles(M, N, K, kind, E) == (name == "large")
    out = torch.full((M, n), 6.0, dtype=kind, device="cuda")
    got = moe.moe_grouped_linear_w4(x, torch.from_numpy(offsets).cuda(), w, s, z, bias=b,
                                    swiglu=swiglu, out=out)
    ref, err = grouped_reference(x, offsets, w, s, z, b, swiglu, swiglu)
    check(got[:M - behind], ref[:M - behind], err[:M - behind])
    assert bool((out[M - behind:] == 6).all())


@pytest.mark.parametrize("M,N,K", [(40, 32, 128), (4100, 1030, 256)])
def test_offsets_are_cut_to_the_rows(M, N, K):
    """Offsets beyond the rows, negative or falling name no row outside x and out."""
    import block_fp8_routed_amd as moe
    w, s, z, _ = weights((4,), N, K, 128, 14)
    x = activations(M, K, 15)
    out = torch.full((M, N), 6.0, dtype=torch.float32, device="cuda")
    offsets = torch.tensor([-5, 10, 4, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    moe.moe_grouped_linear_w4(x, offsets, w, s, z, out=out)
    # expert 0: rows 0 .. 9, expert 1: none, expert 2: 4 .. 39 (over 4 .. 9), expert 3: none
    ref, err = reference(x, w[2], s[2], z[2], None, False, False)
    check(out[10:], ref[10:], err[10:])
    ref, err = reference(x, w[0], s[0], z[0], None, False, False)
    check(out[:4], ref[:4], err[:4])


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [512, 4160])
def test_rows_of_no_expert_take_no_part_in_tiles(out, K):
    """Rows before the first and behind the last expert's, and what the workspace held."""
    import block_fp8_routed_amd as moe
    E, M, N, first, last = 3, 2000, 2048, 37, 911
    w, s, z, b = weights((E,), N, K, 32, 29, bias=True)
    x = activations(M, K, 30)
    assert takes_tiles(M, N, K, out, E)
    offsets = torch.tensor([first, 300, 300, last], dtype=torch.int32).cuda()
    code = moe.MOE_BF16 if out == torch.bfloat16 else moe.MOE_F32
    need = moe.linear_w4_workspace_bytes(M, E, N, K, code)
    got = []
    for fill in (0, 255):
        work = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        y = torch.full((M, N), 5.0, dtype=out, device="cuda")
        rest = x.clone()
        rest[:first] = float("nan") if fill else 1
        rest[last:] = float("nan") if fill else 1
        moe.moe_grouped_linear_w4(rest, offsets, w, s, z, bias=b, out_dtype=out, out=y, workspace=work)
        got.append(y)
    assert torch.equal(*got) and bool((got[0][:first] == 5).all() and (got[0][last:] == 5).all())
    for lo, hi, e in ((first, 300, 0), (300, last, 2)):
        ref, err = reference(x[lo:hi], w[e], s[e], z[e], b[e], False, half=out == torch.bfloat16)
        check(got[0][lo:hi], ref, err)


def test_a_row_does_not_depend_on_the_batch_of_one_kernel():
    """Rows of a batch of one size keep their bits whatever the other rows hold."""
    import block_fp8_routed_amd as moe
    for M, N in ((16, 100), (100, 100), (4100, 700)):
        w, s, z, _ = weights((), N, 512, 64, 16)
        x = activations(M, 512, 17)
        y = x.clone()
        y[M // 2:] = activations(M - M // 2, 512, 18) * 100
        for out in TYPES.values():
            a = moe.moe_linear_w4(x, w, s, z, out_dtype=out)
            b = moe.moe_linear_w4(y, w, s, z, out_dtype=out)
            assert torch.equal(a[:M // 2], b[:M // 2])
            assert torch.equal(b, moe.moe_linear_w4(y, w, s, z, out_dtype=out))


@pytest.mark.parametrize("N,K", [(35, 448), (80, 1024), (16, 2048), (48, 4096), (400, 64), (112, 8320)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_tiles_of_one_stream_are_those_of_calls_of_their_own(N, K, swiglu):
    """An odd number of strips: workgroups go from one tile of 16 rows to the next."""
    import block_fp8_routed_amd as moe
    M = 1000 if N * K < 200_000 else 260
    N += swiglu and N % 2
    w, s, z, _ = weights((), N, K, 64 if K % 64 == 0 else 32, 19, zeros=N % 3 == 0)
    x = activations(M, K, 20)
    assert not takes_tiles(M, N, K, torch.float32)
    whole = moe.moe_linear_w4(x, w, s, z, swiglu=swiglu, out_dtype=torch.float32)
    for r in range(0, M, 16):
        one = moe.moe_linear_w4(x[r:r + 16], w, s, z, swiglu=swiglu, out_dtype=torch.float32)
        assert torch.equal(whole[r:r + 16], one), r
    for _ in range(5):
        assert torch.equal(whole, moe.moe_linear_w4(x, w, s, z, swiglu=swiglu, out_dtype=torch.float32))


def test_offsets_that_fall_count_no_row_twice_over():
    """Offsets back and forth claim every row for every second expert: calls end, and
    what lies outside the rows stays (which expert a row gets is not said)."""
    import block_fp8_routed_amd as moe
    E, M, N, K = 200, 90, 40, 128
    w, s, z, _ = weights((E,), N, K, 128, 23)
    x = activations(M, K, 24)
    whole = torch.full((M + 8, N), 6.0, dtype=torch.float32, device="cuda")
    offsets = torch.tensor([0, M] * (E // 2) + [0], dtype=torch.int32).cuda()
    moe.moe_grouped_linear_w4(x, offsets, w, s, z, out=whole[:M])
    assert bool((whole[M:] == 6).all()) and bool(torch.isfinite(whole).all())


@pytest.mark.parametrize("T,E,k,H,I", [(1, 512, 10, 256, 128), (16, 128, 8, 512, 192), (300, 8, 2, 256, 160),
                                        (2500, 8, 2, 512, 512)])
@pytest.mark.parametrize("share", [False, True])
def test_layer_of_4_bit_experts(T, E, k, H, I, share):
    """dispatch, gate/up with SwiGLU, down, combine, as they are used together; and
    captured, replayed with other inputs beside eager work."""
    import block_fp8_routed_amd as moe
    w1, s1, z1, _ = weights((E,), 2 * I, H, 32, 1, "bf16", True)
    w2, s2, z2, _ = weights((E,), H, I, 32, 2, "bf16", False)
    s1, s2 = s1 * 0.2, s2 * 0.2
    x = activations(T, H, 3)
    idx = torch.from_numpy(choices(T, k, E, 4, "share" if share else "distinct")).cuda()
    gates = torch.rand(T, k, device="cuda")

    def layer():
        rows, offsets, _, inv = moe.moe_dispatch(x, idx, E)
        h = moe.moe_grouped_linear_w4(rows, offsets, w1, s1, z1, swiglu=True)
        y = moe.moe_grouped_linear_w4(h, offsets, w2, s2, z2)
        return h, y, moe.moe_combine(y, gates, inv, out_dtype=torch.float32)

    h, y, out = layer()
    offsets, pair, inv = permutation(idx.cpu().numpy(), E)
    n = int(offsets[-1])
    rows = x[torch.from_numpy(np.maximum(pair, 0).astype(np.int64) // k).cuda()]
    check(h[:n], *(t[:n] for t in grouped_reference(rows, offsets, w1, s1, z1, None, True)))
    # each later step on what the kernels before it gave
    check(y[:n], *(t[:n] for t in grouped_reference(h, offsets, w2, s2, z2, None, False)))
    v = np.where((inv >= 0)[:, :, None], y.double().cpu().numpy()[np.maximum(inv, 0)], 0.0)
    v = v * gates.double().cpu().numpy()[:, :, None]
    check(out, v.sum(axis=1), k * 2.0 ** -24 * np.abs(v).sum(axis=1))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()[2]
    for seed in range(3):
        x.copy_(activations(T, H, 20 + seed))
        idx.copy_(torch.from_numpy(choices(T, k, E, 30 + seed, "share" if share else "any")))
        want = layer()[2]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want)
