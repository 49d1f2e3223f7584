"""The MXFP4 products where their kernels could go wrong unseen, on the GPU, against float64.

Tolerance, as in test_gpu_mx.py: float32 sums of K terms, at worst K 2^-23 of the sum of the
terms' magnitudes, and half a unit of bfloat16 (2^-8) of the result. Y lies between guard
values that start right at its first and behind its last element.
"""

import time

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
PAD = 1024                       # guard elements on either side of Y
# the library's profiling hook names the kernel that a call launches
FEW, T64, T64_128, T128, T256, GEMV = 20, 21, 22, 23, 24, 25


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_lc_amd as P
    P.lib()
    return P


def values(rows, K, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(rows, K, generator=g, device=DEV)
    return x * torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g, device=DEV).float())


def decode(c, s):
    """The float64 values of MXFP4 codes and scale bytes below 255."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=c.device)
    n = torch.stack((c & 15, c >> 4), -1).long().view(c.shape[0], -1, 32)
    v = grid[n & 7] * torch.where(n > 7, -1.0, 1.0)
    return (v * torch.exp2(s.double() - 127).unsqueeze(-1)).flatten(1)


def guarded(M, N, dt):
    """Y [M, N] in the middle of a flat buffer of sevens, and the buffer."""
    buf = torch.full((PAD + M * N + PAD,), 7.0, dtype=dt, device=DEV)
    return buf[PAD:PAD + M * N].view(M, N), buf


def held(Y, buf, X, W, label):
    """Every element of Y against X W^T, and every guard value."""
    assert bool((buf[:PAD] == 7).all()) and bool((buf[PAD + Y.numel():] == 7).all()), label
    half = 2.0 ** -8 * 1.01 if Y.dtype == BF else 0.0
    for r in range(0, Y.shape[0], 512):
        x = X[r:r + 512]
        ref = x @ W.t()
        bound = X.shape[1] * 2.0 ** -23 * (x.abs() @ W.abs().t()) + half * ref.abs()
        bad = (~((Y[r:r + 512].double() - ref).abs() <= bound)).nonzero()
        assert bad.numel() == 0, f"{label}: {len(bad)} elements, first {bad[0].tolist()} + row {r}"


def launches(P, kernel, call):
    """Whether call() launched this kernel: the hook records its two events, which lie 20 ms
    apart before, around the launch."""
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    time.sleep(0.02)
    b.record()
    torch.cuda.synchronize()
    assert P.lib().lcvq_profile_next(kernel, a.cuda_event, b.cuda_event) == 0
    call()
    assert P.lib().lcvq_profile_next(kernel, None, None) == 0
    torch.cuda.synchronize()
    return a.elapsed_time(b) < 15


def product(P, M, N, K, dt, kernel):
    label = f"gemm {M}x{N}x{K} {dt}"
    print(label, flush=True)
    (xc, xs), (wc, ws) = (P.mx_quantize(values(r, K, r), P.LCVQ_MXFP4) for r in (M, N))
    Y, buf = guarded(M, N, dt)
    assert launches(P, kernel, lambda: P.lcvq_mxfp4_gemm(xc, xs, wc, ws, Y)), kernel
    held(Y, buf, decode(xc, xs), decode(wc, ws), label)
    again = torch.empty_like(Y)
    P.lcvq_mxfp4_gemm(xc, xs, wc, ws, again)
    assert torch.equal(again.view(torch.uint8), Y.view(torch.uint8)), label


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(33, 1, 64), (33, 17, 1024), (49, 1, 4128), (65, 65, 544)])
def test_waves_past_the_matrix(P, M, N, K, dt):
    """Tiles whose later waves have no row of W, of X, or of either."""
    product(P, M, N, K, dt, T64)


# Contractions: whole chunks of 512 values; one block, one, three and (15 blocks) four stages
# more; rows of scales on 4-byte boundaries (multiples of 128) and off them.
KS = (1024, 544, 1152, 1408, 2016)
# Rows of Y in 16-byte pieces; odd; even, but no multiple of 8 (bfloat16) or 4 (float32).
TILES = [(T64, 100, 4096), (T64, 70, 4097), (T64, 129, 4098),
         (T64_128, 300, 4096), (T64_128, 259, 4097), (T64_128, 300, 4098),
         (T128, 520, 4000), (T128, 515, 4001), (T128, 530, 4002),
         (T256, 2055, 4104), (T256, 2049, 4101), (T256, 2100, 4098)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("kernel,M,N", TILES)
def test_tiles(P, kernel, M, N, K, dt):
    product(P, M, N, K, dt, kernel)


# 16, 32 and 64 rows of W per workgroup; contractions of one round of the waves, and of more
ROWS = [(100, 2592), (4097, 2592), (5003, 4640), (8192, 544), (8193, 2592), (9002, 4736)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N,K", ROWS)
@pytest.mark.parametrize("M", [1, 16, 17, 32])
def test_few_rows(P, M, N, K, dt):
    product(P, M, N, K, dt, FEW)


@pytest.mark.parametrize("N,K", ROWS)
@pytest.mark.parametrize("M", [1, 4, 5, 16])
def test_decode_product(P, M, N, K):
    label = f"gemv {M}x{N}x{K}"
    print(label, flush=True)
    X, (wc, ws) = values(M, K, M).to(BF), P.mx_quantize(values(N, K, N), P.LCVQ_MXFP4)
    Y, buf = guarded(M, N, BF)
    assert launches(P, GEMV, lambda: P.lcvq_mxfp4_gemv(X, wc, ws, Y))
    held(Y, buf, X.double(), decode(wc, ws), label)


def test_the_hook_tells_kernels_apart(P):
    X, W = (P.mx_quantize(values(r, 64, r), P.LCVQ_MXFP4) for r in (40, 50))
    Y = torch.empty(40, 50, dtype=BF, device=DEV)
    ran = [k for k in (FEW, T64, T64_128, T128, T256, GEMV)
           if launches(P, k, lambda: P.lcvq_mxfp4_gemm(*X, *W, Y))]
    assert ran == [T64]


@pytest.mark.parametrize("M,N", [(12, 5003), (30, 70), (100, 300), (300, 4097), (515, 4001), (2055, 4101)])
def test_nan_blocks_stay_in_their_row_and_column(P, M, N):
    """A NaN block in a whole chunk of X, and one in W's last, partial chunk."""
    K = 1056
    (xc, xs), (wc, ws) = (P.mx_quantize(values(r, K, r), P.LCVQ_MXFP4) for r in (M, N))
    xs[M - 2, 3], ws[N - 3, K // 32 - 1] = 255, 255
    Y = torch.empty(M, N, dtype=F32, device=DEV)
    P.lcvq_mxfp4_gemm(xc, xs, wc, ws, Y)
    want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    want[M - 2], want[:, N - 3] = True, True
    assert torch.equal(torch.isnan(Y), want)


@pytest.mark.parametrize("M", [3, 9])
def test_decode_product_scales_at_the_ends(P, M):
    """W's scale bytes from 0 to 254, one to a row. What lies below the smallest normal float32
    may be flushed; where the terms add up to more than bfloat16 holds the result may be
    infinite."""
    N, K = 255, 416
    g = torch.Generator(DEV).manual_seed(M)
    wc = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV).to(torch.uint8)
    ws = torch.arange(N, device=DEV).to(torch.uint8).view(N, 1).repeat(1, K // 32)
    X = values(M, K, 4).to(BF)
    Y = torch.empty(M, N, dtype=BF, device=DEV)
    P.lcvq_mxfp4_gemv(X, wc, ws, Y)
    x, w = X.double(), decode(wc, ws)
    ref, mag = x @ w.t(), x.abs() @ w.abs().t()
    near = (Y.double() - ref).abs() <= (K * 2.0 ** -23 * mag + 2.0 ** -8 * 1.01 * ref.abs()
                                        + x.abs().sum(1, True) * 2.0 ** -126)
    assert bool((near | (mag >= 2.0 ** 127)).all())


def random_mxfp4(rows, K):
    """Codes and scale bytes at random: values below 2^6, without a float copy of them."""
    g = torch.Generator(DEV).manual_seed(rows)
    c = torch.randint(0, 256, (rows, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    return c, torch.randint(121, 131, (rows, K // 32), generator=g, device=DEV, dtype=torch.uint8)


@pytest.mark.parametrize("M", [1, 16, 40])
def test_offsets_beyond_32_bits_in_the_weight(P, M):
    """5 GiB of codes; rows on either side of 4 GiB and at the end."""
    N, K = 163840, 65536
    wc, ws = random_mxfp4(N, K)
    rows = torch.tensor([0, 1, 131071, 131072, 131073, N - 2, N - 1], device=DEV)
    W = decode(wc[rows], ws[rows])
    c, s = P.mx_quantize(values(M, K, M), P.LCVQ_MXFP4)
    x = P.mx_dequantize(c, s, P.LCVQ_MXFP4)                    # exact in bfloat16
    Y = torch.empty(M, N, dtype=BF, device=DEV)
    for call in ([lambda: P.lcvq_mxfp4_gemv(x, wc, ws, Y)] if M <= 16 else []) + \
                [lambda: P.lcvq_mxfp4_gemm(c, s, wc, ws, Y)]:
        Y.fill_(7)
        call()
        held(Y[:, rows].contiguous(), torch.full((PAD + M * 7 + PAD,), 7.0), x.double(), W, f"{M} rows")


def test_offsets_beyond_32_bits_in_the_output(P):
    """2.5 G elements of Y, 10 GiB of float32."""
    M, N, K = 65537, 40004, 64
    X, W = random_mxfp4(M, K), random_mxfp4(N, K)
    Y = torch.empty(M, N, dtype=F32, device=DEV)
    P.lcvq_mxfp4_gemm(*X, *W, Y)
    rows = torch.tensor([0, 26843, 53685, 53686, 53687, M - 1], device=DEV)   # 2^31 / N = 53681
    held(Y[rows], torch.full((PAD + 6 * N + PAD,), 7.0), decode(*X)[rows], decode(*W), "large Y")


@pytest.mark.parametrize("M", [16, 17, 40])
def test_linear_keeps_its_activations(P, M):
    """mxfp4_linear's activations are those it was given, at any number of rows: against the
    product of X itself (4-bit activations are off by 10% of it), and the same bytes as the
    decode product of each 16 rows."""
    N, K = 200, 416
    X = values(M, K, 5).to(BF)
    W = P.mx_quantize(values(N, K, 6), P.LCVQ_MXFP4)
    Y = P.mxfp4_linear(X, *W)
    Z, buf = guarded(M, N, BF)
    for m in range(0, M, 16):
        P.lcvq_mxfp4_gemv(X[m:m + 16], *W, Z[m:m + 16])
    held(Z, buf, X.double(), decode(*W), f"linear {M}")
    assert torch.equal(Y.view(torch.int16), Z.view(torch.int16))


def test_linear_refuses_rather_than_quantise(P):
    X = values(4, 64, 1)
    W = P.mx_quantize(values(32, 64, 2), P.LCVQ_MXFP4)
    with pytest.raises(TypeError):
        P.mxfp4_linear(X, *W)                       # float32 activations
    Y, Z = P.mxfp4_linear(X, *W, quantize_x=True), torch.empty(4, 32, dtype=BF, device=DEV)
    P.lcvq_mxfp4_gemm(*P.mx_quantize(X, P.LCVQ_MXFP4), *W, Z)
    assert torch.equal(Y, Z)
