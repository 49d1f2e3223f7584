"""The MXFP4 products where their kernels could go wrong unseen, on the GPU, against float64.

Tolerance, as in test_gpu_mx.py: float32 sums of K terms, at worst K 2^-23 of the sum of the
terms' magnitudes, and half a unit of bfloat16 (2^-8) of the result. Y lies between guard
values that start right at its first and behind its last element.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
PAD = 1024                       # guard elements on either side of Y


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


def product(P, M, N, K, dt, seed=0):
    label = f"gemm {M}x{N}x{K} {dt}"
    print(label, flush=True)
    (xc, xs), (wc, ws) = (P.mx_quantize(values(r, K, seed + r), P.LCVQ_MXFP4) for r in (M, N))
    Y, buf = guarded(M, N, dt)
    P.lcvq_mxfp4_gemm(xc, xs, wc, ws, Y)
    held(Y, buf, decode(xc, xs), decode(wc, ws), label)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(33, 1, 64), (33, 17, 1024), (49, 1, 4128), (65, 65, 544)])
def test_waves_past_the_matrix(P, M, N, K, dt):
    """Tiles whose later waves have no row of W, of X, or of either."""
    product(P, M, N, K, dt)


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
