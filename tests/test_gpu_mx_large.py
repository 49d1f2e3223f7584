"""Block-scaled operators on matrices of more than 2^31 elements, on the GPU: offsets beyond
32 bits, and more blocks than one round of a grid. Parts on either side of the limits and at
the ends are compared with float64."""

import numpy as np
import pytest
import torch

import mx_reference as R
from test_gpu_mx_bwd_edges import held

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_lc_amd as P
    P.lib()
    return P


def host(t):
    return t.detach().cpu().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(shape, dt, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.empty(shape, dtype=dt, device=DEV).normal_(generator=g)


# 4.3 G elements: codes beyond 2^31 (MXFP4) and 2^32 (MXINT8) bytes, bfloat16 beyond 2^33
M, K = 131080, 32800
ROWS = torch.tensor([0, 1, 65472, 65473, 65474, 130945, 130946, M - 1])   # 2^31, 2^32 / K


@pytest.mark.parametrize("fmt", [R.FP4, R.INT8])
def test_quantise_and_decode(P, fmt):
    X = normal((M, K), BF, 1)
    c, s = P.mx_quantize(X, fmt)
    rc, rs = R.quantize(f64(X[ROWS]), fmt)
    assert (host(c[ROWS]) == rc).all() and (host(s[ROWS]) == rs).all()
    X.fill_(7)
    P.lcvq_mx_dequantize(c, s, fmt, X)
    assert (f64(X[ROWS]) == R.dequantize(rc, rs, fmt)).all()


def test_gate(P):
    """Tolerances as in test_gpu_mx.py: half a unit of bfloat16, 1e-6 of the terms."""
    G, U = normal((M, K), BF, 2), normal((M, K), BF, 3)
    out = P.silu_gate_fwd(G, U)
    g, u, H = f64(G[ROWS]), f64(U[ROWS]), f64(out["H"][ROWS])
    half = 2.0 ** -8 * 1.01
    ref = R.silu_gate(g, u)
    assert (np.abs(H - ref) <= (half + 1e-6) * np.abs(ref) + 1e-36).all()
    for n, v in (("G8", g), ("U8", u), ("H8", H)):
        rc, rs = R.quantize(v, R.INT8)
        assert (host(out[n][0][ROWS]) == rc).all() and (host(out[n][1][ROWS]) == rs).all(), n
    dG, dU = P.silu_gate_bwd(out["H"], out["G8"], out["U8"])
    g, u = (R.dequantize(*(host(t[ROWS]) for t in out[n]), R.INT8) for n in ("G8", "U8"))
    rG, rU = R.silu_gate_grad(H, g, u)
    s = 1 / (1 + np.exp(-g))
    mag = np.abs(H * u) * s * (1 + abs(g) * (1 - s))
    assert (np.abs(f64(dU[ROWS]) - rU) <= (half + 1e-6) * np.abs(rU) + 1e-36).all()
    assert (np.abs(f64(dG[ROWS]) - rG) <= half * np.abs(rG) + 1e-6 * mag + 1e-36).all()


def weight(N, K, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    packed = torch.randint(0, 256, (N, K // 4), generator=g, device=DEV, dtype=torch.uint8)
    mask = torch.randint(0, 256, (N, K // 8), generator=g, device=DEV, dtype=torch.uint8)
    return packed, mask


def unpack(t, bits):
    """Codes or mask bits of packed rows, as float64."""
    shift = torch.arange(0, 8, bits, dtype=torch.uint8, device=DEV)
    return (t.unsqueeze(-1) >> shift & (1 << bits) - 1).flatten(1).double()


def mixes(d, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return 0.02 * torch.eye(d, device=DEV) + 0.002 * torch.randn(d, d, generator=g, device=DEV), \
        0.01 * torch.randn(d, generator=g, device=DEV)


def test_backward_of_a_large_weight(P):
    """2.2 G weights: dWp beyond 2^33 bytes. Rows of dWp on either side of 2^31 elements, and
    columns of dX at both ends, at the float32 and bfloat16 tolerances of the smaller layers."""
    tokens, N, K, d = 70, 46592, 46592, 8
    packed, mask = weight(N, K, 1)
    A, B = mixes(d, 2)
    dY = normal((tokens, N), BF, 3)
    xc, xs = P.mx_quantize(normal((tokens, K), BF, 4), R.INT8)
    got = P.linear_bwd_ckpt8(dY, xc, xs, packed, mask, A, B, d)
    X = P.mx_dequantize(xc, xs, R.INT8, F32).double()
    y, Ad = dY.double(), A.double()
    rows = torch.tensor([0, 1, 46090, 46091, 46092, 46093, N - 2, N - 1], device=DEV)  # 2^31 / K
    g = (y[:, rows].t() @ X).view(-1, d)
    held(got["dWp"][rows], (g @ Ad).view(len(rows), K) * unpack(mask[rows], 1), 1e-5, "dWp")
    for k0 in (0, K // 2, K - 1024):
        z = unpack(packed[:, k0 // 4:k0 // 4 + 256], 2)
        W = (z.view(-1, d) @ Ad.t() + B.double()).view(N, 1024)
        held(got["dX"][:, k0:k0 + 1024], y @ W, 2.0 ** -8 * 1.01, f"dX {k0}")
    x = X.view(tokens, -1, d)
    held(got["dB"], (y.sum(1).view(-1, 1) * x.sum(1)).sum(0), 1e-5, "dB")
    dA = torch.zeros(d, d, dtype=torch.float64, device=DEV)
    for k0 in range(0, K, 2912):
        yz = y @ unpack(packed[:, k0 // 4:(k0 + 2912) // 4], 2)
        dA += X[:, k0:k0 + 2912].reshape(-1, d).t() @ yz.view(-1, d)
    held(got["dA"], dA, 1e-5, "dA")


def test_backward_over_many_tokens(P):
    """600000 tokens of 4096 values: checkpoint and dX beyond 2^31 elements. dWp and the sums
    run over all of them; dX rows on either side of 2^31 elements and at the end."""
    tokens, N, K, d = 600000, 64, 4096, 8
    packed, mask = weight(N, K, 5)
    A, B = mixes(d, 6)
    dY = normal((tokens, N), BF, 7)
    xc, xs = P.mx_quantize(normal((tokens, K), BF, 8), R.INT8)
    got = P.linear_bwd_ckpt8(dY, xc, xs, packed, mask, A, B, d)
    z, Ad = unpack(packed, 2), A.double()
    W = (z.view(-1, d) @ Ad.t() + B.double()).view(N, K)
    rows = torch.tensor([0, 524286, 524287, 524288, 524289, tokens - 1], device=DEV)  # 2^31 / K
    held(got["dX"][rows], dY[rows].double() @ W, 2.0 ** -8 * 1.01, "dX")
    G = torch.zeros(N, K, dtype=torch.float64, device=DEV)
    for m in range(0, tokens, 50000):
        X = P.mx_dequantize(xc[m:m + 50000], xs[m:m + 50000], R.INT8, F32)
        G += dY[m:m + 50000].double().t() @ X.double()
    g = G.view(-1, d)
    # sums of 600000 terms in four parts, each of 2350 steps of 64 tokens that are rounded to
    # float32: 2350 half units of the sums' size, 1.4e-4, at the very worst
    held(got["dWp"], (g @ Ad).view(N, K) * unpack(mask, 1), 1.4e-4, "dWp")
    held(got["dA"], g.t() @ z.view(-1, d), 1.4e-4, "dA")
    held(got["dB"], g.sum(0), 1.4e-4, "dB")
