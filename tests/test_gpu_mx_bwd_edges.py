"""The backward from 8-bit checkpoints where its kernels could go wrong unseen, on the GPU.

The operators' formulas are evaluated in float64 with torch. Tolerances are counted from the
arithmetic before the bound; U = 2^-24 is half a unit of float32.
"""

import pytest
import torch

import synth_inputs as SI

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_lc_amd as P
    P.lib()
    return P


def layer(P, N, K, d, seed):
    """Codes and mask bits of random proxies, some of them clamped, and A, B; the codes and
    the mask as values too."""
    Wp = SI.make_wp(N, K, seed, DEV, -1.0, 4.0)
    A, B = SI.make_ab(d, seed, DEV)
    packed = torch.empty((N, K // 4), dtype=torch.uint8, device=DEV)
    mask = torch.empty((N, K // 8), dtype=torch.uint8, device=DEV)
    z = torch.empty((N, K), dtype=torch.uint8, device=DEV)
    P.lcvq_quantize(Wp, z, packed, mask)
    bits = torch.arange(8, dtype=torch.uint8, device=DEV)
    m = (mask.unsqueeze(-1) >> bits & 1).view(N, K).bool()
    return packed, mask, A, B, z, m


def checkpoint(P, M, K, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return P.mx_quantize(torch.randn(M, K, generator=g, device=DEV), P.LCVQ_MXINT8)


def few_terms(M, N, seed):
    """dY whose rows hold three values of 8 significant bits each (exact in bfloat16), at
    2^0, 2^-8 and 2^-14: a row's sums are exact or rounded once or twice in float32, and
    the d x d mix is what an error of dX comes from."""
    g = torch.Generator(DEV).manual_seed(seed)
    dY = torch.zeros(M, N, device=DEV)
    at = torch.rand(M, N, generator=g, device=DEV).topk(3, 1)[1]
    v = 1 + torch.randint(0, 128, (M, 3), generator=g, device=DEV) / 128.0
    v *= torch.randint(0, 2, (M, 3), generator=g, device=DEV) * 2 - 1
    return dY.scatter_(1, at, v * torch.tensor([1, 2.0 ** -8, 2.0 ** -14], device=DEV))


# 64 x 64 tiles; 256 x 256 tiles (float32: more than 45000 blocks of 64^3)
@pytest.mark.parametrize("M,N,K", [(300, 320, 256), (4100, 1600, 2432)])
@pytest.mark.parametrize("d", [4, 8, 16])
def test_dx_mix_holds_24_bits(P, M, N, K, d):
    """dX = A C + B r in float32, from C' = dY (2 + z / 2), C = 2 C' - 4 r. C' and r are sums
    of three terms (2 additions, at most 2 U each: 8 U together); the mix's operands hold 24
    bits (2 U each, and the parts' products left out 4 U) and its sums are at most 12
    additions that count (2 U each): 36 U of the terms' magnitudes."""
    print("dx mix", M, N, K, d, flush=True)
    packed, mask, A, B, z, _ = layer(P, N, K, d, 5 * d)
    dY = few_terms(M, N, M + d)
    got = P.linear_bwd_ckpt8(dY, *checkpoint(P, M, K, 1), packed, mask, A, B, d)["dX"].double()
    y, zd, Ad, Bd = dY.double(), z.double(), A.double(), B.double()
    C = (y @ zd).view(M, K // d, d)
    V = (y @ (2 + zd / 2)).view(M, K // d, d)
    r = y.sum(1).view(M, 1, 1)
    ref = C @ Ad.t() + Bd * r
    mag = (2 * V.abs() + 4 * r.abs()) @ Ad.abs().t() + Bd.abs() * r.abs()
    worst = float(((got.view_as(ref) - ref).abs() / mag).max())
    print(f"  {worst / U:.1f} U", flush=True)
    assert worst <= 36 * U


@pytest.mark.parametrize("M,N,K", [(300, 320, 256), (4100, 1600, 2432)])
def test_dx_of_float32_takes_one_dy(P, M, N, K):
    """float32 dY goes into the products as a bfloat16 pair, about 16 bits. With A = I, B = 0
    and one value per row, a multiple of 2^-20 below 2, every step of dX = z (hi + lo) is
    exact (21 bits of the pair, 3 of a code); a row sum of the whole float32 dY would leave 4
    times the rest of the pair in every element, codes 0 too."""
    print("float32 dx", M, N, K, flush=True)
    d = 8
    packed, mask, _, _, z, _ = layer(P, N, K, d, 3)
    A, B = torch.eye(d, device=DEV), torch.zeros(d, device=DEV)
    g = torch.Generator(DEV).manual_seed(8)
    at = torch.randint(0, N, (M, 1), generator=g, device=DEV)
    v = torch.randint(-(1 << 21) + 1, 1 << 21, (M, 1), generator=g, device=DEV) / 2.0 ** 20
    dY = torch.zeros(M, N, device=DEV).scatter_(1, at, v)
    hi = v.to(BF).float()
    pair = hi + (v - hi).to(BF).float()
    assert (pair != v).any()
    got = P.linear_bwd_ckpt8(dY, *checkpoint(P, M, K, 1), packed, mask, A, B, d)["dX"]
    assert torch.equal(got, z[at.view(-1)].float() * pair)
