"""The backward from 8-bit checkpoints where its kernels could go wrong unseen, on the GPU.

The operators' formulas are evaluated in float64 with torch. Tolerances are counted from the
arithmetic before the bound; U = 2^-24 is half a unit of float32.
"""

import time

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


def launches_prologue(P, call):
    """Whether call() took the 256 x 256 tiles, whose prologue the library's profiling hook
    knows (id 6): its two events lie 20 ms apart before."""
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    time.sleep(0.02)
    b.record()
    torch.cuda.synchronize()
    assert P.lib().lcvq_profile_next(6, a.cuda_event, b.cuda_event) == 0
    call()
    assert P.lib().lcvq_profile_next(6, None, None) == 0
    torch.cuda.synchronize()
    return a.elapsed_time(b) < 15


def held(got, ref, tol, label):
    """floatcheck's three figures (tensor, 32 x 32 blocks, elements), on the GPU."""
    got = got.double().view(-1, got.shape[-1])
    ref = ref.view_as(got)
    assert bool(torch.isfinite(got).all()), label
    e = got - ref
    rms = float(ref.square().mean().sqrt())

    def blocks(x):
        x = torch.nn.functional.pad(x.square(), (0, -x.shape[1] % 32, 0, -x.shape[0] % 32))
        return x.view(x.shape[0] // 32, 32, -1, 32).sum((1, 3)).sqrt()

    den = blocks(ref).maximum(1e-3 * rms * blocks(torch.ones_like(ref)))
    figures = (float(e.norm() / ref.norm()), float((blocks(e) / den).max()),
               float((e.abs() / (ref.abs() + 4 * rms)).max()))
    print(f"  {label} {figures[0]:.1e} {figures[1]:.1e} {figures[2]:.1e}", flush=True)
    assert max(figures) <= tol, (label, figures)


def carried(dY):
    """The values the products take for dY: float32 as a bfloat16 pair."""
    hi = dY.to(BF).float()
    return (hi + (dY.float() - hi).to(BF).float()).double()


def formulas(dY, X, z, m, A, B, d):
    y, zd, Ad = carried(dY), z.double(), A.double()
    N, K = z.shape
    What = (zd.view(-1, d) @ Ad.t() + B.double()).view(N, K)
    G = y.t() @ X
    g = G.view(-1, d)
    return {"dX": y @ What, "dWp": (g @ Ad).view(N, K) * m, "dA": g.t() @ zd.view(-1, d),
            "dB": g.sum(0)}


# The kernels that a layer takes, by the launch rules:
#   dW in 256 x 256 tiles: more than 128 of them, one workgroup per tile; up to 128, split over
#     the tokens, with a second launch; more than 256, a multiple of 8, that leave a last round
#     at most half full, from 961 tokens on, the last ones split
#   dX in the same tiles; 64 x 64 tiles for both up to 60000 blocks of 64^3, float32 45000
UNSPLIT, SPLIT, TAIL = (1030, 3904, 4032), (4100, 1600, 2432), (1030, 4544, 4096)
LARGE = [(s, d, dt) for s in (UNSPLIT, SPLIT, TAIL) for d in (4, 8, 16) for dt in (BF, F32)]
SMALL = [((70, 192, 320), d, dt) for d in (4, 8, 16) for dt in (BF, F32)] + \
        [((2050, 2112, 1984), d, BF) for d in (4, 8, 16)] + \
        [((4100, 1344, 2048), d, F32) for d in (4, 8, 16)]       # (bfloat16: two tiles of dY per workgroup)


def run(P, shape, d, dt, want_dx=True):
    M, N, K = shape
    print("bwd", shape, d, dt, "" if want_dx else "without dX", flush=True)
    packed, mask, A, B, z, m = layer(P, N, K, d, M + d)
    g = torch.Generator(DEV).manual_seed(M)
    dY = torch.randn(M, N, generator=g, device=DEV).to(dt)
    xc, xs = checkpoint(P, M, K, 2)
    out = {}

    def call():
        out.update(P.linear_bwd_ckpt8(dY, xc, xs, packed, mask, A, B, d, want_dx))
    large = launches_prologue(P, call)
    first = {n: t.clone() for n, t in out.items() if t is not None}
    call()
    assert all(torch.equal(out[n], t) for n, t in first.items())
    X = P.mx_dequantize(xc, xs, P.LCVQ_MXINT8, F32).double()
    ref = formulas(dY, X, z, m, A, B, d)
    # exact products and operands of 24 bits: float32 sums of up to 4608 terms, 1e-5 is 100
    # units of their result's size; bfloat16 dX is rounded once more, by half a unit
    for n, t in first.items():
        held(t, ref[n], 2.0 ** -8 * 1.01 if n == "dX" and dt == BF else 1e-5, n)
    return large


@pytest.mark.parametrize("shape,d,dt", LARGE)
def test_large_layers(P, shape, d, dt):
    assert run(P, shape, d, dt)


@pytest.mark.parametrize("shape,d,dt", SMALL)
def test_layers_of_few_tiles(P, shape, d, dt):
    assert not run(P, shape, d, dt)


# without dX the rule counts dW's tiles of 64 x 64 too: 1536 of them; float32 20000 blocks
@pytest.mark.parametrize("shape,d,dt,large", [((70, 2496, 2496), 8, BF, False),
                                              ((70, 2560, 2560), 16, BF, True),
                                              ((1, 2560, 2560), 8, BF, True),
                                              ((1000, 2048, 2496), 4, F32, False),
                                              ((1030, 2048, 2496), 8, F32, True),
                                              ((1030, 4544, 4096), 8, BF, True)])
def test_without_dx(P, shape, d, dt, large):
    assert run(P, shape, d, dt, want_dx=False) == large


@pytest.mark.parametrize("shape", [(70, 192, 320), (2050, 2112, 1984), UNSPLIT, SPLIT, TAIL])
@pytest.mark.parametrize("d", [8, 16])
def test_nan_block_of_a_checkpoint(P, shape, d):
    """It reaches dWp of its 32 columns, all of dA and dB, and nothing else: dX and the other
    columns are those of the same call without it."""
    M, N, K = shape
    print("nan block", shape, d, flush=True)
    packed, mask, A, B, _, m = layer(P, N, K, d, 7)
    g = torch.Generator(DEV).manual_seed(M)
    dY = torch.randn(M, N, generator=g, device=DEV).to(BF)
    xc, xs = checkpoint(P, M, K, 4)
    xc[M - 1, 96:128] = 0
    want = P.linear_bwd_ckpt8(dY, xc, xs, packed, mask, A, B, d)
    xs[M - 1, 3] = 255
    got = P.linear_bwd_ckpt8(dY, xc, xs, packed, mask, A, B, d)
    assert torch.equal(got["dX"], want["dX"])
    block = torch.zeros(K, dtype=torch.bool, device=DEV)
    block[96:128] = True
    assert torch.equal(got["dWp"][:, ~block], want["dWp"][:, ~block])
    assert bool(torch.isnan(got["dWp"][:, block][m[:, block]]).all())
    assert bool(torch.isnan(got["dA"]).all()) and bool(torch.isnan(got["dB"]).all())
