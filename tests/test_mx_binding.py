"""The block-scaled binding: what it needs of torch, and of a workspace."""

import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "_cuda_getCurrentRawStream"


@pytest.fixture(scope="module")
def built():
    import bit_weight_only_lc_amd as P
    if not os.path.exists(P.LIB_PATH):
        from bit_weight_only_lc_amd import build
        build.build()


def test_import_without_the_raw_stream(built):
    """The import, the sizes and the refusals of the C ABI need no GPU and no stream."""
    code = (f"import torch\nif hasattr(torch._C, '{NAME}'): del torch._C.{NAME}\n"
            "import bit_weight_only_lc_amd as P\n"
            "assert P.lcvq_linear_bwd_ckpt8_workspace_size(16, 256, 256, 8) > 0\n"
            "assert P.lib().lcvq_mxfp4_gemv(None, 1, 1, 32, None, None, None, None) == 1\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("M,N,K", [(1, 64, 14336), (16, 1, 32), (64, 4096, 14336),
                                   (4096, 4096, 4096), (1 << 20, 1 << 16, 4096), (0, 5, 64)])
def test_product_needs_no_workspace(built, M, N, K):
    import bit_weight_only_lc_amd as P
    assert P.lcvq_mxfp4_gemm_workspace_size(M, N, K) == 0


def test_profile_hook_ids_of_the_products(built):
    """Ids 20 to 25 name their kernels; none lies on either side (no GPU call)."""
    import bit_weight_only_lc_amd as P
    for kid in range(13, 33):
        assert P.lib().lcvq_profile_next(kid, None, None) == (0 if 20 <= kid <= 25 else 2)


@pytest.mark.gpu
def test_product_ignores_its_workspace():
    """NULL, one byte and a large workspace give the same bytes, and leave it as it is."""
    import bit_weight_only_lc_amd as P
    X, W = (P.mx_quantize(torch.randn(r, 512, device="cuda"), P.LCVQ_MXFP4) for r in (70, 90))
    Y = torch.empty(70, 90, dtype=torch.bfloat16, device="cuda")
    P.lcvq_mxfp4_gemm(*X, *W, Y)
    for n in (1, 1 << 20):
        ws, Z = torch.full((n,), 7, dtype=torch.uint8, device="cuda"), torch.zeros_like(Y)
        P.lcvq_mxfp4_gemm(*X, *W, Z, ws)
        assert torch.equal(Y, Z) and bool((ws == 7).all())


@pytest.mark.gpu
def test_both_ways_name_the_same_stream():
    import bit_weight_only_lc_amd as P
    assert P._raw_stream is not P._current_stream
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            i = torch.cuda.current_device()
            assert P._raw_stream(i) == P._current_stream(i) == s.cuda_stream
