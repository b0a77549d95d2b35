"""int8 products and balance loss without a GPU: workspace sizes over whole ranges, the
binding on a torch build without CUDA."""
import ctypes
import subprocess
import sys

import pytest

from conftest import ROOT
from mixture_experts_ffn_15_b200 import _abi
from mixture_experts_ffn_15_b200.build import build


def _lib():
    build()
    return _abi.load()


def never_shrinks(size, values):
    last = 0
    for v in values:
        n = size(v)
        assert n > 0 and n >= last, (v, n, last)
        last = n


@pytest.mark.parametrize("H,E,I", [(128, 128, 64), (128, 256, 64), (32, 1, 32), (64, 200, 96), (2816, 8, 704)])
def test_a_workspace_of_the_ffn_holds_fewer_rows_too(H, E, I):
    """Also across the row counts at which other kernels take over (8 and 48 per expert)."""
    lib = _lib()
    rows = sorted({r for m in (0, 1, 8, 48) for r in range(max(m * E - 70, 0), m * E + 70)} | set(range(0, 20000, 61)))
    never_shrinks(lambda r: lib.moe_expert_ffn_w8a8_workspace_size(r, H, E, I), rows)
    k = min(8, E)
    never_shrinks(lambda t: lib.moe_w8a8_workspace_size(t, H, E, k, I), range(0, 13000 // k))


@pytest.mark.parametrize("E,S", [(8, 1), (60, 3), (128, 1), (256, 65535)])
def test_a_workspace_of_the_balance_loss_holds_fewer_tokens_too(E, S):
    lib = _lib()
    tokens = sorted(set(range(0, 20000, 7)) | set(range(9400, 9600)) | set(range(0, 6000000, 4999)) |
                    {148 * 1024 * 32 * n + d for n in (1, 2, 3) for d in (-1, 0, 1)})
    never_shrinks(lambda t: lib.moe_balance_loss_workspace_size(t, E, S), tokens)
    never_shrinks(lambda s: lib.moe_balance_loss_workspace_size(5000, E, s), range(1, 3000))
    never_shrinks(lambda e: lib.moe_balance_loss_workspace_size(1 << 24, e, S), range(1, 257))


def test_the_package_imports_on_a_torch_build_without_cuda():
    """Such a build has no _cuda_getCurrentRawStream; the argument checks work all the same."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import mixture_experts_ffn_15_b200 as moe\n"
            "try: moe.quantize_rows(torch.zeros(2, 8))\n"
            "except ValueError as e: assert 'CUDA' in str(e)\n"
            "else: raise SystemExit('not refused')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_sizes_whose_tiles_would_pass_32_bits_are_refused():
    lib, P = _lib(), ctypes.c_void_p(4096)
    inv = _abi.MOE_ERR_INVALID_ARG
    for n in ((1 << 30) + 32, (1 << 31) - 32):
        assert lib.moe_matmul_q8(P, P, P, P, None, None, 4, 16, 1, n, 1, P, None, None) == inv
        assert lib.moe_matmul_q8(P, P, P, P, None, P, 4000, 16, 2, n, 1, P, None, None) == inv
    for t in ((1 << 30) + 1, (1 << 31) - 1):
        assert lib.moe_balance_loss_workspace_size(t, 8, 1) == 0
    assert lib.moe_balance_loss_workspace_size(1 << 30, 8, 1) > 0
