"""The feed-forward products at the sizes of tests/feed_forward_paths.py, on the GPU against float64."""

import pytest
import torch

import feed_forward_paths as P
from test_gpu_feed_forward import DT, check_grouped, check_linear, check_weight_gradient, lib, operands  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(P.LINEAR)))
def test_linear(lib, case, dtype):  # noqa: F811
    (m, n, k), half, exact = P.LINEAR[case]
    divided = "divided" in (exact if dtype == "f32" else half)
    assert (lib._lib.mxgemm_block128_workspace_bytes(m, n, k, 1, ("f32", "bf16", "f16").index(dtype)) > 0) == divided
    check_linear(lib, m, n, k, DT[dtype], True, "gelu", True, True, True)
    check_linear(lib, m, n, k, DT[dtype], True, "gelu_tanh", True, True, True, bias_f32=True, pad=(5, 1), seed=2)
    check_linear(lib, m, n, k, DT[dtype], False, "silu", True, False, False, 1, 0, seed=5)
    check_linear(lib, m, n, k, DT[dtype], True, None, False, True, False, 0, 1, seed=9)
    check_linear(lib, m, n, k, DT[dtype], True, "relu", False, False, True, pad=(8, 0), seed=11)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(P.GROUPED)))
def test_grouped(lib, case, dtype):  # noqa: F811
    sizes, n, k, head, tail = P.GROUPED[case][0]
    check_grouped(lib, sizes, n, k, DT[dtype], head, tail)
    check_grouped(lib, sizes, n, k, DT[dtype], head, tail, "silu", True, True, index=torch.int64, seed=7)
    check_grouped(lib, sizes, n, k, DT[dtype], head, tail, "gelu", True, True, fa=1, pad=(5, 1), seed=3)
    check_grouped(lib, sizes, n, k, DT[dtype], head, tail, "gelu_tanh", False, True, fb=1, pad=(8, 8), seed=4)


@pytest.mark.parametrize("case", range(len(P.DEEP)))
def test_weight_gradient(lib, case):  # noqa: F811
    sizes, m, n, head, tail = P.DEEP[case][0]
    assert lib._lib.mxgemm_block128_grouped_weight_gradient_workspace_bytes(P.blocks(sizes, head, tail), len(sizes), m, n) > 0
    check_weight_gradient(lib, sizes, m, n, head, tail)
    check_weight_gradient(lib, sizes, m, n, head, tail, fa=0, fb=1, pad=3, index=torch.int64, seed=5)
    check_weight_gradient(lib, sizes[::-1], m, n, tail, head, seed=6)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("m,n,k", [(64, 513, 7168), (100, 500, 4096), (32, 7168, 2048)])
def test_linear_of_parts_is_the_product_of_parts(lib, m, n, k, dtype):  # noqa: F811
    a, sa, b, sb = operands(lib, m, n, k)
    assert torch.equal(lib.block128_linear(a, sa, b, sb, c_dtype=DT[dtype]), lib.block128_gemm(a, sa, b, sb, c_dtype=DT[dtype]))
