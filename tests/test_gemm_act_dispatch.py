"""Which kernel nvfp4_gemm_act takes, by the library's own rule (host code, no GPU)."""
import os

import pytest

import bit_block_scaled_quantize_amd as nv
from test_gpu_gemm_act_tiles import TILES, few_rows


@pytest.fixture(autouse=True)
def _need_library():
    if not os.path.exists(nv.LIB_PATH):
        pytest.skip("libnvfp4.so not built")


def test_the_tile_kernels_tests_reach_it():
    assert not any(few_rows(*mnk) for mnk in TILES)


def test_few_rows():
    """Up to 64 rows always, and without a workspace; beyond by the number of 64 x 32 workgroups."""
    for n in (1, 5120, 10 ** 6):
        for k in (16, 5120, 20480):
            for m in (1, 16, 17, 64):
                assert few_rows(m, n, k) and nv.workspace_size(nv.OP_GEMM_ACT, m, n, k) == 0
    assert few_rows(768, 4089, 192) and not few_rows(769, 4089, 192)
    assert nv.workspace_size(nv.OP_GEMM_ACT, 768, 4089, 208) == 0 < nv.workspace_size(nv.OP_GEMM_ACT, 769, 4089, 208)
