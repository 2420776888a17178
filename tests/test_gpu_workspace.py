"""A workspace that is not GPU memory, or not all there (host tensors, expanded or strided ones), is
refused by every entry that takes one; one of any element type counts by its bytes."""
import pytest
import torch

import bit_block_scaled_quantize_amd as nv
from bit_block_scaled_quantize_amd.moe import MoETokens
from helpers import log

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _calls():
    """Each entry with a workspace as a function of it, and the bytes it needs."""
    x = torch.randn(256, 512, device="cuda").bfloat16()
    big = torch.randn(4096, 64, device="cuda").bfloat16()
    q, b = nv.quantize(x)[0], nv.quantize(big)[0]
    p = torch.ones(64, device="cuda")
    plan = nv.AdamWPlan([nv.AdamWTensor(p=p, grad=p.clone(), m=p.clone(), v=p.clone())])
    w = torch.randn(4, 32, 64, device="cuda").bfloat16()
    moe = MoETokens.from_bf16(torch.randn(4, 64, device="cuda"), w, w.transpose(1, 2).contiguous(), 2)
    dbias = torch.zeros(512, device="cuda")
    return {
        "quantize": (lambda ws: nv.quantize(x, workspace=ws), nv.workspace_size(nv.OP_QUANTIZE, 256, 512)),
        "rht_rows_quantize": (lambda ws: nv.rht_rows_quantize(x, 1, workspace=ws), nv.workspace_size(nv.OP_QUANTIZE, 256, 512)),
        "rht_quantize": (lambda ws: nv.rht_quantize(x, 1, workspace=ws), nv.workspace_size(nv.OP_RHT_QUANTIZE, 256, 512)),
        "amax": (lambda ws: nv.amax(x, workspace=ws), nv.workspace_size(nv.OP_QUANTIZE, 256, 512)),
        "amax_pair": (lambda ws: nv.amax_pair(x, 1, workspace=ws), nv.workspace_size(nv.OP_AMAX_PAIR, 256, 512)),
        "gemm_ex": (lambda ws: nv.gemm_ex(q, q, workspace=ws), nv.workspace_size(nv.OP_GEMM_EX, 256, 256)),
        "gemm_act": (lambda ws: nv.gemm_act(b, b, workspace=ws), nv.workspace_size(nv.OP_GEMM_ACT, 4096, 4096, 64)),
        "act_grad": (lambda ws: nv.act_grad(x, dbias=dbias, workspace=ws), nv.workspace_size(nv.OP_ACT_GRAD, 256, 512)),
        "adamw": (lambda ws: nv.adamw(plan, 1e-3, max_norm=1.0, workspace=ws), nv.workspace_size(nv.OP_ADAMW, 0, 0)),
        "moe_tokens": (lambda ws: nv.moe_tokens(x[:3, :64], moe.weights, workspace=ws), moe.workspace.numel()),
    }


def test_workspaces():
    for name, (call, need) in _calls().items():
        log(f"workspace of {name}: {need} bytes")
        n = max(need, 256)
        for bad in (torch.zeros((n,), dtype=torch.uint8), torch.zeros((1,), dtype=torch.uint8, device="cuda").expand(n),
                    torch.zeros((2 * n,), dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(nv.NVFP4Error, match="workspace"):
                call(bad)
        call(torch.zeros(((n + 3) // 4,), device="cuda"))
        torch.cuda.synchronize()
