"""The layer's dispatch by one CTA and by three launches: the same order, and the
number of launches that the library states (and bench.py counts)."""
import numpy as np
import pytest
import torch
from cuda.bindings import runtime as rt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from moe_linear_layers_w4a8_b200 import _build
    _build.build()
    import moe_linear_layers_w4a8_b200 as mm
    mm.load_library()
    return mm


def kernels_of(f):
    """Kernel nodes of one call, captured."""
    f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        f()
    raw = rt.cudaGraph_t(g.raw_cuda_graph())
    err, _, n = rt.cudaGraphGetNodes(raw, 0)
    assert err == rt.cudaError_t.cudaSuccess
    err, nodes, n = rt.cudaGraphGetNodes(raw, n)
    assert err == rt.cudaError_t.cudaSuccess
    return sum(rt.cudaGraphNodeGetType(x)[1] == rt.cudaGraphNodeType.cudaGraphNodeTypeKernel for x in nodes[:n])


@pytest.mark.parametrize("E,topk", [(13, 3), (64, 8), (64, 16), (512, 16)])
@pytest.mark.parametrize("T", [1, 255, 256, 257, 333, 400, 512, 513])
def test_dispatch_order_and_launches(m, T, E, topk):
    H, I = 128, 64
    w1 = m.w4a8_pack_expert_weights(lambda e: torch.full((H, 2 * I), 0.01, device="cuda"), E, H, 2 * I, 64, True, "cuda")
    w2 = m.w4a8_pack_expert_weights(lambda e: torch.full((I, H), 0.01, device="cuda"), E, I, H, 64, True, "cuda")
    g = torch.Generator().manual_seed(T + E)
    X, logits = torch.randn(T, H, generator=g).bfloat16().cuda(), torch.randn(T, E, generator=g).cuda()
    r = {}

    def call():
        r.update(m.w4a8_moe_grouped_gemm(X, logits, topk, w1, w2, workspace=r.get("workspace")))

    assert kernels_of(call) == 6 + m.w4a8_moe_dispatch_launches(T, E, topk)
    call()
    flat = r["topk_idx"].reshape(-1).cpu().numpy()
    lay = m.w4a8_moe_workspace_layout(T, E, topk, w1, w2)
    perm, inv = (r["workspace"][lay[k]:lay[k] + 4 * T * topk].view(torch.int32).cpu().numpy() for k in ("perm", "inv"))
    assert np.array_equal(perm, np.argsort(flat, kind="stable"))
    assert np.array_equal(inv[perm], np.arange(T * topk))
    assert np.array_equal(r["expert_offsets"].cpu().numpy(), np.searchsorted(np.sort(flat), np.arange(E + 1)))
