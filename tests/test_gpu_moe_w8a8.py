"""The MoE layer with INT8 experts (w8a8_moe_grouped_gemm, w8a8_moe_experts,
w4a8_moe_dispatch) against 64-bit references and against its own pieces."""
import numpy as np
import pytest
import torch

import oracle as O
from synth import gen_expert_weight, gen_moe_activations
from tests._util import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from moe_linear_layers_w4a8_b200 import _build
    _build.build()
    import moe_linear_layers_w4a8_b200 as mm
    mm.load_library()
    return mm


class Layer:
    def __init__(self, m, E, H, I, seed):
        self.E, self.H, self.I = E, H, I
        mk = lambda which, K, N: lambda e: gen_expert_weight(seed, e, which, K, N, outlier_p=0.001).cuda()  # noqa: E731
        self.w1 = m.w8a8_pack_expert_weights(mk(0, H, 2 * I), E, H, 2 * I, "cuda")
        self.w2 = m.w8a8_pack_expert_weights(mk(1, I, H), E, I, H, "cuda")

    def rows64(self, X_bits, ids, device="cpu"):
        """y of row r through expert ids[r] in 64 bits, with the layer's two
        roundings in between (h to bf16, h to INT8 codes); no bf16 output."""
        q, s, _, _ = O.quant_act(X_bits)
        y = np.zeros((len(ids), self.H))
        for e in np.unique(ids):
            r = np.nonzero(ids == e)[0]
            gu, _, _ = O.w8a8_exact(q[r], s[r], self.w1.q_w[e].cpu().numpy().T, self.w1.s_w[e].cpu().numpy())
            gate, up = gu[:, :self.I], gu[:, self.I:]
            h = O.f64_to_bf16(gate / (1 + np.exp(-gate)) * up)
            qh, sh, _, _ = O.quant_act(h)
            y[r], _, _ = O.w8a8_exact(qh, sh, self.w2.q_w[e].cpu().numpy().T, self.w2.s_w[e].cpu().numpy())
        return y


def rel_rms(got, ref):
    return np.sqrt(np.mean((got - ref) ** 2) / max(np.mean(ref ** 2), 1e-300))


CASES = [
    # (T, E, topk, H, I, zipf)
    (1, 64, 6, 512, 256, None),
    (1, 1, 1, 128, 128, None),
    (2, 8, 8, 256, 128, None),
    (64, 32, 8, 512, 384, 1.1),
    (333, 13, 3, 1152, 640, 1.1),
    (300, 512, 2, 128, 128, None),
    (700, 4, 2, 384, 1408, None),
]


@pytest.mark.parametrize("T,E,topk,H,I,zipf", CASES)
def test_layer(m, T, E, topk, H, I, zipf):
    layer = Layer(m, E, H, I, seed=T + E)
    inp = gen_moe_activations(T, H, E, seed=T * 3 + E, zipf=zipf)
    X, logits = inp.X.cuda(), inp.logits.cuda()
    st = m.new_status("cuda")
    r = m.w8a8_moe_grouped_gemm(X, logits, topk, layer.w1, layer.w2, status=st)
    assert m.w4a8_get_device_status(st) == 0
    idx, wts = m.w4a8_moe_route(logits, topk)
    assert torch.equal(r["topk_idx"], idx) and torch.equal(r["topk_w"], wts)
    offsets, perm, inv = m.w4a8_moe_dispatch(idx, E)
    assert torch.equal(r["expert_offsets"], offsets)
    flat = idx.reshape(-1).cpu().numpy()
    assert np.array_equal(perm.cpu().numpy(), np.argsort(flat, kind="stable"))
    assert np.array_equal(inv.cpu().numpy()[perm.cpu().numpy()], np.arange(T * topk))
    assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(np.sort(flat), np.arange(E + 1)))
    # 64-bit layer on a sample of tokens.  A value of h next to a bf16 tie may
    # round the other way in fp32, and its INT8 code may move by one: 1/127 of
    # the row's largest for a few values, well below 1e-2 of the output's RMS.
    tok = np.unique(np.linspace(0, T - 1, 24).astype(int))
    y = layer.rows64(np.repeat(bits(inp.X)[tok], topk, axis=0), idx.cpu().numpy()[tok].reshape(-1))
    y = O.bf16_to_f32(O.f64_to_bf16(y)).astype(np.float64).reshape(len(tok), topk, H)
    ref = (wts.cpu().numpy().astype(np.float64)[tok][:, :, None] * y).sum(1)
    got = O.bf16_to_f32(bits(r["out"]))[tok].astype(np.float64)
    assert rel_rms(got, ref) <= 1e-2


@pytest.mark.parametrize("R,E,I", [
    (1, 3, 128), (40, 3, 256), (130, 2, 384), (600, 4, 128),
    (4, 1, 1024), (40, 2, 2048), (1200, 20, 1024), (1200, 4, 1664),      # split along k, tiles of 16 to 128 rows
])
def test_gate_up_stage(m, R, E, I):
    """w2 = the identity in codes of 127 and scales of 1/127, so that a row
    comes out as its quantized h: y = s_h q_h / 127 * 127.  The INT8 code of h
    is at most half a step (s_h = max|h| / 127) off, the fp32 products
    2^-22 of it, y one bf16 rounding; h itself was rounded to bf16 once (and
    with it max|h|: 2^-8 of the half step).  Its fp32 value is within 2^-16
    (__expf's error grows with its argument: 2 + 1.2 |x| units of 2^-23, |x| <
    87): the rest of the half step's 2^-7, max|h| 2^-8 / 254, covers that."""
    layer = Layer(m, E, I, I, seed=R + I)
    layer.w2.q_w.zero_()
    layer.w2.q_w[:, torch.arange(I), torch.arange(I)] = 127
    layer.w2.s_w.fill_(1.0 / 127.0)
    inp = gen_moe_activations(R, I, E, seed=R)
    ids = torch.randint(0, E, (R,), generator=torch.Generator().manual_seed(R), dtype=torch.int32)
    st = m.new_status("cuda")
    y = m.w8a8_moe_experts(inp.X.cuda(), ids.cuda(), layer.w1, layer.w2, status=st)
    assert m.w4a8_get_device_status(st) == 0
    y = O.bf16_to_f32(bits(y)).astype(np.float64)
    q, s, _, _ = O.quant_act(bits(inp.X))
    for e in range(E):
        r = np.nonzero(ids.numpy() == e)[0]
        if len(r) == 0:
            continue
        gu, _, _ = O.w8a8_exact(q[r], s[r], layer.w1.q_w[e].cpu().numpy().T, layer.w1.s_w[e].cpu().numpy())
        h = gu[:, :I] / (1 + np.exp(-gu[:, :I])) * gu[:, I:]
        top = np.abs(h).max(1, keepdims=True)
        tol = top / 254 * (1 + 2.0 ** -7) + np.abs(h) * (2 * 2.0 ** -8 + 2.0 ** -19)
        assert (np.abs(y[r] - h) <= tol).all()


def test_experts_equal_layer_rows(m):
    """Routing, experts and combine as separate calls (the expert-parallel
    layer with one rank) give the layer's result bit for bit."""
    from moe_linear_layers_w4a8_b200.ep import ExpertParallelMoE
    for T, E, topk, H, I in [(200, 16, 4, 256, 128), (7, 8, 2, 512, 384)]:
        layer = Layer(m, E, H, I, seed=T)
        inp = gen_moe_activations(T, H, E, seed=T, zipf=1.1)
        X, logits = inp.X.cuda(), inp.logits.cuda()
        r = m.w8a8_moe_grouped_gemm(X, logits, topk, layer.w1, layer.w2)
        out, idx, w = ExpertParallelMoE(E, layer.w1, layer.w2).forward(X, logits, topk)
        assert torch.equal(out, r["out"]) and torch.equal(idx, r["topk_idx"]) and torch.equal(w, r["topk_w"])


def test_grouped_products_compose_to_the_layer(m):
    """The pieces as a user strings them together: route, dispatch, gather,
    grouped gate_up, silu * up, grouped down, combine.  gate_up leaves as bf16
    here and stays fp32 in the layer (one more rounding of 2^-8 of each)."""
    T, E, topk, H, I = 150, 8, 2, 512, 256
    layer = Layer(m, E, H, I, seed=3)
    inp = gen_moe_activations(T, H, E, seed=3)
    X, logits = inp.X.cuda(), inp.logits.cuda()
    idx, w = m.w4a8_moe_route(logits, topk)
    offsets, perm, inv = m.w4a8_moe_dispatch(idx, E)
    rows = X[torch.div(perm, topk, rounding_mode="floor").long()]
    gu = m.w8a8_grouped_linear(rows, offsets, layer.w1).float()
    h = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).bfloat16()
    y = m.w8a8_grouped_linear(h, offsets, layer.w2)
    out = m.w4a8_moe_combine(y[inv.long()], w)
    want = m.w8a8_moe_grouped_gemm(X, logits, topk, layer.w1, layer.w2)["out"]
    assert rel_rms(out.float().cpu().numpy(), want.float().cpu().numpy()) <= 1e-2


def test_bad_ids_and_values_are_reported(m):
    layer = Layer(m, 4, 128, 128, seed=1)
    X = torch.randn(6, 128).bfloat16().cuda()
    st = m.new_status("cuda")
    m.w8a8_moe_experts(X, torch.tensor([0, 1, 2, 3, 4, -1]).cuda(), layer.w1, layer.w2, status=st)
    assert m.w4a8_get_device_status(st) == 1
    for ids in ([0, 9], [0, 2 ** 32], [-2 ** 40, 1]):
        st = m.new_status("cuda")
        m.w4a8_moe_dispatch(torch.tensor(ids).cuda(), 4, status=st)
        assert m.w4a8_get_device_status(st) == 1
    logits = torch.randn(6, 4).cuda()
    for bad in ("x", "logits"):
        Xb, Lb = X.clone(), logits.clone()
        (Xb if bad == "x" else Lb)[3, 2] = float("nan")
        st = m.new_status("cuda")
        m.w8a8_moe_grouped_gemm(Xb, Lb, 2, layer.w1, layer.w2, status=st)
        assert m.w4a8_get_device_status(st) == 4


@pytest.mark.parametrize("T", [3, 40])
def test_two_streams_with_their_own_workspaces(m, T):
    layer = Layer(m, 8, 256, 128, seed=4)
    inp = gen_moe_activations(T, 256, 8, seed=1)
    X, logits = inp.X.cuda(), inp.logits.cuda()
    want = m.w8a8_moe_grouped_gemm(X, logits, 2, layer.w1, layer.w2)["out"]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(m.w8a8_moe_grouped_gemm(X, logits, 2, layer.w1, layer.w2)["out"])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


def test_layer_captured(m):
    layer = Layer(m, 8, 256, 128, seed=2)
    inp = gen_moe_activations(5, 256, 8, seed=1)
    X, logits = inp.X.cuda(), inp.logits.cuda()
    ws = torch.empty(m.w8a8_moe_workspace_size(5, 8, 2, layer.w1, layer.w2), dtype=torch.uint8, device="cuda")
    out = torch.empty(5, 256, dtype=torch.bfloat16, device="cuda")
    m.w8a8_moe_grouped_gemm(X, logits, 2, layer.w1, layer.w2, workspace=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = m.w8a8_moe_grouped_gemm(X, logits, 2, layer.w1, layer.w2, workspace=ws, out=out)
    for seed in range(3):
        new = gen_moe_activations(5, 256, 8, seed=seed + 5)
        X.copy_(new.X)
        logits.copy_(new.logits)
        g.replay()
        want = m.w8a8_moe_grouped_gemm(new.X.cuda(), new.logits.cuda(), 2, layer.w1, layer.w2)
        assert torch.equal(out, want["out"]) and torch.equal(r["topk_idx"], want["topk_idx"])


def test_refusals_of_the_binding(m):
    layer = Layer(m, 4, 128, 128, seed=1)
    X, L = torch.randn(6, 128).bfloat16().cuda(), torch.randn(6, 4).cuda()

    def refused(code, *a, **k):
        with pytest.raises(m.W4A8Error) as e:
            m.w8a8_moe_grouped_gemm(*a, **k)
        assert e.value.code == code

    refused(1, X.float(), L, 2, layer.w1, layer.w2)
    refused(1, X, L.half(), 2, layer.w1, layer.w2)
    refused(1, X, L[:5], 2, layer.w1, layer.w2)
    refused(1, X, torch.randn(6, 5).cuda(), 2, layer.w1, layer.w2)
    refused(1, X, L, 5, layer.w1, layer.w2)
    refused(1, X, L, 0, layer.w1, layer.w2)
    refused(3, X, L, 2, layer.w2, layer.w2)
    refused(1, X, L, 2, layer.w1, layer.w2, out=torch.empty(6, 128, device="cuda"))
    r = m.w8a8_moe_grouped_gemm(X[:0], L[:0], 2, layer.w1, layer.w2)
    assert r["out"].shape == (0, 128) and (r["expert_offsets"] == 0).all()
    with pytest.raises(m.W4A8Error):
        m.w8a8_moe_experts(X, torch.zeros(5, dtype=torch.int32, device="cuda"), layer.w1, layer.w2)
