"""Every tile of the grouped kernels, whole and split along k: each case states
the plan that it is to reach and fails when the planner takes another one (the
plans are also compared without a GPU, tests/test_host_plans.py).  References
in 64 bits, from the definitions.

Tolerances.  INT8: the int32 sum is exact, its conversion and two products round
by 2^-24 each, the output by 2^-8.  W4A16: at most K fp32 additions and a few more
where the sum is split, each rounding by 2^-24 of a running magnitude below
sum |x w|; a tensor-core step adds 16 products at once, so K / 16 + 64 additions,
doubled for the sums inside a step; the output rounds by 2^-8.  One-hot rows have
one term, so they return the bf16 weights unchanged.  h: gate and up as above
(silu moves by |gate| of its argument's error), silu's power 2^-24 |gate| and
2^-22, quotient 2^-22, product 2^-24, then 2^-8."""
from types import SimpleNamespace

import pytest
import torch

pytestmark = pytest.mark.gpu

# (row counts of the experts, K, N, (tile rows, tile columns, split along k))
W8A8 = [
    ([1, 0, 15, 9], 128, 16, (16, 128, False)),
    ([0, 1], 2048, 16, (16, 128, True)),
    ([16, 15, 17] * 12, 128, 272, (16, 256, False)),
    ([1, 17, 9, 17, 3, 9, 3, 0, 17, 16, 3, 17, 17, 9, 17, 15, 9, 8, 15, 3, 17, 17, 3, 17, 17, 1, 17, 16, 8, 0, 3], 896, 1024,
     (16, 256, True)),
    ([32, 31, 33, 32] * 8, 128, 272, (32, 128, False)),
    ([33, 32, 31] * 8, 2048, 144, (32, 128, True)),
    ([32, 31, 33] * 12, 128, 272, (32, 256, False)),
    ([32, 33, 31, 33, 32, 32, 33, 33, 33, 32, 32, 32, 33, 33, 33, 32, 32, 31, 33, 33, 32, 32, 31, 33, 33, 33, 31, 31, 33, 33,
      32, 32, 31, 32, 32], 896, 640, (32, 256, True)),
    ([65, 64, 63, 64] * 8, 128, 272, (64, 128, False)),
    ([65, 63, 65, 65, 33, 32, 1, 33, 17, 33, 64, 32, 65, 128], 1152, 1024, (64, 128, True)),
    ([64, 65, 63] * 12, 128, 272, (64, 256, False)),
    ([65, 64, 65, 65, 65, 64, 65, 64, 64, 65, 64, 65, 65, 65, 63, 64, 65, 64, 65, 64, 63, 65, 65, 65, 64], 896, 1024,
     (64, 256, True)),
    ([128, 127, 129, 128] * 8 + [64, 65, 63], 384, 272, (128, 128, False)),
    ([1500, 300, 1500, 1500, 300, 128, 1000, 1, 1500, 1500, 65, 1], 7168, 16, (128, 128, True)),
    ([128, 127, 129, 128] * 9 + [64, 65, 63], 256, 272, (128, 256, False)),
    ([1, 127, 129, 65, 256, 256, 1, 1, 129, 64, 128, 3, 128, 129, 3, 127, 64, 3, 17, 65, 128, 129, 129, 127, 129, 1, 3, 17,
      128, 127, 64, 64, 128, 256, 127, 129, 65, 64, 17, 3], 2048, 640, (128, 256, True)),
]
# (row counts, H, I, plan of the gate_up product)
GATE_UP = [
    ([1, 0, 17, 16], 128, 256, (16, 128, False)),
    ([1], 1152, 128, (16, 128, True)),
    ([32, 33, 31] * 7, 128, 384, (32, 128, False)),
    ([16, 1, 17, 17, 3, 32, 64, 32, 1, 16, 0, 17, 17], 2048, 128, (32, 128, True)),
    ([65, 64, 63, 64] * 8 + [65, 64], 128, 256, (64, 128, False)),
    ([32, 63, 65, 3, 3, 3, 1, 3, 33, 3, 65, 17, 1, 64, 1, 128, 33, 63, 1, 65, 33, 128, 17, 128, 33], 896, 640,
     (64, 128, True)),
    ([128, 127, 129, 128] * 8 + [128, 129, 64], 256, 256, (128, 128, False)),
    ([1, 127, 1, 17, 1, 1, 129, 127, 128, 129, 17, 17, 17, 17, 127, 17, 129, 65, 129, 17, 256, 127, 3, 3, 0, 3], 1152, 640,
     (128, 128, True)),
]
# tiles of at most 32, 64, 96 and more rows take activation boxes of their own
W4A16 = [
    ([9, 0, 16, 17, 1], 64, 64, (16, 128, False)),
    ([3], 1344, 64, (16, 128, True)),
    ([32, 31, 33, 32] * 8, 64, 192, (32, 128, False)),
    ([1, 33, 17, 17, 1, 17, 3, 17, 0, 0, 1, 16, 3, 16, 64, 1, 0, 17, 0, 3, 17, 17, 0], 2112, 64, (32, 128, True)),
    ([64, 63, 65, 64] * 8, 64, 192, (64, 128, False)),
    ([33, 3, 3, 3, 0, 128, 65, 1, 63, 1, 3, 1, 3, 33, 3, 17, 64, 17, 33, 63, 0, 1], 2112, 192, (64, 128, True)),
    ([127, 1, 127, 65, 129, 1, 65, 127, 17, 64, 0, 64, 17, 127, 0, 129, 65, 64, 256, 1, 256, 128, 17, 256, 256, 65, 128,
      0], 64, 320, (128, 128, False)),
    ([128, 1, 17, 1, 256, 129, 17, 17, 3, 17, 256, 128, 65, 1, 17, 129, 17, 64, 1, 17, 256, 0, 1, 0, 17, 0, 128, 127], 1344,
     640, (128, 128, True)),
    ([1, 97, 96, 64, 129, 33, 1, 129, 32, 129, 0, 33, 192, 97, 0, 33, 97, 1, 191, 33, 0, 191, 65, 32, 0, 65], 64, 640,
     (192, 128, False)),
    ([60, 1, 385, 10, 10, 96, 10, 129, 64, 1, 96, 10, 32], 1344, 1280, (192, 128, True)),
]


@pytest.fixture(scope="module")
def m():
    from moe_linear_layers_w4a8_b200 import _build
    _build.build()
    import moe_linear_layers_w4a8_b200 as mm
    mm.load_library()
    return mm


def ends(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def reached(p):
    return p["tile_rows"], p["tile_cols"], p["range"] > 0


def random_int8(E, K, N, g):
    q = torch.randint(-127, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    return q, (0.5 + torch.rand(E, N, generator=g, device="cuda")) / 100


def random_rows(R, K, g):
    q = torch.randint(-127, 128, (R, K), generator=g, device="cuda", dtype=torch.int8)
    return q, 0.5 + torch.rand(R, generator=g, device="cuda")


@pytest.mark.parametrize("counts,K,N,plan", W8A8)
def test_w8a8(m, counts, K, N, plan):
    g = torch.Generator(device="cuda").manual_seed(K + N)
    at, E, d = ends(counts), len(counts), m.WDesc(8, 1, K, K, N, 1)
    assert reached(m.w8a8_grouped_plan(at, d)) == plan
    qw, sw = random_int8(E, K, N, g)
    q, sx = random_rows(at[-1], K, g)
    st = m.new_status("cuda")
    Y = m.w8a8_grouped_gemm(q, sx, torch.tensor(at, dtype=torch.int32, device="cuda"), m.PackedW8(qw, sw, d, E), status=st)
    assert m.w4a8_get_device_status(st) == 0
    for e in range(E):
        r = slice(at[e], at[e + 1])
        want = sx[r, None].double() * (sw[e].double() * (q[r].double() @ qw[e].double().T))
        assert ((Y[r].double() - want).abs() <= want.abs() * (2.0 ** -8 + 4 * 2.0 ** -24)).all(), f"expert {e}"


@pytest.mark.parametrize("counts,H,I,plan", GATE_UP)
def test_w8a8_gate_up(m, counts, H, I, plan):
    g = torch.Generator(device="cuda").manual_seed(H + I)
    at, E = ends(counts), len(counts)
    R, d1, d2 = at[-1], m.WDesc(8, 1, H, H, 2 * I, 1), m.WDesc(8, 1, I, I, H, 1)
    assert reached(m.w8a8_grouped_plan(at, d1, gate_up=True)) == plan
    qw, sw = random_int8(E, H, 2 * I, g)
    sw = sw * (10.0 / (127 * H ** 0.5))           # gates of a few units
    w1 = m.PackedW8(qw, sw, d1, E)
    w2 = m.PackedW8(torch.zeros(E, H, I, dtype=torch.int8, device="cuda"), torch.ones(E, H, device="cuda"), d2, E)
    X = torch.randn(R, H, generator=g, device="cuda").bfloat16()
    q, sx, _ = m.w4a8_quant_act(X)
    ids = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    st = m.new_status("cuda")
    need = int(m.load_library().w8a8_moe_experts_workspace_size(R, E, d1, d2))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    m.w8a8_moe_experts(X, ids, w1, w2, workspace=ws, status=st)
    assert m.w4a8_get_device_status(st) == 0
    # h lies where the W4A8 layer of the same sizes keeps it
    lay = m.w4a8_moe_workspace_layout(R, E, 1, SimpleNamespace(desc=m.WDesc(4, 1, 64, H, 2 * I, 1)),
                                      SimpleNamespace(desc=m.WDesc(4, 1, 64, I, H, 1)))
    h = ws[lay["h"]:lay["h"] + 2 * R * I].view(torch.bfloat16).view(R, I).double()
    for e in range(E):
        r = slice(at[e], at[e + 1])
        y = sx[r, None].double() * (sw[e].double() * (q[r].double() @ qw[e].double().T))
        gate, up = y[:, :I], y[:, I:]
        want = gate / (1 + torch.exp(-gate)) * up
        rel = 2.0 ** -8 + 2.0 ** -24 * (10 + 4 * gate.abs()) + 2.0 ** -21
        assert ((h[r] - want).abs() <= want.abs() * rel + 1e-30).all(), f"expert {e}"


def random_int4(E, K, N, group, sym, g):
    """Packed codes, scales, zero-points, and the bf16 weights [E, K, N] that they stand for."""
    q = torch.randint(-7, 8, (E, K, N), generator=g, device="cuda") if sym else \
        torch.randint(0, 16, (E, K, N), generator=g, device="cuda")
    G = K // group
    s = (0.5 + torch.rand(E, G, N, generator=g, device="cuda")) / 100
    z = None if sym else torch.randint(0, 16, (E, G, N), generator=g, device="cuda", dtype=torch.uint8)
    v = q.double() if sym else q.double() - z.double().repeat_interleave(group, 1)
    w = (v * s.double().repeat_interleave(group, 1)).float().bfloat16()
    # block (n / 64, group), 16 bytes for (32 k, column): byte b has k = b below and k = b + 16 above
    c = (q & 15).view(E, G, group // 32, 2, 16, N // 64, 64).permute(0, 5, 1, 2, 6, 3, 4)
    packed = (c[..., 0, :] | (c[..., 1, :] << 4)).to(torch.uint8).reshape(E, K * N // 2).contiguous()
    return packed, s, z, w


@pytest.mark.parametrize("group,sym", [(64, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("counts,K,N,plan", W4A16)
def test_w4a16(m, counts, K, N, plan, group, sym):
    if K % group:
        K += 64
    g = torch.Generator(device="cuda").manual_seed(K + N + group)
    at, E, d = ends(counts), len(counts), m.WDesc(4, int(sym), group, K, N, 1)
    assert reached(m.w4a16_grouped_plan(at, d)) == plan
    packed, s, z, w = random_int4(E, K, N, group, sym, g)
    pw, off, R = m.PackedWeight(packed, s, z, d, E), torch.tensor(at, dtype=torch.int32, device="cuda"), at[-1]
    st = m.new_status("cuda")
    X = torch.randn(R, K, generator=g, device="cuda").bfloat16()
    Y = m.w4a16_grouped_gemm(X, off, pw, status=st)
    # one-hot rows, k by k through the rows of an expert and on through the next
    k = (torch.arange(R, device="cuda") * 37) % K
    hot = torch.nn.functional.one_hot(k, K).bfloat16()
    same = m.w4a16_grouped_gemm(hot, off, pw, status=st)
    assert m.w4a8_get_device_status(st) == 0
    bound = 2 * (K / 16 + 64) * 2.0 ** -24
    for e in range(E):
        r = slice(at[e], at[e + 1])
        x, we = X[r].double(), w[e].double()
        want, size = x @ we, x.abs() @ we.abs()
        assert ((Y[r].double() - want).abs() <= 1.01 * bound * size + 2.0 ** -8 * want.abs()).all(), f"expert {e}"
        assert torch.equal(same[r], w[e][k[r]]), f"weights of expert {e}"
