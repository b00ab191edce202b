"""silu(gate) * up of the INT8 MoE layer over the whole range of gates, h read
from the workspace before it is quantized.

Tolerance: gate and up are three fp32 roundings each (2^-24), one of the
gate's moved by silu's slope: relative |gate| of it; the power's argument is
rounded once (2^-24 of |gate|), the power 2^-22, and where numbers are
subnormal 2^-149 absolute (power times gate, product, quotient); quotient and product 2^-22 and 2^-24; then one bf16 rounding, 2^-8."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import oracle as O
from tests._util import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from moe_linear_layers_w4a8_b200 import _build
    _build.build()
    import moe_linear_layers_w4a8_b200 as mm
    mm.load_library()
    return mm


@pytest.mark.parametrize("lo,hi", [(-104.0, -80.0), (-90.0, -85.0), (-60.0, 60.0), (80.0, 120.0), (-2.0, 2.0)])
@pytest.mark.parametrize("R", [5, 128])
def test_silu_times_up(m, R, lo, hi):
    """One-hot rows with codes of 127, so that gate[r, i] = c[r] 127 s_w[i]."""
    H = I = 128
    rows = torch.linspace(0.875, 1.0, R).bfloat16()
    X = torch.zeros(R, H, dtype=torch.bfloat16)
    X[:, 0] = rows
    gates = torch.linspace(lo, hi, I)
    q1 = torch.zeros(1, 2 * I, H, dtype=torch.int8)
    q1[0, :I, 0] = torch.where(gates < 0, -127, 127).to(torch.int8)
    q1[0, I:, 0] = torch.where(torch.arange(I) % 3 == 0, -127, 127).to(torch.int8)
    s1 = torch.cat([gates.abs() / 127, torch.full((I,), 2.0 ** 20)])[None].contiguous()
    w1 = m.PackedW8(q1.cuda(), s1.cuda(), m.WDesc(8, 1, H, H, 2 * I, 1), 1)
    w2 = m.PackedW8(torch.zeros(1, H, I, dtype=torch.int8, device="cuda"), torch.ones(1, H, device="cuda"),
                    m.WDesc(8, 1, I, I, H, 1), 1)
    need = int(m.load_library().w8a8_moe_workspace_size(R, 1, 1, w1.desc, w2.desc))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    st = m.new_status("cuda")
    m.w8a8_moe_grouped_gemm(X.cuda(), torch.zeros(R, 1, device="cuda"), 1, w1, w2, workspace=ws, status=st)
    assert m.w4a8_get_device_status(st) == 0
    # h lies where the W4A8 layer of the same sizes keeps it
    at = m.w4a8_moe_workspace_layout(R, 1, 1, SimpleNamespace(desc=m.WDesc(4, 1, 64, H, 2 * I, 1)),
                                     SimpleNamespace(desc=m.WDesc(4, 1, 64, I, H, 1)))["h"]
    h = O.bf16_to_f32(bits(ws[at:at + 2 * R * I].view(torch.bfloat16).view(R, I))).astype(np.float64)
    qx, sx, _, _ = O.quant_act(bits(X))
    y, _, _ = O.w8a8_exact(qx, sx, q1[0].numpy().T, s1[0].numpy())
    gate, up = y[:, :I], y[:, I:]
    want = gate / (1 + np.exp(-gate)) * up
    rel = 2.0 ** -8 + 2.0 ** -24 * (10 + 4 * np.abs(gate)) + 2.0 ** -21
    assert (np.abs(h - want) <= np.abs(want) * rel + (np.abs(gate) + 2) * np.abs(up) * 2.0 ** -149).all()
