"""w4a8_moe_combine for every batch of slots that it loads together: one at a time,
4 and 8 (one wave of CTAs), 3 (rows from HBM).  Slots are added in order by fp32
fused multiply-adds, each rounding by 2^-24 of a running sum that never exceeds
sum |w y|; the tolerance takes twice that, and one bf16 rounding, 2^-8.  The
order is the same for every batch, so the bits are too."""
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


@pytest.mark.parametrize("topk", list(range(1, 17)))
@pytest.mark.parametrize("T,H", [(1, 8), (3, 136), (37, 2048), (400, 2056), (1000, 1152), (1024, 2048)])
def test_combine(m, T, H, topk):
    g = torch.Generator().manual_seed(T + topk)
    y, w = torch.randn(T * topk, H, generator=g).bfloat16(), torch.rand(T, topk, generator=g)
    out = torch.full((T + 1, H), -7.0, dtype=torch.bfloat16, device="cuda")
    m.w4a8_moe_combine(y.cuda(), w.cuda(), out=out[:T])
    terms = w.numpy().astype(np.float64)[:, :, None] * O.bf16_to_f32(bits(y)).astype(np.float64).reshape(T, topk, H)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    got = O.bf16_to_f32(bits(out[:T])).astype(np.float64)
    assert (np.abs(got - want) <= topk * 2.0 ** -23 * size + 2.0 ** -8 * np.abs(want)).all()
    assert (out[T] == -7).all()
    # the fixed order: the same bits as in a call of few tokens
    pick = sorted({0, T // 2, T - 1})
    rows = torch.cat([y[t * topk:(t + 1) * topk] for t in pick])
    assert torch.equal(m.w4a8_moe_combine(rows.cuda(), w[pick].cuda()), out[pick])


@pytest.mark.parametrize("T,H,topk", [(4096, 2048, 6), (1024, 7168, 7), (700, 7168, 16), (4096, 7168, 2), (4096, 7168, 1)])
def test_combine_of_many_rows(m, T, H, topk):
    """Rows that do not fit L2, against the same tokens a few at a time."""
    g = torch.Generator(device="cuda").manual_seed(T + topk)
    y = torch.randn(T * topk, H, generator=g, device="cuda").bfloat16()
    w = torch.rand(T, topk, generator=g, device="cuda")
    out = m.w4a8_moe_combine(y, w)
    for t0 in list(range(0, T, 32))[:: max(1, T // 1024)]:
        t1 = min(T, t0 + 32)
        assert torch.equal(m.w4a8_moe_combine(y[t0 * topk:t1 * topk], w[t0:t1]), out[t0:t1])
