"""Grouped W8A8 products (rows sorted by expert, ragged) against the oracle.

int32 sums are exact, so the only errors are fp32: the conversion of the sum
and two products (3 * 2^-24 relative) before one bf16 rounding, which stays
within 1 bf16 ulp of the correctly rounded exact value (check_bf16).  The same
arithmetic runs in w8a8_gemm, so each expert's rows must equal it bit for bit."""
import numpy as np
import pytest
import torch

import oracle as O
from synth import gen_linear
from tests._util import bits, check_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from moe_linear_layers_w4a8_b200 import _build
    _build.build()
    import moe_linear_layers_w4a8_b200 as mm
    mm.load_library()
    return mm


def _weights(m, E, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    return m.w8a8_pack_expert_weights(
        lambda e: (torch.randn(K, N, generator=g) * 0.02).cuda(), E, K, N, "cuda")


def _offsets(counts, front=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + front, dtype=torch.int32, device="cuda")


def _one(w, e, m):
    return m.PackedW8(q_w=w.q_w[e], s_w=w.s_w[e], desc=w.desc)


CASES = [
    # (counts, K, N, rows in front, rows behind)
    ([1], 128, 16, 0, 0),                              # one row, one k-block, one piece
    ([0, 1, 0], 256, 256, 0, 0),
    ([0, 0, 0], 256, 64, 0, 5),                        # nobody has rows
    ([1, 1, 1, 1, 1, 1], 2048, 2816, 0, 0),            # a token's six rows: few tiles, split
    ([16, 17, 0, 15, 3], 512, 528, 0, 0),              # around one 16-row tile
    ([33, 1, 64, 65, 2, 0, 31], 384, 1040, 2, 9),      # BN = 32, ragged, rows of nobody
    ([64, 63, 65, 1, 128, 129, 0, 50], 640, 272, 0, 3),  # BN = 64
    ([200, 128, 127, 129, 1], 1152, 400, 1, 1),        # BN = 128
    ([1000], 256, 48, 0, 0),                           # one expert takes every row
    ([3] * 200, 128, 128, 0, 0),                       # many experts
    ([1] * 512, 128, 32, 0, 0),                        # the most experts
    ([5, 0, 90], 7168, 144, 0, 0),                     # long k, few tiles: split with many parts
    ([300, 20, 0, 700], 1408, 2048, 0, 0),
    # tiles of 16 and 32 rows, one box of columns or two, split along k or whole
    ([4], 2048, 208, 0, 0),
    ([1] * 20, 896, 2304, 0, 0),
    ([192] * 12, 128, 64, 0, 0),
    ([40] * 20, 4096, 64, 1, 1),
    ([4] * 16, 128, 2304, 0, 0),
    ([100] * 40, 896, 192, 0, 0),
]


@pytest.mark.parametrize("counts,K,N,front,behind", CASES)
def test_grouped_gemm(m, counts, K, N, front, behind):
    E, used = len(counts), sum(counts)
    R = front + used + behind
    inp = gen_linear(max(R, 1), K, 16, seed=K + N + used)
    w = _weights(m, E, K, N, seed=E * 7 + K)
    st = m.new_status("cuda")
    q, sx, _ = m.w4a8_quant_act(inp.X.cuda()[:R], status=st)
    off = _offsets(counts, front)
    out = torch.full((R, N), -7.0, dtype=torch.bfloat16, device="cuda")
    Y = m.w8a8_grouped_gemm(q, sx, off, w, out=out, status=st)
    assert Y is out and m.w4a8_get_device_status(st) == 0
    qo, so = q.cpu().numpy(), sx.cpu().numpy()
    at = front
    for e, n in enumerate(counts):
        if n:
            rows = slice(at, at + n)
            Ye, A, _ = O.w8a8_exact(qo[rows], so[rows], w.q_w[e].cpu().numpy().T, w.s_w[e].cpu().numpy())
            check_bf16(bits(Y[rows]), Ye, A, what=f"expert {e}")
            assert torch.equal(Y[rows], m.w8a8_gemm(q[rows], sx[rows].clone(), _one(w, e, m)))
        at += n
    # rows of nobody are left as they were
    assert (out[:front] == -7).all() and (out[front + used:] == -7).all()
    # the bf16 entry gives the same
    out2 = torch.full_like(out, -7.0)
    m.w8a8_grouped_linear(inp.X.cuda()[:R], off, w, out=out2, status=st)
    assert m.w4a8_get_device_status(st) == 0 and torch.equal(out2, out)


@pytest.mark.parametrize("counts,K,N", [
    ([192] * 24, 128, 64), ([192] * 24, 2048, 64), ([60] * 40, 128, 320), ([192] * 24, 2048, 192),       # 64 rows
    ([250] * 40, 256, 64), ([120] * 40, 256, 320), ([300, 20, 0, 700, 129] * 5, 256, 768), ([500] * 40, 1664, 128),   # 128
])
def test_taller_tiles_equal_the_dense_product(m, counts, K, N):
    """Tiles of 64 and 128 rows, one box of columns or two, split along k or
    whole: every expert's rows bit for bit as w8a8_gemm gives them."""
    w = _weights(m, len(counts), K, N, seed=len(counts))
    R = sum(counts)
    X = torch.randn(R, K, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    q, sx, _ = m.w4a8_quant_act(X)
    Y = m.w8a8_grouped_gemm(q, sx, _offsets(counts), w)
    at = 0
    for e, n in enumerate(counts):
        if n:
            assert torch.equal(Y[at:at + n], m.w8a8_gemm(q[at:at + n].clone(), sx[at:at + n].clone(), _one(w, e, m)))
        at += n


def test_layer_size_sampled_experts(m):
    """The prompt shape of a 64-expert layer: 24576 rows, K = 1408, N = 2048."""
    g = torch.Generator().manual_seed(3)
    counts = torch.bincount(torch.randint(0, 64, (24576,), generator=g), minlength=64).tolist()
    w = _weights(m, 64, 1408, 2048, seed=1)
    X = torch.randn(24576, 1408, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    Y = m.w8a8_grouped_linear(X, _offsets(counts), w)
    at = 0
    for e, n in enumerate(counts):
        if e in (0, 31, 63):
            assert torch.equal(Y[at:at + n], m.w8a8_linear(X[at:at + n].contiguous(), _one(w, e, m)))
        at += n


def test_rows_of_nobody_may_hold_anything(m):
    w = _weights(m, 3, 256, 64, seed=2)
    X = torch.randn(20, 256, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    want = m.w8a8_grouped_linear(X[2:14].contiguous(), _offsets([5, 0, 7]), w)
    X[:2], X[14:] = float("nan"), float("inf")
    st = m.new_status("cuda")
    out = torch.full((20, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    m.w8a8_grouped_linear(X, _offsets([5, 0, 7], 2), w, out=out, status=st)
    assert m.w4a8_get_device_status(st) == 0
    assert torch.equal(out[2:14], want) and (out[:2] == 3).all() and (out[14:] == 3).all()
    # in a row that is used it is reported
    X[5, 17] = float("nan")
    m.w8a8_grouped_linear(X, _offsets([5, 0, 7], 2), w, out=out, status=st)
    assert m.w4a8_get_device_status(st) == 4


def test_strided_rows_and_outputs(m):
    w = _weights(m, 4, 384, 80, seed=5)
    wide = torch.randn(50, 400, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    X, off = wide[:, :384], _offsets([20, 0, 29, 1])
    want = m.w8a8_grouped_linear(X.contiguous(), off, w)
    for pitch in (80, 88, 83, 200):       # 16-byte rows or not
        buf = torch.full((50, pitch), 9.0, dtype=torch.bfloat16, device="cuda")
        m.w8a8_grouped_linear(X, off, w, out=buf[:, :80])
        assert torch.equal(buf[:, :80], want) and (buf[:, 80:] == 9).all()
    buf = torch.full((50 * 80 + 1,), 9.0, dtype=torch.bfloat16, device="cuda")
    m.w8a8_grouped_linear(X, off, w, out=buf[1:].view(50, 80))   # not 16-byte aligned
    assert torch.equal(buf[1:].view(50, 80), want) and buf[0] == 9


@pytest.mark.parametrize("off", [[0, 5, 3, 12], [-1, 2, 4, 12], [0, 4, 8, 13], [12, 0, 12, 5], [0, 2**31 - 1, 5, 6]])
def test_bad_offsets_are_reported(m, off):
    w = _weights(m, 3, 128, 32, seed=6)
    q, sx, _ = m.w4a8_quant_act(torch.randn(12, 128).bfloat16().cuda())
    st = m.new_status("cuda")
    guard = torch.full((14, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    m.w8a8_grouped_gemm(q, sx, torch.tensor(off, dtype=torch.int32, device="cuda"), w, out=guard[1:13], status=st)
    assert m.w4a8_get_device_status(st) == 1
    assert (guard[0] == 5).all() and (guard[13] == 5).all()


def test_workspace_contents_and_order_do_not_matter(m):
    """Split launches: a workspace full of anything, reused by other shapes,
    gives the same bits every time."""
    shapes = [([1, 1, 2, 1], 2048, 512), ([5, 0, 90, 1], 1024, 144), ([16] * 4, 512, 640)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    todo = []
    for counts, K, N in shapes:
        w = _weights(m, len(counts), K, N, seed=K)
        q, sx, _ = m.w4a8_quant_act(torch.randn(sum(counts), K, generator=torch.Generator().manual_seed(1)).bfloat16().cuda())
        assert 0 < m.w8a8_grouped_workspace_size(sum(counts), w) <= ws.numel()
        todo.append((q, sx, _offsets(counts), w, m.w8a8_grouped_gemm(q, sx, _offsets(counts), w).clone()))
    for fill in (0, 255, None):
        if fill is None:
            ws.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(9))
        else:
            ws.fill_(fill)
        for _ in range(20):
            for q, sx, off, w, want in todo:
                assert torch.equal(m.w8a8_grouped_gemm(q, sx, off, w, workspace=ws), want)


def test_captured_and_eager_calls_share_a_workspace(m):
    """Two graphs and eager calls on one stream, one workspace; offsets change
    between replays."""
    w = _weights(m, 4, 2048, 512, seed=8)
    X = torch.randn(24, 2048, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    off = _offsets([1, 2, 3, 4])
    need = m.w8a8_grouped_linear_workspace_size(24, w)
    ws = torch.randint(0, 255, (need,), dtype=torch.uint8, device="cuda")
    out_a, out_b = (torch.zeros(24, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.w8a8_grouped_linear(X, off, w, out=out_a, workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for out in (out_a, out_b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.w8a8_grouped_linear(X, off, w, out=out, workspace=ws)
        graphs.append(g)
    for counts in ([1, 2, 3, 4], [0, 24, 0, 0], [6, 6, 6, 6], [0, 0, 0, 1]):
        new = _offsets(counts)
        want = m.w8a8_grouped_linear(X, new, w, out=torch.zeros_like(out_a))
        off.copy_(new)
        for g, out in zip(graphs, (out_a, out_b)):
            out.zero_()
            g.replay()
            g.replay()
            eager = m.w8a8_grouped_linear(X, off, w, out=torch.zeros_like(out), workspace=ws)
            assert torch.equal(out, want) and torch.equal(eager, want)


def test_two_streams_with_their_own_workspaces(m):
    w = _weights(m, 8, 2048, 1024, seed=10)
    X = torch.randn(8, 2048, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    off = _offsets([1] * 8)
    want = m.w8a8_grouped_linear(X, off, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(30):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(m.w8a8_grouped_linear(X, off, w))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


@pytest.mark.parametrize("R,K,N", [((1 << 17) + 5, 128, 16400), ((1 << 17) + 5, 16512, 16)])
def test_more_than_2_31_elements(m, R, K, N):
    """Offsets into Y and into the rows that pass 32 bits."""
    w = _weights(m, 2, K, N, seed=12)
    q = torch.randint(-127, 128, (R, K), dtype=torch.int8, device="cuda")
    sx = torch.rand(R, device="cuda") + 0.5
    Y = m.w8a8_grouped_gemm(q, sx, _offsets([9, R - 9]), w)
    assert R * max(K, N) > 2 ** 31
    for e, rows in ((0, slice(0, 9)), (1, slice(9, 200)), (1, slice(R - 300, R))):
        assert torch.equal(Y[rows], m.w8a8_gemm(q[rows].contiguous(), sx[rows].clone(), _one(w, e, m)))


def test_offsets_from_the_kernel_before(m):
    """Offsets and rows written on the stream just before the call, over and over."""
    w = _weights(m, 6, 512, 256, seed=13)
    g = torch.Generator().manual_seed(4)
    X = torch.randn(64, 512, generator=g).bfloat16().cuda()
    ids = [torch.randint(0, 6, (64,), generator=g).cuda() for _ in range(8)]
    want = [m.w8a8_grouped_linear(X[p.long()].contiguous(), o, w) for o, p, _ in
            (m.w4a8_moe_dispatch(i, 6) for i in ids)]
    torch.cuda.synchronize()
    off, rows = torch.zeros(7, dtype=torch.int32, device="cuda"), torch.zeros_like(X)
    for _ in range(10):
        for i, ref in zip(ids, want):
            o, p, _ = m.w4a8_moe_dispatch(i, 6)
            rows.copy_(X[p.long()])
            off.copy_(o)
            assert torch.equal(m.w8a8_grouped_linear(rows, off, w), ref)
            off.zero_()


def test_one_row_of_any_stride(m):
    w = _weights(m, 2, 256, 64, seed=14)
    X = torch.randn(3, 256, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    off = _offsets([0, 1])
    want = m.w8a8_grouped_linear(X[:1].contiguous(), off, w)
    out = torch.zeros(64, 2, dtype=torch.bfloat16, device="cuda").t()[:1]
    with pytest.raises(m.W4A8Error):        # columns not adjacent
        m.w8a8_grouped_linear(X[:1], off, w, out=out)
    row = torch.as_strided(torch.zeros(64, dtype=torch.bfloat16, device="cuda"), (1, 64), (1, 1))
    assert torch.equal(m.w8a8_grouped_linear(X[::2][:1], off, w, out=row), want) and torch.equal(row, want)


def test_refusals_of_the_binding(m):
    w = _weights(m, 4, 256, 64, seed=11)
    q, sx, _ = m.w4a8_quant_act(torch.randn(8, 256).bfloat16().cuda())
    off = _offsets([2, 2, 2, 2])

    def refused(f, *a, **k):
        with pytest.raises(m.W4A8Error) as e:
            f(*a, **k)
        assert e.value.code == 1

    refused(m.w8a8_grouped_gemm, q, sx, off.long(), w)
    refused(m.w8a8_grouped_gemm, q, sx, off[:4], w)
    refused(m.w8a8_grouped_gemm, q, sx, off.cpu(), w)
    refused(m.w8a8_grouped_gemm, q, sx[:7], off, w)
    refused(m.w8a8_grouped_gemm, q, sx.half(), off, w)
    refused(m.w8a8_grouped_gemm, q[:, :128].contiguous(), sx, off, w)
    refused(m.w8a8_grouped_gemm, q.float(), sx, off, w)
    refused(m.w8a8_grouped_gemm, q, sx, off, w, out=torch.empty(8, 64, device="cuda"))
    refused(m.w8a8_grouped_gemm, q, sx, off, w, out=torch.empty(64, 8, device="cuda").bfloat16().t())
    refused(m.w8a8_grouped_gemm, q, sx, off, w, status=torch.zeros(1, dtype=torch.int64, device="cuda"))
    refused(m.w8a8_grouped_gemm, q, sx, off, _one(w, 0, m))              # not stacked
    refused(m.w8a8_gemm, q, sx, w)                                       # stacked
    refused(m.w8a8_linear, torch.randn(8, 256).bfloat16().cuda(), w)
    refused(m.w8a8_grouped_linear, torch.randn(8, 256).cuda(), off, w)
    refused(m.w8a8_pack_weights, torch.randn(256, 64).cuda(), out=w, expert=4)
    refused(m.w8a8_pack_weights, torch.randn(256, 64).cuda(), out=w)
    refused(m.w8a8_pack_weights, torch.randn(256, 64).cuda(), expert=0, out=m.PackedW8(
        w.q_w.cpu(), w.s_w.cpu(), w.desc, 4))                            # slots on another device
    refused(m.w8a8_pack_expert_weights, None, 0, 256, 64, "cuda")
    p4 = m.w4a8_pack_expert_weights(lambda e: torch.randn(256, 64).cuda(), 4, 256, 64, 64, True, "cuda")
    refused(m.w8a8_grouped_gemm, q, sx, off, p4)                         # 4-bit experts
    refused(m.w4a16_grouped_gemm, torch.randn(8, 256).bfloat16().cuda(), off, w)
    refused(m.w4a8_moe_dispatch, torch.zeros(4, device="cuda"), 4)
    refused(m.w4a8_moe_dispatch, torch.zeros(4, dtype=torch.int32), 4)
    refused(m.w4a8_moe_dispatch, torch.zeros(4, dtype=torch.bool, device="cuda"), 4)
    # no rows at all
    assert m.w8a8_grouped_gemm(q[:0], sx[:0], torch.zeros_like(off), w).shape == (0, 64)
