"""Grouped W4A16 products (rows sorted by expert, ragged) against the oracle:
the dequantized weight bit-exact (one-hot rows return it unchanged), outputs
within 1 bf16 ulp of the correctly rounded exact value, or within the fp32
accumulation bound where it nearly cancels.

The bound: at most K fp32 additions and, where the sum is split over k, a few
more, each rounding by 2^-24 of a running magnitude that never exceeds
sum |x w|; a tensor-core step adds 16 products at once, so K / 16 + 64
additions, doubled for the sums inside a step."""
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


def fp32_bound(K):
    return 2.0 * (K / 16 + 64) * 2.0 ** -24


def _weights(m, E, K, N, group, sym, seed):
    g = torch.Generator().manual_seed(seed)
    W = [torch.randn(K, N, generator=g) * 0.02 + (0.0 if sym else 0.01) for _ in range(E)]
    w = m.w4a8_pack_expert_weights(lambda e: W[e].cuda(), E, K, N, group, sym, "cuda")
    return w, W


def _dequant(W, group, sym):
    codes, s, z, bad = O.quant_weights(W.numpy(), group, sym)
    assert not bad
    return O.w4a16_dequant(codes, s, None if sym else z, group)


def _offsets(counts, front=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + front, dtype=torch.int32, device="cuda")


def _one(w, e, m):
    return m.PackedWeight(packed=w.packed[e], s_w=w.s_w[e], z=None if w.z is None else w.z[e], desc=w.desc)


CASES = [
    # (counts, K, N, group, symmetric, rows in front, rows behind)
    ([1], 64, 64, 64, True, 0, 0),
    ([0, 1, 0], 128, 128, 128, False, 0, 0),
    ([0, 0], 128, 64, 64, True, 0, 4),
    ([1] * 6, 2048, 2816, 128, True, 0, 0),                 # a token's six rows
    ([2, 0, 3, 1], 1344, 1088, 64, False, 0, 2),            # K % 128 == 64
    ([16, 17, 0, 15, 8, 9, 7], 512, 320, 64, True, 1, 5),   # around small tiles
    ([33, 1, 64, 65, 2, 0, 31], 448, 576, 64, False, 0, 3),
    ([64, 63, 65, 1, 128, 129], 640, 192, 128, True, 3, 0),
    ([256, 257, 5, 255, 300, 511], 384, 128, 128, False, 0, 7),  # 256-row tiles
    ([700], 256, 64, 64, True, 0, 0),
    ([3] * 150, 128, 64, 128, True, 0, 0),
    ([1, 0, 40], 7168, 128, 64, False, 0, 0),               # long k
    ([24, 0, 1], 4096, 64, 128, True, 0, 0),
    ([30], 1024, 64, 128, True, 0, 0),
    ([30], 1088, 64, 64, False, 1, 0),
    # tiles of 32 to 192 rows, split along k or whole
    ([192] * 12, 128, 64, 128, True, 0, 0),
    ([4] * 40, 896, 64, 64, False, 0, 0),
    ([192] * 24, 128, 64, 64, True, 0, 0),
    ([10] * 12, 1024, 320, 128, False, 0, 1),
    ([10] * 24, 128, 768, 128, False, 0, 0),
    ([10] * 24, 1024, 320, 64, True, 0, 0),
    ([20] * 24, 128, 768, 64, False, 1, 0),
    ([20] * 24, 2048, 320, 128, True, 0, 0),
    # with every number of activation boxes
    ([384, 400, 380, 191, 192, 193, 97, 96, 500, 410, 1, 60, 30, 385, 380, 390], 320, 640, 64, False, 0, 2),
    ([193, 0, 192, 191, 97, 96, 65, 64, 33, 32, 1, 500, 10, 128, 2, 31], 320, 1280, 64, False, 2, 0),
    ([193, 0, 192, 191, 97, 96, 65, 64, 33, 32, 1, 500, 10, 128, 2, 31] * 2, 192, 1280, 64, True, 0, 0),
    ([193, 0, 192, 191, 97, 96, 65, 64, 33, 32, 1, 500, 10, 128, 2, 31], 2048, 640, 128, True, 0, 0),
]


@pytest.mark.parametrize("counts,K,N,group,sym,front,behind", CASES)
def test_grouped_gemm(m, counts, K, N, group, sym, front, behind):
    E, used = len(counts), sum(counts)
    R = front + used + behind
    X = gen_linear(R, K, 64, seed=K + N + used).X
    w, W = _weights(m, E, K, N, group, sym, seed=E * 7 + K)
    st = m.new_status("cuda")
    Xc = X.cuda()
    Xc[:front], Xc[front + used:] = float("nan"), float("inf")   # nobody's rows may hold anything
    out = torch.full((R, N), -7.0, dtype=torch.bfloat16, device="cuda")
    Y = m.w4a16_grouped_gemm(Xc, _offsets(counts, front), w, out=out, status=st)
    assert Y is out and m.w4a8_get_device_status(st) == 0
    at = front
    for e, n in enumerate(counts):
        if n:
            Ye, A = O.w4a16_gemm(bits(X[at:at + n]), _dequant(W[e], group, sym))
            check_bf16(bits(Y[at:at + n]), Ye, A, rel=fp32_bound(K), what=f"expert {e}")
        at += n
    assert (out[:front] == -7).all() and (out[front + used:] == -7).all()
    # the same bits in every run
    again = m.w4a16_grouped_gemm(Xc, _offsets(counts, front), w, out=torch.full_like(out, -7.0))
    assert torch.equal(again, out)


@pytest.mark.parametrize("K,N,group,sym", [
    (256, 192, 128, True), (256, 192, 128, False), (320, 128, 64, True), (320, 128, 64, False),
])
@pytest.mark.parametrize("rows", [5, 16, 40, 256])
def test_dequantized_weight_is_exact(m, K, N, group, sym, rows):
    """One-hot rows (`rows` of them for each expert) return weight rows unchanged."""
    E = 2 * ((K + rows - 1) // rows)
    w, W = _weights(m, 2, K, N, group, sym, seed=K + rows)
    pick = torch.arange(E) % 2       # experts alternate between the two weights
    big = m.PackedWeight(packed=w.packed[pick].contiguous(), s_w=w.s_w[pick].contiguous(),
                         z=None if sym else w.z[pick].contiguous(), desc=w.desc, experts=E)
    eye = torch.eye(K, dtype=torch.bfloat16, device="cuda")
    parts = [eye[(e // 2) * rows:(e // 2 + 1) * rows] for e in range(E)]
    Y = m.w4a16_grouped_gemm(torch.cat(parts), _offsets([len(p) for p in parts]), big)
    Wh = [_dequant(x, group, sym) for x in W]
    at = 0
    for e, part in enumerate(parts):
        assert np.array_equal(bits(Y[at:at + len(part)]), Wh[e % 2][(e // 2) * rows:(e // 2) * rows + len(part)])
        at += len(part)


def test_layer_size_sampled_experts(m):
    g = torch.Generator().manual_seed(3)
    counts = torch.bincount(torch.randint(0, 64, (12288,), generator=g), minlength=64).tolist()
    w, W = _weights(m, 64, 1408, 2048, 128, True, seed=1)
    X = gen_linear(12288, 1408, 64, seed=4).X
    Y = m.w4a16_grouped_gemm(X.cuda(), _offsets(counts), w)
    at = 0
    for e, n in enumerate(counts):
        if e in (0, 63):
            Ye, A = O.w4a16_gemm(bits(X[at:at + n]), _dequant(W[e], 128, True))
            check_bf16(bits(Y[at:at + n]), Ye, A, rel=fp32_bound(1408), what=f"expert {e}")
        at += n


@pytest.mark.parametrize("K,N,group,sym", [(192, 2112, 64, False), (128, 2176, 128, True), (320, 2304, 64, True)])
def test_many_tiles(m, K, N, group, sym):
    """Many tiles for each CTA; the last columns half a box, an odd and an even number of boxes."""
    counts = [5000, 0, 3, 9000, 193, 2500, 40, 8100, 5900]
    w, W = _weights(m, len(counts), K, N, group, sym, seed=K)
    X = gen_linear(sum(counts), K, 64, seed=N).X
    Y = m.w4a16_grouped_gemm(X.cuda(), _offsets(counts), w)
    at = 0
    for e, n in enumerate(counts):
        pick = sorted(set(range(0, n, 97)) | set(range(max(n - 3, 0), n)))
        if pick:
            Ye, A = O.w4a16_gemm(bits(X[at:at + n][pick]), _dequant(W[e], group, sym))
            check_bf16(bits(Y[at:at + n][pick]), Ye, A, rel=fp32_bound(K), what=f"expert {e}")
        at += n


def test_many_tiles_of_few_rows(m):
    """Many tiles of 16 rows for each CTA: one row for each of 300 experts, wide N."""
    E, K, N = 300, 64, 16064
    w, W = _weights(m, 2, K, N, 64, True, seed=3)
    pick = torch.arange(E) % 2
    big = m.PackedWeight(packed=w.packed[pick].contiguous(), s_w=w.s_w[pick].contiguous(), z=None, desc=w.desc, experts=E)
    X = gen_linear(E, K, 64, seed=5).X
    Y = m.w4a16_grouped_gemm(X.cuda(), _offsets([1] * E), big)
    for e in (0, 1):
        Ye, A = O.w4a16_gemm(bits(X[e::2]), _dequant(W[e], 64, True))
        check_bf16(bits(Y[e::2]), Ye, A, rel=fp32_bound(K), what=f"weight {e}")


def test_strided_rows_and_outputs(m):
    for counts in ([20, 0, 29, 1], [2, 1, 0, 2]):
        R = sum(counts)
        w, _ = _weights(m, 4, 384, 128, 64, False, seed=5)
        wide = torch.randn(R, 400, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
        X, off = wide[:, :384], _offsets(counts)
        want = m.w4a16_grouped_gemm(X.contiguous(), off, w)
        for pitch in (128, 136, 131):
            buf = torch.full((R, pitch), 9.0, dtype=torch.bfloat16, device="cuda")
            m.w4a16_grouped_gemm(X, off, w, out=buf[:, :128])
            assert torch.equal(buf[:, :128], want) and (buf[:, 128:] == 9).all()


@pytest.mark.parametrize("off", [[0, 5, 3, 12], [-1, 2, 4, 12], [0, 4, 8, 13], [12, 0, 12, 5], [0, 2**31 - 1, 5, 6]])
def test_bad_offsets_are_reported(m, off):
    w, _ = _weights(m, 3, 128, 64, 64, True, seed=6)
    st = m.new_status("cuda")
    guard = torch.full((14, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    m.w4a16_grouped_gemm(torch.randn(12, 128).bfloat16().cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"),
                         w, out=guard[1:13], status=st)
    assert m.w4a8_get_device_status(st) == 1
    assert (guard[0] == 5).all() and (guard[13] == 5).all()


def test_nonfinite_rows_stay_in_their_row(m):
    """A NaN or infinite activation reaches its own row of the output alone."""
    for counts in ([3, 2], [40, 30]):
        R = sum(counts)
        w, _ = _weights(m, 2, 256, 128, 128, True, seed=7)
        X = torch.randn(R, 256, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
        off = _offsets(counts)
        want = m.w4a16_grouped_gemm(X, off, w)
        X[1, 7], X[R - 2, 100] = float("nan"), float("inf")
        got = m.w4a16_grouped_gemm(X, off, w)
        keep = [r for r in range(R) if r not in (1, R - 2)]
        assert torch.equal(got[keep], want[keep])
        assert torch.isnan(got[1]).all() and not torch.isfinite(got[R - 2]).any()


def test_workspace_contents_and_order_do_not_matter(m):
    """Split launches: a workspace full of anything, reused by other shapes,
    gives the same bits every time."""
    shapes = [([1, 1, 2, 1], 2048, 512), ([5, 0, 90, 1], 1024, 192), ([16] * 4, 1216, 640), ([200], 4096, 64)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    todo = []
    for counts, K, N in shapes:
        w, _ = _weights(m, len(counts), K, N, 64, False, seed=K)
        X = torch.randn(sum(counts), K, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        assert 0 < m.w4a16_grouped_workspace_size(sum(counts), w) <= ws.numel()
        todo.append((X, _offsets(counts), w, m.w4a16_grouped_gemm(X, _offsets(counts), w).clone()))
    for fill in (0, 255, None):
        if fill is None:
            ws.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(9))
        else:
            ws.fill_(fill)
        for _ in range(20):
            for X, off, w, want in todo:
                assert torch.equal(m.w4a16_grouped_gemm(X, off, w, workspace=ws), want)


def test_captured_with_changing_offsets(m):
    w, _ = _weights(m, 4, 512, 256, 128, True, seed=8)
    X = torch.randn(48, 512, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    off, out = _offsets([12, 12, 12, 12]), torch.zeros(48, 256, dtype=torch.bfloat16, device="cuda")
    m.w4a16_grouped_gemm(X, off, w, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.w4a16_grouped_gemm(X, off, w, out=out)
    for counts in ([12, 12, 12, 12], [0, 48, 0, 0], [1, 0, 0, 2]):
        off.copy_(_offsets(counts))
        want = m.w4a16_grouped_gemm(X, off, w, out=torch.zeros_like(out))
        out.zero_()
        g.replay()
        assert torch.equal(out, want)


def test_two_streams_with_their_own_workspaces(m):
    w, _ = _weights(m, 8, 1024, 256, 128, True, seed=10)
    X = torch.randn(8, 1024, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    off = _offsets([1] * 8)
    want = m.w4a16_grouped_gemm(X, off, w)
    assert m.w4a16_grouped_workspace_size(8, w) > 0
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(30):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(m.w4a16_grouped_gemm(X, off, w))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


def test_more_than_2_31_elements(m):
    """Offsets into Y that pass 32 bits: rows at both ends against small calls."""
    R, K, N = (1 << 17) + 5, 64, 16448
    w, _ = _weights(m, 2, K, N, 64, True, seed=12)
    X = torch.randn(R, K, device="cuda").bfloat16()
    Y = m.w4a16_grouped_gemm(X, _offsets([9, R - 9]), w)
    assert R * N > 2 ** 31
    for e, rows in ((0, slice(0, 9)), (1, slice(9, 200)), (1, slice(R - 300, R))):   # K = 64: one sum, one order
        n = rows.stop - rows.start
        assert torch.equal(Y[rows], m.w4a16_grouped_gemm(X[rows].contiguous(), _offsets([n, 0] if e == 0 else [0, n]), w))


def test_experts_of_a_layer(m):
    """Route, dispatch, gather, gate_up, silu * up, down, combine with the
    packed weights a W4A8 layer uses; against the same steps in fp64 on the
    dequantized weights.  bf16 roundings, each at most 2^-8 of its value and
    independent of the others: gate and up (h moves by at most twice that), h,
    the expert rows; the fp32 sums and the last rounding are covered by their
    root mean squares being at most 2^-8 / sqrt(3)."""
    T, E, topk, H, I, group = 40, 6, 2, 512, 256, 128
    w1, W1 = _weights(m, E, H, 2 * I, group, True, seed=1)
    w2, W2 = _weights(m, E, I, H, group, True, seed=2)
    g = torch.Generator().manual_seed(5)
    X = torch.randn(T, H, generator=g).bfloat16().cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    idx, wt = m.w4a8_moe_route(logits, topk)
    offsets, perm, inv = m.w4a8_moe_dispatch(idx, E)
    rows = X[torch.div(perm, topk, rounding_mode="floor").long()]
    gu = m.w4a16_grouped_gemm(rows, offsets, w1).float()
    h = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).bfloat16()
    out = m.w4a8_moe_combine(m.w4a16_grouped_gemm(h, offsets, w2)[inv.long()], wt)
    f64 = lambda W: torch.from_numpy(O.bf16_to_f32(_dequant(W, group, True)).astype(np.float64))  # noqa: E731
    ref = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(topk):
            e = int(idx[t, j])
            y = X[t].double().cpu() @ f64(W1[e])
            y = (y[:I] / (1 + torch.exp(-y[:I])) * y[I:]) @ f64(W2[e])
            ref[t] += float(wt[t, j]) * y
    err = (out.double().cpu() - ref).norm() / ref.norm()
    assert err <= 4 * 2.0 ** -8


def test_refusals_of_the_binding(m):
    w, _ = _weights(m, 4, 256, 64, 64, False, seed=11)
    X, off = torch.randn(8, 256).bfloat16().cuda(), _offsets([2, 2, 2, 2])

    def refused(code, *a, **k):
        with pytest.raises(m.W4A8Error) as e:
            m.w4a16_grouped_gemm(*a, **k)
        assert e.value.code == code

    refused(1, X.float(), off, w)
    refused(1, X.t().contiguous().t(), off, w)
    refused(1, X[:, 1:], off, w)
    refused(1, X, off.long(), w)
    refused(1, X, off[:4], w)
    refused(1, X, off, _one(w, 0, m))
    refused(1, X, off, w, out=torch.empty(8, 64, device="cuda"))
    refused(3, X, off, m.PackedWeight(w.packed, w.s_w, None, w.desc, 4))
    refused(1, X, off, m.PackedWeight(w.packed, w.s_w[:, :1], w.z, w.desc, 4))
    refused(1, X, off, m.PackedWeight(w.packed[:2], w.s_w, w.z, w.desc, 4))
    odd = torch.randn(8, 260).bfloat16().cuda()[:, :256]      # pitch not a multiple of 16 bytes
    refused(1, odd, off, w)
    assert m.w4a16_grouped_gemm(X[:0], torch.zeros_like(off), w).shape == (0, 64)
