"""Host-side choices that can be asked for without a GPU."""
import pytest


@pytest.fixture(scope="module")
def m():
    from moe_linear_layers_w4a8_b200 import _build
    _build.build()
    import moe_linear_layers_w4a8_b200 as mm
    mm.load_library()
    return mm


@pytest.mark.parametrize("T,E,topk,launches", [
    (1, 64, 6, 1), (256, 512, 16, 1), (257, 512, 16, 1), (320, 512, 3, 1), (333, 13, 3, 1), (400, 64, 8, 1),
    (512, 512, 1, 1),
    # one CTA's second chunk of tokens has too many pairs
    (320, 512, 8, 3), (400, 256, 16, 3), (512, 64, 8, 3), (512, 64, 16, 3), (512, 512, 16, 3),
    (513, 64, 1, 3), (4096, 64, 6, 3),
    (0, 64, 6, 0), (-1, 64, 6, 0), (5, 0, 1, 0), (5, 513, 1, 0), (5, 64, 17, 0), (5, 4, 5, 0), (5, 4, 0, 0),
])
def test_dispatch_launches(m, T, E, topk, launches):
    assert m.w4a8_moe_dispatch_launches(T, E, topk) == launches


@pytest.mark.parametrize("T,E,topk,launches", [(64, 256, 8, 7), (333, 13, 3, 7), (512, 512, 16, 9), (4096, 64, 6, 9)])
def test_bench_counts_the_dispatch_launches(m, T, E, topk, launches):
    import bench
    wl = bench.MoEWorkload("moe_sym")
    wl.T, wl.E, wl.topk = T, E, topk
    assert wl.launches_per_step == launches


def test_grouped_cases_reach_every_kernel(m):
    """On 148 SMs: the cases of tests/test_gpu_grouped_heights.py reach the plans
    that they state, and between them every tile height, whole and split, of
    every kernel, and in W4A16 every activation box under both."""
    from tests import test_gpu_grouped_heights as t
    seen = set()
    for counts, K, N, plan in t.W8A8:
        assert t.reached(m.w8a8_grouped_plan(t.ends(counts), m.WDesc(8, 1, K, K, N, 1), sms=148)) == plan
        seen.add(("plain",) + plan)
    for counts, H, I, plan in t.GATE_UP:
        p = m.w8a8_grouped_plan(t.ends(counts), m.WDesc(8, 1, H, H, 2 * I, 1), gate_up=True, sms=148)
        assert t.reached(p) == plan
        seen.add(("gate_up",) + plan)
    boxes = {16: (16,), 32: (32,), 64: (32, 64), 128: (32, 64, 128), 192: (32, 64, 96, 192)}
    for counts, K, N, plan in t.W4A16:
        for group in (64, 128):
            Kg = K + 64 if K % group else K
            for sym in (0, 1):
                p = m.w4a16_grouped_plan(t.ends(counts), m.WDesc(4, sym, group, Kg, N, 1), sms=148)
                assert t.reached(p) == plan
                # a split's segments begin inside a stage of activations
                assert not p["range"] or p["units"] % p["range"]
        seen.add(("w4a16",) + plan)
        rows = {min(plan[0], n - i) for n in counts for i in range(0, n, plan[0])}
        for lo, hi in zip((0,) + boxes[plan[0]], boxes[plan[0]]):
            assert any(lo < r <= hi for r in rows), (plan, lo, hi)
    want = {("plain", bn, cols, split) for bn in (16, 32, 64, 128) for cols in (128, 256) for split in (False, True)}
    want |= {("gate_up", bn, 128, split) for bn in (16, 32, 64, 128) for split in (False, True)}
    want |= {("w4a16", bn, 128, split) for bn in (16, 32, 64, 128, 192) for split in (False, True)}
    assert seen == want


def test_grouped_plan_refusals(m):
    d8, d4 = m.WDesc(8, 1, 256, 256, 64, 1), m.WDesc(4, 1, 64, 256, 64, 1)
    for plan, d, wrong in ((m.w8a8_grouped_plan, d8, d4), (m.w4a16_grouped_plan, d4, d8)):
        for offsets, kw, desc, code in [([0, 5, 3], {}, d, 1), ([-1, 5], {}, d, 1), ([0, 5], dict(R=4), d, 1),
                                        ([0, 5], dict(sms=-1), d, 1), ([0], {}, d, 1), ([0, 5], {}, wrong, 3),
                                        ([0] * 514, {}, d, 2), ([], {}, d, 1), ([0, 2**32 + 5], {}, d, 1), ([0, 5], dict(R=2**32 + 5), d, 1),
                                        ([0, 5], dict(R=(1 << 24) + 1), d, 2)]:
            with pytest.raises(m.W4A8Error) as e:
                plan(offsets, desc, **{"sms": 148, **kw})
            assert e.value.code == code
    with pytest.raises(m.W4A8Error) as e:
        m.w8a8_grouped_plan([0, 5], m.WDesc(8, 1, 256, 256, 64, 2), sms=148)
    assert e.value.code == 3
    assert m.w8a8_grouped_plan([0, 0], d8, R=0, sms=148)["tiles"] == 0


def test_too_many_rows_are_refused(m):
    """More (token, slot) rows than the kernels number in 32 bits: refused before
    anything is launched (the pointers are never dereferenced)."""
    lib, fake = m.load_library(), 256
    for T, topk in [(1 << 27, 16), ((1 << 31) - 1, 2)]:
        assert lib.w4a8_moe_combine(fake, fake, T, topk, 8, fake, None) == 2
    for T in ((1 << 27) + 1, (1 << 31) - 1):
        assert lib.w4a8_moe_route(fake, T, 16, 1, fake, fake, None, None) == 2
