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
