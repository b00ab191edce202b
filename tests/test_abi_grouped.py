"""Host-side checks of the grouped products and the INT8 MoE layer: every
refusal below happens before any CUDA call, so no GPU is needed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from moe_linear_layers_w4a8_b200 import _build
    _build.build()
    import moe_linear_layers_w4a8_b200 as m
    return m.load_library()


def _d8(K=512, N=512, **kw):
    import moe_linear_layers_w4a8_b200 as m
    d = dict(bits=8, symmetric=1, group=K, K=K, N=N, layout_version=1)
    d.update(kw)
    return m.WDesc(**d)


FAKE = ctypes.c_void_p(256)   # never dereferenced
ODD = ctypes.c_void_p(264)    # not 16-byte aligned
BIG = 1 << 40


def _gemm(lib, qx=FAKE, sx=FAKE, off=FAKE, R=16, E=4, qw=FAKE, sw=FAKE, d=None, Y=FAKE, ldy=512, ws=FAKE, wsb=BIG):
    d = _d8() if d is None else d
    return lib.w8a8_grouped_gemm(qx, sx, off, R, E, qw, sw, ctypes.byref(d), Y, ldy, ws, wsb, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d="bits"), 3), (dict(d="K"), 3), (dict(d="N"), 3), (dict(d="group"), 3),
    (dict(R=-1), 1), (dict(E=0), 1), (dict(E=513), 2), (dict(R=(1 << 24) + 1), 2),
    (dict(Y=None), 1), (dict(ldy=511), 1), (dict(qx=None), 1), (dict(sx=None), 1), (dict(off=None), 1),
    (dict(qw=None), 1), (dict(sw=None), 1), (dict(qx=ODD), 1), (dict(qw=ODD), 1),
    (dict(ws=None, wsb=0), 7), (dict(ws=ODD), 7), (dict(R=0), 0),
])
def test_grouped_gemm_refusals(lib, kw, code):
    kw = dict(kw)
    if "d" in kw:
        kw["d"] = {"bits": _d8(bits=4), "K": _d8(K=520), "N": _d8(N=520), "group": _d8(group=128)}[kw["d"]]
    assert _gemm(lib, **kw) == code


def test_grouped_sizes(lib):
    d = _d8()
    need = lib.w8a8_grouped_workspace_size(16, 4, ctypes.byref(d))
    assert need > 0 and _gemm(lib, wsb=need - 1) == 7
    # many more tiles than SMs whatever the offsets say: nothing is split
    assert lib.w8a8_grouped_workspace_size(1 << 20, 4, ctypes.byref(d)) == 0
    assert lib.w8a8_grouped_workspace_size(0, 4, ctypes.byref(d)) == 0
    assert lib.w8a8_grouped_workspace_size(16, 513, ctypes.byref(d)) == 0
    lin = lib.w8a8_grouped_linear_workspace_size(16, 4, ctypes.byref(d))
    assert lin >= need + 16 * 512 + 16 * 4


@pytest.mark.parametrize("kw,code", [
    (dict(), 7), (dict(X=None), 1), (dict(ldx=500), 1), (dict(ldx=516), 2), (dict(X=ODD), 2), (dict(qw=ODD), 1),
    (dict(off=None), 1), (dict(ldy=100), 1), (dict(R=0), 0), (dict(R=-1), 1),
])
def test_grouped_linear_refusals(lib, kw, code):
    a = dict(X=FAKE, R=16, ldx=512, off=FAKE, E=4, qw=FAKE, sw=FAKE, Y=FAKE, ldy=512)
    a.update(kw)
    d = _d8()
    assert lib.w8a8_grouped_linear(a["X"], a["R"], a["ldx"], a["off"], a["E"], a["qw"], a["sw"], ctypes.byref(d),
                                   a["Y"], a["ldy"], FAKE, 16, None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(topk=65), 1), (dict(topk=0), 1), (dict(E=513, topk=4), 2), (dict(topk=17), 2), (dict(T=-1), 1),
    (dict(w1=_d8), 3), (dict(w2="K"), 3), (dict(w2="N"), 3), (dict(H=8320), 2), (dict(T=1 << 24, topk=2), 2),
    (dict(X=None), 1), (dict(logits=None), 1), (dict(out=ODD), 1), (dict(ws=None), 7), (dict(wsb=100), 7), (dict(T=0), 0),
])
def test_moe_w8_refusals(lib, kw, code):
    H = kw.get("H", 2048)
    w1, w2 = _d8(H, 2816), _d8(1408, H)
    if kw.get("w1"):
        w1 = _d8(H, 2816, bits=4)
    if kw.get("w2") == "K":
        w2 = _d8(1280, H)
    if kw.get("w2") == "N":
        w2 = _d8(1408, 1024)
    a = dict(X=FAKE, logits=FAKE, T=16, E=64, topk=6, out=FAKE, ws=FAKE, wsb=BIG)
    a.update({k: v for k, v in kw.items() if k in a})
    r = lib.w8a8_moe_grouped_gemm(a["X"], a["logits"], a["T"], a["E"], a["topk"], FAKE, FAKE, ctypes.byref(w1), FAKE,
                                  FAKE, ctypes.byref(w2), a["out"], FAKE, FAKE, FAKE, a["ws"], a["wsb"], None, None)
    assert r == code


def test_moe_w8_experts_refusals(lib):
    w1, w2 = _d8(256, 256), _d8(128, 256)
    call = lambda X=FAKE, ids=FAKE, R=8, E=4, y=FAKE, ws=FAKE, wsb=BIG: lib.w8a8_moe_experts(  # noqa: E731
        X, ids, R, E, FAKE, FAKE, ctypes.byref(w1), FAKE, FAKE, ctypes.byref(w2), y, ws, wsb, None, None)
    assert call(X=None) == 1 and call(ids=None) == 1 and call(y=None) == 1 and call(X=ODD) == 1
    assert call(E=0) == 1 and call(E=600) == 2 and call(R=-1) == 1
    assert call(ws=None) == 7 and call(wsb=16) == 7
    assert call(R=0) == 0


def test_dispatch_refusals(lib):
    call = lambda ids=FAKE, P=8, E=4, o=FAKE, ws=FAKE, wsb=BIG: lib.w4a8_moe_dispatch(  # noqa: E731
        ids, P, E, o, FAKE, FAKE, ws, wsb, None, None)
    assert call(ids=None) == 1 and call(P=-1) == 1 and call(E=0) == 1 and call(E=513) == 2 and call(o=None) == 1
    assert call(ws=None) == 7 and call(wsb=16) == 7 and call(ws=ODD) == 7


def test_binding_refusals():
    import torch
    import moe_linear_layers_w4a8_b200 as m
    w = m.PackedW8(q_w=torch.zeros(4, 16, 128, dtype=torch.int8), s_w=torch.ones(4, 16),
                   desc=m.WDesc(8, 1, 128, 128, 16, 1), experts=4)
    off = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(m.W4A8Error) as e:   # CPU tensors
        m.w8a8_grouped_gemm(torch.zeros(2, 128, dtype=torch.int8), torch.ones(2), off, w)
    assert e.value.code == 1
    with pytest.raises(m.W4A8Error):
        m.w8a8_grouped_linear(torch.zeros(2, 128, dtype=torch.bfloat16), off, w)
    with pytest.raises(m.W4A8Error):
        m.w8a8_moe_grouped_gemm(torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(2, 4), 2, w, w)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), 1), (dict(X=ODD), 1), (dict(ldx=500), 1), (dict(ldx=516), 1), (dict(off=None), 1), (dict(ldy=511), 1),
    (dict(Y=None), 1), (dict(pk=None), 1), (dict(pk=ODD), 1), (dict(sw=None), 1), (dict(sw=ODD), 1),
    (dict(z=FAKE), 3), (dict(sym=0), 3), (dict(bits=8), 3), (dict(group=32), 3), (dict(N=500), 3),
    (dict(R=-1), 1), (dict(E=0), 1), (dict(E=513), 2), (dict(R=(1 << 24) + 1), 2), (dict(R=0), 0),
    (dict(N=128, ws=None), 7), (dict(N=128, ws=ODD), 7), (dict(N=128, wsb=100), 7),
])
def test_w4a16_grouped_refusals(lib, kw, code):
    import moe_linear_layers_w4a8_b200 as m
    a = dict(X=FAKE, R=16, ldx=512, off=FAKE, E=4, pk=FAKE, sw=FAKE, z=None, Y=FAKE, ldy=512, sym=1, bits=4, group=128,
             N=512, ws=FAKE, wsb=BIG)
    a.update(kw)
    d = m.WDesc(a["bits"], a["sym"], a["group"], 512, a["N"], 1)
    assert lib.w4a16_grouped_gemm(a["X"], a["R"], a["ldx"], a["off"], a["E"], a["pk"], a["sw"], a["z"],
                                  ctypes.byref(d), a["Y"], a["ldy"], a["ws"], a["wsb"], None, None) == code
