"""Argument checks of the products on FP4 weights; they run before any CUDA
call, so no GPU is needed, and nothing is enqueued."""
import ctypes

import pytest
import torch

BIG = 2 ** 31


@pytest.fixture(scope="module")
def fq():
    from fp4_post_weight_grid_b200 import build
    build.build()
    import fp4_post_weight_grid_b200 as m
    m.load()
    return m


@pytest.fixture(scope="module")
def q():
    buf = ctypes.create_string_buffer(512)
    p = ctypes.addressof(buf)
    q.keep = buf
    return p + (-p % 16)


def _calls(fq, q):
    """The four calls with sound arguments, any of them replaced by name."""
    lib = fq.load()

    def linear(**kw):
        a = dict(fmt=0, x=q, m=2, w=q, ws=q, S=q, n=3, k=64, ep=None, y=q, dt=1, st=q)
        a.update(kw)
        return lib.fp4q_linear(a["fmt"], a["x"], a["m"], a["w"], a["ws"], a["S"], a["n"], a["k"], a["ep"], a["y"],
                               a["dt"], a["st"], None)

    def linear_group(**kw):
        a = dict(fmt=0, x=q, m=2, off=q, g=2, w=q, ws=q, S=q, n=3, k=64, ep=None, y=q, dt=1, st=q)
        a.update(kw)
        return lib.fp4q_linear_group(a["fmt"], a["x"], a["m"], a["off"], a["g"], a["w"], a["ws"], a["S"], a["n"],
                                     a["k"], a["ep"], a["y"], a["dt"], a["st"], None)

    def matmul(**kw):
        a = dict(fmt=0, x=q, xs=q, xS=q, m=2, w=q, ws=q, S=q, n=3, k=64, ep=None, y=q, dt=1, st=q)
        a.update(kw)
        return lib.fp4q_matmul(a["fmt"], a["x"], a["xs"], a["xS"], a["m"], a["w"], a["ws"], a["S"], a["n"], a["k"],
                               a["ep"], a["y"], a["dt"], a["st"], None)

    def matmul_group(**kw):
        a = dict(fmt=0, x=q, xs=q, xS=q, m=2, off=q, g=2, w=q, ws=q, S=q, n=3, k=64, ep=None, y=q, dt=1, st=q)
        a.update(kw)
        return lib.fp4q_matmul_group(a["fmt"], a["x"], a["xs"], a["xS"], a["m"], a["off"], a["g"], a["w"], a["ws"],
                                     a["S"], a["n"], a["k"], a["ep"], a["y"], a["dt"], a["st"], None)

    return dict(linear=linear, linear_group=linear_group, matmul=matmul, matmul_group=matmul_group)


@pytest.mark.parametrize("name", ["linear", "linear_group", "matmul", "matmul_group"])
def test_refusals(fq, q, name):
    call = _calls(fq, q)[name]
    assert call(fmt=2) == fq.ERR_DTYPE and call(dt=2) == fq.ERR_DTYPE
    for kw in (dict(m=-1), dict(n=-1), dict(k=-32), dict(k=0), dict(k=48), dict(k=16), dict(m=BIG), dict(n=BIG),
               dict(k=BIG), dict(m=BIG - 256), dict(m=2 ** 62), dict(n=2 ** 62)):
        assert call(**kw) == fq.ERR_SHAPE, kw
    for f in ("x", "w", "ws", "S", "y", "st"):
        assert call(**{f: None}) == fq.ERR_NULL, f
        assert call(**{f: q + 2}) == fq.ERR_ALIGN, f
    for f in ("x", "w", "ws", "y"):
        assert call(**{f: q + 8}) == fq.ERR_ALIGN, f
    # S is not read for MXFP4; the next check is reached
    assert call(fmt=1, S=None, y=q + 8) == fq.ERR_ALIGN
    if name.startswith("matmul"):
        assert call(xs=None) == fq.ERR_NULL and call(xS=None) == fq.ERR_NULL
        assert call(xs=q + 2) == fq.ERR_ALIGN and call(xS=q + 2) == fq.ERR_ALIGN
        assert call(fmt=1, xS=None, y=q + 8) == fq.ERR_ALIGN
    if name.endswith("group"):
        assert call(off=None) == fq.ERR_NULL and call(off=q + 2) == fq.ERR_ALIGN
        assert call(g=-1) == fq.ERR_SHAPE and call(g=1025) == fq.ERR_ARG
        assert call(g=1024, n=1 << 21) == fq.ERR_SHAPE
    for f in ("bias", "mul", "residual"):
        ep = fq.Epilogue(None, None, None, 0)
        setattr(ep, f, q + 8)
        assert call(ep=ctypes.byref(ep)) == fq.ERR_ALIGN, f
    for act in (-1, 5):
        assert call(ep=ctypes.byref(fq.Epilogue(None, None, None, act))) == fq.ERR_ARG


@pytest.mark.parametrize("name", ["linear", "linear_group", "matmul", "matmul_group"])
def test_empty_products_touch_nothing(fq, q, name):
    call = _calls(fq, q)[name]
    nothing = dict(x=None, w=None, ws=None, S=None, y=None, st=None)
    assert call(m=0, **nothing) == fq.OK
    assert call(n=0, **nothing) == fq.OK
    if name.endswith("group"):
        assert call(g=0, **nothing) == fq.OK


def test_the_binding_refuses(fq):
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(3, 32, dtype=torch.uint8)
    y, st = torch.zeros(2, 3, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    S, ws = torch.ones(1), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp4q_linear(fq.NVFP4, x, w, ws, S, y, st)
    with pytest.raises(ValueError, match="do not fit"):
        fq.fp4q_linear(fq.NVFP4, x[:, :32], w, ws, S, y, st)
    with pytest.raises(ValueError, match="do not fit"):
        fq.fp4q_linear(fq.NVFP4, x, w, ws, S, y[:1], st)
    with pytest.raises(ValueError, match="2-D"):
        fq.fp4q_linear_group(fq.NVFP4, x, torch.zeros(2, dtype=torch.int32), w, ws, S, y, st)
    with pytest.raises(fq.Fp4qError) as e:
        fq.fp4q_linear(7, x, w, ws, S, y, st)
    assert e.value.status == fq.ERR_DTYPE
    with pytest.raises(fq.Fp4qError) as e:
        fq.fp4q_linear(fq.NVFP4, x, w, ws, None, y, st)
    assert e.value.status == fq.ERR_NULL
    with pytest.raises(fq.Fp4qError) as e:
        fq.fp4q_linear(fq.NVFP4, x[:, :48], w[:, :24], ws, S, y, st)
    assert e.value.status == fq.ERR_SHAPE
    with pytest.raises(TypeError):
        fq.fp4q_matmul(fq.NVFP4, w[:2], None, S, w, ws, S, y, st)


@pytest.mark.parametrize("name", ["linear", "linear_group", "matmul", "matmul_group"])
def test_rows_too_long_for_a_tile_are_refused(fq, q, name):
    call = _calls(fq, q)[name]
    for k in (2 ** 26 + 32, 2 ** 29, 2 ** 30, 2 ** 30 + 64):
        assert call(k=k, m=1, n=1) == fq.ERR_SHAPE, k
    assert call(k=2 ** 26, m=1, n=1, y=q + 8) == fq.ERR_ALIGN         # the next check is reached


def test_check_status_raises_every_flag(fq):
    wants = {fq.FLAG_NONFINITE: fq.ERR_NONFINITE, fq.FLAG_RANGE: fq.ERR_RANGE, fq.FLAG_OFFSETS: fq.ERR_ARG,
             fq.FLAG_TIMEOUT: fq.ERR_CUDA}
    for flag, error in wants.items():
        with pytest.raises(fq.Fp4qError, match="device status") as e:
            fq.check_status(torch.tensor([flag], dtype=torch.int32))
        assert e.value.status == error
    assert fq.check_status(torch.zeros(1, dtype=torch.int32)) == 0
