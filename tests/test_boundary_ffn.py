"""Refusals of the block norm, the codes by row and column, the product of codes and the gated
activation, through the C ABI on invented addresses (nothing is launched) and through the
binding's own checks."""
import pytest
import torch

from bitwise_reproducible_int8_gb300 import build_lib, repro
from test_boundary_blocks import B, BAD, INF, NAN, call

NORM = dict(x=B, x_ld=64, y=2 * B, y_ld=64, type=0, gate=None, gate_ld=0, gain_post=None, gain_pre=3 * B, alpha=1.0,
            beta=1.0, eps=1e-6, n=10, D=64, flags=0, h=4 * B, h_ld=64, u=5 * B, u_type=0, u_ld=64, stats=6 * B,
            stream=None)


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return repro.lib()


def test_block_norm_fwd(L):
    f = lambda **kw: call(L.repro_block_norm_fwd, NORM, **kw)  # noqa: E731
    for kw in (dict(), dict(flags=4, gain_post=7 * B), dict(gate=7 * B), dict(gate=7 * B, gate_ld=64, flags=8),
               dict(y=None, h=None), dict(u=None, gain_pre=None), dict(stats=None), dict(h=B), dict(type=1, u_type=1),
               dict(D=16384, x_ld=16384, y_ld=16384, h_ld=16384, u_ld=16384), dict(x=B + 4), dict(n=1, x_ld=1 << 40)):
        assert f(**kw) not in BAD, kw                       # only the device is missing here
    for kw in (dict(x=None), dict(h=None), dict(y=None), dict(y=None, h=None, u=None, gain_pre=None), dict(u=None),
               dict(type=2), dict(u_type=2), dict(flags=1), dict(flags=16), dict(flags=8), dict(gain_post=7 * B),
               dict(y=None, h=None, gate=7 * B), dict(y=None, h=None, flags=4), dict(alpha=NAN), dict(beta=INF),
               dict(eps=-1.0), dict(eps=NAN), dict(eps=INF)):
        assert f(**kw) == -1, kw
    for kw in (dict(n=-1), dict(D=0), dict(D=16385, x_ld=20000, y_ld=20000, h_ld=20000, u_ld=20000), dict(x_ld=63),
               dict(y_ld=63), dict(h_ld=63), dict(u_ld=63), dict(n=(1 << 31) + 1), dict(x_ld=(1 << 28) + 1),
               dict(gate=7 * B, gate_ld=63, flags=8)):
        assert f(**kw) == -2, kw
    for kw in (dict(x=B + 2), dict(y=2 * B + 1), dict(h=4 * B + 2), dict(u=5 * B + 2), dict(gain_pre=3 * B + 2),
               dict(stats=6 * B + 1), dict(gate=7 * B + 2), dict(type=1, x=B + 1, gate=None)):
        assert f(**kw) == -3, kw
    for kw in (dict(h=2 * B), dict(u=B), dict(u=4 * B + 256), dict(h=B + 64), dict(h=B, h_ld=128), dict(stats=5 * B),
               dict(u=3 * B), dict(h=3 * B + 4 * 60)):
        assert f(**kw) == -8, kw
    assert f(n=0, x=None) == 0 and f(n=0, y=None, h=None, u=None, gain_pre=None) == 0


def test_block_norm_bwd(L):
    ws = repro.repro_block_norm_bwd_ws_bytes(1000, 64)
    ok = dict(dh=B, dh_ld=64, du=2 * B, u_type=0, du_ld=64, h=3 * B, h_ld=64, y=4 * B, y_ld=64, type=0, gate=None,
              gate_ld=0, gain_post=None, gain_pre=5 * B, stats=6 * B, alpha=1.0, beta=1.0, n=1000, D=64, flags=0,
              dx=7 * B, dx_ld=64, dy=8 * B, dy_ld=64, dgate=None, dgate_ld=0, dgain_post=None, dgain_pre=9 * B,
              ws=10 * B, ws_bytes=ws, stream=None)
    f = lambda **kw: call(L.repro_block_norm_bwd, ok, **kw)  # noqa: E731
    none = dict(gain_pre=None, dgain_pre=None)
    for kw in (dict(), dict(dh=None), dict(du=None, h=None, **none), dict(y=None, dy=None), dict(dx=B), dict(flags=1),
               dict(gate=11 * B, dgate=12 * B), dict(gate=11 * B, dgate=12 * B, flags=8, gate_ld=64, dgate_ld=80),
               dict(flags=4, gain_post=11 * B, dgain_post=12 * B), dict(ws=None, ws_bytes=0, **none)):
        assert f(**kw) not in BAD, kw
    for kw in (dict(dh=None, du=None, h=None, **none), dict(du=None), dict(h=None), dict(dx=None), dict(dy=None),
               dict(y=None), dict(stats=None), dict(dgain_pre=None), dict(gain_pre=None), dict(gate=11 * B),
               dict(dgate=11 * B), dict(gain_post=11 * B, dgain_post=12 * B), dict(gain_post=11 * B, flags=4),
               dict(du=None, h=None), dict(flags=2), dict(flags=8), dict(type=3), dict(u_type=2), dict(alpha=INF)):
        assert f(**kw) == -1, kw
    for kw in (dict(n=-1), dict(D=0), dict(dh_ld=1), dict(du_ld=1), dict(h_ld=1), dict(y_ld=1), dict(dx_ld=1), dict(dy_ld=1),
               dict(gate=11 * B, dgate=12 * B, flags=8, gate_ld=64, dgate_ld=60)):
        assert f(**kw) == -2, kw
    for kw in (dict(dh=B + 1), dict(du=2 * B + 2), dict(dx=7 * B + 2), dict(dgain_pre=9 * B + 2), dict(ws=10 * B + 8),
               dict(stats=6 * B + 2), dict(y=4 * B + 2)):
        assert f(**kw) == -3, kw
    assert f(ws=None) == -7 and f(ws_bytes=ws - 1) == -7
    for kw in (dict(dx=2 * B), dict(dx=B + 64), dict(dx=B, dx_ld=80), dict(dy=7 * B), dict(dy=4 * B), dict(dx=3 * B),
               dict(dgain_pre=5 * B), dict(ws=B), dict(ws=9 * B), dict(dgain_pre=6 * B)):
        assert f(**kw) == -8, kw
    assert f(n=0, flags=1, ws=None, dh=None, du=None, h=None, dx=None, stats=None) == 0
    size = repro.repro_block_norm_bwd_ws_bytes
    assert size(0, 64) == 0 and size(10, 0) == 0 and size(10, 16385) == 0 and size(17, 5) >= 3 * 8 * 4 * 3


def test_quant_rows(L):
    ok = dict(x=B, type=0, x_ld=64, mul=2 * B, n=10, D=64, flags=1, q=3 * B, q_ld=64, scales=4 * B, ws=5 * B, ws_bytes=256,
              stream=None)
    f = lambda **kw: call(L.repro_quant_rows_i8, ok, **kw)  # noqa: E731
    for kw in (dict(), dict(flags=0, ws=None, ws_bytes=0), dict(mul=None), dict(q=3 * B + 1), dict(x=B + 4), dict(type=1)):
        assert f(**kw) not in BAD, kw
    for kw in (dict(x=None), dict(q=None), dict(scales=None), dict(type=2), dict(flags=2)):
        assert f(**kw) == -1, kw
    for kw in (dict(n=-1), dict(D=0), dict(x_ld=63), dict(q_ld=63), dict(n=(1 << 31) + 1), dict(x_ld=(1 << 28) + 1),
               dict(D=(1 << 28) + 1, x_ld=1 << 29, q_ld=1 << 29)):
        assert f(**kw) == -2, kw
    for kw in (dict(x=B + 2), dict(mul=2 * B + 2), dict(scales=4 * B + 2), dict(ws=5 * B + 4)):
        assert f(**kw) == -3, kw
    assert f(ws=None) == -7 and f(ws_bytes=255) == -7
    for kw in (dict(q=B), dict(scales=B + 100), dict(scales=3 * B), dict(ws=2 * B), dict(q=2 * B)):
        assert f(**kw) == -8, kw
    assert f(n=0, flags=0, x=None, q=None, scales=None) == 0
    assert repro.repro_quant_rows_i8_ws_bytes(10, 64) == 0 and repro.repro_quant_rows_i8_ws_bytes(10, 64, True) == 256
    assert repro.repro_quant_rows_i8_ws_bytes(10, 0, True) == 0


def test_matmul(L):
    ws = repro.repro_matmul_i8_ws_bytes(100, 64, 128)
    ok = dict(a=B, a_ld=128, b=2 * B, b_ld=128, s_a=3 * B, s_b=4 * B, M=100, N=64, K=128, flags=0, y=5 * B, y_type=0,
              y_ld=64, ws=6 * B, ws_bytes=ws, stream=None)
    f = lambda **kw: call(L.repro_matmul_i8, ok, **kw)  # noqa: E731
    for kw in (dict(), dict(s_a=None, s_b=None), dict(y_type=1), dict(flags=1), dict(flags=2), dict(flags=6, b_ld=64),
               dict(a=B + 1, b=2 * B + 3, a_ld=129, b_ld=1001), dict(y=5 * B + 4, y_ld=65), dict(M=4, ws=None, ws_bytes=0)):
        assert f(**kw) not in BAD, kw
    for kw in (dict(a=None), dict(b=None), dict(y=None), dict(y_type=2), dict(flags=8), dict(flags=1, y_type=1)):
        assert f(**kw) == -1, kw
    top = repro.REPRO_MM_MAX_ROWS
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(K=133145, a_ld=140000, b_ld=140000), dict(M=top + 1),
               dict(N=top + 1, y_ld=top + 1), dict(a_ld=127), dict(b_ld=127), dict(y_ld=63), dict(flags=2, a_ld=99),
               dict(flags=4, b_ld=63), dict(y_ld=(1 << 28) + 1)):
        assert f(**kw) == -2, kw
    for kw in (dict(y=5 * B + 2), dict(s_a=3 * B + 2), dict(s_b=4 * B + 1), dict(ws=6 * B + 8)):
        assert f(**kw) == -3, kw
    assert f(ws=None) == -7 and f(ws_bytes=ws - 1) == -7
    for kw in (dict(y=B), dict(y=2 * B + 4), dict(y=3 * B), dict(ws=5 * B), dict(ws=B), dict(ws=4 * B)):
        assert f(**kw) == -8, kw
    assert f(M=0, a=None, y=None) == 0 and f(N=0) == 0 and f(K=0, flags=1, a=None, b=None) == 0
    size = repro.repro_matmul_i8_ws_bytes
    assert size(4, 64, 128) == 0 and size(16, 64, 127) == 0 and size(0, 64, 128) == 0 and size(17, 64, 133145) == 0
    assert size(1000, 2000, 515) >= 2 * 3000 * 520 and size(1, 64, 128, trans_b=True) > 0


def test_swiglu(L):
    G = 2
    ok = dict(gu=B, type=0, gu_ld=400, n=10, F=200, a=2 * B, a_type=0, a_ld=200, codes=3 * B, scales=4 * B, stream=None)
    f = lambda **kw: call(L.repro_swiglu_fwd, ok, **kw)  # noqa: E731
    for kw in (dict(), dict(codes=None, scales=None), dict(type=1, a_type=1), dict(gu=B + 4, gu_ld=401)):
        assert f(**kw) not in BAD, kw
    for kw in (dict(gu=None), dict(a=None), dict(codes=None), dict(scales=None), dict(type=2), dict(a_type=2)):
        assert f(**kw) == -1, kw
    for kw in (dict(n=-1), dict(F=0), dict(gu_ld=399), dict(a_ld=199), dict(F=(1 << 27) + 1, gu_ld=1 << 29, a_ld=1 << 29)):
        assert f(**kw) == -2, kw
    for kw in (dict(gu=B + 2), dict(a=2 * B + 2), dict(codes=3 * B + 8), dict(scales=4 * B + 2)):
        assert f(**kw) == -3, kw
    for kw in (dict(a=B), dict(codes=B), dict(scales=3 * B + 10 * 2 * G * 128 - 16), dict(scales=2 * B)):
        assert f(**kw) == -8, kw
    assert f(n=0, gu=None, a=None) == 0
    okb = dict(da=B, a_type=0, da_ld=200, gu=None, gu_ld=400, codes=3 * B, scales=4 * B, n=10, F=200, dgu=5 * B, type=0,
               dgu_ld=400, stream=None)
    f = lambda **kw: call(L.repro_swiglu_bwd, okb, **kw)  # noqa: E731
    for kw in (dict(), dict(gu=2 * B, codes=None, scales=None)):
        assert f(**kw) not in BAD, kw
    for kw in (dict(da=None), dict(dgu=None), dict(codes=None, scales=None), dict(gu=2 * B), dict(scales=None), dict(type=3)):
        assert f(**kw) == -1, kw
    for kw in (dict(n=-1), dict(F=0), dict(da_ld=199), dict(dgu_ld=399), dict(gu=2 * B, gu_ld=399)):
        assert f(**kw) == -2, kw
    assert f(dgu=5 * B + 2) == -3 and f(da=B + 2) == -3
    for kw in (dict(dgu=B), dict(dgu=3 * B), dict(dgu=4 * B), dict(dgu=2 * B, gu=2 * B, codes=None, scales=None)):
        assert f(**kw) == -8, kw
    assert f(n=0, da=None, dgu=None) == 0


def test_binding_checks(monkeypatch):
    """Shapes and types are refused before the library is reached."""
    class Reached:
        def __getattr__(self, name):
            def call(*a):
                raise AssertionError("not refused")
            return call

    class Device(torch.Tensor):              # host memory that passes for a device's
        is_cuda = property(lambda self: True)

    monkeypatch.setattr(repro, "lib", Reached)
    t = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt).as_subclass(Device)  # noqa: E731
    i8, bf = torch.int8, torch.bfloat16
    x = t(3, 8)
    bad = [
        lambda: repro.repro_block_norm_fwd(x, t(3, 8, dt=bf), t(3, 8), x),
        lambda: repro.repro_block_norm_fwd(x, t(2, 8), t(3, 8), x),
        lambda: repro.repro_block_norm_fwd(x, None, None, x, stats=t(3, 3)),
        lambda: repro.repro_block_norm_fwd(x, x, x, x, gate=t(7)),
        lambda: repro.repro_block_norm_fwd(x, x, x, x, gate=t(3, 8, dt=bf)),
        lambda: repro.repro_block_norm_fwd(x, None, None, x, g_pre=t(7)),
        lambda: repro.repro_block_norm_fwd(t(3, 8, dt=torch.float16), None, None, x),
        lambda: repro.repro_block_norm_bwd(x, x, x, x, t(3, 2), x, x, gate=t(8), dgate=t(3, 8)),
        lambda: repro.repro_block_norm_bwd(x, x, x, x, t(5), x, x),
        lambda: repro.repro_block_norm_bwd(x, x, x, x, t(3, 2), x, t(3, 9)),
        lambda: repro.repro_quant_rows_i8(x, t(3, 8), t(3)),
        lambda: repro.repro_quant_rows_i8(x, t(3, 8, dt=i8), t(8)),
        lambda: repro.repro_quant_rows_i8(x, t(3, 8, dt=i8), t(3), mul=t(3)),
        lambda: repro.repro_quant_rows_i8(x, t(3, 7, dt=i8), t(3)),
        lambda: repro.repro_matmul_i8(t(3, 8, dt=i8), t(5, 9, dt=i8), t(3, 5)),
        lambda: repro.repro_matmul_i8(t(3, 8, dt=i8), t(5, 8, dt=i8), t(5, 3)),
        lambda: repro.repro_matmul_i8(t(3, 8), t(5, 8, dt=i8), t(3, 5)),
        lambda: repro.repro_matmul_i8(t(3, 8, dt=i8), t(5, 8, dt=i8), t(3, 5), s_a=t(5)),
        lambda: repro.repro_matmul_i8(t(3, 8, dt=i8), t(5, 8, dt=i8), t(3, 5, dt=i8)),
        lambda: repro.repro_swiglu_fwd(t(3, 8), t(3, 5)),
        lambda: repro.repro_swiglu_fwd(t(3, 8), t(3, 4), t(3, 2, 1, 128, dt=i8)),
        lambda: repro.repro_swiglu_fwd(t(3, 8), t(3, 4), t(3, 2, 1, 127, dt=i8), t(3, 2, 1)),
        lambda: repro.repro_swiglu_bwd(t(3, 4), t(3, 8), gu=t(3, 8, dt=bf)),
        lambda: repro.repro_swiglu_bwd(t(3, 4), t(4, 8)),
    ]
    for f in bad:
        with pytest.raises(ValueError) as e:
            f()
        assert "CUDA" not in str(e.value), e.value
