"""Refusals of the embedding, the per-head norm with rotation and the distillation
loss, through the C ABI on invented addresses (nothing is launched) and through
the binding's own checks."""
import ctypes

import pytest
import torch

from bitwise_reproducible_int8_gb300 import build_lib, repro

NAN, INF = float("nan"), float("inf")
B = 1 << 40       # invented buffers, far apart
BAD = (-1, -2, -3, -7, -8)


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return repro.lib()


def call(fn, base, **kw):
    """fn with the named arguments of `base`, in order, some replaced."""
    assert set(kw) <= set(base), set(kw) - set(base)
    return fn(*{**base, **kw}.values())


def test_embed_fwd(L):
    ok = dict(table=B, table_type=0, table_ld=64, s_w=None, tokens=2 * B, index_bytes=8, n=10, V=100, D=64,
              scale=1.0, pad=-1, out=3 * B, out_type=0, out_ld=64, stream=None)
    f = lambda **kw: call(L.repro_embed_fwd, ok, **kw)  # noqa: E731
    assert f() not in BAD                                    # only the device is missing here
    for kw in (dict(table=None), dict(tokens=None), dict(out=None), dict(table_type=3), dict(out_type=2),
               dict(index_bytes=2), dict(scale=NAN), dict(scale=INF), dict(table_type=2), dict(s_w=4 * B)):
        assert f(**kw) == -1, kw
    for kw in (dict(n=-1), dict(V=0), dict(D=0), dict(table_ld=63), dict(out_ld=10), dict(n=1 << 31),
               dict(table_ld=1 << 29)):
        assert f(**kw) == -2, kw
    for kw in (dict(table=B + 2), dict(out=3 * B + 1), dict(tokens=2 * B + 4)):
        assert f(**kw) == -3, kw
    assert f(out=B + 4 * 64 * 99) == -8 and f(out=2 * B) == -8
    assert f(n=0, table=None, tokens=None, out=None) == 0
    assert f(table=B + 4) not in BAD                         # rows need only their type's alignment


def test_embed_bwd(L):
    ws = repro.repro_embed_bwd_ws_bytes(1000, 100, 64)
    ok = dict(dout=B, dout_type=0, dout_ld=64, tokens=2 * B, index_bytes=4, n=1000, V=100, D=64, scale=1.0,
              pad=-1, dtable=3 * B, dtable_ld=64, flags=0, ws=4 * B, ws_bytes=ws, stream=None)
    f = lambda **kw: call(L.repro_embed_bwd, ok, **kw)  # noqa: E731
    assert f() not in BAD
    for kw in (dict(dout=None), dict(tokens=None), dict(dtable=None), dict(dout_type=2), dict(flags=2),
               dict(index_bytes=1), dict(scale=-INF)):
        assert f(**kw) == -1, kw
    for kw in (dict(n=-1), dict(V=0), dict(V=repro.REPRO_EMBED_MAX_V + 1), dict(D=0), dict(dout_ld=1),
               dict(n=repro.REPRO_EMBED_MAX_N + 1),
               dict(dtable_ld=63)):
        assert f(**kw) == -2, kw
    assert f(ws=None) == -7 and f(ws_bytes=ws - 1) == -7
    assert f(ws=4 * B + 8) == -3 and f(dtable=3 * B + 2) == -3
    assert f(ws=3 * B) == -8 and f(dtable=B) == -8 and f(ws=2 * B) == -8
    assert f(n=0, flags=1, ws=None) == 0
    assert repro.repro_embed_bwd_ws_bytes(-1, 10, 10) == 0
    assert repro.repro_embed_bwd_ws_bytes(10, repro.REPRO_EMBED_MAX_V + 1, 10) == 0
    # no partial rows where no token can have a second chunk
    assert repro.repro_embed_bwd_ws_bytes(64, 10, 4096) < repro.repro_embed_bwd_ws_bytes(65, 10, 4096)


QK = dict(q=B, q_ld=24 * 64, q_hs=64, k=2 * B, k_ld=24 * 64, k_hs=64, type=0, gain_q=None, gain_k=None,
          rope=3 * B, P=128, positions=None, T=10, eps=1e-6, n=20, Hq=16, Hkv=4, D=64, R=64, flags=0)
QK_BAD = [(dict(q=None), -1), (dict(k=None), -1), (dict(rope=None), -1), (dict(type=2), -1), (dict(eps=-1.0), -1),
          (dict(eps=NAN), -1), (dict(eps=INF), -1), (dict(flags=4), -1), (dict(n=-1), -2), (dict(Hq=0), -2),
          (dict(Hkv=-1), -2), (dict(D=513, q_hs=600, k_hs=600), -2), (dict(D=0), -2), (dict(R=63), -2),
          (dict(R=66), -2), (dict(P=0), -2), (dict(T=0), -2), (dict(q_hs=63), -2), (dict(k_ld=0), -2),
          (dict(n=1 << 30), -2), (dict(q=B + 2), -3), (dict(rope=3 * B + 4), -3), (dict(positions=4 * B + 2), -3)]


def test_qk_norm_rope_fwd(L):
    ok = dict(QK, q_out=5 * B, k_out=6 * B, stream=None)
    f = lambda **kw: call(L.repro_qk_norm_rope_fwd, ok, **kw)  # noqa: E731
    assert f() not in BAD
    for kw, status in QK_BAD + [(dict(flags=1), -1), (dict(q_out=None), -1), (dict(k_out=None), -1),
                                (dict(q_out=5 * B + 4), -3), (dict(q_out=B + 64), -8), (dict(k_out=5 * B + 1024), -8),
                                (dict(q_out=3 * B), -8)]:
        assert f(**kw) == status, kw
    assert f(n=0, q=None, k=None, q_out=None, k_out=None) == 0
    assert f(Hkv=0, k=None, k_out=None) not in BAD
    assert f(Hkv=0, k=None, k_out=None, gain_k=7 * B) == -1
    assert f(R=0, rope=None, P=0, T=0) not in BAD


def test_qk_norm_rope_bwd(L):
    need = repro.repro_qk_norm_rope_bwd_ws_bytes(20, 16, 4, 64)
    ok = dict(dq_out=5 * B, dk_out=6 * B, **dict(QK, gain_q=7 * B, gain_k=8 * B), dq=9 * B, dq_ld=1024, dq_hs=64,
              dk=10 * B, dk_ld=256, dk_hs=64, dgain_q=11 * B, dgain_k=12 * B, ws=13 * B, ws_bytes=need, stream=None)
    f = lambda **kw: call(L.repro_qk_norm_rope_bwd, ok, **kw)  # noqa: E731
    assert need == (5 + 2) * 64 * 4
    assert f() not in BAD and f(flags=1) not in BAD
    for kw, status in QK_BAD + [(dict(dq_out=None), -1), (dict(dk=None), -1), (dict(dgain_q=None), -1),
                                (dict(gain_k=None), -1), (dict(dq_hs=32), -2), (dict(dk_ld=0), -2),
                                (dict(ws=None), -7), (dict(ws_bytes=need - 4), -7), (dict(ws=13 * B + 4), -3),
                                (dict(dq=B), -8), (dict(dk=6 * B), -8), (dict(dgain_q=12 * B), -8),
                                (dict(ws=9 * B), -8), (dict(dk=9 * B), -8)]:
        assert f(**kw) == status, kw
    # the gradient of the fused output: q's and k's heads side by side in one buffer
    fused = dict(dq=9 * B, dq_ld=24 * 64, dk=9 * B + 16 * 64 * 4, dk_ld=24 * 64)
    assert f(**fused) not in BAD
    assert f(**dict(fused, dk=9 * B + 15 * 64 * 4)) == -8     # k's first head over q's last
    assert f(**dict(fused, dk_ld=23 * 64)) == -8
    assert f(gain_q=None, dgain_q=None, gain_k=None, dgain_k=None, ws=None) not in BAD
    assert f(n=0, flags=1, dq=None, dk=None) == 0
    assert repro.repro_qk_norm_rope_bwd_ws_bytes(1, 1, 0, 513) == 0


def hp(tau=1.0, w_kd=1.0, w_ce=0.0, w_z=0.0):
    return ctypes.byref(repro.DistillHparams(tau, w_kd, w_ce, w_z))


DISTILL_BAD = [(dict(z=None), -1), (dict(t_idx=None), -1), (dict(z_type=2), -1), (dict(index_bytes=3), -1),
               (dict(hp=None), -1), (dict(hp=hp(tau=0.0)), -1), (dict(hp=hp(tau=NAN)), -1), (dict(hp=hp(tau=-1.0)), -1),
               (dict(hp=hp(tau=INF)), -1), (dict(hp=hp(w_kd=NAN)), -1), (dict(hp=hp(w_z=INF)), -1),
               (dict(hp=hp(w_ce=0.5), labels=None), -1), (dict(n=-1), -2), (dict(V=0), -2), (dict(K=-1), -2),
               (dict(K=65537), -2), (dict(z_ld=4999), -2), (dict(n=1 << 30), -2), (dict(z=B + 2), -3),
               (dict(t_idx=2 * B + 2), -3), (dict(labels=4 * B + 2), -3)]


def test_distill(L):
    ws = repro.repro_distill_ws_bytes(40, 5000)
    assert ws == 40 * (5 * 12 + 32)
    ok = dict(z=B, z_type=0, z_ld=5000, t_idx=2 * B, t_val=3 * B, t_type=0, labels=4 * B, index_bytes=4, n=40,
              V=5000, K=16, hp=hp(), flags=0, loss=5 * B, stats=6 * B, ws=7 * B, ws_bytes=ws, stream=None)
    f = lambda **kw: call(L.repro_distill_fwd, ok, **kw)  # noqa: E731
    assert f() not in BAD and f(flags=1) not in BAD and f(labels=None) not in BAD
    for kw, status in DISTILL_BAD + [(dict(t_val=None), -1), (dict(t_type=2), -1), (dict(flags=2), -1),
                                     (dict(loss=None), -1), (dict(stats=None), -1), (dict(ws=None), -7),
                                     (dict(ws_bytes=ws - 1), -7), (dict(ws=7 * B + 4), -3), (dict(loss=5 * B + 2), -3),
                                     (dict(loss=6 * B), -8), (dict(stats=B), -8), (dict(ws=3 * B), -8)]:
        assert f(**kw) == status, kw
    assert f(n=0, z=None, loss=None) == 0
    assert f(K=0, t_idx=None, t_val=None) not in BAD
    ok = dict(z=B, z_type=0, z_ld=5000, t_idx=2 * B, labels=4 * B, index_bytes=4, n=40, V=5000, K=16, hp=hp(),
              stats=6 * B, g=8 * B, g_n=40, dz=9 * B, dz_ld=5000, stream=None)
    f = lambda **kw: call(L.repro_distill_bwd, ok, **kw)  # noqa: E731
    assert f() not in BAD and f(g_n=1) not in BAD and f(dz=B) not in BAD       # in place
    for kw, status in DISTILL_BAD + [(dict(stats=None), -1), (dict(g=None), -1), (dict(dz=None), -1), (dict(g_n=2), -1),
                                     (dict(dz_ld=4999), -2), (dict(dz=9 * B + 1), -3), (dict(dz=B + 16), -8),
                                     (dict(dz=B, dz_ld=5004), -8), (dict(dz=6 * B), -8), (dict(dz=8 * B), -8)]:
        assert f(**kw) == status, kw


def test_binding_refuses(L):
    """Shapes, types and layouts the binding turns away before the library sees them."""
    t = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):                       # not on the device
        repro.repro_embed_fwd(t(10, 4), i(3), t(3, 4))
    with pytest.raises(ValueError):                       # widths differ
        repro.repro_embed_fwd(t(10, 4), i(3), t(3, 5))
    with pytest.raises(ValueError):                       # codes without a scale
        repro.repro_embed_fwd(t(10, 4, dt=torch.int8), i(3), t(3, 4))
    with pytest.raises(ValueError):                       # columns apart
        repro.repro_embed_fwd(t(4, 10).t(), i(3), t(3, 4))
    with pytest.raises(ValueError):                       # rows at two strides
        repro.repro_embed_fwd(t(10, 4), i(6), t(2, 5, 4)[:, :3])
    with pytest.raises(ValueError):                       # gradients are binary32
        repro.repro_embed_bwd(t(3, 4), i(3), t(10, 4, dt=torch.bfloat16))
    with pytest.raises(ValueError):
        repro.repro_qk_norm_rope_fwd(t(3, 2, 8), t(4, 2, 8), t(9, 8), t(3, 2, 8), t(4, 2, 8))
    with pytest.raises(ValueError):
        repro.repro_qk_norm_rope_fwd(t(3, 2, 8), None, t(9, 8), t(3, 2, 8), None, g_q=t(7))
    with pytest.raises(ValueError):
        repro.repro_qk_norm_rope_fwd(t(3, 2, 8, dt=torch.float16), None, t(9, 8), t(3, 2, 8), None)
    with pytest.raises(ValueError):                       # indexes and labels of two types
        repro.repro_distill_fwd(t(3, 50), i(3, 4), t(3, 4), t(3), t(3, 12), labels=i(3).long())
    with pytest.raises(ValueError):
        repro.repro_distill_fwd(t(3, 50), i(3, 4), t(3, 4), t(3), t(3, 11))
    with pytest.raises(ValueError):
        repro.repro_distill_bwd(t(3, 50), i(3, 4), t(3, 12), t(1), t(3, 50, dt=torch.bfloat16))
