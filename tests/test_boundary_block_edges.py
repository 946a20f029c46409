"""More refusals and admissions of the embedding, the per-head norm with rotation and the
distillation loss, through the C ABI on invented addresses: nothing is launched."""
import pytest

from bitwise_reproducible_int8_gb300 import repro
from test_boundary_blocks import B, BAD, QK, L, call, hp  # noqa: F401


@pytest.fixture
def qk_bwd(L):  # noqa: F811
    """The head norm's backward of 20 tokens of 16 and 4 heads of 64, some arguments replaced."""
    need = repro.repro_qk_norm_rope_bwd_ws_bytes(20, 16, 4, 64)
    ok = dict(dq_out=5 * B, dk_out=6 * B, **dict(QK, gain_q=7 * B, gain_k=8 * B), dq=9 * B, dq_ld=1024, dq_hs=64,
              dk=10 * B, dk_ld=256, dk_hs=64, dgain_q=11 * B, dgain_k=12 * B, ws=13 * B, ws_bytes=need, stream=None)
    return lambda **kw: call(L.repro_qk_norm_rope_bwd, ok, **kw)


def test_gradients_over_themselves(qk_bwd):
    """Strides that put two heads or tokens of dq (dk) in one place are refused: the writes race."""
    f = qk_bwd
    for kw in (dict(dq_ld=64), dict(dq_ld=1023), dict(dk_ld=255), dict(dq_ld=1), dict(dq_hs=128),
               dict(dk_hs=20 * 64 - 1, dk_ld=64), dict(dk_hs=20 * 64, dk_ld=63),
               dict(Hkv=1, dk_ld=63), dict(dq_hs=65, dq_ld=1024 + 14)):
        assert f(**kw) == -8, kw
    # token after token, head after head, with room between; a single token's or head's other stride
    for kw in (dict(dq_hs=65, dq_ld=1024 + 15), dict(dq_hs=20 * 64, dq_ld=64), dict(dk_hs=20 * 70, dk_ld=70),
               dict(Hkv=1, dk_ld=64), dict(n=1, dq_ld=1, dk_ld=3)):
        assert f(**kw) not in BAD, kw
    # inputs may share what they like
    assert f(q_ld=64, k_ld=1) not in BAD


def test_gradients_between_one_another(qk_bwd):
    """A fused gradient with q, k (and v) of each head side by side, tokens or heads outermost."""
    def f(slots, k_slot, n=20, heads_first=False, **kw):
        s = slots * 64
        ld, hs = (s, n * s) if heads_first else (4 * s, s)
        return qk_bwd(**{**dict(n=n, Hq=4, Hkv=4, dq_ld=ld, dq_hs=hs, dk=9 * B + k_slot * 64 * 4, dk_ld=ld, dk_hs=hs), **kw})

    for heads_first in (False, True):
        for slots, k_slot in ((2, 1), (3, 1), (3, 2), (3, -1)):
            assert f(slots, k_slot, heads_first=heads_first) not in BAD
        assert f(3, 0, heads_first=heads_first) == -8
        for off in (-4, 4):                                   # an element into the neighbour
            assert f(2, 1, heads_first=heads_first, dk=9 * B + 64 * 4 + off) == -8
        assert f(3, 1, heads_first=heads_first, dk=9 * B + 64 * 4 - 4) == -8
        assert f(3, 1, heads_first=heads_first, Hkv=2) not in BAD
    assert f(3, 1, dk_ld=4 * 3 * 64 + 64) == -8               # tokens at another distance
    assert f(3, 1, dq_ld=4 * 3 * 64 + 64, dk_ld=4 * 3 * 64 + 64) == -8    # no whole number of heads
    assert f(3, 1, n=1, dq_ld=1, dk_ld=5) not in BAD


def test_temperature_range(L):  # noqa: F811
    """The header's range of tau, both calls."""
    ws = repro.repro_distill_ws_bytes(40, 5000)
    common = dict(z=B, z_type=0, z_ld=5000, t_idx=2 * B)
    fwd = dict(common, t_val=3 * B, t_type=0, labels=None, index_bytes=4, n=40, V=5000, K=16, hp=hp(), flags=0,
               loss=5 * B, stats=6 * B, ws=7 * B, ws_bytes=ws, stream=None)
    bwd = dict(common, labels=None, index_bytes=4, n=40, V=5000, K=16, hp=hp(), stats=6 * B, g=8 * B, g_n=1,
               dz=9 * B, dz_ld=5000, stream=None)
    for fn, base in ((L.repro_distill_fwd, fwd), (L.repro_distill_bwd, bwd)):
        for tau in (1e-4, 0.5, 1e4):
            assert call(fn, base, hp=hp(tau=tau)) not in BAD, tau
        for tau in (9.9e-5, 1e-30, 1.01e4, 1e30):
            assert call(fn, base, hp=hp(tau=tau)) == -1, tau


def test_stride_of_a_single_row(L, qk_bwd):  # noqa: F811
    """The distance to a next row that is not there may be anything (a slice of a long cache)."""
    far = 1 << 40
    assert qk_bwd(n=1, q_ld=far, k_ld=far, dq_ld=far, dk_ld=far) not in BAD
    for kw in (dict(q_ld=far), dict(dk_ld=far)):
        assert qk_bwd(**kw) == -2, kw
    embed = dict(table=B, table_type=0, table_ld=far, s_w=None, tokens=2 * B, index_bytes=8, n=1, V=1, D=64, scale=1.0,
                 pad=-1, out=3 * B, out_type=0, out_ld=far, stream=None)
    assert call(L.repro_embed_fwd, embed) not in BAD
    assert call(L.repro_embed_fwd, embed, V=2) == -2 and call(L.repro_embed_fwd, embed, n=2) == -2
    loss = dict(z=B, z_type=0, z_ld=far, t_idx=None, labels=None, index_bytes=4, n=1, V=5000, K=0, hp=hp(), stats=6 * B,
                g=8 * B, g_n=1, dz=9 * B, dz_ld=far, stream=None)
    assert call(L.repro_distill_bwd, loss) not in BAD and call(L.repro_distill_bwd, loss, n=2) == -2
