"""A workspace that a call makes itself is allocated for the call's stream.  Memory of
the current stream may still have that stream's work to come (its former owner's), and
would be handed to the next owner there while the call runs."""
import contextlib

import pytest
import torch

from bitwise_reproducible_int8_gb300 import build_lib, repro

f32, i8, i32, u8 = torch.float32, torch.int8, torch.int32, torch.uint8


def t(*shape, dt=f32):
    return torch.zeros(shape, dtype=dt)


def attention(stream):
    x, rows = t(1, 70, 2, 128), t(1, 70, 2)
    repro.repro_attn_bwd(x, x, t(1, 70, 2, 128, dt=i8), t(1), x, x, rows, rows, x, x, x, stream=stream)


CALLS = {
    "wscale": lambda s: repro.repro_wscale(t(100), 0, t(1), stream=s),
    "linear_fwd": lambda s: repro.repro_linear_fwd(t(64, 64, dt=i8), t(64, 64, dt=i8), t(1), t(1), t(64, 64), stream=s),
    "linear_bwd": lambda s: repro.repro_linear_bwd(t(64, 64), t(64, 64, dt=i8), t(64, 64, dt=i8), t(1), t(1), t(64, 64),
                                                   t(64, 64), stream=s),
    "attn_bwd": attention,
    "sumsq": lambda s: repro.repro_sumsq(t(100), t(1), stream=s),
    "selftest": lambda s: repro.repro_selftest(torch.device("cpu"), stream=s),
    "embed_bwd": lambda s: repro.repro_embed_bwd(t(3, 4), t(3, dt=i32), t(10, 4), stream=s),
    "qk_norm_rope_bwd": lambda s: repro.repro_qk_norm_rope_bwd(t(3, 2, 8), None, t(3, 2, 8), None, None, t(3, 2, 8), None,
                                                               g_q=t(8), dg_q=t(8), stream=s),
    "distill_fwd": lambda s: repro.repro_distill_fwd(t(3, 50), t(3, 4, dt=i32), t(3, 4), t(3), t(3, 12), stream=s),
}


@pytest.fixture
def made(monkeypatch):
    """The streams that workspaces were made on (None: the current one)."""
    build_lib.build()
    current, made = [None], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (made.append(current[-1]), empty(*a, **k))[1])
    return made


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream,want", [(None, None), (0x5555, ("external", 0x5555)), (0, "default")])
def test_made_on_the_calls_stream(made, name, stream, want):
    with pytest.raises(ValueError, match="CUDA tensor"):      # after the workspace: these are host tensors
        CALLS[name](stream)
    assert made == [want]
