"""The workspaces that the feed-forward half's calls make themselves belong to the call's stream."""
import pytest
import torch

from bitwise_reproducible_int8_gb300 import repro
from test_workspace_stream import made, t  # noqa: F401

i8 = torch.int8


class Device(torch.Tensor):                  # host memory that passes the shape and type checks
    is_cuda = property(lambda self: True)


def d(*shape, dt=torch.float32):
    return t(*shape, dt=dt).as_subclass(Device)


CALLS = {
    "block_norm_bwd": lambda s: repro.repro_block_norm_bwd(d(3, 8), d(3, 8), d(3, 8), None, d(3, 2), d(3, 8), None, g_pre=d(8),
                                                           dg_pre=d(8), stream=s),
    "quant_columns": lambda s: repro.repro_quant_rows_i8(d(3, 8), d(3, 8, dt=i8), d(8), columns=True, stream=s),
    "matmul": lambda s: repro.repro_matmul_i8(d(30, 8, dt=i8), d(5, 8, dt=i8), d(30, 5), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream,want", [(None, None), (0x5555, ("external", 0x5555)), (0, "default")])
def test_made_on_the_calls_stream(made, name, stream, want):  # noqa: F811
    with pytest.raises(ValueError, match="CUDA tensor"):      # the workspace is a host tensor
        CALLS[name](stream)
    assert made == [want]
