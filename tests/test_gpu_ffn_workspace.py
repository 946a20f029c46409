"""GPU: the feed-forward calls in workspaces of exactly the stated size on any 16-byte boundary, as one
cut out of a caller's arena lies: the same bits as in a workspace of their own, and nothing written
around it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
import test_gpu_ffn as T  # noqa: E402
from gpu_helpers import dev, host  # noqa: E402
from test_gpu_blocks import same  # noqa: E402
from test_oracle_ffn import norm_case  # noqa: E402

pytestmark = pytest.mark.gpu
GUARD = 256


def arena(nbytes, off):
    """(workspace of nbytes, `off` past a 256-byte boundary; the bytes around it)."""
    buf = torch.full((2 * GUARD + off + nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0
    return buf[GUARD + off:GUARD + off + nbytes], (buf[:GUARD + off], buf[GUARD + off + nbytes:])


def untouched(around):
    return all(bool((b == 0xA5).all()) for b in around)


# products cut along K on pairs of SMs (all layouts), whole ones, of few tokens, and by transposed weights
MM = [(300, 260, 8192, True, True), (1024, 512, 8200, True, True), (200, 300, 4100, False, False), (150, 520, 3100, False, True),
      (500, 300, 96, False, False), (40, 300, 2064, False, False), (100, 129, 2064, False, False), (3, 528, 700, False, True)]


@pytest.mark.parametrize("M,N,K,a_t,b_t", MM)
@pytest.mark.parametrize("off", [0, 16, 32, 48, 240])
@pytest.mark.parametrize("kind,accumulate", [(T.F32, False), (T.F32, True), (T.BF, False)])
def test_matmul(M, N, K, a_t, b_t, off, kind, accumulate):
    a, b, sa, sb = T.mm_case(M, N, K)
    at, bt = (dev(np.ascontiguousarray(v.T) if t else v) for v, t in ((a, a_t), (b, b_t)))
    sa, sb = dev(sa), dev(sb)
    old = torch.linspace(-1, 1, M * N, device="cuda").view(M, N).to(kind)
    want, got = old.clone(), old.clone()
    R.repro_matmul_i8(at, bt, want, sa, sb, a_t, b_t, accumulate)
    ws, around = arena(R.repro_matmul_i8_ws_bytes(M, N, K, a_t, b_t), off)
    R.repro_matmul_i8(at, bt, got, sa, sb, a_t, b_t, accumulate, ws=ws)
    assert torch.equal(got, want) and untouched(around)
    if not accumulate and kind is T.F32:
        acc = (torch.from_numpy(a).double() @ torch.from_numpy(b).double().T).numpy().astype(np.float32)
        same(host(got), acc * host(sa)[:, None] * host(sb))
    assert R.repro_device_check() == R.REPRO_OK


@pytest.mark.parametrize("off", [16, 48, 240])
@pytest.mark.parametrize("n,D", [(40, 300), (19, 2048), (9000, 255)])
def test_block_norm_bwd(off, n, D):
    c = norm_case(n, D, "channel", True, True)
    t = {k: dev(v) for k, v in c.items() if isinstance(v, np.ndarray)}
    st = torch.rand((n, 2), device="cuda") + 0.5
    out = []
    for ws, around in ((None, ()), arena(R.repro_block_norm_bwd_ws_bytes(n, D), off)):
        o = [torch.empty((n, D), device="cuda") for _ in range(2)] + [torch.empty(D, device="cuda") for _ in range(3)]
        R.repro_block_norm_bwd(t["dh"], t["du"], t["x"], t["y"], st, o[0], o[1], gate=t["gate"], dgate=o[2], g_post=t["g_post"],
                               g_pre=t["g_pre"], dg_post=o[3], dg_pre=o[4], post=True, ws=ws)
        out.append(o)
        assert untouched(around)
    assert all(torch.equal(p, q) for p, q in zip(*out))


@pytest.mark.parametrize("off", [16, 48, 240])
@pytest.mark.parametrize("n,D", [(7, 33), (300, 1001), (100, 512)])
def test_quant_columns(off, n, D):
    x = torch.randn((n, D), device="cuda")
    out = []
    for ws, around in ((None, ()), arena(R.repro_quant_rows_i8_ws_bytes(n, D, True), off)):
        o = [torch.empty((n, D), dtype=torch.int8, device="cuda"), torch.empty(D, device="cuda")]
        R.repro_quant_rows_i8(x, *o, columns=True, ws=ws)
        out.append(o)
        assert untouched(around)
    assert all(torch.equal(p, q) for p, q in zip(*out))


@pytest.mark.parametrize("off", [16, 48, 240])
def test_selftest(off):
    ws, around = arena(R.lib().repro_selftest_ws_bytes(), off)
    assert R.lib().repro_selftest(ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == R.REPRO_OK
    assert untouched(around)
