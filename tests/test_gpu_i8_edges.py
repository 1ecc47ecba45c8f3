"""The 8-bit token path on the GPU where its arithmetic is narrowest: gates of every finite size, the bias in every
form of the product, rows whose squares are lost one at a time, and calls after a failed one.

Tolerances count roundings; u = 2^-24 is half a step of fp32, relative.
- silu(g) x: 2^t off by 4 u (2^-22, the approximate instruction), its correction, the sum with 1, the reciprocal
  (2^-23), and two products: 4 + 1 + 1 + 2 + 1 + 1 = 10 u; the scale's division adds one.
"""
import ctypes

import numpy as np
import pytest

from gpu_inputs import torch_mod
from test_gpu_i8 import U, _code, _dt, _gen, _i8_case, _pad16, _quantize, _rows, wr  # noqa: F401  (wr: fixture)

pytestmark = pytest.mark.gpu
FLT_MAX = float(np.finfo(np.float32).max)
SILU = 10 * U


def _silu64(g):
    """silu in 64 bits, without an overflow on either side."""
    torch = torch_mod()
    e = torch.exp(-g.abs())
    return torch.where(g >= 0, g / (1 + e), g * e / (1 + e))


def _gated_check(wr, gate, x, dt, ld=None):
    q, s = _quantize(wr, x.to(_dt(dt)), gate=gate.to(_dt(dt)), dt=dt, ld=ld, ldg=ld)
    torch = torch_mod()
    v = _silu64(gate.to(_dt(dt)).double()) * x.to(_dt(dt)).double()
    A = v.abs().amax(1)
    assert bool(torch.isfinite(s).all())
    # (scales below 2^-126 round to a step of 2^-149)
    assert bool(((s.double() - A / 127).abs() <= (SILU + U) * 1.01 * A / 127 + 2.0 ** -149).all()), \
        float(((s.double() * 127 / A - 1).abs() / U).nan_to_num().max())
    t = 127 * v / A[:, None]
    assert float((q.double() - t).abs().max()) <= 0.5 + 127 * (2 * SILU + U)


# ---------------------------------------------------------------- gates

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K,ld", [(1, 1), (5, 5), (7, 9), (320, 320), (2560, 2560), (9728, 9729), (40000, 40000)])
def test_very_large_gates_are_numbers(wr, dt, K, ld):  # noqa: F811
    """Gates up to the largest finite one: silu(g) = g there, and only a product past fp32 is an infinity."""
    torch = torch_mod()
    big = [60.0, 88.0, 89.0, 104.0, 130.0, 1e4, 1e10, 1e30, 2.2e38, 2.4e38, 3e38, 3.38e38]
    gate = torch.randn(len(big), K, device="cuda", generator=_gen(K))
    x = torch.randn(len(big), K, device="cuda", generator=_gen(K + 1))
    gate[:, K // 2] = torch.tensor(big, device="cuda")
    x[:, K // 2] = torch.where(torch.arange(len(big), device="cuda") % 2 == 0, 0.5, -0.75)
    _gated_check(wr, gate, x, dt, ld)


def test_a_gate_of_the_largest_number_and_infinities(wr):  # noqa: F811
    torch = torch_mod()
    gate = torch.full((7, 40), 1.0, device="cuda")
    x = torch.ones(7, 40, device="cuda")
    gate[0, 3] = FLT_MAX          # a number
    gate[1, 3], x[1, 3] = FLT_MAX, 2.0   # the product is not
    gate[2, 3] = float("inf")
    gate[3, 3] = float("nan")
    gate[4, 3], x[4, 3] = -FLT_MAX, FLT_MAX   # silu reads as 0
    gate[5] = -FLT_MAX
    gate[6, 3] = -float("inf")    # -inf / inf
    q, s = _quantize(wr, x, gate=gate)
    assert abs(float(s[0]) * 127 / FLT_MAX - 1) <= 12 * U and int(q[0, 3]) == 127 and not q[0, 4:].any()
    assert bool(torch.isnan(s[1:4]).all()) and not q[1:4].any()
    assert int(q[4, 3]) == 0 and bool((q[4, 4:] == 127).all())
    assert float(s[5]) == 0 and not q[5].any()
    assert bool(torch.isnan(s[6])) and not q[6].any()


@pytest.mark.parametrize("lo,hi", [(-87.3, -80), (-80, -60), (-60, -40), (-40, -20), (-20, -5), (-5, 5), (5, 88), (88, 300)])
def test_silu_of_one_band_of_gates(wr, lo, hi):  # noqa: F811
    """Rows of one value, so that each scale shows one silu: within its bound in every band of gates."""
    torch = torch_mod()
    M = 60000
    gate = (lo + (hi - lo) * torch.rand(M, 1, device="cuda", generator=_gen(int(hi)), dtype=torch.float64)).float()
    x = (1 + torch.rand(M, 1, device="cuda", generator=_gen(3))) * 2.0 ** 60
    _gated_check(wr, gate, x, "f32")


def test_rows_of_negative_gates(wr):  # noqa: F811
    torch = torch_mod()
    for at in (-10.0, -40.0, -80.0, -86.0):
        gate = at + torch.rand(9, 2560, device="cuda", generator=_gen(int(-at)))
        x = torch.randn(9, 2560, device="cuda", generator=_gen(5)) * 2.0 ** 50
        _gated_check(wr, gate, x, "f32")


# ---------------------------------------------------------------- the product's roundings

SHAPES = [(1, 200, 2000), (2, 513, 4100), (1, 5400, 2560), (3, 640, 2560), (8, 2560, 4096), (12, 4000, 1000), (16, 640, 300),
          (9, 8192, 640), (17, 300, 128), (64, 256, 4096), (64, 2560, 9728), (40, 6144, 640), (128, 130, 77), (300, 2560, 2560),
          (333, 2560, 4096), (256, 19456, 640), (512, 9728, 300), (1024, 2560, 512), (2048, 2560, 640)]


# both sides of where short rows go from one kernel to another
SHORT_ROWS = [(m, n, k) for m in (1, 2) for n, k in ((1024, 1024), (1025, 1024), (1030, 1025), (5328, 1025), (5329, 1025), (5328, 2048), (5329, 2048),
                                                   (5329, 2049), (8193, 1023), (8193, 1024), (12288, 1025), (12289, 1025), (12289, 1791), (12289, 1792), (12289, 2049), (20000, 1100))]
SHORT_ROWS += [(m, n, k) for m in (3, 8, 9) for n, k in ((8193, 1023), (8193, 1024), (12288, 2048), (12289, 1791), (12289, 1792), (12301, 2049), (8193, 4096))]


@pytest.mark.parametrize("ydt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES + SHORT_ROWS)
def test_gemm_i8_rounds_each_step_once(wr, M, N, K, ydt):  # noqa: F811
    """The conversion, two products and the bias round one after the other, in every form: the bits of the same steps
    as separate operations."""
    torch = torch_mod()
    x, w, xs, ws = _i8_case(M, N, K, M + N + K)
    bias = torch.randn(N, device="cuda", generator=_gen(N)) * 0.1
    _, xv = _rows(x, _pad16(K), extra=0)
    _, wv = _rows(w, _pad16(K), extra=0)
    acc = (x.double() @ w.double().t()).float()
    for ld in (N, N + 3):
        y = torch.empty(M, ld, dtype=_dt(ydt), device="cuda")[:, :N]
        wr.wr_gemm_i8(M, N, K, xv, _pad16(K), xs, wv, _pad16(K), ws, _code(wr, ydt), y, ld, None, 0, bias=bias)
        want = acc * xs[:, None]
        want = want * ws
        want = want + bias
        assert torch.equal(y, want.to(_dt(ydt)))


def test_gemm_i8_same_bits_for_every_batch_with_a_bias(wr):  # noqa: F811
    torch = torch_mod()
    N, K = 2560, 4096
    x, w, xs, ws = _i8_case(700, N, K, 9)
    bias = torch.randn(N, device="cuda", generator=_gen(2)) * 0.1
    rows = []
    for M in (700, 1, 2, 3, 8, 9, 16, 17, 64, 100, 256, 333):
        y = torch.empty(M, N, device="cuda")
        wr.wr_gemm_i8(M, N, K, x, K, xs, w, K, ws, wr.WR_F32, y, N, None, 0, bias=bias)
        rows.append(y)
    for y in rows[1:]:
        assert torch.equal(y, rows[0][:y.shape[0]])


# ---------------------------------------------------------------- sums of squares

@pytest.mark.parametrize("D", [2048, 4096, 16384, 32768])
@pytest.mark.parametrize("M", [1, 400])
def test_norm_of_a_row_whose_small_squares_come_one_at_a_time(wr, M, D):  # noqa: F811
    """One value of 1 and, at the start of 256-value stretches, values whose squares are just under half a step of 1:
    added to the large one after the other all are lost. The sum is a chain of at most 16 squares in a thread and then
    a tree: 16 + 1 + 5 + 5 roundings, and two of the mean; a root keeps half of these, and adds 4 u of its own (2 ulp);
    the product after it 1: 19.5 u."""
    torch = torch_mod()
    small = float(np.sqrt(np.float64(2.0 ** -24 * 0.98)))
    for part in (1, 2, 4):
        h = torch.zeros(M, D, device="cuda")
        h[:, : D // part : 256] = small
        for near in (8, 16, 32, 64, 128, *(i * D // part + j for i in range(part) for j in (0, 2, 4, 6))):
            h[:, near] = small
        h[:, 0] = 1.0
        y = torch.empty(M, D, device="cuda")
        wr.wr_residual_norm(M, D, residual=h, ld_residual=D, y=y, ld_y=D, eps=0.0)
        v = h.double()
        ref = v / torch.sqrt((v * v).mean(1, keepdim=True))
        err = ((y.double() - ref).abs() / ref.abs().clamp_min(1e-30)).max()
        assert float(err) <= 19.5 * U, float(err) / U


# ---------------------------------------------------------------- after a call that failed

def _driver():
    lib = ctypes.CDLL("libcuda.so.1")
    lib.cuStreamBeginCapture_v2.argtypes = [ctypes.c_void_p, ctypes.c_int]
    lib.cuStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]
    return lib


def test_a_failed_call_does_not_fail_the_next(wr):  # noqa: F811
    """A product issued into a capture that has been broken off reports that; the calls after it, on other streams, are
    not blamed for it."""
    torch = torch_mod()
    M, N, K = 40, 64, 256
    x, w, xs, ws = _i8_case(M, N, K, 1)
    y, h = torch.zeros(M, N, device="cuda"), torch.randn(M, K, device="cuda", generator=_gen(1))
    q, s, z = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, K, device="cuda")

    def product(m, stream):
        wr.wr_gemm_i8(m, N, K, x, K, xs, w, K, ws, wr.WR_F32, y, N, None, 0, stream=stream)

    stream = torch.cuda.Stream()
    for m in (1, 8, 40):   # each of the product's launches
        product(m, None)
    torch.cuda.synchronize()
    driver = _driver()
    relaxed = 2
    for m in (1, 8, 40):
        assert driver.cuStreamBeginCapture_v2(stream.cuda_stream, relaxed) == 0
        assert wr.wr_get_device_error(stream) == 3   # a wait for a stream that is being captured: breaks the capture off
        try:
            with pytest.raises(wr.WrError) as e:
                product(m, stream)
            assert e.value.status == 3
            wr.wr_quantize_rows(wr.WR_F32, M, K, h, K, q, K, s)
            wr.wr_residual_norm(M, K, residual=h, ld_residual=K, y=z, ld_y=K)
            product(m, None)
        finally:
            graph = ctypes.c_void_p()
            assert driver.cuStreamEndCapture(stream.cuda_stream, ctypes.byref(graph)) != 0 and not graph.value
    # a failure that is not the path's own
    assert driver.cuStreamBeginCapture_v2(stream.cuda_stream, relaxed) == 0
    assert wr.wr_get_device_error(stream) == 3
    driver.cuStreamEndCapture(stream.cuda_stream, ctypes.byref(ctypes.c_void_p()))
    wr.wr_residual_norm(M, K, residual=h, ld_residual=K, y=z, ld_y=K)
    torch.cuda.synchronize()
    assert wr.wr_get_device_error() == 0


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("M,N,K", [
    (40, 20000, 65536),     # a CTA a tile
    (17, 300, 131071),      # clusters that share a tile
    (200, 2560, 131071),
    (300, 2560, 131071),    # clusters of pairs
    (64, 10240, 65536),     # pairs that take tiles in turn
    (512, 9728, 65536),     # and cut tiles
])
def test_a_product_whose_waits_run_out_ends_and_says_so(wr, M, N, K):  # noqa: F811
    """The failure path of each tcgen05 form, with copies and MMAs in flight: the kernel ends, the error word tells, and
    the calls behind it, one of the same form at once among them, are what they should be."""
    torch = torch_mod()
    ld = _pad16(K)
    x = torch.randint(-128, 128, (M, ld), device="cuda", generator=_gen(M), dtype=torch.int8)
    w = torch.randint(-128, 128, (N, ld), device="cuda", generator=_gen(N), dtype=torch.int8)
    xs, ws = torch.full((M,), 2.0 ** -20, device="cuda"), torch.ones(N, device="cuda")
    y, z, lost = (torch.full((M, N), float("nan"), device="cuda") for _ in range(3))
    assert wr.wr_get_device_error() == 0
    wr.wr_gemm_i8(M, N, K, x, ld, xs, w, ld, ws, wr.WR_F32, y, N, None, 0)
    assert wr.wr_get_device_error() == 0
    for _ in range(3):
        wr.wr_selftest_gemm_i8_timeout(M, N, K, x, ld, xs, w, ld, ws, lost, N)
        wr.wr_gemm_i8(M, N, K, x, ld, xs, w, ld, ws, wr.WR_F32, z, N, None, 0)
        assert wr.wr_get_device_error() == 4
        assert wr.wr_get_device_error() == 0
        assert torch.equal(y, z)
        z.fill_(float("nan"))
    rows = slice(0, N, max(1, N // 50))
    ref = (x[:, :K].double() @ w[rows, :K].double().t()) * 2.0 ** -20
    assert bool(((y[:, rows].double() - ref).abs() <= U * ref.abs()).all())


# ---------------------------------------------------------------- the workspace that is not needed

@pytest.mark.parametrize("M", [1, 8, 16, 40, 300, 1500])
def test_gemm_i8_with_and_without_a_workspace(wr, M):  # noqa: F811
    """No size needs a workspace: y is the same without one and with one, which is left as it was."""
    torch = torch_mod()
    N, K = 640, 2048
    x, w, xs, ws = _i8_case(M, N, K, M)
    space = torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda")
    ys = []
    for workspace, size in ((None, 0), (space, space.numel()), (space.data_ptr() + 8, 4)):
        y = torch.full((M, N), float("nan"), device="cuda")
        wr.wr_gemm_i8(M, N, K, x, K, xs, w, K, ws, wr.WR_F32, y, N, workspace, size)
        ys.append(y)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2]) and bool((space == 7).all())
