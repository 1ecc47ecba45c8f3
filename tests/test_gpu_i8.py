"""The 8-bit token path on the GPU (wr_quantize_rows, wr_gemm_i8, wr_residual_norm) against plain
implementations in 64 bits.

Tolerances count roundings; u = 2^-24 is half a step of fp32, relative.
- wr_gemm_i8: the integer sum is exact; its conversion, two products and the bias round once each:
  4 u of |sum * scales| + |bias|, then half a step of y's type.
- wr_quantize_rows without a gate: no tolerance (codes are the exact decision, the scale is one
  rounded division). With a gate v = silu(g) x is off by at most 8 u: expf 1 step (2 u), the sum u, the
  division 2 steps (4 u), the product u.
- wr_residual_norm: a mean of squares is a chain of at most 32 additions a thread and a tree of 10:
  42 u, and 2 for the squares and the division by D; its root halves that (22 u), and root, reciprocal
  and the three products after it add 6: under 32 u relative for a norm of exact inputs.
"""
import numpy as np
import pytest

from gpu_inputs import torch_mod

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SENTINEL = 77


@pytest.fixture(scope="module")
def wr():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_weight_only_wr_b200 as lib
    return lib


def _dt(name):
    torch = torch_mod()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}[name]


def _code(wr, name):
    return {"f32": wr.WR_F32, "bf16": wr.WR_BF16, "f16": wr.WR_F16, "i8": wr.WR_I8}[name]


def _half_step(dtype):
    """(relative, absolute) rounding of a type: half a step of normal and of subnormal values."""
    torch = torch_mod()
    f = torch.finfo(dtype)
    return f.eps / 2, f.tiny * f.eps / 2


def _rows(t, ld, extra=1, fill=SENTINEL):
    """t copied into rows ld apart inside a buffer with `extra` more rows; (buffer, view)."""
    torch = torch_mod()
    M, K = t.shape
    buf = torch.full((M + extra, ld), fill, dtype=t.dtype, device="cuda")
    buf[:M, :K] = t
    return buf, buf[:M, :K]


def _empty_rows(M, K, ld, dtype):
    torch = torch_mod()
    buf = torch.full((M + 1, ld), SENTINEL, dtype=dtype, device="cuda")
    return buf, buf[:M, :K]


def _untouched(buf, M, K):
    """Nothing behind the rows' ends and nothing behind the last row was written."""
    assert bool((buf[:M, K:] == SENTINEL).all()) and bool((buf[M:] == SENTINEL).all())


def _pad16(n):
    return (n + 15) // 16 * 16


def _gen(seed):
    torch = torch_mod()
    return torch.Generator(device="cuda").manual_seed(seed)


# ---------------------------------------------------------------- wr_gemm_i8

def _i8_case(M, N, K, seed, extreme=False):
    torch = torch_mod()
    g = _gen(seed)
    x = torch.randint(-128, 128, (M, K), device="cuda", generator=g, dtype=torch.int32).to(torch.int8)
    w = torch.randint(-128, 128, (N, K), device="cuda", generator=g, dtype=torch.int32).to(torch.int8)
    if extreme:
        x.fill_(-128)
        w.fill_(-128)
    xs = torch.rand(M, device="cuda", generator=g) * 0.05
    ws = torch.rand(N, device="cuda", generator=g) * 1e-3
    return x, w, xs, ws


def _i8_workspace(wr, M, N, K):
    torch = torch_mod()
    n = wr.wr_gemm_i8_workspace_bytes(M, N, K)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda"), n


def _i8_check(wr, x, w, xs, ws, ydt="f32", bias=None, ldx=None, ldw=None, ldy=None, workspace=None, stream=None):
    torch = torch_mod()
    (M, K), N = x.shape, w.shape[0]
    ldx, ldw, ldy = ldx or _pad16(K), ldw or _pad16(K), ldy or N
    _, xv = _rows(x, ldx, extra=0)
    _, wv = _rows(w, ldw, extra=0)
    buf, y = _empty_rows(M, N, ldy, _dt(ydt))
    space, nb = workspace or _i8_workspace(wr, M, N, K)
    wr.wr_gemm_i8(M, N, K, xv, ldx, xs, wv, ldw, ws, _code(wr, ydt), y, ldy, space, nb, bias=bias, stream=stream)
    acc = x.double() @ w.double().t()
    p = acc * xs.double()[:, None] * ws.double()
    ref = p if bias is None else p + bias.double()
    rel, sub = _half_step(y.dtype)
    mag = p.abs() if bias is None else p.abs() + bias.double().abs()
    tol = 4.01 * U * mag + rel * ref.abs() * 1.001 + sub
    if ydt == "f16":
        over = ref.abs() >= 65519   # rounds to infinity near there
        assert bool((y[over].abs() >= 65504).all())
        tol[over] = float("inf")
    err = (y.double() - ref).abs()
    if ydt == "f16":
        err[over] = 0
    assert bool((err <= tol).all()), float((err / tol).max())
    _untouched(buf, M, N)
    assert wr.wr_get_device_error() == 0
    return y


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 64, 65, 100, 128, 129, 192, 255, 256, 257, 300])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 15), (129, 272), (260, 1259)])
def test_gemm_i8_tokens(wr, M, N, K):
    _i8_check(wr, *_i8_case(M, N, K, 100 + M * 7 + N))


@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 31, 32, 63, 64, 100, 127, 128, 129, 255, 256, 257, 1000, 2560, 4097, 9728])
@pytest.mark.parametrize("M", [1, 6, 20, 70, 270])
def test_gemm_i8_depths(wr, M, K):
    _i8_check(wr, *_i8_case(M, 77, K, 3 * K + M), ydt="f32")


@pytest.mark.parametrize("N", [1, 3, 16, 31, 33, 127, 128, 129, 255, 256, 257, 640, 2560])
@pytest.mark.parametrize("M", [1, 8, 40, 130, 513])
def test_gemm_i8_channels(wr, M, N):
    _i8_check(wr, *_i8_case(M, N, 640, 5 * N + M), ydt="bf16")


@pytest.mark.parametrize("ydt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 200, 300), (7, 200, 300), (50, 200, 300), (600, 520, 700)])
def test_gemm_i8_types_bias_strides(wr, ydt, M, N, K):
    torch = torch_mod()
    x, w, xs, ws = _i8_case(M, N, K, M + N + K)
    bias = torch.randn(N, device="cuda", generator=_gen(1))
    _i8_check(wr, x, w, xs, ws, ydt, bias=bias, ldx=_pad16(K) + 48, ldw=_pad16(K) + 112, ldy=N + 5)
    _i8_check(wr, x, w, xs, ws, ydt, bias=None, ldy=N + 1)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 2560), (32, 6144, 2560), (333, 2560, 9728), (1, 2560, 9728), (16, 1024, 2560),
                                   (512, 9728, 2560), (1000, 1024, 4096), (2048, 2560, 2560), (3, 19456, 2560), (4100, 300, 200)])
def test_gemm_i8_layer_shapes(wr, M, N, K):
    _i8_check(wr, *_i8_case(M, N, K, M + N + K), ydt="bf16" if M % 2 else "f32")


@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_gemm_i8_largest_sums(wr, M):
    """Every product 16384 at the largest K: the sum is 2^31 - 16384, the most an int32 holds here."""
    x, w, xs, ws = _i8_case(M, 130, 131071, 5, extreme=True)
    _i8_check(wr, x, w, xs, ws)


def test_gemm_i8_same_bits_for_every_batch(wr):
    """A token's row does not depend on the batch it is in, nor on the run."""
    torch = torch_mod()
    x, w, xs, ws = _i8_case(300, 384, 2000, 9)
    whole = _i8_check(wr, x, w, xs, ws).clone()
    for M in (1, 3, 8, 9, 30, 70, 128, 200):
        assert torch.equal(_i8_check(wr, x[:M], w, xs[:M], ws), whole[:M])
    for _ in range(3):
        assert torch.equal(_i8_check(wr, x, w, xs, ws), whole)


def test_gemm_i8_scales_of_zero_and_nan(wr):
    """A padding token (scale 0) gives zeros, a poisoned token or channel (scale NaN) NaN, and only there."""
    torch = torch_mod()
    for M in (4, 50, 300):
        x, w, xs, ws = _i8_case(M, 150, 256, M)
        xs[1], xs[2], ws[7] = 0.0, float("nan"), float("nan")
        x[2] = 0
        y = torch.empty(M, 150, device="cuda")
        space, nb = _i8_workspace(wr, M, 150, 256)
        wr.wr_gemm_i8(M, 150, 256, x, 256, xs, w, 256, ws, wr.WR_F32, y, 150, space, nb)
        bad = torch.zeros(M, 150, dtype=torch.bool, device="cuda")
        bad[2] = True
        bad[:, 7] = True
        assert torch.equal(torch.isnan(y), bad)
        assert bool((y[1][~bad[1]] == 0).all())


def test_gemm_i8_rows_past_32_bits(wr):
    """Rows 2^30 bytes apart: the last starts behind 2^32."""
    torch = torch_mod()
    ld, K = 1 << 30, 300
    for M, N in ((2, 6), (40, 6), (6, 40)):
        x, w, xs, ws = _i8_case(M, N, K, 4)
        big = max(M, N)
        if M > 6:
            _i8_check_rows(wr, x, w, xs, ws, _pad16(K), ld)
        else:
            _i8_check_rows(wr, x, w, xs, ws, ld, ld if big == N and N <= 6 else _pad16(K))


def _i8_check_rows(wr, x, w, xs, ws, ldx, ldw):
    torch = torch_mod()
    (M, K), N = x.shape, w.shape[0]
    xb = torch.empty((M - 1) * ldx + _pad16(K), dtype=torch.int8, device="cuda").as_strided((M, K), (ldx, 1))
    wb = torch.empty((N - 1) * ldw + _pad16(K), dtype=torch.int8, device="cuda").as_strided((N, K), (ldw, 1))
    xb.copy_(x)
    wb.copy_(w)
    y = torch.empty(M, N, device="cuda")
    space, nb = _i8_workspace(wr, M, N, K)
    wr.wr_gemm_i8(M, N, K, xb, ldx, xs, wb, ldw, ws, wr.WR_F32, y, N, space, nb)
    p = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    assert bool(((y.double() - p).abs() <= 4.01 * U * p.abs()).all())


def test_gemm_i8_reads_nothing_behind_the_rows(wr):
    """The last row ends at its last element: the operands sit at the very end of their storage, and
    what stands between rows (K not a multiple of 16) does not matter."""
    torch = torch_mod()
    for M, N, K in ((1, 5, 33), (8, 130, 77), (40, 130, 77), (300, 260, 1001)):
        x, w, xs, ws = _i8_case(M, N, K, K)
        y0 = _i8_check(wr, x, w, xs, ws)
        ld = _pad16(K)
        xb = torch.full(((M - 1) * ld + K,), 99, dtype=torch.int8, device="cuda").as_strided((M, K), (ld, 1))
        wb = torch.full(((N - 1) * ld + K,), -55, dtype=torch.int8, device="cuda").as_strided((N, K), (ld, 1))
        xb.copy_(x)
        wb.copy_(w)
        y = torch.empty(M, N, device="cuda")
        space, nb = _i8_workspace(wr, M, N, K)
        wr.wr_gemm_i8(M, N, K, xb, ld, xs, wb, ld, ws, wr.WR_F32, y, N, space, nb)
        assert torch.equal(y, y0)


def test_gemm_i8_workspace_serves_many_calls_and_streams(wr):
    """One zeroed workspace for calls of several sizes in stream order; two streams with their own."""
    torch = torch_mod()
    shapes = [(64, 256, 4096), (300, 1024, 640), (20, 640, 9728), (64, 256, 4096)]
    nb = max(wr.wr_gemm_i8_workspace_bytes(*s) for s in shapes)
    space = torch.zeros(max(nb, 16), dtype=torch.uint8, device="cuda")
    for i, s in enumerate(shapes):
        _i8_check(wr, *_i8_case(*s, 50 + i), workspace=(space, nb))
    streams = [torch.cuda.Stream() for _ in range(2)]
    cases = [_i8_case(*shapes[i], 60 + i) for i in range(2)]
    spaces = [_i8_workspace(wr, *shapes[i]) for i in range(2)]
    ys = [torch.empty(s[0], s[1], device="cuda") for s in shapes[:2]]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, st in enumerate(streams):
            (M, N, K), (x, w, xs, ws) = shapes[i], cases[i]
            wr.wr_gemm_i8(M, N, K, x, K, xs, w, K, ws, wr.WR_F32, ys[i], N, *spaces[i], stream=st)
    torch.cuda.synchronize()
    for i in range(2):
        x, w, xs, ws = cases[i]
        assert torch.equal(ys[i], _i8_check(wr, x, w, xs, ws))


def test_i8_path_in_a_graph(wr):
    """Quantizer and product captured once and replayed on new inputs."""
    torch = torch_mod()
    for M in (1, 40, 300):
        N, K = 384, 2560
        h = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
        q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        _, w, _, ws = _i8_case(M, N, K, 3)
        y = torch.empty(M, N, device="cuda")
        space, nb = _i8_workspace(wr, M, N, K)

        def step(stream=None):
            wr.wr_quantize_rows(wr.WR_BF16, M, K, h, K, q, K, s, stream=stream)
            wr.wr_gemm_i8(M, N, K, q, K, s, w, K, ws, wr.WR_F32, y, N, space, nb, stream=stream)

        h.copy_(torch.randn(M, K, device="cuda", generator=_gen(1)))
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for seed in (2, 3):
            h.copy_(torch.randn(M, K, device="cuda", generator=_gen(seed)))
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            got = y.clone()
            step()
            torch.cuda.synchronize()
            assert torch.equal(got, y) and bool((got != 0).any())


# ---------------------------------------------------------------- wr_quantize_rows

def _codes64(v):
    """(codes, scale) of fp32 rows v (numpy), decided in 64 bits."""
    A = np.abs(v).max(axis=1).astype(np.float32)
    safe = np.where(A > 0, A, 1).astype(np.float64)
    q = np.rint(v.astype(np.float64) * 127 / safe[:, None])
    return q.astype(np.int8), A / np.float32(127)


def _quantize(wr, x, ld=None, ldq=None, gate=None, ldg=None, dt="f32"):
    torch = torch_mod()
    M, K = x.shape
    ld, ldq = ld or K, ldq or K
    _, xv = _rows(x, ld, extra=0)
    gv = None
    if gate is not None:
        _, gv = _rows(gate, ldg or K, extra=0)
    buf, q = _empty_rows(M, K, ldq, torch.int8)
    s = torch.full((M + 1,), float(SENTINEL), device="cuda")
    wr.wr_quantize_rows(_code(wr, dt), M, K, xv, ld, q, ldq, s, gate=gv, ldg=ldg or K)
    _untouched(buf, M, K)
    assert float(s[M]) == SENTINEL
    return q, s[:M]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 31), (7, 100), (2, 255), (33, 256), (3, 1259), (17, 2560),
                                 (2, 4096), (2, 4097), (3, 8192), (2, 8200), (3, 9728), (2, 16384), (2, 16392), (2, 32768),
                                 (2, 32769), (2, 50000), (3, 50008), (2000, 320)])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_quantize_rows_exact(wr, dt, M, K, pad):
    torch = torch_mod()
    x = (torch.randn(M, K, device="cuda", generator=_gen(M + K)) * 3).to(_dt(dt))
    q, s = _quantize(wr, x, ld=K + pad, ldq=K + pad, dt=dt)
    qr, sr = _codes64(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)


def test_quantize_rows_ties_and_their_neighbours(wr):
    """Values at the middle of two codes (to the even one) and the fp32 values next to them, for largest
    values that 127 divides and that it does not, of every magnitude down to subnormals."""
    torch = torch_mod()
    rng = np.random.default_rng(0)
    rows = []
    for A in [127.0, 1.0, 254.0, 3.0, 1e30, 3e38, 1e-30, 1e-37, 1e-40, 5e-45, 127 * 2.0 ** -140, 2.0 ** -126] + list(rng.uniform(0.5, 2, 20)):
        A = np.float32(A)
        mid = ((np.arange(-127, 127) + 0.5) * np.float64(A) / 127).astype(np.float32)
        near = [mid]
        for k in (1, 2, 3):
            up, dn = mid.copy(), mid.copy()
            for _ in range(k):
                up, dn = np.nextafter(up, np.float32(np.inf)), np.nextafter(dn, np.float32(-np.inf))
            near += [up, dn]
        r = np.concatenate(near + [[A]]).astype(np.float32)
        rows.append(np.clip(r, -A, A))
    v = np.stack(rows)
    q, s = _quantize(wr, torch.from_numpy(v).cuda())
    qr, sr = _codes64(v)
    assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)


@pytest.mark.parametrize("K", [5, 2560, 12000, 40000])
def test_quantize_rows_zero_and_poisoned_rows(wr, K):
    torch = torch_mod()
    x = torch.randn(6, K, device="cuda", generator=_gen(K))
    x[1] = 0
    x[2, K // 2] = float("nan")
    x[3, K - 1] = float("inf")
    x[4, 0] = float("-inf")
    q, s = _quantize(wr, x)
    assert float(s[1]) == 0 and bool((q[1:5] == 0).all())
    assert bool(torch.isnan(s[2:5]).all())
    qr, sr = _codes64(x[[0, 5]].cpu().numpy())
    assert np.array_equal(q[[0, 5]].cpu().numpy(), qr) and np.array_equal(s[[0, 5]].cpu().numpy(), sr)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,ld,ldg", [(1, 9728, 9728, 9728), (5, 1, 1, 1), (4, 77, 80, 77), (9, 2560, 5120, 5120), (3, 333, 335, 340),
                                        (2, 16000, 16000, 16000), (2, 40001, 40001, 40001)])
def test_quantize_rows_gated(wr, dt, M, K, ld, ldg):
    torch = torch_mod()
    g = _gen(M * K)
    x = (torch.randn(M, K, device="cuda", generator=g) * 2).to(_dt(dt))
    gate = (torch.randn(M, K, device="cuda", generator=g) * 4).to(_dt(dt))
    gate[0, 0] = -60000 if dt == "f16" else -2e5   # exp overflows: silu is -0
    q, s = _quantize(wr, x, ld=ld, gate=gate, ldg=ldg, dt=dt)
    gd = gate.double()
    v = x.double() * torch.nan_to_num(gd * torch.sigmoid(gd))
    A = v.abs().amax(1)
    tiny = 2.0 ** -119   # where expf overflows, silu below e^-88 reads as 0
    assert bool(((s.double() - A / 127).abs() <= 10 * U * A / 127 + tiny).all())
    t = torch.where(A[:, None] > 0, 127 * v / torch.where(A > 0, A, 1)[:, None], torch.zeros_like(v))
    if float(A.min()) > 2.0 ** -90:
        assert float((q.double() - t).abs().max()) <= 0.5 + 127 * 17 * U


# ---------------------------------------------------------------- wr_residual_norm

def _norm_case(M, D, block="bf16", residual="bf16", gate="none", gdt="bf16", weights="bf16", seed=0):
    torch = torch_mod()
    g = _gen(seed + M + 3 * D)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    c = {"b": r(M, D).to(_dt(block)) if block else None, "h": (r(M, D) * 2).to(_dt(residual)) if residual else None,
         "wp": (1 + 0.2 * r(D)).to(_dt(weights)), "wn": (1 + 0.2 * r(D)).to(_dt(weights)), "g": None}
    if gate != "none":
        c["g"] = torch.tanh(r(1 if gate == "row" else M, D)).to(_dt(gdt))
    return c


def _norm_check(wr, c, M, D, ydt="bf16", post=True, wpost=True, wnorm=True, offset=0.0, scale=1.0, eps=1e-6, pad=0, rdt="bf16",
                bdt="bf16", gdt="bf16", wdt="bf16", in_place=False, want_residual=True, stream=None):
    torch = torch_mod()
    ld = D + pad
    kw = {}
    if c["b"] is not None:
        kw.update(block=_rows(c["b"], ld, extra=0)[1], ld_block=ld, block_type=_code(wr, bdt))
    hv = None
    if c["h"] is not None:
        hbuf, hv = _rows(c["h"], ld)
        kw.update(residual=hv, ld_residual=ld)
    kw["residual_type"] = _code(wr, rdt)
    if want_residual:
        robuf, ro = (hbuf, hv) if in_place else _empty_rows(M, D, ld, _dt(rdt))
        kw.update(residual_out=ro, ld_residual_out=ld)
    if c["g"] is not None:
        one = c["g"].shape[0] == 1 and M != 1
        gv = c["g"] if one else _rows(c["g"], ld, extra=0)[1]
        kw.update(gate=gv, ld_gate=0 if one else ld, gate_type=_code(wr, gdt))
    if post:
        kw.update(post_norm=True, post_weight=c["wp"] if wpost else None)
    if ydt:
        ldy = _pad16(D) if ydt == "i8" and not pad else ld
        ybuf, y = _empty_rows(M, D, ldy, _dt(ydt))
        ys = torch.full((M + 1,), float(SENTINEL), device="cuda") if ydt == "i8" else None
        kw.update(y=y, ld_y=ldy, y_type=_code(wr, ydt), y_scale=ys, norm_weight=c["wn"] if wnorm else None)
    wr.wr_residual_norm(M, D, weight_type=_code(wr, wdt), weight_offset=offset, residual_scale=scale, eps=eps, stream=stream, **kw)
    torch.cuda.synchronize()

    def norm(v, w):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * w

    one = torch.ones(D, dtype=torch.float64, device="cuda")
    branch = torch.zeros(M, D, dtype=torch.float64, device="cuda")
    if c["b"] is not None:
        branch = c["b"].double()
        if post:
            branch = norm(branch, c["wp"].double() + offset if wpost else one)
        if c["g"] is not None:
            branch = branch * c["g"].double()
    keep = c["h"].double() * scale if c["h"] is not None else torch.zeros_like(branch)
    h = keep + branch
    # the branch is off by 33 u (a norm and the gate), the sum of both rounds once
    eh = 33 * U * branch.abs() + U * (keep.abs() + h.abs()) + 2.0 ** -140
    if want_residual:
        rel, sub = _half_step(ro.dtype)
        err = (ro.double() - h).abs()
        assert bool((err <= eh + rel * (h.abs() + eh) + sub).all()), float((err / (eh + rel * h.abs())).max())
        _untouched(robuf, M, D)
    if not ydt:
        return
    wn = c["wn"].double() + offset if wnorm else one
    ref = norm(h, wn)
    root = torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    rr = torch.sqrt((eh * eh).mean(1, keepdim=True)) / root + 32 * U     # of the root, relative
    ey = (eh / root) * wn.abs() + rr * ref.abs()
    ey = ey * 1.001
    if ydt != "i8":
        rel, sub = _half_step(y.dtype)
        err = (y.double() - ref).abs()
        assert bool((err <= ey + rel * (ref.abs() + ey) + sub).all()), float((err / (ey + rel * ref.abs())).max())
    else:
        A, eA = ref.abs().amax(1), ey.amax(1)
        s = ys[:M].double()
        assert bool(((s * 127 - A).abs() <= eA + 2 * U * A + 2.0 ** -140).all())
        off = (y.double() * s[:, None] - ref).abs()
        assert bool((off <= 0.5 * s[:, None] * (1 + 1e-4) + ey + 2 * U * ref.abs() + 2.0 ** -140).all())
        assert float(ys[M]) == SENTINEL and bool((y.abs().int().amax(1)[A > 0] == 127).all())
    _untouched(ybuf, M, D)


@pytest.mark.parametrize("M,D", [(1, 1), (3, 2), (2, 8), (4, 33), (5, 100), (2, 256), (1, 2560), (33, 2560), (7, 1237), (3, 4096), (3, 4104),
                                 (2, 8192), (2, 8193), (2, 9728), (2, 16384), (3, 20000), (2, 32768), (2, 32767), (3000, 128)])
@pytest.mark.parametrize("ydt", ["bf16", "i8", "f32"])
@pytest.mark.parametrize("post", [False, True])
def test_norm_sizes(wr, M, D, ydt, post):
    _norm_check(wr, _norm_case(M, D), M, D, ydt=ydt, post=post)


@pytest.mark.parametrize("bdt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rdt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ydt", ["f32", "bf16", "f16", "i8"])
@pytest.mark.parametrize("gate,gdt,wdt", [("none", "f32", "f32"), ("row", "f16", "bf16"), ("token", "f32", "f16")])
def test_norm_types_and_gates(wr, bdt, rdt, ydt, gate, gdt, wdt):
    M, D = 9, 500
    c = _norm_case(M, D, bdt, rdt, gate, gdt, wdt)
    _norm_check(wr, c, M, D, ydt, bdt=bdt, rdt=rdt, gdt=gdt, wdt=wdt, scale=0.75, offset=-0.25)


@pytest.mark.parametrize("pad", [1, 8, 24])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D", [640, 1237, 6000])
def test_norm_strides_and_in_place(wr, pad, in_place, D):
    _norm_check(wr, _norm_case(11, D, gate="token"), 11, D, "i8" if pad == 8 else "bf16", pad=pad, in_place=in_place)


def test_norm_parts(wr):
    """Each part alone: no block, no residual, no weights, no residual output, no norm output."""
    for M, D in ((1, 2560), (6, 77), (3, 5000)):
        _norm_check(wr, _norm_case(M, D, block=None), M, D, post=False)
        _norm_check(wr, _norm_case(M, D, residual=None), M, D)
        _norm_check(wr, _norm_case(M, D, residual=None, gate="token"), M, D, post=False, want_residual=False)
        _norm_check(wr, _norm_case(M, D), M, D, wpost=False, wnorm=False, offset=3.0)
        _norm_check(wr, _norm_case(M, D), M, D, want_residual=False, ydt="i8")
        _norm_check(wr, _norm_case(M, D), M, D, ydt=None)


def test_norm_zero_and_poisoned_rows(wr):
    torch = torch_mod()
    M, D = 6, 300
    for ydt in ("f32", "i8"):
        c = _norm_case(M, D, "f32", "f32")
        for k, v in ((1, 0.0), (2, float("nan")), (3, float("inf"))):
            c["b"][k] = 0 if v == 0 else c["b"][k]
            c["h"][k] = 0 if v == 0 else c["h"][k]
            if v != 0:
                c["b"][k, 17] = v
        y = torch.empty(M, 304, dtype=_dt(ydt), device="cuda")[:, :D]
        s = torch.empty(M, device="cuda") if ydt == "i8" else None
        ro = torch.empty(M, D, device="cuda")
        wr.wr_residual_norm(M, D, block=c["b"], ld_block=D, residual=c["h"], ld_residual=D, residual_out=ro, ld_residual_out=D,
                            post_weight=c["wp"], norm_weight=c["wn"], weight_type=wr.WR_BF16, y=y, ld_y=304,
                            y_type=_code(wr, ydt), y_scale=s)
        assert bool((ro[1] == 0).all()) and bool((y[1] == 0).all())
        if ydt == "f32":
            assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3, 17]))
            assert bool(torch.isfinite(y[[0, 1, 4, 5]]).all())
        else:
            assert float(s[1]) == 0 and bool(torch.isnan(s[2:4]).all()) and bool((y[2:4] == 0).all())
            assert bool(torch.isfinite(s[[0, 4, 5]]).all())


def test_norm_rows_past_32_bits(wr):
    torch = torch_mod()
    M, D, ld = 4, 300, 1 << 30
    b = torch.empty(3 * ld + D, dtype=torch.bfloat16, device="cuda").as_strided((M, D), (ld, 1))
    q = torch.empty(3 * ld + 304, dtype=torch.int8, device="cuda").as_strided((M, D), (ld, 1))
    s = torch.empty(M, device="cuda")
    b.copy_(torch.randn(M, D, device="cuda", generator=_gen(2)))
    wr.wr_residual_norm(M, D, block=b, ld_block=ld, block_type=wr.WR_BF16, y=q, ld_y=ld, y_type=wr.WR_I8, y_scale=s)
    near = torch.empty(M, 304, dtype=torch.int8, device="cuda")
    s2 = torch.empty(M, device="cuda")
    wr.wr_residual_norm(M, D, block=b.contiguous(), ld_block=D, block_type=wr.WR_BF16, y=near, ld_y=304, y_type=wr.WR_I8, y_scale=s2)
    assert torch.equal(s, s2) and torch.equal(q, near[:, :D])
    x = b.contiguous()
    wr.wr_quantize_rows(wr.WR_BF16, M, D, b, ld, q, ld, s)
    wr.wr_quantize_rows(wr.WR_BF16, M, D, x, D, near, 304, s2)
    assert torch.equal(s, s2) and torch.equal(q, near[:, :D])


def test_norm_and_quantizer_same_codes(wr):
    """The codes that the norm writes are the quantizer's of the fp32 values that it writes."""
    torch = torch_mod()
    for M, D in ((1, 2560), (5, 1237), (3, 9000)):
        c = _norm_case(M, D, "f32", "bf16")
        y, q, q2 = torch.empty(M, D, device="cuda"), *(torch.empty(M, _pad16(D), dtype=torch.int8, device="cuda") for _ in range(2))
        s, s2 = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        args = dict(block=c["b"], ld_block=D, residual=c["h"], ld_residual=D, residual_type=wr.WR_BF16, norm_weight=c["wn"],
                    weight_type=wr.WR_BF16)
        wr.wr_residual_norm(M, D, y=y, ld_y=D, **args)
        wr.wr_residual_norm(M, D, y=q, ld_y=_pad16(D), y_type=wr.WR_I8, y_scale=s, **args)
        wr.wr_quantize_rows(wr.WR_F32, M, D, y, D, q2, _pad16(D), s2)
        assert torch.equal(s, s2) and torch.equal(q[:, :D], q2[:, :D])


# ---------------------------------------------------------------- together, and where they run

@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_mlp_block_in_8_bits(wr, M):
    """norm -> gate/up -> silu, product, codes -> down -> residual + norm, as a server runs it, on a side
    stream, against the same steps in 64 bits on the codes that were made."""
    torch = torch_mod()
    H, F = 512, 1300
    g = _gen(M)
    Fp = _pad16(F)
    h = torch.randn(M, H, device="cuda", generator=g).bfloat16()
    wn = (1 + 0.1 * torch.randn(H, device="cuda", generator=g)).bfloat16()
    W1 = 0.05 * torch.randn(2 * Fp, H, device="cuda", generator=g)
    W2 = 0.05 * torch.randn(H, F, device="cuda", generator=g)
    q1, s1 = torch.empty(2 * Fp, H, dtype=torch.int8, device="cuda"), torch.empty(2 * Fp, device="cuda")
    q2, s2 = torch.empty(H, Fp, dtype=torch.int8, device="cuda"), torch.empty(H, device="cuda")
    a, sa = torch.empty(M, H, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    m, sm = torch.empty(M, Fp, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    gu = torch.empty(M, 2 * Fp, device="cuda")
    d = torch.empty(M, H, device="cuda")
    out, y = torch.empty_like(h), torch.empty_like(h)
    sp1, n1 = _i8_workspace(wr, M, 2 * Fp, H)
    sp2, n2 = _i8_workspace(wr, M, H, F)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    k = dict(stream=st)
    wr.wr_quantize_rows(wr.WR_F32, 2 * Fp, H, W1, H, q1, H, s1, **k)
    wr.wr_quantize_rows(wr.WR_F32, H, F, W2, F, q2, Fp, s2, **k)
    wr.wr_residual_norm(M, H, residual=h, ld_residual=H, residual_type=wr.WR_BF16, norm_weight=wn, weight_type=wr.WR_BF16,
                        y=a, ld_y=H, y_type=wr.WR_I8, y_scale=sa, **k)
    wr.wr_gemm_i8(M, 2 * Fp, H, a, H, sa, q1, H, s1, wr.WR_F32, gu, 2 * Fp, sp1, n1, **k)
    wr.wr_quantize_rows(wr.WR_F32, M, F, gu[:, Fp:], 2 * Fp, m, Fp, sm, gate=gu, ldg=2 * Fp, **k)
    wr.wr_gemm_i8(M, H, F, m, Fp, sm, q2, Fp, s2, wr.WR_F32, d, H, sp2, n2, **k)
    wr.wr_residual_norm(M, H, block=d, ld_block=H, residual=h, ld_residual=H, residual_out=out, ld_residual_out=H,
                        residual_type=wr.WR_BF16, norm_weight=wn, weight_type=wr.WR_BF16, y=y, ld_y=H, y_type=wr.WR_BF16, **k)
    st.synchronize()
    gu64 = (a.double() @ q1.double().t()) * sa.double()[:, None] * s1.double()
    assert bool(((gu.double() - gu64).abs() <= 3.01 * U * gu64.abs()).all())
    v = torch.nn.functional.silu(gu.double()[:, :F]) * gu.double()[:, Fp:Fp + F]
    assert float((m[:, :F].double() - 127 * v / v.abs().amax(1, keepdim=True)).abs().max()) <= 0.5 + 127 * 17 * U
    d64 = (m[:, :F].double() @ q2[:, :F].double().t()) * sm.double()[:, None] * s2.double()
    assert bool(((d.double() - d64).abs() <= 3.01 * U * d64.abs()).all())
    h64 = h.double() + d.double()
    assert bool(((out.double() - h64).abs() <= (2.0 ** -9 + 4 * U) * h64.abs() * 1.01 * 2 + 2 * U * (h.double().abs() + d.double().abs())).all())
    y64 = h64 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + 1e-6) * wn.double()
    assert float(((y.double() - y64).abs() / y64.abs().clamp_min(1e-2)).max()) <= 2.0 ** -8 + 1e-4
    # against the block with no 8-bit rounding at all: each rounding of rows is off by at most half a
    # step of its largest value; together a few percent of the output's size
    x = h.double() / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + 1e-6) * wn.double()
    t = x @ W1.double().t()
    full = (torch.nn.functional.silu(t[:, :F]) * t[:, Fp:Fp + F]) @ W2.double().t()
    assert float((d.double() - full).norm() / full.norm()) < 0.1


def test_norm_between_packed_linears(wr):
    """fp32 outputs of a packed decode call -> residual + norm -> bf16 activations of the next."""
    torch = torch_mod()
    from gpu_inputs import q_case
    from oracle import wr_oracle as o
    import wr_synth
    M, H = 3, 512
    codes, scales, packed, s_d = q_case(wr, 2, H, H, 5)
    x_bits = wr_synth.activations_bf16(3, M, H)
    x = torch.from_numpy(x_bits.view(np.int16)).cuda().view(torch.bfloat16)
    h = torch.randn(M, H, device="cuda", generator=_gen(1)).bfloat16()
    w = (1 + 0.1 * torch.randn(H, device="cuda", generator=_gen(2))).bfloat16()
    nb = wr.wr_gemv_workspace_bytes(M, H, H, 2)
    space = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    y1, y2, a = torch.empty(M, H, device="cuda"), torch.empty(M, H, device="cuda"), torch.empty_like(h)
    wr.wr_gemv(M, H, H, x, packed, s_d, 2, y1, space, nb)
    wr.wr_residual_norm(M, H, block=y1, ld_block=H, residual=h, ld_residual=H, residual_out=h, ld_residual_out=H,
                        residual_type=wr.WR_BF16, norm_weight=w, weight_type=wr.WR_BF16, y=a, ld_y=H, y_type=wr.WR_BF16)
    wr.wr_gemv(M, H, H, a, packed, s_d, 2, y2, space, nb)
    torch.cuda.synchronize()
    ref, bound = o.gemm_codes(a.view(torch.int16).cpu().numpy().view(np.uint16), codes, scales, 2)
    assert np.all(np.abs(y2.cpu().numpy() - ref) <= 1e-4 * bound)


def test_host_tensors_are_refused(wr):
    torch = torch_mod()
    x, q, s = torch.randn(2, 32), torch.empty(2, 32, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    with pytest.raises(ValueError):
        wr.wr_quantize_rows(wr.WR_F32, 2, 32, x, 32, q, 32, s)


def test_gemm_i8_forms_on_two_streams(wr):
    """Products of every form (whole tiles by pairs, tiles shared by clusters, single CTAs) issued on two
    streams at once, so that their CTAs share SMs: all of them end, with the results of one stream."""
    torch = torch_mod()
    shapes = [(256, 19456, 640), (16, 640, 4096), (300, 2560, 2560), (64, 2560, 9728), (1024, 2560, 512), (9, 300, 128), (2, 512, 300),
              (333, 2560, 4096), (40, 6144, 640)]
    cases = []
    for i, (M, N, K) in enumerate(shapes):
        x, w, xs, ws = _i8_case(M, N, K, 70 + i)
        xv, wv = _rows(x, _pad16(K), extra=0)[1], _rows(w, _pad16(K), extra=0)[1]
        ys = [torch.empty(M, N, device="cuda") for _ in range(3)]
        cases.append((M, N, K, xv, xs, wv, ws, ys, _i8_workspace(wr, M, N, K)))

    def run(c, slot, stream=None):
        M, N, K, xv, xs, wv, ws, ys, (space, nb) = c
        wr.wr_gemm_i8(M, N, K, xv, _pad16(K), xs, wv, _pad16(K), ws, wr.WR_F32, ys[slot], N, space, nb, stream=stream)

    for c in cases:
        run(c, 2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(40):
        for k in range(len(cases)):
            run(cases[k], 0, streams[0])
            run(cases[(5 * k + rep) % len(cases)], 1, streams[1])
    torch.cuda.synchronize()
    for c in cases:
        assert torch.equal(c[7][0], c[7][2]) and torch.equal(c[7][1], c[7][2])
    assert wr.wr_get_device_error() == 0


def _chain(wr, M, steps, sync, graph=False):
    """A run in which every call reads what the call before it wrote, products behind products among them:
    codes of h, a product, its first row as the bias of another, and norms in place."""
    torch = torch_mod()
    H = 640
    g = _gen(7)
    h = torch.randn(M, H, device="cuda", generator=g)
    h0 = h.clone()
    W = torch.randint(-127, 128, (H, H), device="cuda", generator=g, dtype=torch.int32).to(torch.int8)
    ws = torch.full((H,), 1e-4, device="cuda")
    wn = torch.ones(H, device="cuda")
    q, s = torch.empty(M, H, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    y, z = torch.empty(M, H, device="cuda"), torch.empty(M, H, device="cuda")
    space, nb = _i8_workspace(wr, M, H, H)

    def step():
        wr.wr_quantize_rows(wr.WR_F32, M, H, h, H, q, H, s)
        sync()
        wr.wr_gemm_i8(M, H, H, q, H, s, W, H, ws, wr.WR_F32, y, H, space, nb)
        sync()
        wr.wr_gemm_i8(M, H, H, q, H, s, W, H, ws, wr.WR_F32, z, H, space, nb, bias=y)
        sync()
        wr.wr_gemm_i8(M, H, H, q, H, s, W, H, ws, wr.WR_F32, y, H, space, nb, bias=z)
        sync()
        wr.wr_residual_norm(M, H, block=y, ld_block=H, residual=h, ld_residual=H, residual_out=h, ld_residual_out=H, norm_weight=wn,
                            y=z, ld_y=H, residual_scale=0.5)
        sync()
        wr.wr_residual_norm(M, H, block=z, ld_block=H, residual=h, ld_residual=H, residual_out=h, ld_residual_out=H, residual_scale=0.5)
        sync()

    if graph:
        step()
        torch.cuda.synchronize()
        h.copy_(h0)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        h.copy_(h0)
        for _ in range(steps):
            gr.replay()
    else:
        for _ in range(steps):
            step()
    torch.cuda.synchronize()
    return h.clone(), y.clone(), z.clone()


@pytest.mark.parametrize("M", [1, 2, 7, 40, 300, 1500])
def test_calls_that_follow_one_another(wr, M):
    """The products start before the call in front of them has ended: with nothing between the calls, in a graph,
    and with a wait after each call the results are the same bits."""
    torch = torch_mod()
    waited = _chain(wr, M, 12, torch.cuda.synchronize)
    for got in (_chain(wr, M, 12, lambda: None), _chain(wr, M, 12, lambda: None, graph=True)):
        assert all(torch.equal(a, b) for a, b in zip(got, waited))
    assert bool(torch.isfinite(waited[0]).all()) and wr.wr_get_device_error() == 0


def test_many_short_rows(wr):
    torch = torch_mod()
    for M, K in ((100001, 24), (70000, 3)):
        x = torch.randn(M, K, device="cuda", generator=_gen(M))
        q, s = _quantize(wr, x)
        qr, sr = _codes64(x.cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)
        _norm_check(wr, _norm_case(M, K, gate="row"), M, K, "i8")


@pytest.mark.parametrize("M,D", [(2, 12000), (3, 20000), (700, 9000), (400, 17000)])
def test_norm_long_rows_in_place(wr, M, D):
    _norm_check(wr, _norm_case(M, D, gate="token"), M, D, "bf16", in_place=True, pad=8)
    _norm_check(wr, _norm_case(M, D, "f32", "f32", gdt="f32", weights="f32"), M, D, "i8", in_place=True, rdt="f32", bdt="f32", wdt="f32", pad=1)


def test_tensors_of_another_device_are_refused(wr):
    class Other:   # what the binding asks of a tensor
        def get_device(self):
            return 1 + torch_mod().cuda.current_device()

        def data_ptr(self):
            return 1 << 20

    with pytest.raises(ValueError, match="current device"):
        wr.wr_quantize_rows(wr.WR_F32, 2, 32, Other(), 32, 1 << 20, 32, 1 << 20)


@pytest.mark.parametrize("D", [7, 300, 2560, 9000, 20000])
@pytest.mark.parametrize("M", [2, 400])
def test_norm_of_very_large_and_very_small_rows(wr, M, D):
    """Rows whose squares leave fp32's range are normed like any other (rows of ordinary size beside them)."""
    torch = torch_mod()
    for size, eps in ((1e25, 1e-6), (3e37, 0.0), (1e-22, 0.0), (1e-30, 0.0)):
        c = _norm_case(M, D, "f32", "f32")
        for k in ("b", "h"):
            c[k][0] *= size / 8
        c["b"][1] *= size / 8   # the block alone: the post-norm brings it back
        _norm_check(wr, c, M, D, "f32", rdt="f32", bdt="f32", eps=eps)
        h = torch.zeros(M, D, device="cuda")
        h[0], h[1] = c["h"][0], 1.0
        y = torch.empty(M, D, device="cuda")
        wr.wr_residual_norm(M, D, residual=h, ld_residual=D, y=y, ld_y=D, eps=eps)
        v = h[:2].double()
        ref = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
        assert bool(((y[:2].double() - ref).abs() <= 33 * U * ref.abs()).all())


def test_two_host_threads(wr):
    """Two threads that call at once, each on its own stream with its own tensors."""
    import threading
    torch = torch_mod()
    shapes = [(3, 640, 2560), (300, 512, 1024)]
    work = []
    for i, (M, N, K) in enumerate(shapes):
        x, w, xs, ws = _i8_case(M, N, K, 90 + i)
        h = torch.randn(M, K, device="cuda", generator=_gen(i))
        work.append((M, N, K, h, w, ws, torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"),
                     [torch.empty(M, N, device="cuda") for _ in range(2)], torch.cuda.Stream()))
    errors = []

    def run(i, slot, stream, times):
        M, N, K, h, w, ws, q, s, ys, _ = work[i]
        for _ in range(times):
            wr.wr_quantize_rows(wr.WR_F32, M, K, h, K, q, K, s, stream=stream)
            wr.wr_gemm_i8(M, N, K, q, K, s, w, K, ws, wr.WR_F32, ys[slot], N, None, 0, stream=stream)

    def thread(i):
        try:
            run(i, 0, work[i][9], 200)
        except Exception as e:   # seen by the main thread below
            errors.append(e)

    for i in range(2):
        run(i, 1, None, 1)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in range(2):
        assert torch.equal(work[i][8][0], work[i][8][1])


def test_products_behind_copies_fills_and_other_streams(wr):
    """A product captured (and issued) right behind a fill, a copy, a torch kernel, an event of another stream:
    what is in front of it in the stream need not be one of this library's kernels."""
    torch = torch_mod()
    for M in (1, 40, 1500):
        N, K = 512, 640
        x, w, xs, ws = _i8_case(M, N, K, M)
        want = _i8_check(wr, x, w, xs, ws).clone()
        xq, y, other = torch.empty_like(x), torch.empty(M, N, device="cuda"), torch.cuda.Stream()
        host = x.cpu().pin_memory()

        def product():
            wr.wr_gemm_i8(M, N, K, xq, K, xs, w, K, ws, wr.WR_F32, y, N, None, 0)

        def behind_fill():
            xq.copy_(x)
            y.zero_()          # a memset
            product()

        def behind_copy():
            xq.copy_(x)        # device to device
            product()

        def behind_upload():
            xq.copy_(host, non_blocking=True)
            product()

        def behind_kernel():
            torch.neg(x, out=xq)
            torch.neg(xq, out=xq)   # (-128 is its own negative: twice is the identity)
            product()

        def behind_event():
            cur = torch.cuda.current_stream()
            other.wait_stream(cur)
            with torch.cuda.stream(other):
                xq.copy_(x)
                y.zero_()
            cur.wait_stream(other)
            product()

        for f in (behind_fill, behind_copy, behind_upload, behind_kernel, behind_event):
            for _ in range(3):
                xq.zero_()
                f()
                torch.cuda.synchronize()
                assert torch.equal(y, want)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                f()
                product()
            for _ in range(3):
                xq.zero_()
                y.zero_()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 2, 3, 8, 9, 16, 17])
@pytest.mark.parametrize("N,K", [(1024, 1024), (1025, 1025), (4096, 1000), (4097, 4096), (4096, 4097), (4111, 300), (8192, 4096),
                                 (8193, 513), (12300, 260), (2561, 4100), (40, 20000)])
def test_gemm_i8_where_the_kernel_changes(wr, M, N, K):
    """Both sides of the sizes at which another kernel takes over, in every type."""
    x, w, xs, ws = _i8_case(M, N, K, M + 2 * N + K)
    for ydt in ("f32", "bf16", "f16"):
        _i8_check(wr, x, w, xs, ws, ydt, ldy=N + (M % 2))


@pytest.mark.parametrize("M", [250, 256, 289, 505, 512, 1030])
@pytest.mark.parametrize("N,K", [(19456, 300), (19301, 2560), (9728, 2560), (19200, 130), (22000, 1)])
def test_gemm_i8_tiles_left_over(wr, M, N, K):
    """Large products whose tiles come out a few more than whole rounds of the GPU."""
    x, w, xs, ws = _i8_case(M, N, K, M + 2 * N + K)
    for ydt in ("f32", "bf16"):
        _i8_check(wr, x, w, xs, ws, ydt, ldy=N + (M % 2))


@pytest.mark.parametrize("M", [1, 2, 3, 8, 9, 16])
@pytest.mark.parametrize("N,K", [(4736, 6144), (4737, 6144), (4736, 6145), (2048, 2048), (2049, 2040), (1030, 2049), (4736, 1500), (4737, 2561), (5328, 2560), (5329, 2560),
                                 (5329, 2561), (7104, 5000), (7105, 2049), (7105, 4097), (7200, 2000)])
def test_gemm_i8_few_tokens_all_forms(wr, M, N, K):
    """Few tokens on both sides of the sizes that choose among dp4a and the forms of the warps' MMA."""
    x, w, xs, ws = _i8_case(M, N, K, M + 2 * N + K)
    for ydt in ("f32", "bf16"):
        _i8_check(wr, x, w, xs, ws, ydt, ldy=N + (M % 2))


def test_gemm_i8_tiles_left_over_on_two_streams_and_replayed(wr):
    """Products whose last tiles are cut, at once on two streams, then replayed from a graph with new tokens."""
    torch = torch_mod()
    M, N, K = 256, 19456, 384
    cases = [_i8_case(M, N, K, seed) for seed in (5, 6)]
    want = [(x.double() @ w.double().t()).float() * xs[:, None] * ws[None, :] for x, w, xs, ws in cases]
    ys = [torch.zeros(M, N, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]

    def call(i):
        x, w, xs, ws = cases[i]
        wr.wr_gemm_i8(M, N, K, x, K, xs, w, K, ws, wr.WR_F32, ys[i], N, None, 0, stream=streams[i].cuda_stream)

    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            call(i)
    torch.cuda.synchronize()
    for y, v in zip(ys, want):
        assert torch.equal(y, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        call(0)
    cases[0][0][:100].zero_()
    ys[0].fill_(float("nan"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert not ys[0][:100].any()
    assert torch.equal(ys[0][100:], want[0][100:])
