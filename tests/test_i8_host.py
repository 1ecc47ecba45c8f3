"""Argument checks of the 8-bit token path, on the CPU: every refusal comes before any launch, so the
addresses below are never followed."""
import ctypes

import pytest

import bit_weight_only_wr_b200 as wr

P = 1 << 20   # an aligned address
BAD, UNSUPPORTED = 1, 2


def _status(call, *a, **k):
    with pytest.raises(wr.WrError) as e:
        call(*a, stream=0, **k)
    return e.value.status


QUANT = dict(type=wr.WR_BF16, M=4, K=100, x=P, ldx=100, q=P, ldq=112, scale=P)


@pytest.mark.parametrize("change,status", [
    (dict(type=wr.WR_I8), UNSUPPORTED), (dict(type=9), UNSUPPORTED), (dict(type=-1), UNSUPPORTED),
    (dict(M=0), BAD), (dict(M=-1), BAD), (dict(K=0), BAD), (dict(K=1 << 31), BAD), (dict(M=1 << 31), BAD),
    (dict(ldx=99), BAD), (dict(ldq=99), BAD), (dict(gate=P, ldg=99), BAD), (dict(ldx=-100), BAD), (dict(ldx=1 << 40), BAD),
    (dict(x=None), BAD), (dict(q=None), BAD), (dict(scale=None), BAD),
    (dict(x=P + 2), BAD), (dict(q=P + 8), BAD), (dict(scale=P + 4), BAD), (dict(gate=P + 2, ldg=100), BAD),
])
def test_quantize_rows_refusals(change, status):
    assert _status(wr.wr_quantize_rows, **{**QUANT, **change}) == status


GEMM = dict(M=40, N=70, K=100, x=P, ldx=112, x_scale=P, w=P, ldw=112, w_scale=P, y_type=wr.WR_F32, y=P, ldy=70, workspace=P,
            workspace_bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(y_type=wr.WR_I8), UNSUPPORTED), (dict(y_type=7), UNSUPPORTED), (dict(K=131072, ldx=131072, ldw=131072), UNSUPPORTED),
    (dict(M=0), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(M=1 << 31), BAD), (dict(N=1 << 31, ldy=1 << 31), BAD),
    (dict(ldx=96), BAD), (dict(ldx=104), BAD), (dict(ldw=96), BAD), (dict(ldw=104), BAD), (dict(ldy=69), BAD), (dict(ldx=-112), BAD),
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(x_scale=None), BAD), (dict(w_scale=None), BAD), (dict(y=None), BAD),
    (dict(x=P + 1), BAD), (dict(w=P + 4), BAD), (dict(x_scale=P + 4), BAD), (dict(w_scale=P + 8), BAD), (dict(y=P + 2), BAD),
    (dict(bias=P + 4), BAD),
])
def test_gemm_i8_refusals(change, status):
    assert _status(wr.wr_gemm_i8, **{**GEMM, **change}) == status


def test_gemm_i8_workspace():
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 131072), (-1, 1, 1)):
        assert wr.wr_gemm_i8_workspace_bytes(*bad) == 0
    for M, N, K in ((1, 64, 64), (40, 70, 9728), (333, 2560, 9728), (4096, 19456, 2560)):
        need = wr.wr_gemm_i8_workspace_bytes(M, N, K)
        if need:
            a = {**GEMM, "M": M, "N": N, "K": K, "ldx": K, "ldw": K, "ldy": N}
            assert _status(wr.wr_gemm_i8, **{**a, "workspace_bytes": need - 1}) == BAD
            assert _status(wr.wr_gemm_i8, **{**a, "workspace": None}) == BAD
            assert _status(wr.wr_gemm_i8, **{**a, "workspace": P + 8}) == BAD


NORM = dict(M=4, D=100, block=P, ld_block=100, block_type=wr.WR_F32, residual=P, ld_residual=100, residual_type=wr.WR_BF16,
            residual_out=P, ld_residual_out=100, norm_weight=P, weight_type=wr.WR_BF16, y=P, ld_y=100, y_type=wr.WR_BF16)


@pytest.mark.parametrize("change,status", [
    (dict(block_type=wr.WR_I8), UNSUPPORTED), (dict(residual_type=5), UNSUPPORTED), (dict(weight_type=wr.WR_I8), UNSUPPORTED),
    (dict(y_type=4), UNSUPPORTED), (dict(gate=P, gate_type=3), UNSUPPORTED),
    (dict(D=32769, ld_block=32769, ld_residual=32769, ld_residual_out=32769, ld_y=32769), UNSUPPORTED),
    (dict(M=0), BAD), (dict(D=0), BAD), (dict(M=1 << 31), BAD),
    (dict(block=None, residual=None), BAD), (dict(residual_out=None, y=None, norm_weight=None), BAD),
    (dict(block=None, post_norm=True), BAD), (dict(block=None, gate=P), BAD), (dict(post_weight=P, post_norm=False), BAD),
    (dict(y=None), BAD), (dict(y_type=wr.WR_I8), BAD), (dict(y_scale=P), BAD), (dict(y=None, norm_weight=None, y_scale=P), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(residual_scale=float("inf")), BAD),
    (dict(weight_offset=float("nan")), BAD),
    (dict(ld_block=99), BAD), (dict(ld_residual=50), BAD), (dict(ld_residual_out=99), BAD), (dict(ld_y=99), BAD),
    (dict(gate=P, ld_gate=99), BAD), (dict(ld_residual_out=101), BAD),
    (dict(block=P + 4), BAD), (dict(residual=P + 2), BAD), (dict(norm_weight=P + 2), BAD), (dict(y=P + 8), BAD), (dict(post_weight=P + 2), BAD),
    (dict(gate=P + 2), BAD), (dict(residual_out=P + 4), BAD), (dict(y_type=wr.WR_I8, y_scale=P + 4), BAD),
])
def test_residual_norm_refusals(change, status):
    assert _status(wr.wr_residual_norm, **{**NORM, **change}) == status


def test_residual_norm_struct():
    """The binding's struct has the C layout; a reserved field and a null struct are refused."""
    assert ctypes.sizeof(wr.WrResidualNormArgs) == 8 * 15 + 4 * 10
    a = wr.WrResidualNormArgs(M=1, D=16, block=P, ld_block=16, y=P, ld_y=16, eps=1e-6, residual_scale=1.0, reserved=1)
    assert wr._lib.wr_residual_norm(a, 0) == BAD
    assert wr._lib.wr_residual_norm(None, 0) == BAD


def test_host_tensors_are_refused():
    import torch
    with pytest.raises(ValueError):
        wr.wr_quantize_rows(wr.WR_F32, 2, 16, torch.zeros(2, 16), 16, P, 16, P, stream=0)


def test_arguments_by_name_and_by_place():
    """The extension module takes arguments as a Python function does."""
    with pytest.raises(TypeError, match="missing"):
        wr.wr_quantize_rows(wr.WR_F32, 2, 16)
    with pytest.raises(TypeError, match="unexpected"):
        wr.wr_quantize_rows(**QUANT, stream=0, colour=3)
    with pytest.raises(TypeError, match="multiple"):
        wr.wr_quantize_rows(wr.WR_F32, **QUANT, stream=0)
    with pytest.raises(TypeError, match="positional"):
        wr.wr_residual_norm(1, 2, 3)
    with pytest.raises(TypeError):
        wr.wr_quantize_rows(**{**QUANT, "M": "4"}, stream=0)
    with pytest.raises(OverflowError):
        wr.wr_quantize_rows(**{**QUANT, "type": 1 << 40}, stream=0)
    name = "".join(["l", "dx"])   # an equal string that is not the interned one
    assert _status(wr.wr_quantize_rows, **{**{k: v for k, v in QUANT.items() if k != "ldx"}, name: 99}) == BAD
    q = dict(QUANT)
    place = [q.pop(k) for k in ("type", "M", "K", "x", "ldx")]
    assert _status(wr.wr_quantize_rows, *place[:-1], 99, **q) == BAD


def test_the_message_of_a_refusal():
    e = None
    try:
        wr.wr_gemm_i8(**{**GEMM, "M": 0}, stream=0)
    except wr.WrError as err:
        e = err
    assert e is not None and e.status == BAD and str(e) == "wr_gemm_i8: invalid argument (status 1)"
