"""Argument checks of the 8-bit token path's self-test, on the CPU (see test_i8_host.py)."""
import pytest

import bit_weight_only_wr_b200 as wr
from test_i8_host import BAD, GEMM, P, UNSUPPORTED, _status


SELFTEST = {k: GEMM[k] for k in ("M", "N", "K", "x", "ldx", "x_scale", "w", "ldw", "w_scale", "y", "ldy")}


@pytest.mark.parametrize("change,status", [
    (dict(M=1), UNSUPPORTED), (dict(M=8), UNSUPPORTED), (dict(K=131072, ldx=131072, ldw=131072), UNSUPPORTED),
    (dict(M=0), BAD), (dict(ldx=104), BAD), (dict(x=None), BAD), (dict(y=P + 4), BAD), (dict(ldy=69), BAD),
])
def test_selftest_refusals(change, status):
    assert _status(wr.wr_selftest_gemm_i8_timeout, **{**SELFTEST, **change}) == status
