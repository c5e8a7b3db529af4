"""Refusals of norm calls in place, on the host before any CUDA call."""
import pytest

import test_expert_abi as A
from structured_activation_sparsity_b200 import _lib as L

Y, X, OUT = A.FAKE, 2 * A.FAKE, 3 * A.FAKE


@pytest.mark.parametrize("over,strides", [
    (Y, dict(ld_n=72)), (X, dict(ld_n=72)), (Y, dict(ld_y=72)), (X, dict(ld_x=72)),
    (Y, dict(ld_y=80, ld_n=72)), (X, dict(ld_x=80, ld_n=64)),
])
def test_n_over_y_or_x_needs_its_stride(over, strides):
    cfg = L.make_norm_cfg(**{**A.OK_NORM, **strides})
    assert A._norm(cfg, y=Y, x=X, x_out=OUT, n=over) == L.SS_EINVAL
