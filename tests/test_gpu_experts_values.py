"""Values at which the forms of the expert product and the MXFP4 Linear could part: infinities."""

import numpy as np
import pytest
import torch

from tests._linear_ref import assert_within_bound, expert_values, f64, mx_values
from tests.test_gpu_experts import FMTS, _acts, _offsets, _stack

pytestmark = pytest.mark.gpu

# rows of each expert and N: few rows (CUDA cores), few rows of many experts (mma.sync), many rows (tcgen05)
FORMS = {"cores": ([2, 0, 1], 150), "mma_sync": ([1, 0, 2, 2] * 10, 525), "tcgen05": ([90, 0, 70], 150)}


def _experts_of(counts):
    return np.repeat(np.arange(len(counts)), counts)


def _nonfinite_product(x, w):
    """What the non-finite elements of x [K] make of x w[N, K]^T: an infinity, or NaN."""
    k = np.flatnonzero(~np.isfinite(x))
    with np.errstate(invalid="ignore"):
        return (x[k] * w[:, k]).sum(1)


def _same_nonfinite(y, ref, what):
    assert (np.isnan(y) == np.isnan(ref)).all(), what
    some = ~np.isnan(ref)
    assert (y[some] == ref[some]).all(), what


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("form", FORMS)
def test_infinite_activations(lib, fmt, form):
    # inf times a weight is an infinity of its sign, times zero NaN; the other rows do not notice
    counts, N = FORMS[form]
    T, K = sum(counts), 384
    p = _stack(lib, fmt, len(counts), N, K, 21)
    X = _acts(T, K, 22)
    X[0, 7] = float("inf")
    X[1, 130], X[1, 131] = float("-inf"), float("inf")
    X[T - 1, 383] = float("-inf")
    if T > 3:
        X[5, 64], X[5, 300] = float("inf"), float("nan")
    Y = f64(lib.wq_linear_experts(X.cuda(), _offsets(counts).cuda(), p))
    x = f64(X)
    for i, e in enumerate(_experts_of(counts)):
        if np.isfinite(x[i]).all():
            assert np.isfinite(Y[i]).all(), (i, e)
        else:
            _same_nonfinite(Y[i], _nonfinite_product(x[i], expert_values(p, e)), f"row {i} expert {e}")


@pytest.mark.parametrize("M", [1, 2, 5, 40])
def test_infinite_activations_under_scales_far_apart(lib, M):
    N, K = 48, 512
    g = torch.Generator().manual_seed(4)
    W = torch.randn(N, K // 32, 32, generator=g) * torch.exp2(torch.randint(-50, 50, (N, K // 32, 1), generator=g).float())
    W[5, 2:] = 0
    p = lib.wq_quantize_mxfp4(W.reshape(N, K).to(torch.bfloat16).cuda())
    X = _acts(M, K, M)
    X[M - 1, 40] = float("inf")
    Y, x = f64(lib.wq_linear_mxfp4(X.cuda(), p)), f64(X)
    _same_nonfinite(Y[M - 1], _nonfinite_product(x[M - 1], mx_values(p)), "the row")
    if M > 1:
        assert_within_bound(torch.from_numpy(Y[:M - 1]), x[:M - 1], mx_values(p), False)
