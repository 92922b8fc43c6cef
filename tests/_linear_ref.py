"""fp64 references and error bounds of the MXFP4 and expert-grouped Linears.

Bound of one output against the exact product of the same packed weights,
with S = sum_k |x_k w_k| (all roundings relative, half a step each):
  * the bf16 result: 2^-8 |y|;
  * fp32 accumulation of K exact products, in any order: K 2^-24 S, twice that
    for adders that truncate;
  * one bf16 rounding per term where a kernel's comment says so (INT4 weights
    times an fp16 scale; activations or weights times act_inv_s): 2^-8 S.
"""
import numpy as np
import torch

import oracle
from tests._parity import bits


def mx_values(p) -> np.ndarray:
    return oracle.dequant_mxfp4(dict(codes=bits(p.codes), bscale=bits(p.bscale), N=p.N, K=p.K))


def expert_values(p, e: int) -> np.ndarray:
    """fp64 weights [N, K] of expert e of a PackedExperts."""
    if p.fmt == "int4":
        return oracle.dequant_int4(dict(qweight=bits(p.packed[e]), scales=bits(p.scales[e]),
                                        zeros=None if p.zeros is None else bits(p.zeros[e]), N=p.N, K=p.K,
                                        group_size=p.group_size, zero_point=p.zero_point))
    if p.fmt == "nvfp4":
        return oracle.dequant_nvfp4(dict(codes=bits(p.packed[e]), bscale=bits(p.bscale[e]),
                                         g=float(p.global_scale[e]), N=p.N, K=p.K))
    return oracle.dequant_mxfp4(dict(codes=bits(p.packed[e]), bscale=bits(p.bscale[e]), N=p.N, K=p.K))


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def assert_within_bound(Y, x: np.ndarray, w: np.ndarray, rounded_terms: bool, what=""):
    """Y (bf16 [M, N]) against x [M, K] w[N, K]^T in fp64, elementwise."""
    ref = x @ w.T
    S = np.abs(x) @ np.abs(w).T
    # a tensor-core accumulator may also drop what lies 2^-24 below the largest term of its sum
    tol = 2.0**-8 * np.abs(ref) + (2 * x.shape[1] * 2.0**-24 + (2.0**-8 if rounded_terms else 0.0)) * S
    y = f64(Y)
    assert y.shape == ref.shape, (what, y.shape, ref.shape)
    bad = ~(np.abs(y - ref) <= tol + 2.0**-133)
    assert not bad.any(), (what, np.argwhere(bad)[:5].tolist(), y[bad][:5], ref[bad][:5], tol[bad][:5])
