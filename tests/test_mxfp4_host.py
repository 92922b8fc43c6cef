"""MXFP4 and expert-grouped entry points on the host: the oracle's pack against
a search over all scales, sizes, argument checks (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import w4a16_gemm_wq_b200 as wq
from w4a16_gemm_wq_b200 import build

P = ctypes.c_void_p
GOOD, BAD, ODD = P(1 << 20), P((1 << 20) + 8), P((1 << 20) + 2)


@pytest.fixture(scope="module")
def clib():
    build.build()
    return wq.load()


def test_e8m0_values():
    assert oracle.e8m0_decode(127) == 1.0 and oracle.e8m0_decode(0) == 2.0**-127
    assert oracle.e8m0_decode(254) == 2.0**127 and math.isnan(oracle.e8m0_decode(255))


@pytest.mark.parametrize("seed,spread", [(0, 0.0), (1, 8.0), (2, 40.0)])
def test_oracle_pack_is_the_specified_rounding(seed, spread):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(7, 96, generator=g) * torch.exp2(spread * torch.randn(7, 96, generator=g))).to(torch.bfloat16)
    W[0, :32] = 0.0
    W[1, 5] = -0.0
    p = oracle.quantize_mxfp4(W)
    v = oracle.dequant_mxfp4(p)
    w = W.double().numpy()
    mags = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    for r in range(7):
        for b in range(3):
            blk = w[r, 32 * b:32 * b + 32]
            m = np.abs(blk).max()
            e = -127 if m == 0 else min(127, max(-127, math.frexp(m)[1] - 3))
            assert p["bscale"][r, b] == e + 127
            scale = 2.0**e
            if m > 0 and e > -127:
                assert 4.0 <= m / scale < 8.0
            # no other magnitude is nearer than the chosen one
            got = np.abs(v[r, 32 * b:32 * b + 32]) / scale
            assert np.isin(got, mags).all()
            dist = np.abs(np.abs(blk)[:, None] / scale - mags[None])
            assert (np.abs(np.abs(blk) / scale - got) == dist.min(axis=1)).all()


def test_oracle_pack_ties_signs_and_saturation():
    # block maximum 4 -> e = 0: the values are E2M1 quotients themselves
    vals = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -0.0, 0.0, -4.0]
    want = [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -0.0, -1.0, -1.0, -2.0, -2.0, -4.0, -0.0, 0.0, -4.0]
    v = oracle.dequant_mxfp4(oracle.quantize_mxfp4(torch.tensor([vals * 2], dtype=torch.bfloat16)))[0]
    assert v.tolist() == want * 2 and (np.signbit(v) == np.signbit(np.array(want * 2))).all()
    # 7.75 has the exponent of 4 too: 5 is a tie (to 4), 5.03 and above saturate at 6
    v = oracle.dequant_mxfp4(oracle.quantize_mxfp4(torch.tensor([[7.75, 5.0, 5.03125, -7.0] * 8], dtype=torch.bfloat16)))
    assert v[0, :4].tolist() == [6.0, 4.0, 6.0, -6.0]


def test_oracle_pack_of_non_finite_blocks():
    W = torch.ones(1, 96, dtype=torch.bfloat16)
    W[0, 3], W[0, 40] = float("inf"), float("nan")
    p = oracle.quantize_mxfp4(W)
    assert p["bscale"][0].tolist() == [255, 255, 125] and not p["codes"][0, :32].any()


def test_sizes(clib):
    assert wq.mxfp4_sizes(2048, 11008) == (2048 * 5504, 2048 * 344)
    for K in (0, 16, 100):
        with pytest.raises(wq.WQError):
            wq.mxfp4_sizes(16, K)
    # W4A16: room for the activations times act_inv_s, for more rows than the forms for few rows take
    assert wq.linear_workspace_size(8, 11008, 2048, wq.WQ_FMT_MXFP4, 0) == 0
    assert wq.linear_workspace_size(2048, 11008, 2048, wq.WQ_FMT_MXFP4, 0) == 2048 * 2048 * 2
    # W4A4: at least the activations' codes and scales
    assert wq.linear_workspace_size(100, 256, 2048, wq.WQ_FMT_MXFP4, 1) >= 100 * (1024 + 64)
    with pytest.raises(wq.WQError):
        wq.linear_workspace_size(16, 16, 64, wq.WQ_FMT_INT4, 1)
    with pytest.raises(wq.WQError):
        wq.linear_workspace_size(16, 16, 64, 3, 0)


def test_mxfp4_arguments_are_checked_before_any_launch(clib):
    assert clib.wq_quantize_mxfp4(None, 16, 64, None, GOOD, GOOD, None) == wq.WQ_ERR_ARG
    assert clib.wq_quantize_mxfp4(BAD, 16, 64, None, GOOD, GOOD, None) == wq.WQ_ERR_ARG
    assert clib.wq_quantize_mxfp4(GOOD, 16, 48, None, GOOD, GOOD, None) == wq.WQ_ERR_ARG
    assert clib.wq_quantize_mxfp4(GOOD, 0, 64, None, GOOD, GOOD, None) == wq.WQ_ERR_ARG
    assert clib.wq_quantize_mxfp4(GOOD, 16, 64, BAD, GOOD, GOOD, None) == wq.WQ_ERR_ARG
    assert clib.wq_dequantize_mxfp4(GOOD, None, 16, 64, GOOD, None) == wq.WQ_ERR_ARG
    assert clib.wq_dequantize_mxfp4(GOOD, GOOD, 16, 64, BAD, None) == wq.WQ_ERR_ARG
    lin = clib.wq_linear_mxfp4
    assert lin(GOOD, 0, 16, 64, GOOD, GOOD, 0, None, GOOD, None, 0, None) == wq.WQ_ERR_ARG
    assert lin(GOOD, 1, 16, 64, GOOD, GOOD, 2, None, GOOD, None, 0, None) == wq.WQ_ERR_ARG
    assert lin(GOOD, 1, 16, 64, GOOD, None, 0, None, GOOD, None, 0, None) == wq.WQ_ERR_ARG
    assert lin(GOOD, 1, 16, 64, GOOD, GOOD, 0, BAD, GOOD, None, 0, None) == wq.WQ_ERR_ARG
    # W4A4: K % 64, a missing, too small or misaligned workspace
    assert lin(GOOD, 1, 16, 96, GOOD, GOOD, 1, None, GOOD, GOOD, 1 << 30, None) == wq.WQ_ERR_ARG
    assert lin(GOOD, 1, 16, 64, GOOD, GOOD, 1, None, GOOD, None, 0, None) == wq.WQ_ERR_ARG
    assert lin(GOOD, 1, 16, 64, GOOD, GOOD, 1, None, GOOD, GOOD, 16, None) == wq.WQ_ERR_ARG
    assert "workspace" in clib.wq_last_error().decode()
    assert lin(GOOD, 1, 16, 64, GOOD, GOOD, 1, None, GOOD, BAD, 1 << 30, None) == wq.WQ_ERR_ARG


def _stack(fmt, **kw):
    w = wq.ExpertStack(format=fmt, E=4, N=16, K=128, packed=1 << 20)
    if fmt == wq.WQ_FMT_INT4:
        w.scales, w.zeros, w.group_size, w.zero_point = 1 << 20, 1 << 20, 64, 1
    else:
        w.bscale = 1 << 20
    if fmt == wq.WQ_FMT_NVFP4:
        w.global_scale = 1 << 20
    for k, v in kw.items():
        setattr(w, k, v)
    return w


@pytest.mark.parametrize("fmt,kw,status", [
    (0, dict(format=7), wq.WQ_ERR_ARG), (0, dict(E=0), wq.WQ_ERR_ARG), (0, dict(E=1025), wq.WQ_ERR_ARG),
    (0, dict(N=0), wq.WQ_ERR_ARG), (0, dict(K=100), wq.WQ_ERR_ARG), (2, dict(E=1024, N=1 << 21), wq.WQ_ERR_ARG),
    (0, dict(group_size=16), wq.WQ_ERR_UNSUPPORTED), (0, dict(K=96), wq.WQ_ERR_ARG),
    (0, dict(zeros=None), wq.WQ_ERR_ARG), (0, dict(zero_point=0), wq.WQ_ERR_ARG), (0, dict(zero_point=2), wq.WQ_ERR_ARG),
    (0, dict(scales=None), wq.WQ_ERR_ARG), (1, dict(bscale=None), wq.WQ_ERR_ARG),
    (1, dict(global_scale=None), wq.WQ_ERR_ARG), (1, dict(global_scale=(1 << 20) + 2), wq.WQ_ERR_ARG),
    (2, dict(packed=None), wq.WQ_ERR_ARG), (2, dict(packed=(1 << 20) + 8), wq.WQ_ERR_ARG),
    (2, dict(bscale=(1 << 20) + 8), wq.WQ_ERR_ARG)])
def test_expert_stacks_are_checked(clib, fmt, kw, status):
    w = _stack(fmt, **kw)
    assert clib.wq_linear_experts(ctypes.byref(w), GOOD, 8, GOOD, GOOD, None) == status


def test_expert_call_arguments_are_checked(clib):
    w = _stack(wq.WQ_FMT_MXFP4)
    call = clib.wq_linear_experts
    assert call(None, GOOD, 8, GOOD, GOOD, None) == wq.WQ_ERR_ARG
    assert call(ctypes.byref(w), GOOD, -1, GOOD, GOOD, None) == wq.WQ_ERR_ARG
    assert call(ctypes.byref(w), GOOD, 8, None, GOOD, None) == wq.WQ_ERR_ARG
    assert call(ctypes.byref(w), GOOD, 8, ODD, GOOD, None) == wq.WQ_ERR_ARG
    assert call(ctypes.byref(w), BAD, 8, GOOD, GOOD, None) == wq.WQ_ERR_ARG
    assert call(ctypes.byref(w), GOOD, 8, GOOD, None, None) == wq.WQ_ERR_ARG
    assert call(ctypes.byref(w), None, 0, None, None, None) == wq.WQ_OK  # no rows: nothing is launched


def test_group_takes_mxfp4_items(clib):
    it = wq.LinearItem(format=wq.WQ_FMT_MXFP4, N=16, K=64, X=1 << 20, packed=1 << 20, Y=1 << 20)
    assert clib.wq_linear_group(ctypes.byref(it), 1, 1, None) == wq.WQ_ERR_ARG  # no block scales
    it.format = 3
    assert clib.wq_linear_group(ctypes.byref(it), 1, 1, None) == wq.WQ_ERR_ARG


def test_binding_refuses_packs_and_host_tensors():
    p = wq.PackedMXFP4(None, None, 1, 32)
    for fn in (wq.wq_quantize_mxfp4, wq.wq_quantize_experts, wq.wq_quantize_nvfp4):
        with pytest.raises(ValueError):
            fn(p)
    W = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: wq.wq_quantize_mxfp4(W), lambda: wq.wq_quantize_experts(W.view(1, 4, 64)),
                 lambda: wq.wq_linear_mxfp4(W, p), lambda: wq.wq_dequantize_mxfp4(W),
                 lambda: wq.wq_linear_experts(W, torch.zeros(2, dtype=torch.int32), p)):
        with pytest.raises(ValueError):
            call()
