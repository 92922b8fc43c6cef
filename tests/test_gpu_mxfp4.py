"""MXFP4 on the GPU: the pack bit for bit against the oracle, its values, and the
MXFP4 Linear (bf16 and 4-bit activations) against fp64 products of the same packs."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests._linear_ref import assert_within_bound, f64, mx_values
from tests._parity import bits

pytestmark = pytest.mark.gpu


def _weights(N, K, seed, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(N, K, generator=g) / math.sqrt(K)
    if spread:
        w = w * torch.exp2(spread * torch.randn(N, K, generator=g))
    return w.to(torch.bfloat16)


def _acts(M, K, seed):
    return torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _inv_s(K, seed):
    return torch.exp(0.5 * torch.randn(K, generator=torch.Generator().manual_seed(seed)))


def _same_pack(p, W, s=None):
    ref = oracle.quantize_mxfp4(W, None if s is None else s.numpy())
    np.testing.assert_array_equal(bits(p.bscale), ref["bscale"])
    np.testing.assert_array_equal(bits(p.codes), ref["codes"])
    return ref


@pytest.mark.parametrize("N,K", [(1, 32), (1, 64), (3, 96), (37, 2048), (1003, 1376), (130, 11008)])
@pytest.mark.parametrize("spread", [0.0, 6.0, 60.0])
@pytest.mark.parametrize("scaled", [False, True])
def test_pack_is_the_oracles(lib, N, K, spread, scaled):
    # spread 60 reaches bf16's subnormals and, times s, fp32's
    W = _weights(N, K, N + K, spread)
    W = torch.where(torch.isfinite(W), W, torch.zeros_like(W))
    s = _inv_s(K, 3) if scaled else None
    p = lib.wq_quantize_mxfp4(W.cuda(), scale_s=None if s is None else s.cuda())
    ref = _same_pack(p, W, s)
    v = lib.wq_dequantize_mxfp4(p)
    np.testing.assert_array_equal(f64(v), oracle.dequant_mxfp4(ref))


def test_pack_of_edge_blocks(lib):
    W = torch.zeros(8, 128, dtype=torch.bfloat16)
    W[0, :16] = torch.tensor([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -0.0, -7.75])
    W[1, 7] = float("inf")
    W[2, 40] = float("nan")
    W[3, 70] = float("-inf")
    W[4, :] = torch.finfo(torch.bfloat16).max
    W[5, ::3] = torch.finfo(torch.bfloat16).tiny
    W[6, 5] = 2.0**-133  # bf16's smallest subnormal
    W[7, :] = -0.0
    p = lib.wq_quantize_mxfp4(W.cuda())
    ref = _same_pack(p, W)
    v = f64(lib.wq_dequantize_mxfp4(p))
    np.testing.assert_array_equal(v, oracle.dequant_mxfp4(ref))
    assert np.isnan(v[1, :32]).all() and (v[1, 32:] == 0).all()
    # s overflows the product: the block is not finite either
    s = torch.ones(128)
    s[100] = 1e38
    p = lib.wq_quantize_mxfp4((W[4:5] + 0).cuda(), scale_s=s.cuda())
    _same_pack(p, W[4:5], s)
    assert p.bscale[0, 3].item() == 255


def test_values_of_every_scale_and_code(lib):
    codes = torch.arange(16, dtype=torch.uint8).repeat(256, 1)  # bytes 0..15 -> codes (0..15, 0)
    codes = codes | (torch.arange(16, dtype=torch.uint8).flip(0) << 4)
    bscale = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(256, 1)
    p = lib.PackedMXFP4(codes.contiguous().cuda(), bscale.cuda(), 256, 32)
    v = f64(lib.wq_dequantize_mxfp4(p))
    ref = oracle.dequant_mxfp4(dict(codes=codes.numpy(), bscale=bscale.numpy(), N=256, K=32))
    with np.errstate(over="ignore"):
        ref = np.where(np.abs(ref) >= 2.0**128, np.copysign(np.inf, ref), ref)
    np.testing.assert_array_equal(v, ref)
    np.testing.assert_array_equal(np.signbit(v[:255]), np.signbit(ref[:255]))


@pytest.mark.parametrize("M", [1, 2, 3, 8, 13, 16, 17, 31, 33, 64, 65, 100, 129, 192, 193, 260, 515])
@pytest.mark.parametrize("N,K", [(1, 32), (5, 96), (203, 1056), (384, 512), (130, 2080), (264, 2048)])
def test_linear(lib, M, N, K):
    W, X = _weights(N, K, N * K, 1.0), _acts(M, K, M + K)
    p = lib.wq_quantize_mxfp4(W.cuda())
    Y = lib.wq_linear_mxfp4(X.cuda(), p)
    assert lib.wq_device_error() == 0
    assert_within_bound(Y, f64(X), mx_values(p), False, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M", [1, 5, 16, 40, 200])
@pytest.mark.parametrize("N,K", [(3, 32), (129, 1056), (256, 2048)])
def test_linear_with_act_inv_s(lib, M, N, K):
    s = _inv_s(K, 11)
    W, X = _weights(N, K, 5), _acts(M, K, M)
    p = lib.wq_quantize_mxfp4(W.cuda(), scale_s=s.cuda())
    inv = (1.0 / s).float()
    Y = lib.wq_linear_mxfp4(X.cuda(), p, act_inv_s=inv.cuda())
    assert_within_bound(Y, f64(X) * inv.double().numpy(), mx_values(p), True, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(1, 2048, 11008), (16, 2051, 11008), (300, 2048, 2048)])
def test_linear_at_block_shapes(lib, M, N, K):
    W, X = _weights(N, K, 1), _acts(M, K, 2)
    p = lib.wq_quantize_mxfp4(W.cuda())
    Y = lib.wq_linear_mxfp4(X.cuda(), p)
    assert_within_bound(Y, f64(X), mx_values(p), False)
    again = lib.wq_linear_mxfp4(X.cuda(), p)
    assert torch.equal(Y.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("M", [1, 7, 16, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(1, 64), (5, 192), (203, 1088), (136, 512), (256, 2048)])
@pytest.mark.parametrize("scaled", [False, True])
def test_linear_with_fp4_activations(lib, M, N, K, scaled):
    W, X = _weights(N, K, N + K, 1.0), _acts(M, K, M)
    inv = _inv_s(K, 17) if scaled else None
    p = lib.wq_quantize_mxfp4(W.cuda())
    need = lib.linear_workspace_size(M, N, K, lib.WQ_FMT_MXFP4, 1)
    ws = torch.full((need,), 0xAB, dtype=torch.uint8, device="cuda")
    Y = lib.wq_linear_mxfp4(X.cuda(), p, act_fp4=1, act_inv_s=None if inv is None else inv.cuda(), ws=ws)
    assert lib.wq_device_error() == 0
    x = oracle.dequant_mxfp4(oracle.quantize_mxfp4(X, None if inv is None else inv.numpy()))
    assert_within_bound(Y, x, mx_values(p), False, f"{M}x{N}x{K}")


@pytest.mark.parametrize("act_fp4", [0, 1])
@pytest.mark.parametrize("M", [4, 150])
def test_extreme_scales(lib, M, act_fp4):
    # weights near 2^100 against activations near 2^-100, and the other way round
    N, K = 40, 256
    for up in (100, -100):
        W = (_weights(N, K, 3).double() * 2.0**up).to(torch.bfloat16)
        X = (_acts(M, K, 4).double() * 2.0**-up).to(torch.bfloat16)
        p = lib.wq_quantize_mxfp4(W.cuda())
        Y = lib.wq_linear_mxfp4(X.cuda(), p, act_fp4=act_fp4)
        x = oracle.dequant_mxfp4(oracle.quantize_mxfp4(X)) if act_fp4 else f64(X)
        assert_within_bound(Y, x, mx_values(p), False, f"2^{up}")


@pytest.mark.parametrize("act_fp4", [0, 1])
@pytest.mark.parametrize("M", [2, 12, 150])
def test_not_a_number_stays_in_its_row_and_column(lib, M, act_fp4):
    N, K = 140, 320
    W, X = _weights(N, K, 8), _acts(M, K, 9)
    W[17, 100] = float("nan")
    X[1, 5] = float("nan")
    X[0, 6] = float("inf")
    p = lib.wq_quantize_mxfp4(W.cuda())
    Y = f64(lib.wq_linear_mxfp4(X.cuda(), p, act_fp4=act_fp4))
    rows, cols = np.arange(M) > 1, np.arange(N) != 17
    assert np.isnan(Y[:, 17]).all() and np.isnan(Y[1]).all()
    assert not np.isfinite(Y[0]).any()
    assert np.isfinite(Y[np.ix_(rows, cols)]).all()


def test_group_items(lib):
    K = 512
    X = _acts(2, K, 1).cuda()
    ps = [lib.wq_quantize_mxfp4(_weights(N, K, N).cuda()) for N in (64, 203)]
    pn = lib.wq_quantize_nvfp4(_weights(96, K, 7).cuda())
    outs = [torch.empty(2, p.N, dtype=torch.bfloat16, device="cuda") for p in (*ps, pn)]
    lib.wq_linear_group([(X, p, y) for p, y in zip((*ps, pn), outs)])
    for p, y in zip(ps, outs):
        assert torch.equal(y.view(torch.int16), lib.wq_linear_mxfp4(X, p).view(torch.int16))
    assert torch.isfinite(outs[2].float()).all()


def test_other_stream_and_captured_replay(lib):
    N, K, M = 200, 512, 24
    W, X = _weights(N, K, 1).cuda(), _acts(M, K, 2).cuda()
    ws = torch.empty(lib.linear_workspace_size(M, N, K, lib.WQ_FMT_MXFP4, 1), dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(2):
            p = lib.wq_quantize_mxfp4(W)
            y16, y4 = lib.wq_linear_mxfp4(X, p), lib.wq_linear_mxfp4(X, p, act_fp4=1, ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            p = lib.wq_quantize_mxfp4(W)
            y16, y4 = lib.wq_linear_mxfp4(X, p), lib.wq_linear_mxfp4(X, p, act_fp4=1, ws=ws)
    torch.cuda.current_stream().wait_stream(st)
    for seed in (5, 6):
        W.copy_(_weights(N, K, seed))
        X.copy_(_acts(M, K, seed + 1))
        g.replay()
        torch.cuda.synchronize()
        assert_within_bound(y16, f64(X), mx_values(p), False)
        x = oracle.dequant_mxfp4(oracle.quantize_mxfp4(X.cpu()))
        assert_within_bound(y4, x, mx_values(p), False)


def test_binding_refuses_wrong_tensors(lib):
    W = _weights(16, 64, 1).cuda()
    p = lib.wq_quantize_mxfp4(W)
    X = _acts(3, 64, 1).cuda()
    bad = [lambda: lib.wq_quantize_mxfp4(W.t()), lambda: lib.wq_quantize_mxfp4(W.half()),
           lambda: lib.wq_quantize_mxfp4(W[0]), lambda: lib.wq_quantize_mxfp4(W, scale_s=torch.ones(63).cuda()),
           lambda: lib.wq_linear_mxfp4(X.float(), p), lambda: lib.wq_linear_mxfp4(X[:, :32].contiguous(), p),
           lambda: lib.wq_linear_mxfp4(X, p, out=torch.empty(3, 15, dtype=torch.bfloat16, device="cuda")),
           lambda: lib.wq_linear_mxfp4(X, lib.PackedMXFP4(p.codes, p.bscale[:, :1].contiguous(), 16, 64)),
           lambda: lib.wq_dequantize_mxfp4(p, out=torch.empty(16, 63, dtype=torch.bfloat16, device="cuda"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(lib.WQError):
        lib.wq_quantize_mxfp4(torch.zeros(4, 48, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(lib.WQError):
        lib.wq_linear_mxfp4(X, p, act_fp4=1, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
