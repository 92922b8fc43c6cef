"""The forms of the MXFP4 Linear and the expert product where sizes change from one to the
next, and what they share: K over a cluster, activations held in fp16, first calls in a capture."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests._linear_ref import assert_within_bound, f64, mx_values
from tests.test_gpu_experts import FMTS, _acts, _check, _offsets, _run, _stack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [128, 384, 1152, 2048])
@pytest.mark.parametrize("lead,tail", [(0, 0), (3, 20)])
def test_few_rows_of_many_experts(lib, fmt, K, lead, tail):
    counts = [0, 1, 2, 9, 0, 3, 17, 1, 8, 0] * 4
    _run(lib, _stack(lib, fmt, len(counts), 525, K, K), counts, 8, lead, tail)


@pytest.mark.parametrize("fmt", ["int4_g32", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("K", [32, 96, 160, 2080])
def test_few_rows_of_many_experts_at_odd_lengths(lib, fmt, K):
    counts = [1, 0, 13, 2] * 10
    _run(lib, _stack(lib, fmt, len(counts), 525, K, K), counts, 9)


@pytest.mark.parametrize("fmt,K", [("int4_g32", 5888), ("int4_g32", 5920), ("nvfp4", 6656), ("mxfp4", 6656),
                                   ("mxfp4", 6688)])
def test_the_longest_k_of_few_rows(lib, fmt, K):
    counts = [0] * 30
    counts[2], counts[7], counts[29] = 13, 1, 19
    _run(lib, _stack(lib, fmt, len(counts), 525, K, 1), counts, 10)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [1152, 2048, 4224])
@pytest.mark.parametrize("counts", [[20, 0, 45], [1, 200, 0], [7, 5, 8]])
def test_k_shared_by_a_cluster(lib, fmt, K, counts):
    _run(lib, _stack(lib, fmt, 3, 131, K, K), counts, 11, 5, 30)


@pytest.mark.parametrize("M", [1, 2, 3, 8, 9, 200])
@pytest.mark.parametrize("K", [6656, 6688, 11008])
def test_long_k_with_and_without_room_for_scaled_rows(lib, M, K):
    N = 67
    W = torch.randn(N, K, generator=torch.Generator().manual_seed(K)).to(torch.bfloat16)
    inv = torch.exp(0.5 * torch.randn(K, generator=torch.Generator().manual_seed(1)))
    X = _acts(M, K, M)
    p = lib.wq_quantize_mxfp4(W.cuda())
    w, x, n = mx_values(p), f64(X), lib.linear_workspace_size(M, N, K, lib.WQ_FMT_MXFP4, 0)
    assert_within_bound(lib.wq_linear_mxfp4(X.cuda(), p), x, w, False)
    for room in {0, max(0, n - 1), n, n + 16}:
        ws = torch.full((room,), 0xAB, dtype=torch.uint8, device="cuda") if room else \
            torch.empty(16, dtype=torch.uint8, device="cuda")
        Y = lib.wq_linear_mxfp4(X.cuda(), p, act_inv_s=inv.cuda(), ws=ws)
        assert_within_bound(Y, x * inv.double().numpy(), w, True, f"{room} of {n} bytes")
        if room > n:
            assert (ws[n:] == 0xAB).all()


@pytest.mark.parametrize("M", [1, 2, 8, 16])
def test_group_items_with_act_inv_s(lib, M):
    N, K = 133, 1056
    X = _acts(M, K, 1)
    inv = torch.exp(0.5 * torch.randn(K, generator=torch.Generator().manual_seed(2)))
    p = lib.wq_quantize_mxfp4(torch.randn(N, K, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda())
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    lib.wq_linear_group([(X.cuda(), p, Y, inv.cuda())])
    assert_within_bound(Y, f64(X) * inv.double().numpy(), mx_values(p), True)


@pytest.mark.parametrize("M", [1, 2, 5, 40])
@pytest.mark.parametrize("spread", [8, 30, 60])
def test_activations_of_a_wide_range(lib, M, spread):
    # fp16 staging of few rows: exact down to 2^-31 of the row's largest magnitude, and what is
    # below is off by half a step of fp16's smallest, 2^-25 where the largest is 2^14 or more
    N, K = 70, 1056
    g = torch.Generator().manual_seed(spread)
    X = (torch.randn(M, K, generator=g) * torch.exp2(-spread * torch.rand(M, K, generator=g))).to(torch.bfloat16)
    X[0, 3] = 1e30
    X[-1, 5] = 1e-38
    p = lib.wq_quantize_mxfp4(torch.randn(N, K, generator=g).to(torch.bfloat16).cuda())
    Y, w, x = f64(lib.wq_linear_mxfp4(X.cuda(), p)), mx_values(p), f64(X)
    ref, S = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = 2.0**-8 * np.abs(ref) + 2 * K * 2.0**-24 * S
    tol = tol + 2.0**-39 * np.abs(x).max(1, keepdims=True) * np.abs(w).sum(1)[None]
    assert (np.abs(Y - ref) <= tol).all()


@pytest.mark.parametrize("M", [1, 2, 5, 40])
def test_scales_far_apart_in_a_row(lib, M):
    N, K = 48, 512
    g = torch.Generator().manual_seed(4)
    W = torch.randn(N, K // 32, 32, generator=g) * torch.exp2(torch.randint(-50, 50, (N, K // 32, 1), generator=g).float())
    W[3] = 0
    W[5, 2:] = 0
    p = lib.wq_quantize_mxfp4(W.reshape(N, K).to(torch.bfloat16).cuda())
    X = _acts(M, K, M)
    assert_within_bound(lib.wq_linear_mxfp4(X.cuda(), p), f64(X), mx_values(p), False)


def test_a_pack_of_more_than_two_gib(lib):
    E, N, K = 40, 16384, 7168
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    bscale = torch.randint(118, 124, (E, N, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    assert codes.numel() > 1 << 31
    p = lib.PackedExperts("mxfp4", E, N, K, codes, bscale=bscale)
    for counts in ([0] * 38 + [1, 2], [0] * 38 + [30, 9], [0] * 38 + [4, 40]):
        T = sum(counts)
        X = _acts(T, K, T)
        Y = lib.wq_linear_experts(X.cuda(), _offsets(counts).cuda(), p)
        assert lib.wq_device_error() == 0
        r = 0
        for e in (38, 39):  # the last 64 rows of the last experts
            q = lib.PackedMXFP4(codes[e, -64:].contiguous(), bscale[e, -64:].contiguous(), 64, K)
            n = counts[e]
            assert_within_bound(Y[r:r + n, -64:], f64(X[r:r + n]), mx_values(q), False, f"expert {e}")
            r += n


def test_first_calls_inside_a_capture():
    # a process whose first launches, with their one-time queries, are captured
    code = """
import torch, w4a16_gemm_wq_b200 as wq
torch.manual_seed(0)
W = torch.randn(3, 131, 2048, device="cuda").to(torch.bfloat16)
X = torch.randn(48, 2048, device="cuda").to(torch.bfloat16)
inv = torch.rand(2048, device="cuda") + 0.5
off = torch.tensor([0, 20, 20, 48], dtype=torch.int32, device="cuda")
packs = [wq.PackedExperts("mxfp4", 3, 131, 2048, torch.randint(0, 256, (3, 131, 1024), dtype=torch.uint8, device="cuda"),
                          bscale=torch.full((3, 131, 64), 120, dtype=torch.uint8, device="cuda"))]
one = wq.PackedMXFP4(packs[0].packed[0].contiguous(), packs[0].bscale[0].contiguous(), 131, 2048)
torch.cuda.synchronize()
def calls():
    return [wq.wq_linear_experts(X, off, packs[0]), wq.wq_linear_experts(X[:9], off[:1].repeat(4).contiguous(), packs[0]),
            wq.wq_linear_mxfp4(X[:1], one), wq.wq_linear_mxfp4(X[:5], one), wq.wq_linear_mxfp4(X, one, act_inv_s=inv),
            wq.wq_linear_mxfp4(X, one, act_fp4=1), wq.wq_dequantize_mxfp4(wq.wq_quantize_mxfp4(W[0]))]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = calls()
g.replay()
torch.cuda.synchronize()
assert wq.wq_device_error() == 0
for x, y in zip(a, calls()):
    assert torch.equal(x.view(torch.int16), y.view(torch.int16))
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_streams_at_once(lib):
    # the same pack from two streams, forms with and without clusters in flight together
    p = _stack(lib, "mxfp4", 3, 131, 4224, 1)
    sizes = [[20, 0, 45], [1, 0, 3], [200, 100, 0], [9, 9, 9]]
    X = [_acts(sum(c), 4224, i) for i, c in enumerate(sizes)]
    dev = [(x.cuda(), _offsets(c).cuda()) for x, c in zip(X, sizes)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    out = [[], []]
    for _ in range(5):
        for s, st in enumerate(streams):
            with torch.cuda.stream(st):
                out[s] += [lib.wq_linear_experts(x, o, p) for x, o in (dev if s else dev[::-1])]
    torch.cuda.synchronize()
    assert lib.wq_device_error() == 0
    for s in range(2):
        for i, y in enumerate(out[s]):
            k = i % 4 if s else 3 - i % 4
            assert torch.equal(y.view(torch.int16), out[1][k].view(torch.int16))
    for k, c in enumerate(sizes):
        _check(out[1][k], X[k], p, c)
