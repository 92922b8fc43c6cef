"""Values at which the forms of the expert product and the MXFP4 Linear could part: infinities,
INT4 rows of a wide range, what few INT4 rows keep of their bits, magnitudes near the ends of fp32."""
import math

import numpy as np
import pytest
import torch

from tests._linear_ref import assert_within_bound, expert_values, f64, mx_values
from tests.test_gpu_experts import FMTS, _acts, _offsets, _run, _stack

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


def _int4_stack(lib, E, N, K, G, seed):
    """Random codes and zero points, scales within a factor of two."""
    g = torch.Generator().manual_seed(seed)
    ng = K // G
    words = lambda *s: torch.randint(-2**31, 2**31, s, generator=g).to(torch.int32).cuda()
    zeros = words(E, N, (ng + 7) // 8)
    if ng % 8:
        zeros[..., -1] &= (1 << 4 * (ng % 8)) - 1
    scales = (2.0**-7 * (1 + torch.rand(E, N, ng, generator=g))).half().cuda()
    return lib.PackedExperts("int4", E, N, K, words(E, N, K // 8), scales=scales, zeros=zeros, group_size=G,
                             zero_point=1)


def _scale_of_terms(p, e):
    """The scale of each weight, [N, K] in fp64."""
    return np.repeat(f64(p.scales[e]), p.group_size, axis=1)


def _int4_sum_error(p, e, x, form):
    """Bound of the error of the fp32 sums of an INT4 row, [M, N] for x [M, K], from S = sum_k s |x_k|.

    cores: per 32 k two chains of 16 multiply-adds of terms below 2 |x| (17 roundings), times 16;
    31 adds of x times 16 + z <= 31; four more roundings of both: under 2^11 2^-24 S.
    mma_sync: G / 16 steps of terms up to 1264 |x| (1024 + 16 * 15), each off by two units of
    2^-23 of its partial sum at most; the sums of x times 1024 + z, 12 roundings.
    """
    S = np.abs(x) @ _scale_of_terms(p, e).T
    if form == "cores":
        return 2.0**11 * 2.0**-24 * S
    return ((p.group_size / 16) * 2 * 1264 * 2.0**-23 + 12 * 1039 * 2.0**-24) * S


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("form", ["cores", "mma_sync"])
def test_int4_elements_far_below_the_rows_largest(lib, G, form):
    # group 0 holds the row's largest element and has scale 0; the elements of the other groups, 2^-34 of
    # it, all lie between two fp16 values of the row's staging on the same side
    counts, N = FORMS[form]
    T, K = sum(counts), 1024
    p = _int4_stack(lib, len(counts), N, K, G, 31)
    p.scales[:, :, 0] = 0
    X = torch.full((T, K), 2.0**-14 * 131 / 128, dtype=torch.bfloat16)
    X[:, :G] = 0.0
    X[:, 5] = 2.0**20
    Y = f64(lib.wq_linear_experts(X.cuda(), _offsets(counts).cuda(), p))
    x = f64(X)
    for e in np.unique(_experts_of(counts)):
        rows = _experts_of(counts) == e
        w = expert_values(p, e)
        ref = x[rows] @ w.T
        # elements are held to 2^-35 of the row's largest
        tol = 2.0**-8 * np.abs(ref) + 2.0**-35 * 2.0**20 * np.abs(w).sum(1) + _int4_sum_error(p, e, x[rows], form)
        bad = np.abs(Y[rows] - ref) > tol
        assert not bad.any(), (e, np.abs(Y[rows] - ref).max(), tol.min(), bad.mean())


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("form", ["cores", "mma_sync"])
@pytest.mark.parametrize("outlier", [0, 64.0, 1e4])
def test_int4_of_few_rows_rounds_no_weight(lib, G, form, outlier):
    counts, N = FORMS[form]
    T, K = sum(counts), 2048
    p = _int4_stack(lib, len(counts), N, K, G, 32)
    X = _acts(T, K, 33)
    if outlier:
        X[:, 77] = outlier
        X[:, 1500] = -outlier
        # half the weight rows have q = z under the first: its term is zero
        z = (p.zeros[:, ::2, (77 // G) // 8] >> (4 * ((77 // G) % 8))) & 15
        word, at = 77 // 8, 4 * (77 % 8)
        old = p.packed[:, ::2, word]
        p.packed[:, ::2, word] = (old & ~(15 << at)) | (z << at)
    Y = f64(lib.wq_linear_experts(X.cuda(), _offsets(counts).cuda(), p))
    x, err, norm = f64(X), 0.0, 0.0
    for e in np.unique(_experts_of(counts)):
        rows = _experts_of(counts) == e
        ref = x[rows] @ expert_values(p, e).T
        S = np.abs(x[rows]) @ np.abs(expert_values(p, e)).T
        tol = 2.0**-8 * np.abs(ref) + K * 2.0**-24 * S + _int4_sum_error(p, e, x[rows], form)
        assert (np.abs(Y[rows] - ref) <= tol).all(), e
        err, norm = err + ((Y[rows] - ref) ** 2).sum(), norm + (ref**2).sum()
    if not outlier:
        # one rounding to bf16 (2^-8 at most, evenly spread) and a tenth for the sums
        assert math.sqrt(err / norm) <= 1.1 * 2.0**-8 / math.sqrt(3), math.sqrt(err / norm)


@pytest.mark.parametrize("fmt", ["int4_g128", "int4_g64", "int4_g32"])
def test_int4_of_many_rows_rounds_a_weight_once(lib, fmt):
    counts, N = FORMS["tcgen05"]
    p = _stack(lib, fmt, len(counts), N, 2048, 34)
    X = _acts(sum(counts), 2048, 35)
    Y, x = f64(lib.wq_linear_experts(X.cuda(), _offsets(counts).cuda(), p)), f64(X)
    ref = np.concatenate([x[:90] @ expert_values(p, 0).T, x[90:] @ expert_values(p, 2).T])
    # two independent roundings to bf16, of the weights and of the result
    assert math.sqrt(((Y - ref) ** 2).sum() / (ref**2).sum()) <= 1.1 * math.sqrt(2) * 2.0**-8 / math.sqrt(3)


@pytest.mark.parametrize("fmt,form,wexp,xexp", [
    ("nvfp4", "cores", -20, 115), ("nvfp4", "mma_sync", -20, 115), ("nvfp4", "cores", -100, 120),
    ("nvfp4", "mma_sync", -100, 120), ("nvfp4", "cores", 100, -110), ("nvfp4", "mma_sync", 100, -110),
    ("mxfp4", "cores", -30, 123), ("mxfp4", "mma_sync", -30, 123), ("mxfp4", "tcgen05", -30, 123),
    ("mxfp4", "cores", 121, -115), ("mxfp4", "mma_sync", 121, -115), ("mxfp4", "tcgen05", 121, -115),
    ("mxfp4", "cores", -115, 123), ("mxfp4", "mma_sync", -115, 123), ("mxfp4", "mma_sync", -110, -15),
    ("int4_g64", "cores", -4, 121), ("int4_g32", "cores", -4, 121), ("int4_g64", "mma_sync", -4, 121),
    ("int4_g64", "cores", -4, -118), ("int4_g64", "mma_sync", -4, -118)])
def test_magnitudes_near_the_ends_of_the_range(lib, fmt, form, wexp, xexp):
    # finite products of factors whose exponents are far from zero
    counts, N = FORMS[form]
    T, K = sum(counts), 1152
    g = torch.Generator().manual_seed(36)
    W = (torch.randn(len(counts), N, K, generator=g).double() * 2.0**wexp).to(torch.bfloat16).cuda()
    G = 32 if fmt == "int4_g32" else 64
    p = lib.wq_quantize_experts(W, "int4", G) if fmt.startswith("int4") else lib.wq_quantize_experts(W, fmt)
    X = (_acts(T, K, 37).double() * 2.0**xexp).to(torch.bfloat16)
    Y, x = lib.wq_linear_experts(X.cuda(), _offsets(counts).cuda(), p), f64(X)
    for e in np.unique(_experts_of(counts)):
        rows = torch.from_numpy(_experts_of(counts) == e)
        assert_within_bound(Y[rows.cuda()], x[rows.numpy()], expert_values(p, e), p.fmt == "int4", f"expert {e}")


@pytest.mark.parametrize("M", [1, 2, 5, 8, 40])
@pytest.mark.parametrize("wexp,xexp", [(-30, 123), (121, -115), (-115, 123), (-110, -15), (123, -130)])
def test_mxfp4_magnitudes_near_the_ends_of_the_range(lib, M, wexp, xexp):
    N, K = 70, 1056
    g = torch.Generator().manual_seed(38)
    p = lib.wq_quantize_mxfp4((torch.randn(N, K, generator=g).double() * 2.0**wexp).to(torch.bfloat16).cuda())
    X = (_acts(M, K, 39).double() * 2.0**xexp).to(torch.bfloat16)
    assert_within_bound(lib.wq_linear_mxfp4(X.cuda(), p), f64(X), mx_values(p), False)


@pytest.mark.parametrize("N,K", [(150, 512), (2051, 2048)])
def test_one_expert_is_the_plain_product(lib, N, K):
    # one expert that holds all rows runs as the product without offsets does: the same bits
    p = _stack(lib, "mxfp4", 1, N, K, 51)
    one = lib.PackedMXFP4(p.packed[0], p.bscale[0], N, K)
    for M in (1, 2, 3, 5, 8, 9, 13, 16, 17, 40):
        X = _acts(M, K, M).cuda()
        Y = lib.wq_linear_experts(X, _offsets([M]).cuda(), p)
        assert torch.equal(Y.view(torch.int16), lib.wq_linear_mxfp4(X, one).view(torch.int16)), M


@pytest.mark.parametrize("fmt", ["int4_g64", "int4_g32", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("N,K", [(2100, 4096), (4099, 2112), (700, 7168)])
@pytest.mark.parametrize("counts", [[0, 1, 0, 0, 0, 0, 1, 0], [3, 0, 1, 2, 0, 4, 1, 5], [0, 0, 16, 0, 0, 0, 0, 0]])
def test_few_rows_of_few_large_experts(lib, fmt, N, K, counts):
    _run(lib, _stack(lib, fmt, len(counts), N, K, 52), counts, 53, 0, 0)


# few rows of many experts: the mma.sync form
MANY = dict(E=40, N=525, K=512)


def _many(lib, fmt, seed):
    return _stack(lib, fmt, MANY["E"], MANY["N"], MANY["K"], seed)


@pytest.mark.parametrize("fmt", ["int4_g64", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("change", [(3, -1), (20, 0), (7, 1 << 30), (40, 61), (0, 5)])
def test_bad_offsets_of_many_experts_compute_nothing(lib, fmt, change):
    p, T = _many(lib, fmt, 41), 60
    offsets = torch.tensor([i * T // 40 for i in range(41)], dtype=torch.int32)
    offsets[change[0]] = change[1]
    out = torch.full((T, p.N), 3.0, dtype=torch.bfloat16, device="cuda")
    lib.wq_linear_experts(_acts(T, p.K, 1).cuda(), offsets.cuda(), p, out=out)
    with pytest.raises(lib.WQError) as e:
        lib.wq_device_error()
    assert e.value.status == lib.WQ_ERR_ARG and "offsets" in str(e.value)
    assert (out == 3.0).all() and lib.wq_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_many_experts_give_the_same_bits_every_time(lib, fmt):
    p, counts = _many(lib, fmt, 42), [0, 1, 2, 3] * 10
    X, o = _acts(sum(counts), p.K, 2).cuda(), _offsets(counts).cuda()
    ys = [lib.wq_linear_experts(X, o, p).view(torch.int16) for _ in range(4)]
    assert all(torch.equal(ys[0], y) for y in ys[1:])


@pytest.mark.parametrize("M", [5, 8])
def test_nan_scale_of_a_block_stays_in_its_column(lib, M):
    N, K = 140, 320
    p = lib.wq_quantize_mxfp4((torch.randn(N, K, generator=torch.Generator().manual_seed(1)) / 16).to(torch.bfloat16).cuda())
    p.bscale[17, 4] = 255
    p.codes[33, 32:48] = 0  # a block of zeros under a NaN scale is NaN too
    p.bscale[33, 2] = 255
    X = _acts(M, K, 3)
    X[2, 9] = float("nan")
    Y = f64(lib.wq_linear_mxfp4(X.cuda(), p))
    assert np.isnan(Y[:, [17, 33]]).all() and np.isnan(Y[2]).all()
    cols = ~np.isin(np.arange(N), [17, 33])
    assert np.isfinite(Y[np.ix_(np.arange(M) != 2, cols)]).all()


def test_nan_scale_of_one_of_many_experts(lib):
    p, counts = _many(lib, "mxfp4", 43), [1, 2] * 20
    p.bscale[7, 11, 3] = 255
    T = sum(counts)
    Y = f64(lib.wq_linear_experts(_acts(T, p.K, 3).cuda(), _offsets(counts).cuda(), p))
    mine = _experts_of(counts) == 7
    assert np.isnan(Y[mine, 11]).all()
    Y[mine, 11] = 0
    assert np.isfinite(Y).all()


@pytest.mark.parametrize("fmt", ["int4_g64", "nvfp4", "mxfp4"])
def test_many_experts_replayed_with_other_offsets_and_on_two_streams(lib, fmt):
    p, T = _many(lib, fmt, 44), 60
    X, o = _acts(T, p.K, 1).cuda(), _offsets([0, 1, 2, 3] * 10).cuda()
    outs = [torch.zeros(T, p.N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        lib.wq_linear_experts(X, o, p, out=outs[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            lib.wq_linear_experts(X, o, p, out=outs[0])
    torch.cuda.current_stream().wait_stream(st)

    def check(Y, X, counts):
        r = 0
        for e, n in enumerate(counts):
            if n:
                assert_within_bound(Y[r:r + n], f64(X[r:r + n]), expert_values(p, e), p.fmt == "int4", f"expert {e}")
            r += n

    sizes = [[60] + [0] * 39, [0] * 39 + [60], [3, 0] * 20, [0] * 40, [1, 2, 1, 2] * 10]
    for i, counts in enumerate(sizes):
        outs[0].fill_(5.0)
        X.copy_(_acts(T, p.K, i + 5))
        o.copy_(_offsets(counts))
        g.replay()
        check(outs[0], X, counts)
        assert (outs[0][sum(counts):] == 5.0).all()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, y in zip(streams, outs):
        with torch.cuda.stream(s):
            for _ in range(4):
                lib.wq_linear_experts(X, o, p, out=y)
    torch.cuda.synchronize()
    assert lib.wq_device_error() == 0
    check(outs[0], X, sizes[-1])
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


# ---------------------------------------------------------------- refusals of the binding
def test_binding_refuses_workspaces_and_group_items_it_cannot_hold(lib):
    X, W = _acts(12, 64, 1).cuda(), _acts(16, 64, 2).cuda()
    p = lib.wq_quantize_mxfp4(W)
    need = lib.linear_workspace_size(12, 16, 64, lib.WQ_FMT_MXFP4, 1)
    out = torch.empty(12, 16, dtype=torch.bfloat16, device="cuda")
    short = lib.PackedMXFP4(p.codes, p.bscale[:, :1].contiguous(), 16, 64)
    bad = [lambda: lib.wq_linear_mxfp4(X, p, act_fp4=1, ws=torch.empty(1, dtype=torch.uint8, device="cuda").expand(need)),
           lambda: lib.wq_linear_mxfp4(X, p, act_fp4=1, ws=torch.empty(need, dtype=torch.uint8)),
           lambda: lib.make_group([(X, short, out)]),
           lambda: lib.make_group([(X, lib.wq_quantize_experts(W.view(1, 16, 64)), out)])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
