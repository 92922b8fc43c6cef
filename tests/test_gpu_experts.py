"""Products grouped by expert on the GPU against fp64 products of the same packs."""
import math

import numpy as np
import pytest
import torch

from tests._linear_ref import assert_within_bound, expert_values, f64

pytestmark = pytest.mark.gpu

FMTS = ["int4_g128", "int4_g64", "int4_g32", "int4_sym", "nvfp4", "mxfp4"]


def _stack(lib, fmt, E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(E, N, K, generator=g) / math.sqrt(K)).to(torch.bfloat16).cuda()
    if fmt.startswith("int4"):
        G = {"int4_g128": 128, "int4_g32": 32}.get(fmt, 64)
        return lib.wq_quantize_experts(W, "int4", G, 0 if fmt == "int4_sym" else 1)
    return lib.wq_quantize_experts(W, fmt)


def _acts(T, K, seed):
    return torch.randn(T, K, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _offsets(counts, lead=0):
    return torch.tensor(np.concatenate([[lead], lead + np.cumsum(counts)]), dtype=torch.int32)


def _check(Y, X, p, counts, lead=0, what=""):
    r = lead
    for e, n in enumerate(counts):
        if n:
            assert_within_bound(Y[r:r + n], f64(X[r:r + n]), expert_values(p, e), p.fmt == "int4", f"{what} expert {e}")
        r += n


def _run(lib, p, counts, seed, lead=0, tail=0):
    T = lead + sum(counts) + tail
    X = _acts(T, p.K, seed)
    X[:lead] = float("nan")       # rows of no expert: neither read into others nor written
    X[T - tail:] = float("inf") if tail else 0.0
    out = torch.full((T, p.N), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = lib.wq_linear_experts(X.cuda(), _offsets(counts, lead).cuda(), p, out=out)
    assert lib.wq_device_error() == 0
    assert Y.data_ptr() == out.data_ptr()
    _check(Y, X, p, counts, lead)
    assert (Y[:lead] == 7.0).all() and (Y[T - tail:] == 7.0).all() if tail else (Y[:lead] == 7.0).all()
    return X, Y


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K", [(1, 128), (96, 384), (203, 1152), (264, 2048)])
@pytest.mark.parametrize("counts", [[1, 0, 0, 0], [3, 1, 0, 17], [0, 33, 64, 5], [130, 0, 1, 260]])
def test_formats_and_sizes(lib, fmt, N, K, counts):
    _run(lib, _stack(lib, fmt, len(counts), N, K, N + K), counts, 3)


@pytest.mark.parametrize("fmt", ["int4_g32", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("K", [32, 64, 96, 160, 288, 1056, 2080])
@pytest.mark.parametrize("counts", [[2, 5], [70, 9]])
def test_odd_lengths_of_k(lib, fmt, K, counts):
    _run(lib, _stack(lib, fmt, 2, 77, K, K), counts, 4)


@pytest.mark.parametrize("fmt", ["int4_g64", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("lead,tail", [(0, 1), (5, 0), (40, 300)])
def test_rows_of_no_expert_stay(lib, fmt, lead, tail):
    _run(lib, _stack(lib, fmt, 3, 130, 256, 1), [20, 0, 45], 5, lead, tail)


@pytest.mark.parametrize("fmt", ["int4_g64", "mxfp4"])
@pytest.mark.parametrize("E,counts", [
    (1, {0: 1}), (1, {0: 700}), (130, {0: 1, 129: 1}), (130, {64: 500}), (1024, {3: 2, 1000: 40, 1023: 1}),
    (300, {e: 1 + e % 3 for e in range(300)})])
def test_numbers_of_experts(lib, fmt, E, counts):
    c = [counts.get(e, 0) for e in range(E)]
    _run(lib, _stack(lib, fmt, E, 40, 128, E), c, 6)


@pytest.mark.parametrize("fmt", ["int4_g64", "nvfp4", "mxfp4"])
def test_every_row_count_around_the_tiles(lib, fmt):
    p = _stack(lib, fmt, 4, 150, 256, 9)
    for n in list(range(14, 19)) + list(range(30, 35)) + [47, 48, 49, 63, 64, 65, 95, 96, 97, 127, 128, 129, 191, 192,
                                                          193, 255, 256, 257, 384, 385]:
        _run(lib, p, [n, 1, 0, n + 1], n)


def test_no_rows(lib):
    p = _stack(lib, "mxfp4", 3, 64, 128, 1)
    Y = lib.wq_linear_experts(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"),
                              torch.zeros(4, dtype=torch.int32, device="cuda"), p)
    assert Y.shape == (0, 64)
    X = _acts(9, 128, 1).cuda()
    out = torch.full((9, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lib.wq_linear_experts(X, torch.full((4,), 4, dtype=torch.int32, device="cuda"), p, out=out)
    assert (out == 3.0).all()
    # without `out`, rows of no expert are zero
    Y = lib.wq_linear_experts(X, torch.tensor([2, 3, 3, 5], dtype=torch.int32, device="cuda"), p)
    assert (Y[:2] == 0).all() and (Y[5:] == 0).all() and (Y[2:5] != 0).any()


@pytest.mark.parametrize("T", [9, 2000])
@pytest.mark.parametrize("offsets", [[0, 5, 4, 9], [-1, 2, 3, 9], [0, 2, 3, 1 << 30], [0, 1 << 30, 3, 9], [9, 8, 7, 6]])
def test_bad_offsets_compute_nothing(lib, T, offsets):
    p = _stack(lib, "mxfp4", 3, 200, 128, 1)
    X = _acts(T, 128, 1).cuda()
    out = torch.full((T, 200), 3.0, dtype=torch.bfloat16, device="cuda")
    lib.wq_linear_experts(X, torch.tensor(offsets, dtype=torch.int32, device="cuda"), p, out=out)
    with pytest.raises(lib.WQError) as e:
        lib.wq_device_error()
    assert e.value.status == lib.WQ_ERR_ARG and "offsets" in str(e.value)
    assert (out == 3.0).all()
    assert lib.wq_device_error() == 0


@pytest.mark.parametrize("fmt", ["int4_g64", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("counts", [[2, 3], [90, 70]])
def test_not_a_number_stays_in_its_row(lib, fmt, counts):
    p = _stack(lib, fmt, 2, 150, 256, 2)
    T = sum(counts)
    X = _acts(T, 256, 3)
    X[1, 7] = float("nan")
    X[counts[0], 9] = float("inf")
    Y = f64(lib.wq_linear_experts(X.cuda(), _offsets(counts).cuda(), p))
    ok = np.ones(T, bool)
    ok[[1, counts[0]]] = False
    assert np.isfinite(Y[ok]).all() and np.isnan(Y[1]).all()
    assert not np.isfinite(Y[counts[0]]).all()


def test_nan_scale_of_one_expert(lib):
    p = _stack(lib, "mxfp4", 2, 130, 256, 2)
    p.bscale[1, 5, 3] = 255
    X = _acts(40, 256, 3)
    Y = f64(lib.wq_linear_experts(X.cuda(), _offsets([20, 20]).cuda(), p))
    assert np.isnan(Y[20:, 5]).all()
    Y[20:, 5] = 0
    assert np.isfinite(Y).all()


@pytest.mark.parametrize("fmt", ["int4_g64", "nvfp4"])
@pytest.mark.parametrize("counts", [[1, 0, 4, 2], [300, 20, 0, 150]])
def test_same_bits_every_time(lib, fmt, counts):
    p = _stack(lib, fmt, 4, 520, 1024, 1)
    X = _acts(sum(counts), 1024, 2).cuda()
    o = _offsets(counts).cuda()
    ys = [lib.wq_linear_experts(X, o, p).view(torch.int16) for _ in range(4)]
    assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_replayed_with_other_offsets_and_on_two_streams(lib):
    E, N, K, T = 5, 264, 512, 150
    p, q = _stack(lib, "mxfp4", E, N, K, 1), _stack(lib, "int4_g64", E, N, K, 2)
    X, o = _acts(T, K, 1).cuda(), _offsets([30] * 5).cuda()
    outs = [torch.zeros(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        lib.wq_linear_experts(X, o, p, out=outs[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            lib.wq_linear_experts(X, o, p, out=outs[0])
    torch.cuda.current_stream().wait_stream(st)
    for counts in ([0, 0, 150, 0, 0], [1, 2, 3, 4, 5], [100, 0, 0, 0, 50]):
        outs[0].zero_()
        X.copy_(_acts(T, K, sum(counts)))
        o.copy_(_offsets(counts))
        g.replay()
        _check(outs[0], X, p, counts)
    # both stacks at once, on two streams
    counts = [40, 0, 60, 1, 49]
    o.copy_(_offsets(counts))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, w, y in zip(streams, (p, q), outs):
        with torch.cuda.stream(s):
            for _ in range(3):
                lib.wq_linear_experts(X, o, w, out=y)
    torch.cuda.synchronize()
    for w, y in zip((p, q), outs):
        _check(y, X, w, counts)


@pytest.mark.parametrize("tokens", [1, 9, 120])
@pytest.mark.parametrize("fmt", ["int4", "nvfp4", "mxfp4"])
def test_a_mixture_of_experts_block(lib, tokens, fmt):
    # packs, routing, both products and the combination as a block runs them; each product
    # against the fp64 product of the rows that it was given
    E, top, D, F = 8, 2, 256, 384
    g = torch.Generator().manual_seed(tokens)
    up = lib.wq_quantize_experts((torch.randn(E, 2 * F, D, generator=g) / 16).to(torch.bfloat16).cuda(), fmt)
    down = lib.wq_quantize_experts((torch.randn(E, D, F, generator=g) / 16).to(torch.bfloat16).cuda(), fmt)
    x = torch.randn(tokens, D, generator=g).to(torch.bfloat16).cuda()
    weight, ids = torch.topk(torch.softmax(torch.randn(tokens, E, generator=g), -1).cuda(), top)
    order = torch.argsort(ids.flatten(), stable=True)
    counts = torch.bincount(ids.flatten(), minlength=E)
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
    rows = x[order // top]
    h = lib.wq_linear_experts(rows, offsets, up)
    act = (torch.nn.functional.silu(h[:, :F].float()) * h[:, F:].float()).to(torch.bfloat16)
    y = lib.wq_linear_experts(act, offsets, down)
    out = torch.zeros(tokens, D, device="cuda").index_add_(0, order // top, y.float() * weight.flatten()[order, None])
    assert lib.wq_device_error() == 0 and torch.isfinite(out).all()
    _check(h, rows, up, counts.tolist())
    _check(y, act, down, counts.tolist())


def test_each_expert_is_the_single_linear(lib):
    # the same pack as one expert, and through its own entry point
    N, K, T = 264, 512, 100
    X = _acts(T, K, 1).cuda()
    p = _stack(lib, "mxfp4", 1, N, K, 1)
    Y = lib.wq_linear_experts(X, _offsets([T]).cuda(), p)
    Z = lib.wq_linear_mxfp4(X, lib.PackedMXFP4(p.packed[0], p.bscale[0], N, K))
    assert (Y.float() - Z.float()).abs().max() <= 2.0**-7 * Z.float().abs().max()


def test_binding_refuses_wrong_tensors(lib):
    p = _stack(lib, "int4_g64", 3, 64, 128, 1)
    X, o = _acts(9, 128, 1).cuda(), _offsets([3, 3, 3]).cuda()
    bad = [lambda: lib.wq_linear_experts(X.float(), o, p), lambda: lib.wq_linear_experts(X, o.long(), p),
           lambda: lib.wq_linear_experts(X, o[:3], p), lambda: lib.wq_linear_experts(X, o.cpu(), p),
           lambda: lib.wq_linear_experts(X[:, :64].contiguous(), o, p), lambda: lib.wq_linear_experts(X.t(), o, p),
           lambda: lib.wq_linear_experts(X, o, p, out=torch.empty(8, 64, dtype=torch.bfloat16, device="cuda")),
           lambda: lib.wq_linear_experts(X, o, lib.PackedExperts("int4", 3, 64, 128, p.packed, group_size=64)),
           lambda: lib.wq_linear_experts(X, o, lib.PackedExperts("fp8", 3, 64, 128, p.packed)),
           lambda: lib.wq_quantize_experts(X), lambda: lib.wq_quantize_experts(X.view(1, 9, 128), "fp8")]
    for call in bad:
        with pytest.raises(ValueError):
            call()
