"""Cases of the MXFP4 and expert-grouped operators: how they are called, and their plain form.

    quantise  W (bf16 [N, K]) -> MXFP4 pack -> the values the pack stands for (bf16 [N, K])
    linear    Y = (X inv_s) W^T for an MXFP4 pack, activations in bf16 or (act_fp4) packed to MXFP4 too
    experts   Y[i] = X[i] W_e^T for offsets[e] <= i < offsets[e+1] over a stack of 4-bit packs

`own` False computes the plain form in elementary torch operations; True calls the library.
"""
import math
import random

import torch

own = False

# magnitudes of the eight E2M1 codes (the sign is bit 3)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one small projection (the k projection of a 2048-wide block): the time of the launches
        dict(name="quantise_small", op="quantise", N=256, K=2048, scaled=False),
        # odd row count, K not a power of two, with an input-channel scale as an AWQ pack has it
        dict(name="quantise_scaled_odd", op="quantise", N=1003, K=1376, scaled=True),
        # a large matrix of a whole-model pass
        dict(name="quantise_large", op="quantise", N=16384, K=8192, scaled=False),
        # one token through the gate projection of a decode step
        dict(name="linear_token", op="linear", M=1, N=11008, K=2048, act_fp4=0, scaled=False),
        # a small decode batch through a down projection, odd N, 1/s left on the activations
        dict(name="linear_batch_odd", op="linear", M=13, N=2051, K=11008, act_fp4=0, scaled=True),
        # prefill of 2048 tokens through the gate projection, bf16 activations and 4-bit ones
        dict(name="linear_prefill", op="linear", M=2048, N=11008, K=2048, act_fp4=0, scaled=False),
        dict(name="linear_prefill_a4", op="linear", M=2048, N=11008, K=2048, act_fp4=1, scaled=False),
        # one token, eight experts: the smallest decode step of a mixture of experts
        dict(name="experts_token", op="experts", fmt="mxfp4", E=64, active=8, T=8, tail=0, N=1408, K=2048, G=0,
             skew=0.0),
        # 32 tokens, eight experts each: nearly every expert holds a few rows
        dict(name="experts_batch", op="experts", fmt="int4", E=64, active=61, T=256, tail=0, N=1408, K=2048, G=64,
             skew=1.0),
        # padded batch: rows behind the last sequence stay; odd N, an odd number of groups of 32
        dict(name="experts_padded_odd", op="experts", fmt="int4", E=60, active=37, T=1931, tail=117, N=1003, K=2080,
             G=32, skew=2.0),
        # prefill of 2048 tokens, eight experts each, near-even routing
        dict(name="experts_prefill", op="experts", fmt="nvfp4", E=64, active=64, T=16384, tail=0, N=1408, K=2048, G=0,
             skew=0.3),
        # the way back to the model's width with uneven routing
        dict(name="experts_down_uneven", op="experts", fmt="mxfp4", E=64, active=64, T=8192, tail=0, N=2048, K=1408,
             G=0, skew=2.0),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["quantise", "linear", "linear", "experts", "experts"])
    if op == "quantise":
        return dict(op=op, N=_logint(rng, 1, 16384), K=32 * _logint(rng, 1, 256), scaled=rng.random() < 0.4)
    if op == "linear":
        a4 = int(rng.random() < 0.3)
        K = 64 * _logint(rng, 1, 172) if a4 else 32 * _logint(rng, 1, 344)
        N = _logint(rng, 1, 11008)
        top = min(2048, (2048 * 11008 * 2048) // (N * K))
        return dict(op=op, M=_logint(rng, 1, max(1, top)), N=N, K=K, act_fp4=a4, scaled=rng.random() < 0.4)
    fmt = rng.choice(["int4", "nvfp4", "mxfp4"])
    G = rng.choice([32, 64, 128]) if fmt == "int4" else 0
    step = max(G, 32)
    K = step * _logint(rng, 1, 2048 // step)
    N = _logint(rng, 1, 2048)
    E = _logint(rng, 1, 128)
    T = _logint(rng, 1, min(16384, max(1, (16384 * 1408 * 2048) // (N * K))))
    active = rng.randint(1, min(E, T))
    return dict(op=op, fmt=fmt, E=E, active=active, T=T, tail=rng.choice([0, 0, rng.randint(1, 200)]), N=N, K=K, G=G,
                skew=round(rng.uniform(0.0, 2.5), 2))


def work(case):
    c = case
    if c["op"] == "quantise":
        n = c["N"] * c["K"]
        return {"bytes": 4.0 * n + (4.0 * c["K"] if c["scaled"] else 0.0), "flops": 4.0 * n}
    if c["op"] == "linear":
        w = c["N"] * c["K"] * (0.5 + 1 / 32)
        return {"bytes": w + 2.0 * c["M"] * (c["K"] + c["N"]) + (4.0 * c["K"] if c["scaled"] else 0.0),
                "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    if c["fmt"] == "int4":
        per_row = c["K"] / 2 + c["K"] / c["G"] * 2 + (c["K"] / c["G"] + 7) // 8 * 4
    else:
        per_row = c["K"] / 2 + c["K"] / (16 if c["fmt"] == "nvfp4" else 32)
    w = c["active"] * c["N"] * per_row
    return {"bytes": w + 2.0 * c["T"] * (c["K"] + c["N"]) + 4.0 * (c["E"] + 1), "flops": 2.0 * c["T"] * c["N"] * c["K"]}


# ---------------------------------------------------------------- plain forms
def _e2m1_codes(v):
    """Nearest E2M1 code of fp32 values: ties to the even code, saturating at 6, sign kept."""
    a = v.abs()
    c = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (c + 8 * torch.signbit(v)).to(torch.uint8)


def _e2m1_values(codes):
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float32, device=codes.device)
    return table[codes.long()]


def _mx_quantise(A, s=None):
    """bf16 [R, C] (times s per column, fp32) -> (codes uint8 [R, C], exponents int [R, C / 32])."""
    a = A.float()
    if s is not None:
        a = a * s
    b = a.view(a.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = torch.frexp(amax)[1] - 3  # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    codes = _e2m1_codes(torch.ldexp(b, -e.unsqueeze(-1)))
    return codes.view_as(a), e


def _mx_values(codes, e):
    v = _e2m1_values(codes).view(codes.shape[0], -1, 32)
    return torch.ldexp(v, e.unsqueeze(-1)).view(codes.shape)


def _pack_nibbles(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def _unpack_nibbles(packed):
    return torch.stack((packed & 15, packed >> 4), dim=-1).view(packed.shape[0], -1)


def _e4m3_values(b):
    return b.view(torch.float8_e4m3fn).float()


def _int4_words(q):  # codes [R, C] -> int32 words of eight codes, the first in the low bits
    w = torch.zeros(q.shape[0], q.shape[1] // 8, dtype=torch.int64, device=q.device)
    for j in range(8):
        w |= q[:, j::8].long() << (4 * j)
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32)


def _int4_nibbles(w, n):  # int32 words [R, C] -> the first n nibbles of each row
    sh = torch.arange(0, 32, 4, device=w.device)
    return ((w.unsqueeze(-1) >> sh) & 15).view(w.shape[0], -1)[:, :n]


def _int4_values(w, r0, r1, G):
    scales, zeros = w["scales"][r0:r1].float(), w["zeros"][r0:r1]
    q = _int4_nibbles(w["packed"][r0:r1], w["K"]).view(r1 - r0, -1, G)
    z = _int4_nibbles(zeros, scales.shape[1])
    return ((q - z.unsqueeze(-1)).float() * scales.unsqueeze(-1)).view(r1 - r0, -1)


def _expert_values(w, e, dtype=torch.float32):
    """The weights [N, K] of expert e of a stack, as the values the pack stands for."""
    N, K = w["N"], w["K"]
    r0, r1 = e * N, (e + 1) * N
    if w["fmt"] == "int4":
        return _int4_values(w, r0, r1, w["G"]).to(dtype)
    v = _e2m1_values(_unpack_nibbles(w["packed"][r0:r1]))
    if w["fmt"] == "mxfp4":
        return _mx_values_of_bytes(v, w["bscale"][r0:r1]).to(dtype)
    sb = _e4m3_values(w["bscale"][r0:r1]).unsqueeze(-1)
    return (v.view(N, -1, 16) * sb).view(N, K).to(dtype) * w["g"][e].to(dtype)


def _mx_values_of_bytes(v, bscale):
    return torch.ldexp(v.view(v.shape[0], -1, 32), (bscale.int() - 127).unsqueeze(-1)).view(v.shape)


def _plain(state):
    op = state["op"]
    if op == "quantise":
        codes, e = _mx_quantise(state["W"], state["s"])
        return _mx_values(codes, e).to(torch.bfloat16)
    if op == "linear":
        Wv = _mx_values_of_bytes(_e2m1_values(_unpack_nibbles(state["codes"])), state["bscale"])
        if state["act_fp4"]:
            Xv = _mx_values(*_mx_quantise(state["X"], state["inv_s"]))
        else:
            Xv = state["X"].float()
            if state["inv_s"] is not None:
                Xv = Xv * state["inv_s"]
        return (Xv @ Wv.t()).to(torch.bfloat16)
    Y = state["Y"]
    for e, (r0, r1) in enumerate(zip(state["bounds"][:-1], state["bounds"][1:])):
        if r1 > r0:
            Y[r0:r1] = (state["X"][r0:r1].float() @ _expert_values(state["w"], e).t()).to(torch.bfloat16)
    return Y


def _own(state):
    import w4a16_gemm_wq_b200 as wq

    op = state["op"]
    if op == "quantise":
        return wq.wq_dequantize_mxfp4(wq.wq_quantize_mxfp4(state["W"], scale_s=state["s"]))
    if op == "linear":
        return wq.wq_linear_mxfp4(state["X"], state["pack"], act_fp4=state["act_fp4"], act_inv_s=state["inv_s"],
                                  ws=state["ws"])
    return wq.wq_linear_experts(state["X"], state["offsets"], state["pack"], out=state["Y"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weights(rows, K, g):
    return (torch.randn(rows, K, device="cuda", generator=g) / math.sqrt(K)).to(torch.bfloat16)


def _activations(rows, K, g):
    # unit normal with a few strong channels, as the output of a norm has them
    x = torch.randn(rows, K, device="cuda", generator=g)
    ch = 1.0 + 4.0 * (torch.rand(K, device="cuda", generator=g) < 0.02).float()
    return (x * ch).to(torch.bfloat16)


def _channel_scale(K, g):
    return torch.exp(0.4 * torch.randn(K, device="cuda", generator=g))


def _bounds(case, seed):
    """Row bounds of the experts: `active` of them (chosen by the seed) share T rows, unevenly by `skew`."""
    r = random.Random(seed)
    E, A, T = case["E"], case["active"], case["T"]
    chosen = r.sample(range(E), A)
    share = [math.exp(case["skew"] * r.gauss(0.0, 0.5)) for _ in range(A)]
    rest, total = T - A, sum(share)
    counts = [1 + int(rest * s / total) for s in share]
    for i in range(T - sum(counts)):
        counts[i % A] += 1
    per = [0] * E
    for e, n in zip(chosen, counts):
        per[e] = n
    bounds = [0]
    for n in per:
        bounds.append(bounds[-1] + n)
    return bounds


def _stack(case, g):
    """The packed weights of all experts, rows [E * N]."""
    E, N, K, fmt, G = case["E"], case["N"], case["K"], case["fmt"], case["G"]
    w = dict(fmt=fmt, E=E, N=N, K=K, G=G, packed=[], bscale=[], scales=[], zeros=[], g=[])
    for _ in range(E):
        W = _weights(N, K, g).float()
        if fmt == "int4":
            b = W.view(N, -1, G)
            mx, mn = b.amax(-1), b.amin(-1)
            s = ((mx - mn) / 15.0).clamp(1e-5, 65504.0).half()
            z = torch.round(-mn / s.float()).clamp(0, 15)
            q = (torch.round(b / s.float().unsqueeze(-1)) + z.unsqueeze(-1)).clamp(0, 15)
            zp = torch.nn.functional.pad(z.int(), (0, -z.shape[1] % 8))
            w["packed"].append(_int4_words(q.view(N, K).int()))
            w["scales"].append(s)
            w["zeros"].append(_int4_words(zp))
        elif fmt == "mxfp4":
            codes, e = _mx_quantise(W)
            w["packed"].append(_pack_nibbles(codes))
            w["bscale"].append((e + 127).to(torch.uint8))
        else:
            gs = W.abs().amax() / (6 * 448)
            b = W.view(N, -1, 16)
            sb = (b.abs().amax(-1) / 6 / gs).to(torch.float8_e4m3fn)
            d = sb.float().unsqueeze(-1) * gs
            codes = torch.where(d > 0, _e2m1_codes(b / d), torch.zeros((), dtype=torch.uint8, device="cuda"))
            w["packed"].append(_pack_nibbles(codes.view(N, K)))
            w["bscale"].append(sb.view(torch.uint8))
            w["g"].append(gs.view(1))
    for k in ("packed", "bscale", "scales", "zeros", "g"):
        w[k] = torch.cat(w[k]) if w[k] else None
    return w


def prepare(case, seed):
    g = _gen(seed)
    op, K = case["op"], case["K"]
    if op == "quantise":
        s = _channel_scale(K, g) if case["scaled"] else None
        return dict(op=op, W=_weights(case["N"], K, g), s=s)
    if op == "linear":
        M, N = case["M"], case["N"]
        codes, e = _mx_quantise(_weights(N, K, g))
        st = dict(op=op, X=_activations(M, K, g), codes=_pack_nibbles(codes), bscale=(e + 127).to(torch.uint8),
                  act_fp4=case["act_fp4"], inv_s=_channel_scale(K, g) if case["scaled"] else None)
        if own:
            import w4a16_gemm_wq_b200 as wq

            st["pack"] = wq.PackedMXFP4(st["codes"], st["bscale"], N, K)
            nbytes = wq.linear_workspace_size(M, N, K, wq.WQ_FMT_MXFP4, case["act_fp4"])
            st["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None
        return st
    w = _stack(case, g)
    rows = case["T"] + case["tail"]
    bounds = _bounds(case, seed)
    st = dict(op=op, w=w, X=_activations(rows, K, g), bounds=bounds,
              offsets=torch.tensor(bounds, dtype=torch.int32, device="cuda"),
              Y=torch.randn(rows, case["N"], device="cuda", generator=g).to(torch.bfloat16))
    if own:
        import w4a16_gemm_wq_b200 as wq

        E, N = case["E"], case["N"]

        def view(t):
            return None if t is None else t.view(E, N, -1)

        st["pack"] = wq.PackedExperts(case["fmt"], E, N, K, view(w["packed"]), scales=view(w["scales"]),
                                      zeros=view(w["zeros"]), group_size=case["G"], zero_point=1,
                                      bscale=view(w["bscale"]), global_scale=w["g"])
    return st


# ---------------------------------------------------------------- the definition, in 64 bits
def _mx_exact(A, s=None):
    """The MXFP4 values of A (times s, rounded to fp32), from the nearest entry of the table of magnitudes."""
    out = torch.empty(A.shape, dtype=torch.float64, device=A.device)
    mags = torch.tensor(E2M1, dtype=torch.float64, device=A.device)
    rows = max(1, (1 << 24) // A.shape[1])
    for r in range(0, A.shape[0], rows):
        a = A[r:r + rows].float()
        a = (a if s is None else a * s).double().view(a.shape[0], -1, 32)
        top = a.abs().amax(-1, keepdim=True)
        p = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
        # the logarithm may be off by one at a power of two
        p = p + (torch.exp2(p + 1) <= top).double() - (torch.exp2(p) > top).double()
        scale = torch.exp2(torch.where(top > 0, p - 2, torch.full_like(p, -127.0)).clamp(-127, 127))
        x = (a / scale).abs()
        best, dist = torch.zeros_like(x), x.clone()
        for c in range(1, 8):
            d = (x - mags[c]).abs()
            # the closer one; at a tie the even code
            take = (d < dist) | ((d == dist) & (c % 2 == 0))
            best, dist = torch.where(take, mags[c], best), torch.where(take, d, dist)
        out[r:r + rows] = (torch.copysign(best, a) * scale).view(a.shape[0], -1)
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "quantise":
        return _mx_exact(st["W"], st["s"])
    mags = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def e2m1(packed):  # low nibble first
        nib = torch.empty(packed.shape[0], packed.shape[1] * 2, dtype=torch.long, device="cuda")
        nib[:, 0::2], nib[:, 1::2] = (packed % 16).long(), (packed // 16).long()
        return torch.where(nib >= 8, -mags[nib % 8], mags[nib % 8])

    def spread(scale, K):
        return scale.repeat_interleave(K // scale.shape[1], dim=1)

    K = case["K"]
    if case["op"] == "linear":
        W = e2m1(st["codes"]) * spread(torch.exp2(st["bscale"].double() - 127), K)
        if case["act_fp4"]:
            X = _mx_exact(st["X"], st["inv_s"])
        else:
            X = st["X"].double() if st["inv_s"] is None else st["X"].double() * st["inv_s"].double()
        return X @ W.t()
    Y, w, N = st["Y"].double(), st["w"], case["N"]
    for e in range(case["E"]):
        r0, r1 = st["bounds"][e], st["bounds"][e + 1]
        if r0 == r1:
            continue
        rows = slice(e * N, (e + 1) * N)
        if case["fmt"] == "int4":
            q = torch.empty(N, K, dtype=torch.float64, device="cuda")
            for j in range(8):
                q[:, j::8] = ((w["packed"][rows].long() % 2**32) // 16**j % 16).double()
            ng = K // case["G"]
            z = torch.stack([(w["zeros"][rows][:, i // 8].long() % 2**32) // 16**(i % 8) % 16 for i in range(ng)], 1)
            W = (q - spread(z.double(), K)) * spread(w["scales"][rows].double(), K)
        elif case["fmt"] == "mxfp4":
            W = e2m1(w["packed"][rows]) * spread(torch.exp2(w["bscale"][rows].double() - 127), K)
        else:
            W = e2m1(w["packed"][rows]) * spread(w["bscale"][rows].view(torch.float8_e4m3fn).double(), K)
            W = W * w["g"][e].double()
        Y[r0:r1] = st["X"][r0:r1].double() @ W.t()
    return Y
