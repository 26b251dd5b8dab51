"""What a 4-bit refiner block does around its linear layers, as measurable cases.

Four operators of lora_gemm_b200 that one denoising step calls in a row:

  quantize   mxfp4_quantize / mxfp4_dequantize: bf16 rows to OCP MXFP4 (E2M1
             codes, one E8M0 scale per 32 values along K) and back
  linear     lora_linear_mxfp4: y = deq(x) deq(W)^T + (x A_cat^T) B_cat^T, the
             activations quantized within the call as each stage does it
  norm       block_norm: h' = alpha h + gate * N(b) and n = N(h') (1 + scale) +
             shift, with n also as MXFP4 where the next layer takes it so
  backward   block_norm_backward: the gradients of all of norm's inputs

`own` false: the plain form, elementary torch operations in FP32.  `own` true:
the library's calls.  Both take the same state.  listed() names the cases,
draw() gives more of the same ranges, exact() is the definition in FP64.
"""

import math

import torch

own = False
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases.  d = 1024 and 7168, 4d = 28672, 3d = 21504, the adapter ranks (sums of
# 384, 128 and 64) and the 2,304-token and 14,400-token frames (36 x 64 and
# 90 x 160 cells) are this repository's own workload sizes.
# ---------------------------------------------------------------------------
def listed():
    return [
        # One token's activations: all launch latency.
        dict(name="quantize 1x1024", op="quantize", M=1, K=1024),
        # A ragged slice of a 2K clip before its d -> d layer.
        dict(name="quantize 33001x7168", op="quantize", M=33001, K=7168),
        # A single token through a wide layer with all three adapters: bound by reading the weights.
        dict(name="linear 1x7168x7168 r576", op="linear", M=1, K=7168, N=7168, R=576),
        # A few conditioning tokens through the d -> 3d projection, one adapter pair.
        dict(name="linear 19x7168x21504 r192", op="linear", M=19, K=7168, N=21504, R=192),
        # One small frame at the narrow width: the smallest grid the repository runs.
        dict(name="linear 2304x1024x1024 r576", op="linear", M=2304, K=1024, N=1024, R=576),
        # A ragged batch through d -> 3d with the adapters merged away.
        dict(name="linear 5003x7168x21504 r0", op="linear", M=5003, K=7168, N=21504, R=0),
        # Part of a 2K clip through the MLP's output projection: the largest product.
        dict(name="linear 16384x28672x7168 r576", op="linear", M=16384, K=28672, N=7168, R=576),
        # One token between two blocks, handed on in 4 bits.
        dict(name="norm 1x7168 bf16 q", op="norm", M=1, D=7168, seg=1, fp32=False, post="rms", pre="rms", alpha=1.0,
             quant=True),
        # One small frame with an FP32 stream and layer norms.
        dict(name="norm 2304x1024 fp32", op="norm", M=2304, D=1024, seg=2304, fp32=True, post="none", pre="layer",
             alpha=1.0, quant=False),
        # Four and a half 2K frames, modulated per frame, handed on in 4 bits.
        dict(name="norm 66601x7168 bf16 q", op="norm", M=66601, D=7168, seg=14400, fp32=False, post="rms", pre="rms",
             alpha=0.7071, quant=True),
        # A short training slice with an odd frame length and layer norms.
        dict(name="backward 777x1024 fp32", op="backward", M=777, D=1024, seg=301, fp32=True, post="layer",
             pre="layer", alpha=1.0, quant=False),
        # Two 2K frames and a ragged rest, in training.
        dict(name="backward 33001x7168 bf16", op="backward", M=33001, D=7168, seg=14400, fp32=False, post="rms",
             pre="rms", alpha=0.7071, quant=False),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "norm", "backward"])
    if op == "quantize":
        return dict(op=op, M=_log_uniform(rng, 1, 33001), K=128 * _log_uniform(rng, 1, 56))
    if op == "linear":
        K = 128 * _log_uniform(rng, 1, 224)
        N = 32 * _log_uniform(rng, 1, 672)
        R = 64 * rng.randint(0, 9)
        most = 16384 * (28672 * 7168 + 576 * (28672 + 7168)) // (K * N + R * (K + N))
        return dict(op=op, M=_log_uniform(rng, 1, min(16384, most)), K=K, N=N, R=R)
    quant = op == "norm" and rng.random() < 0.5
    D = 128 * _log_uniform(rng, 1, 80) if quant else 8 * _log_uniform(rng, 8, 1280)
    most = 66601 if op == "norm" else 33001
    M = _log_uniform(rng, 1, min(most, most * 7168 // D))
    return dict(op=op, M=M, D=D, seg=_log_uniform(rng, max(1, M // 16), M), fp32=rng.random() < 0.5,
                post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "layer"]),
                alpha=rng.choice([1.0, 0.7071]), quant=quant)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _activations(g, M, K):
    """Normal activations with a spread over rows and a few large channels."""
    x = torch.randn(M, K, generator=g, device=DEV)
    x *= torch.exp2(torch.randn(M, 1, generator=g, device=DEV))
    x[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device=DEV)] *= 8.0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, M = case["op"], case["M"]
    s = dict(case)
    if op == "quantize":
        s["x"] = _activations(g, M, case["K"])
    elif op == "linear":
        K, N, R = case["K"], case["N"], case["R"]
        s["x"] = _activations(g, M, K)
        w = (torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16)
        # The weights in 4 bits, as a program holds them after loading.
        codes, exps = _plain_quantize(w)
        s["W"] = (_pack(codes), _blocked(exps))
        # FP32 merged factors; the adapters' term comes to about half the base term.
        s["A"] = torch.randn(R, K, generator=g, device=DEV) * K ** -0.5 if R else None
        s["B"] = torch.randn(N, R, generator=g, device=DEV) * (0.5 * R ** -0.5) if R else None
    else:
        D, seg = case["D"], case["seg"]
        S = -(-M // seg)
        stream = torch.float32 if case["fp32"] else torch.bfloat16
        s["h"] = (_activations(g, M, D).float() * 2.0).to(stream)
        s["b"] = _activations(g, M, D)
        s["gate"] = torch.randn(S, D, generator=g, device=DEV) * 0.3
        s["scale"] = torch.randn(S, D, generator=g, device=DEV) * 0.2
        s["shift"] = torch.randn(S, D, generator=g, device=DEV) * 0.2
        if op == "backward":
            s["dn"] = (torch.randn(M, D, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
            s["dh"] = (torch.randn(M, D, generator=g, device=DEV) * 0.1).to(stream)
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(s):
    return _own_run(s) if own else _plain_run(s)


def _own_run(s):
    import lora_gemm_b200 as lg

    op = s["op"]
    if op == "quantize":
        codes, scales = lg.mxfp4_quantize(s["x"])
        return {"values": lg.mxfp4_dequantize(codes, scales)}
    if op == "linear":
        return {"y": lg.lora_linear_mxfp4(s["x"], lg.mxfp4_quantize(s["x"]), s["W"], s["A"], s["B"])}
    kinds = dict(alpha=s["alpha"], post=None if s["post"] == "none" else s["post"], pre=s["pre"],
                 segment_tokens=s["seg"])
    if op == "norm":
        h, n, q = lg.block_norm(s["h"], s["b"], s["gate"], s["scale"], s["shift"],
                                quant="mxfp4" if s["quant"] else None, **kinds)
        return {"h": h, "n": n, "q": lg.mxfp4_dequantize(*q)} if s["quant"] else {"h": h, "n": n}
    dh, db, dgate, dscale, dshift = lg.block_norm_backward(s["dn"], s["dh"], s["h"], s["b"], s["gate"], s["scale"],
                                                           **kinds)
    return {"dh": dh, "db": db, "dgate": dgate, "dscale": dscale, "dshift": dshift}


# E2M1 code (sign in bit 3) -> value.
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _power(e):
    """2^e in FP64 from the bits (a power function rounds)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _plain_quantize(x):
    """Codes [rows, K] (one per value) and block exponents [rows, K / 32]."""
    rows, K = x.shape
    v = x.float().view(rows, K // 32, 32)
    amax = v.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)  # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    a = (v.double().abs() * _power(-e)[..., None]).float()  # exact
    # Round to nearest, ties to the even code.
    c = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).byte()
    c += 8 * torch.signbit(v).byte()
    return c.view(rows, K), e


def _values(codes, exps):
    """The FP32 values that codes and exponents stand for (exact)."""
    rows, K = codes.shape
    v = torch.tensor(_E2M1, device=codes.device)[codes.int()].view(rows, K // 32, 32)
    return (v * _power(exps)[..., None]).float().view(rows, K)


def _pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), -1).view(packed.shape[0], -1)


def _blocked(exps):
    """E8M0 bytes in the blocked layout: 128 rows x 4 blocks are 512 bytes,
    row r and block b of a group at 16 (r mod 32) + 4 (r / 32) + b."""
    rows, kb = exps.shape
    pad = -rows % 128
    byte = torch.nn.functional.pad((exps + 127).to(torch.uint8), (0, 0, 0, pad))
    return byte.view(-1, 4, 32, kb // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _unblocked(scales, rows, kb):
    byte = scales.view(-1, kb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, kb)
    return byte[:rows].int() - 127


def _plain_norm(v, kind):
    """(normalised rows, 1 / deviation)."""
    if kind == "none":
        return v, None
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)
    return v * r, r


def _plain_norm_grad(g, u, r, kind):
    """Gradient of the rows from that of the normalised rows u."""
    if kind == "none":
        return g
    d = g - u * (g * u).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(-1, keepdim=True)
    return d * r


def _segment_sums(v, seg):
    M, D = v.shape
    S = -(-M // seg)
    return torch.nn.functional.pad(v, (0, 0, 0, S * seg - M)).view(S, seg, D).sum(1)


def _plain_run(s):
    op, M = s["op"], s["M"]
    if op == "quantize":
        return {"values": _values(*_plain_quantize(s["x"])).to(torch.bfloat16)}
    if op == "linear":
        x, (codes, scales) = s["x"], s["W"]
        N, K = codes.shape[0], s["K"]
        y = _values(*_plain_quantize(x)) @ _values(_unpack(codes), _unblocked(scales, N, K // 32)).T
        if s["R"]:
            y += (x.float() @ s["A"].T) @ s["B"].T
        return {"y": y.to(torch.bfloat16)}
    seg = torch.arange(M, device=s["h"].device) // s["seg"]
    gate, scale = s["gate"][seg], s["scale"][seg]
    if op == "norm":
        u, _ = _plain_norm(s["b"].float(), s["post"])
        h = (s["alpha"] * s["h"].float() + gate * u).to(s["h"].dtype)
        # The pre-norm reads the stream as it is stored.
        n = _plain_norm(h.float(), s["pre"])[0] * (1.0 + scale) + s["shift"][seg]
        n = n.to(torch.bfloat16)
        if not s["quant"]:
            return {"h": h, "n": n}
        # The 4-bit copy is that of the bf16 n.
        return {"h": h, "n": n, "q": _values(*_plain_quantize(n)).to(torch.bfloat16)}
    dn = s["dn"].float()
    xhat, r = _plain_norm(s["h"].float(), s["pre"])
    dh = s["dh"].float() + _plain_norm_grad(dn * (1.0 + scale), xhat, r, s["pre"])
    u, rb = _plain_norm(s["b"].float(), s["post"])
    db = _plain_norm_grad(gate * dh, u, rb, s["post"])
    return {"dh": (s["alpha"] * dh).to(s["h"].dtype), "db": db.to(torch.bfloat16),
            "dgate": _segment_sums(dh * u, s["seg"]), "dscale": _segment_sums(dn * xhat, s["seg"]),
            "dshift": _segment_sums(dn, s["seg"])}


# ---------------------------------------------------------------------------
# Work of one pass: each input read once, each output written once.
# ---------------------------------------------------------------------------
def work(case):
    op, M = case["op"], case["M"]
    if op == "quantize":
        n = M * case["K"]
        # bf16 in; codes and scales written; bf16 values out.
        return {"bytes": 2 * n + n * 17 / 32 + 2 * n, "flops": 0}
    if op == "linear":
        K, N, R = case["K"], case["N"], case["R"]
        return {"bytes": 2 * M * K + N * K * 17 / 32 + 4 * R * (K + N) + 2 * M * N,
                "flops": 2 * M * (K * N + R * (K + N))}
    D = case["D"]
    n, S, w = M * D, -(-M // case["seg"]), 4 if case["fp32"] else 2
    if op == "norm":
        # h, b in; h', n out; the 4-bit copy written and its values out.
        return {"bytes": n * (w + 2 + w + 2) + 3 * 4 * S * D + (n * 17 / 32 + 2 * n if case["quant"] else 0),
                "flops": 0}
    # dn, dh', h', b in; dh, db out; gate, scale in; dgate, dscale, dshift out.
    return {"bytes": n * (2 + w + w + 2 + w + 2) + 5 * 4 * S * D, "flops": 0}


# ---------------------------------------------------------------------------
# The definition in FP64.
# ---------------------------------------------------------------------------
def _exact_power(e):
    return torch.tensor([2.0 ** k for k in range(-140, 141)], dtype=torch.float64, device=e.device)[e.long() + 140]


def _exact_mxfp4(v):
    """Values of the MXFP4 copy of FP64 rows: per 32 values 2^e with e =
    floor(log2 max) - 2; E2M1 has steps of 1/2 below 2, 1 below 4 and 2 to 6."""
    rows, K = v.shape
    t = v.reshape(rows, -1, 32)
    top = t.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top)).clamp(-130.0, 130.0)
    e = e - (_exact_power(e) > top).double()  # the logarithm rounded up to a whole number,
    e = e + (_exact_power(e + 1) <= top).double()  # or down past one
    e = (e - 2.0).clamp(-127.0, 127.0)
    t = t * _exact_power(-e)
    step = 0.5 + 0.5 * (t.abs() >= 2.0) + 1.0 * (t.abs() >= 4.0)
    t = (torch.round(t / step) * step).clamp(-6.0, 6.0)  # torch.round takes ties to even
    return (t * _exact_power(e)).reshape(rows, K)


def _exact_weights(packed, scales, N, K):
    n = torch.arange(N, device=packed.device)[:, None]
    k = torch.arange(K // 32, device=packed.device)[None, :]
    at = ((n // 128) * (K // 128) + k // 4) * 512 + 16 * (n % 32) + 4 * ((n % 128) // 32) + k % 4
    power = _exact_power(scales[at].double() - 127.0)
    w = torch.empty(N, K, dtype=torch.float64, device=packed.device)
    for half in (0, 1):
        c = ((packed >> (4 * half)) & 15).double()
        m, sign = torch.remainder(c, 8.0), 1.0 - 2.0 * torch.floor(c / 8.0)
        frac, ex = torch.remainder(m, 2.0), torch.floor(m / 2.0)
        w[:, half::2] = sign * torch.where(ex > 0, (1.0 + frac / 2.0) * _exact_power((ex - 1.0).clamp(min=0.0)), frac / 2.0)
    return w * power.repeat_interleave(32, 1)


def _exact_center(v, kind):
    return v - v.mean(1, keepdim=True) if kind == "layer" else v


def exact(case, seed):
    s = prepare(case, seed)
    op, M = case["op"], case["M"]
    if op == "quantize":
        return {"values": _exact_mxfp4(s["x"].double())}
    if op == "linear":
        w = _exact_weights(s["W"][0], s["W"][1], case["N"], case["K"])
        y = torch.empty(M, case["N"], dtype=torch.float64, device=DEV)
        for i in range(0, M, 4096):
            x = s["x"][i:i + 4096].double()
            y[i:i + 4096] = _exact_mxfp4(x) @ w.T
            if case["R"]:
                y[i:i + 4096] += (x @ s["A"].double().T) @ s["B"].double().T
        return {"y": y}
    D, seg, eps = case["D"], case["seg"], 1e-6
    stream = s["h"].dtype
    out = {}
    if op == "norm":
        out = {k: torch.empty(M, D, dtype=torch.float64, device=DEV) for k in ("h", "n", "q")}
        for f in range(-(-M // seg)):
            for i in range(f * seg, min((f + 1) * seg, M), 4096):
                at = slice(i, min(i + 4096, (f + 1) * seg, M))
                u = s["b"][at].double()
                if case["post"] != "none":
                    c = _exact_center(u, case["post"])
                    u = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
                h = case["alpha"] * s["h"][at].double() + s["gate"][f].double() * u
                out["h"][at] = h
                c = _exact_center(h.to(stream).double(), case["pre"])
                n = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * (1.0 + s["scale"][f].double())
                n = n + s["shift"][f].double()
                out["n"][at] = n
                if case["quant"]:
                    out["q"][at] = _exact_mxfp4(n.to(torch.bfloat16).double())
        if not case["quant"]:
            del out["q"]
        return out
    S = -(-M // seg)
    out = {k: torch.empty(M, D, dtype=torch.float64, device=DEV) for k in ("dh", "db")}
    out |= {k: torch.zeros(S, D, dtype=torch.float64, device=DEV) for k in ("dgate", "dscale", "dshift")}
    for f in range(S):
        gate, mul = s["gate"][f].double(), 1.0 + s["scale"][f].double()
        for i in range(f * seg, min((f + 1) * seg, M), 4096):
            at = slice(i, min(i + 4096, (f + 1) * seg, M))
            dn = s["dn"][at].double()
            out["dshift"][f] += dn.sum(0)
            c = _exact_center(s["h"][at].double(), case["pre"])
            var = (c * c).mean(1, keepdim=True) + eps
            out["dscale"][f] += (dn * c / torch.sqrt(var)).sum(0)
            t = dn * mul
            t = t / torch.sqrt(var) - c * (t * c).mean(1, keepdim=True) / var ** 1.5
            dh = s["dh"][at].double() + _exact_center(t, case["pre"])
            out["dh"][at] = case["alpha"] * dh
            u = s["b"][at].double()
            t = gate * dh
            if case["post"] != "none":
                c = _exact_center(u, case["post"])
                var = (c * c).mean(1, keepdim=True) + eps
                t = _exact_center(t / torch.sqrt(var) - c * (t * c).mean(1, keepdim=True) / var ** 1.5, case["post"])
                u = c / torch.sqrt(var)
            out["db"][at] = t
            out["dgate"][f] += (dh * u).sum(0)
    return out
