"""block_norm_backward over many rows a CTA: its ring of row stages refilled, its
meeting places and their barriers' phases used again and again, its column sums
carried over dozens to thousands of rows, on one CTA and on clusters of 2, 4 and 8.
And its gradients against differences of block_norm.

The reference is the formula in FP64 on the GPU.  Tolerances as in
test_gpu_block_norm.py: half a step of the output type plus 2^-16 of the magnitudes
that enter; a column sum adds one rounding of 2^-24 for each addition on its longest
chain: the rows of a CTA, then an eighth of the CTAs of a segment, then eight."""

import pytest
import torch

import lora_gemm_b200 as lg

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP = 2.0 ** -16
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
KINDS = [(post, pre) for post in ("rms", "layer") for pre in ("rms", "layer")]


def _near(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


def _norm(v, kind, eps):
    """(N(v), 1 / deviation, the magnitude that enters a value) of FP64 rows; kind "rms" or "layer"."""
    mean = v.abs().mean(1, keepdim=True) if kind == "layer" else 0.0
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    u = v * r
    return u, r, u.abs() + r * mean


def _norm_gradient(g, u, r, kind):
    d = g - u * (g * u).mean(1, keepdim=True)
    return r * (d - d.mean(1, keepdim=True) if kind == "layer" else d)


def _check(t, got, post, pre, alpha, eps, seg, chain):
    """Rows against the formula, segment by segment; column sums with a longest chain of `chain` additions."""
    dh, db, dgate, dscale, dshift = got
    stream, M = t["h"].dtype, t["h"].shape[0]
    rounds = chain * 2.0 ** -24
    for s in range(-(-M // seg)):
        gate, mul = t["gate"][s].double(), 1.0 + t["scale"][s].double()
        sums = [0.0] * 6
        for i in range(s * seg, min((s + 1) * seg, M), 16384):
            at = slice(i, min(i + 16384, (s + 1) * seg, M))
            dn = t["dn"][at].double()
            x, r, xm = _norm(t["h"][at].double(), pre, eps)
            g = dn * mul
            dho = t["dh"][at].double() if t["dh"] is not None else torch.zeros_like(g)
            d = dho + _norm_gradient(g, x, r, pre)
            gm = g.abs()
            mag = dho.abs() + r * (gm + gm.mean(1, keepdim=True) + xm * (gm * xm).mean(1, keepdim=True))
            _near(dh[at], alpha * d, STEP[stream] * (alpha * d).abs() + FP * abs(alpha) * mag, "dh")
            u, r, um = _norm(t["b"][at].double(), post, eps)
            want = _norm_gradient(gate * d, u, r, post)
            w = gate.abs() * mag
            tol = 2 * FP * r * (w + w.mean(1, keepdim=True) + um * (w * um).mean(1, keepdim=True))
            _near(db[at], want, 2.0 ** -8 * want.abs() + tol, "db")
            for k, v in enumerate((d * u, mag * um, dn * x, dn.abs() * xm, dn, dn.abs())):
                sums[k] = sums[k] + v.sum(0)
        _near(dgate[s], sums[0], (2 * FP + rounds) * sums[1], "dgate")
        _near(dscale[s], sums[2], (FP + rounds) * sums[3], "dscale")
        _near(dshift[s], sums[4], rounds * sums[5], "dshift")


def _inputs(M, D, S, stream, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    return {"h": (randn(M, D) * torch.exp2(randn(M, 1)) + 0.25).to(stream), "b": (randn(M, D) - 0.25).to(torch.bfloat16),
            "gate": randn(S, D) * 0.5, "scale": randn(S, D) * 0.3, "dn": randn(M, D).to(torch.bfloat16),
            "dh": randn(M, D).to(stream)}


# Rows a CTA: about 50 to 75; segments that end inside one.
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post,pre", KINDS)
@pytest.mark.parametrize("M,D,seg", [(50001, 1024, 20003), (9001, 7168, 3517), (6001, 9216, 2411), (4001, 16384, 1699)])
def test_many_rows_a_cta(M, D, seg, post, pre, stream):
    t = _inputs(M, D, -(-M // seg), stream, seed=D)
    got = lg.block_norm_backward(t["dn"], t["dh"], t["h"], t["b"], t["gate"], t["scale"], alpha=0.7, post=post, pre=pre,
                                 segment_tokens=seg)
    # At most 128 rows in a row, then at most 8 x 64 CTAs of a segment.
    _check(t, got, post, pre, 0.7, 1e-6, seg, chain=128 + 64 + 8)
    assert lg.get_last_device_error() == lg.LG_OK


def test_column_sums_past_32_bit_offsets():
    """305,000 x 7168: about 2,061 rows on each of 148 clusters, all of them different."""
    M, D = 305_000, 7168
    t = _inputs(8, D, 1, torch.bfloat16, seed=1)
    t["dh"] = None
    for k in ("h", "b", "dn"):
        t[k] = torch.empty(M, D, dtype=torch.bfloat16, device=DEV)
        for i in range(0, M, 50_000):
            n = min(50_000, M - i)
            t[k][i:i + n] = torch.randn(n, D, generator=torch.Generator(device=DEV).manual_seed(i + len(k)), device=DEV)
    got = lg.block_norm_backward(t["dn"], None, t["h"], t["b"], t["gate"], t["scale"])
    _check(t, got, "rms", "rms", 1.0, 1e-6, M, chain=2200 + 32 + 8)
    del t, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("post", ["rms", "layer"])
@pytest.mark.parametrize("D", [512, 7168])
def test_db_against_differences_of_the_kernel(post, D):
    """db . v against central differences of the kernel's own h', through the norm.

    b and b +- v / 32 are bf16 numbers (b in sixteenths below 4).  The formula's own difference quotient in FP64
    gives the truncation; an FP32 h' is off by 2^-16 of gate |u| and by its rounding, which the quotient turns into
    2^5 times as much: four deviations of their sum as independent errors; db itself is rounded to bf16.  v = sign(db) makes every value count, and
    along v = sign(b) a projection left out would show."""
    M, seg = 6, 3
    g = torch.Generator().manual_seed(D)
    b = (torch.randn(M, D, generator=g).clamp(-3.5, 3.5) * 16).round() / 16
    h, dho, gate = (torch.randn(n, D, generator=g).to(DEV) for n in (M, M, 2))
    b = b.to(DEV)
    _, db, _, _, _ = lg.block_norm_backward(None, dho, h, b.to(torch.bfloat16), gate, post=post, pre=None,
                                            segment_tokens=seg)
    gate_rows = gate.double().repeat_interleave(seg, 0)
    u, r, _ = _norm(b.double(), post, 1e-6)
    exact = _norm_gradient(gate_rows * dho.double(), u, r, post)
    size = float(exact.abs().sum())

    def loss(v):
        out, _, _ = lg.block_norm(h, v.to(torch.bfloat16), gate, post=post, pre=None, segment_tokens=seg)
        return float((out.double() * dho.double()).sum())

    def formula(v):
        return float((gate_rows * _norm(v.double(), post, 1e-6)[0] * dho.double()).sum())

    noise = 2.0 ** 5 * FP * float(((gate_rows * u).abs() * dho.double().abs()).square().sum().sqrt()) * 4
    noise += 2.0 ** 5 * 2.0 ** -24 * float((dho.double() * (h.double().abs() + 4)).square().sum().sqrt()) * 4
    for v in (torch.sign(exact).float(), torch.sign(b)):
        step = v / 32
        num = (loss(b + step) - loss(b - step)) * 16
        truncation = abs((formula(b + step) - formula(b - step)) * 16 - float((exact * v).sum()))
        got = float((db.double() * v.double()).sum())
        assert abs(num - got) <= truncation + noise + 2.0 ** -8 * size, (num, got, truncation, noise, size)
