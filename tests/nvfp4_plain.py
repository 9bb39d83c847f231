"""Plain 64-bit forms of the NVFP4 cache, the attention over it and the
matrix-vector product, written from their definitions with elementary torch
operations, for the GPU tests (any device)."""
import math

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def sf_values(sf):
    """e4m3 bytes -> 64-bit values (0x7F and 0xFF are NaN)."""
    return sf.view(torch.float8_e4m3fn).double()


def decode(codes, sf, gs):
    """codes [..., n/2], sf [..., n/16] -> code * sf * gs [..., n] in 64 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    return table[c] * sf_values(sf).repeat_interleave(16, -1) * float(gs)


def sf_rows(sf4, capacity):
    """Cache factors [ceil(capacity/4), Hkv, hd/16, 4] -> [capacity, Hkv, hd/16]."""
    return sf4.permute(0, 3, 1, 2).flatten(0, 1)[:capacity]


def sf_pack(sf):
    """[capacity, Hkv, hd/16] -> the cache's layout; the factors of slots that pad the last quad are NaN."""
    pad = -sf.shape[0] % 4
    sf = torch.cat((sf, torch.full((pad,) + sf.shape[1:], 0x7F, dtype=torch.uint8, device=sf.device)))
    return sf.unflatten(0, (-1, 4)).permute(0, 2, 3, 1).contiguous()


def quantise(y, gs):
    """32-bit y [..., n] -> (codes [..., n/2], sf [..., n/16]) by the library's decisions: 32-bit products with
    rounded reciprocals; a block that holds a NaN or an infinity gets factor 0x7F and zero codes."""
    gs = torch.tensor(float(gs), dtype=torch.float32, device=y.device)
    b = y.float().unflatten(-1, (-1, 16))
    fine = torch.isfinite(b).all(-1)
    b = torch.where(fine.unsqueeze(-1), b, 0.0)
    sf = (b.abs().amax(-1) * (1.0 / (6.0 * gs))).clamp(max=448.0).to(torch.float8_e4m3fn)
    eff = sf.float() * gs
    r = torch.where(eff > 0, 1.0 / eff, 0.0)
    v = b * r.unsqueeze(-1)
    a = v.abs()
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=y.device)
    ties_up = torch.tensor([False, True, False, True, False, True, False], device=y.device)
    code = ((a.unsqueeze(-1) > edges) | ((a.unsqueeze(-1) == edges) & ties_up)).sum(-1).to(torch.uint8)
    code = (code + 8 * torch.signbit(v).to(torch.uint8)).flatten(-2)
    sf = torch.where(fine, sf.view(torch.uint8), torch.tensor(0x7F, dtype=torch.uint8, device=y.device))
    code = torch.where(fine.repeat_interleave(16, -1), code, torch.zeros_like(code))
    return code[..., 0::2] | (code[..., 1::2] << 4), sf


def norm_rope(x, w, cos, sin, eps):
    """Per-head RMSNorm (w None: none) and rotate-half RoPE of x [M, H, hd] in 64 bits; cos, sin [M, hd/2]."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32))) * \
            w.double()
    a, b = x.chunk(2, -1)
    c, s = cos.double().unsqueeze(1), sin.double().unsqueeze(1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def attention(q, k, v, spans, slot_of, scale, head_of):
    """out [M, Hq, hd], and per (token, head) the largest |v| and the largest sum |q||k| it sees (for bounds).
    k, v 64-bit [capacity, Hkv, hd]; spans[i] = (lo, hi); slot_of(i, positions) -> slots, -1 left out."""
    M, Hq, hd = q.shape
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    vmax = torch.zeros((M, Hq), dtype=torch.float64, device=q.device)
    smax = torch.zeros((M, Hq), dtype=torch.float64, device=q.device)
    qd = q.double()
    heads = torch.tensor([head_of(h) for h in range(Hq)], device=q.device)
    for i, (lo, hi) in enumerate(spans):
        if hi <= lo:
            continue
        pos = torch.arange(lo, hi, device=q.device)
        slots = slot_of(i, pos)
        slots = slots[slots >= 0]
        if slots.numel() == 0:
            continue
        ki, vi = k[slots][:, heads], v[slots][:, heads]           # [n, Hq, hd]
        s = torch.einsum("hd,nhd->hn", qd[i], ki) * scale
        out[i] = torch.einsum("hn,nhd->hd", torch.softmax(s, -1), vi)
        vmax[i] = vi.abs().amax((0, 2))
        smax[i] = torch.einsum("hd,nhd->hn", qd[i].abs(), ki.abs()).amax(-1) * abs(scale)
    return out, vmax, smax


def attention_bound(ref, vmax, smax, n_keys, hd, dt):
    """Bound on |out - ref|.  A weight's relative error d is at most half a binary16 step (2^-11), the error of its
    exponent (the score's 32-bit sum of hd products, 2^-23 each as the tensor core may cut instead of round, and 2
    roundings of the scaled argument) and the exponential's 2^-22; numerator and denominator use the same rounded
    weights, so their quotient moves by at most 2 d max|v|.  The output's sums add n_keys roundings of 2^-23 (twice:
    numerator and denominator), tiny weights n_keys 2^-36 max|v|, the result half a step of its type."""
    d = 2.0 ** -11 + 2.0 ** -22 + (hd + 2) * 2.0 ** -23 * smax
    n = n_keys * (2.0 ** -22 + 2.0 ** -36)
    half_step = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * half_step
    return (2 * d + n).unsqueeze(-1) * vmax.unsqueeze(-1) + half_step * 1.01 * ref.abs() + tiny


def sf_swizzle(sf):
    n, c = sf.shape
    pad = torch.zeros((math.ceil(n / 128) * 128, math.ceil(c / 4) * 4), dtype=torch.uint8, device=sf.device)
    pad[:n, :c] = sf
    return pad.view(-1, 4, 32, pad.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().flatten()


def matvec_bound(x, w, ref, dt, group=128):
    """Bound on |y - ref| (bias included in ref): products are exact, each of K sums and the group factors err by
    2^-23 of the running magnitude; bf16 rows are carried to 2^-39 of a group's largest magnitude; half a step of the
    result."""
    K = x.shape[1]
    mag = x.abs() @ w.abs().t()
    pad = torch.nn.functional.pad(x.abs(), (0, -K % group)).unflatten(-1, (-1, group))
    top = pad.amax(-1, keepdim=True).expand_as(pad).flatten(-2)[:, :K]
    half_step = torch.finfo(dt).eps / 2
    return (K + 8) * 2.0 ** -23 * mag + 2.0 ** -39 * (top @ w.abs().t()) + 1.01 * half_step * ref.abs() + \
        torch.finfo(dt).smallest_normal * half_step


def attention_norm_bound(smax, hd, depth, dt):
    """Bound on |out - ref| / |ref| as norms over a head's outputs, for values v that are independent of the scores
    (zero-mean, one variance).  With weights p fixed, ref = sum p v / sum p has the expected square sum p^2 / (sum p)^2
    and an error sum d p v / sum p of relative weight errors |d| <= D has at most D^2 times that, so their norms'
    ratio is D, and the common error of the denominator adds another D.  D is half a binary16 step, the exponential's
    2^-22, the score's (hd + 2) 2^-23 smax, and 2^-23 for each of the `depth` additions that follow one another in a
    sum.  The result adds half a step of its type.  Both norms are of hd numbers or more: they are off their expectations by
    1 / sqrt(2 hd), far inside the factor of 2."""
    d = 2.0 ** -11 + 2.0 ** -22 + (hd + 2) * 2.0 ** -23 * smax + depth * 2.0 ** -23
    return 2 * (2 * d + torch.finfo(dt).eps / 2)
