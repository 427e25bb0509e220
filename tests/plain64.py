"""Attention over a cache in 64 bits, by its definition (torch on the CPU).

The operators' tests take the rows that a cache holds as values and compare the
library's outputs with this. It shares no code with the library or the oracle.
"""
import math

import torch


def visible(pos: int, window: int, first_tokens: int) -> list[int]:
    """Positions that a token at `pos` sees: all up to its own, or with a window
    the first tokens and the window's."""
    if window <= 0:
        return list(range(pos + 1))
    return [j for j in range(pos + 1) if j > pos - window or j < first_tokens]


def attend(q, keys, values, lens, window=0, first_tokens=0, softcap=0.0, sink=None, scale=None):
    """q [B][T][Hq][D] (rotated); keys, values [B][Hkv][cap][D]; lens [B]: tokens
    cached before the T new ones, which sit at lens[b] + t. Returns [B][T][Hq][D]
    in float64."""
    q, keys, values = q.double().cpu(), keys.double().cpu(), values.double().cpu()
    B, T, Hq, D = q.shape
    Hkv = keys.shape[1]
    G = Hq // Hkv
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64)
    for b in range(B):
        for t in range(T):
            use = torch.tensor(visible(int(lens[b]) + t, window, first_tokens))
            for h in range(Hkv):
                z = q[b, t, h * G:(h + 1) * G] @ keys[b, h, use].T * (scale or 1.0 / math.sqrt(D))
                if softcap:
                    z = softcap * torch.tanh(z / softcap)
                lse = torch.logsumexp(z, -1)
                if sink is not None:
                    lse = torch.logaddexp(lse, sink[h * G:(h + 1) * G].double().cpu())
                out[b, t, h * G:(h + 1) * G] = torch.exp(z - lse.unsqueeze(-1)) @ values[b, h, use]
    return out


def q4_quantize(x):
    """4-bit codes in [-7, 7] and fp16 scales (one per 32 dims) of rows x [..., D], by
    the storage rule: the scale's division and roundings are single IEEE
    operations of fp32, so are the codes'."""
    g = x.float().cpu().unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / 7.0).to(torch.bfloat16).float().clamp(max=2720.0).to(torch.float16)
    f = s.float().unsqueeze(-1)
    codes = torch.where(f > 0, (g / torch.where(f > 0, f, torch.ones_like(f))).round().clamp(-7, 7), torch.zeros_like(g))
    return codes.flatten(-2).to(torch.int8), s


def q4_nibbles(codes):
    """Stored bytes [..., D / 2] as codes in [-8, 7], [..., D]."""
    c = codes.cpu()
    return torch.stack([(c & 15).to(torch.int8) - 8, (c >> 4).to(torch.int8) - 8], -1).flatten(-2)


def q4_values(codes, scales):
    """Stored bytes and scales as float64 values."""
    return q4_nibbles(codes).double() * scales.double().cpu().repeat_interleave(32, -1)


def rope_rows(x, lens, theta, rotary_dim=0, interleaved=False):
    """Rows x [B][T][H][D] turned by their positions lens[b] + t, in float64 (no scaling)."""
    x = x.double().cpu().clone()
    B, T, _, D = x.shape
    R = rotary_dim or D
    f = theta ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    pos = torch.as_tensor(lens, dtype=torch.float64).reshape(B, 1) + torch.arange(T, dtype=torch.float64)
    ang = (pos.unsqueeze(-1) * f).unsqueeze(2)
    ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    ib = ia + 1 if interleaved else ia + R // 2
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia] = a * ang.cos() - b * ang.sin()
    x[..., ib] = a * ang.sin() + b * ang.cos()
    return x


def rms_norm(x, w, eps, offset=0.0):
    x = x.double().cpu()
    return x * (w.double().cpu() + offset) / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)


def cached_values(layer):
    """The rows of a layer's caches as float64 values, [B][Hkv][cap][D]."""
    got = []
    for name in ("k", "v"):
        x, s = layer.logical(name + "_cache"), layer.logical(name + "_scale")
        if x.dtype == torch.uint8:
            got.append(q4_values(x, s))
            continue
        x = x.double().cpu()
        got.append(x if s is None else x * s.double().cpu().unsqueeze(-1))
    return got
