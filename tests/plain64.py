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


def cached_values(layer):
    """The rows of a layer's caches as float64 values, [B][Hkv][cap][D]."""
    got = []
    for name in ("k", "v"):
        x, s = layer.logical(name + "_cache"), layer.logical(name + "_scale")
        x = x.double().cpu()
        got.append(x if s is None else x * s.double().cpu().unsqueeze(-1))
    return got
