"""Sliding-window attention with sinks from its definition in 64 bits, with the
bound that fp32 arithmetic over exact bf16 products allows (torch, any device)."""
from __future__ import annotations

import math

import torch


def visible(length, rows, window, sinks, device):
    """[rows][length] truth values: row r sits at length - rows + r."""
    at = torch.arange(length - rows, length, device=device)[:, None]
    pos = torch.arange(length, device=device)[None, :]
    return (pos <= at) & ((at - pos < window) | (pos < sinks))


def attend(q, k, v, window, sinks, scale):
    """q [W][Hq][d], k and v [n][Hkv][d] (one stream, the linear cache; bf16).
    Returns the output [W][Hq][d] in 64 bits and, for every element, how far an
    fp32 evaluation may be off:

      scores   d products, exact in fp32, added with an error of at most
               2^-23 of the sum of their magnitudes each: ds = d 2^-23 scale
               max |q|.|k| (and 2^-22 |s| for the scale and log2 e);
      weights  exp2 to 2^-21, kept as two bf16 parts to 2^-18;
      sums     at most n additions, of 2^-23 each;
      so every output is within sum w |v| (e^(2 ds) - 1 + 2^-17 + n 2^-22).
    """
    W, Hq, d = q.shape
    n, Hkv, _ = k.shape
    G = Hq // Hkv
    sees = visible(n, W, window, sinks, q.device)
    cols = sees.any(0).nonzero()[:, 0]         # invisible slots may hold anything
    sees = sees[:, cols][:, None, None, :]
    q = q.double().view(W, Hkv, G, d)
    k, v = k[cols].double(), v[cols].double()
    s = torch.einsum("whgd,nhd->whgn", q, k) * scale
    s = s.masked_fill(~sees, -math.inf)
    w = torch.softmax(s, -1)
    out = torch.einsum("whgn,nhd->whgd", w, v)
    mags = torch.einsum("whgd,nhd->whgn", q.abs(), k.abs()) * abs(scale)
    mags = mags.masked_fill(~sees, 0.0).amax(-1)
    ds = mags * (d * 2.0 ** -23 + 2.0 ** -22)
    rel = torch.expm1(2 * ds) + 2.0 ** -17 + cols.numel() * 2.0 ** -22
    bound = torch.einsum("whgn,nhd->whgd", w, v.abs()) * rel[..., None]
    return out.reshape(W, Hq, d), bound.reshape(W, Hq, d)
