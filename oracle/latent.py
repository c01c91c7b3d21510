"""Float64 references of the latent-cache operators and of the draft verification,
written token by token from their definitions (include/kda.h).  CPU, for tests."""
from __future__ import annotations

import math

import torch


def sequences(N, L, T, cu):
    """(first token, count) of each sequence: uniform L, or cu_seqlens over T tokens."""
    if cu is None:
        return [(n * L, L) for n in range(N)]
    cu = [min(max(int(c), 0), T) for c in cu]
    return [(cu[n], max(cu[n + 1] - cu[n], 0)) for n in range(N)]


def cached(cache, table, n, length):
    """The first `length` rows of sequence n, in order."""
    page = cache.shape[1]
    return torch.stack([cache[int(table[n, j // page]), j % page] for j in range(length)]) \
        if length else cache[0, :0]


def attend(q, cache, table, lens, rank, scale, cu=None):
    """out, lse of every row, and per row what bounds its error: sum_j p_j |c_j| per column
    and the largest scale * sum |q| |c_j|.  Rows of no sequence are None (NaN here)."""
    B, T, H, D = q.shape
    rows = q.double().reshape(B * T, H, D)
    out = torch.full((B * T, H, rank), math.nan, dtype=torch.float64)
    mag = torch.zeros((B * T, H, rank), dtype=torch.float64)
    lse = torch.full((B * T, H), math.nan, dtype=torch.float64)
    size = torch.zeros((B * T, H), dtype=torch.float64)
    for n, (first, cnt) in enumerate(sequences(len(lens), T, B * T, cu)):
        length = min(int(lens[n]), table.shape[1] * cache.shape[1])
        c = cached(cache, table, n, length).double()
        for i in range(cnt):
            sees = length - cnt + i + 1
            if sees <= 0:
                out[first + i], lse[first + i] = 0.0, -math.inf
                continue
            x, k = rows[first + i], c[:sees]
            s = scale * (x @ k.T)
            lse[first + i] = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            out[first + i] = p @ k[:, :rank]
            mag[first + i] = p @ k[:, :rank].abs()
            size[first + i] = scale * (x.abs() @ k.abs().T).amax(-1)
    sh = (B, T, H)
    return out.reshape(*sh, rank), lse.reshape(sh), mag.reshape(*sh, rank), size.reshape(sh)


def turn(x, pos, inv_freq, interleaved):
    """x [.., rope] at position pos."""
    if inv_freq is None:
        return x
    a = pos * inv_freq.double()
    c, s = torch.cos(a), torch.sin(a)
    y = torch.empty_like(x)
    half = x.shape[-1] // 2
    u, v = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, half), slice(half, None))
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., u] * s + x[..., v] * c
    return y


def append(kv, cache, table, lens, rank, cu=None, norm_weight=None, eps=1e-6, inv_freq=None,
           interleaved=False, q_pe=None, q_pe_out=None):
    """The cache (float64 copy) after the call, and q_pe_out; rows of no sequence keep
    q_pe_out's values."""
    B, T, D = kv.shape
    cache = cache.double().clone()
    page = cache.shape[1]
    x = kv.double().reshape(B * T, D)
    q_out = None
    if q_pe is not None:
        qi = q_pe.double().reshape(B * T, q_pe.shape[2], D - rank)
        q_out = q_pe_out.double().clone().reshape(qi.shape)
    for n, (first, cnt) in enumerate(sequences(len(lens), T, B * T, cu)):
        for i in range(cnt):
            pos = int(lens[n]) - cnt + i
            y = x[first + i].clone()
            if norm_weight is not None:
                y[:rank] = y[:rank] / torch.sqrt(y[:rank].square().mean() + eps) * norm_weight.double()
            y[rank:] = turn(y[rank:], pos, inv_freq, interleaved)
            if q_out is not None:
                q_out[first + i] = turn(qi[first + i], pos, inv_freq, interleaved)
            if 0 <= pos < table.shape[1] * page and 0 <= int(table[n, pos // page]) < cache.shape[0]:
                cache[int(table[n, pos // page]), pos % page] = y
    return cache, None if q_out is None else q_out.reshape(q_pe.shape)


def verify(target, draft, tokens, uniforms, draft_lens=None):
    N, L1, V = target.shape
    out = torch.full((N, L1), -1, dtype=torch.int32)
    acc = torch.zeros(N, dtype=torch.int32)
    for n in range(N):
        Ln = L1 - 1 if draft_lens is None else min(max(int(draft_lens[n]), 0), L1 - 1)
        a = 0
        while a < Ln:
            x = int(tokens[n, a])
            if not 0 <= x < V:
                break
            qx = 1.0 if draft is None else float(draft[n, a, x])
            if not float(uniforms[n, a]) * qx < float(target[n, a, x]):
                break
            out[n, a] = x
            a += 1
        w = target[n, a].double().clone()
        if a < Ln:
            x = int(tokens[n, a])
            if draft is not None:
                w -= draft[n, a].double()
            elif 0 <= x < V:
                w[x] = 0.0
        w = torch.where(w > 0, w, torch.zeros_like(w))
        cum = torch.cumsum(w, 0)
        if float(cum[-1]) > 0:
            over = torch.nonzero((cum > float(uniforms[n, L1 - 1]) * float(cum[-1])) & (w > 0))
            out[n, a] = int(over[0]) if len(over) else int(torch.nonzero(w > 0)[-1])
        elif a < Ln and 0 <= int(tokens[n, a]) < V:
            out[n, a] = int(tokens[n, a])
        acc[n] = a
    return out, acc
