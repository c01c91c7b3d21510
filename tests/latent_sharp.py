"""Sharper checks of the latent attention than worst-case bounds an element: the error's root mean
square, and inputs whose exact result shows a single token lost, doubled or misplaced.

Root mean square.  U is half a step of the type.  An fp32 sum of D products of random signs has
partial sums of |q * c| (the norm of the products) and is off by at most 2^-24 of them a step, in
random directions: sqrt(D) 2^-24 scale |q * c|.  The scaled score takes two roundings, 2^-23 |s|,
and the exponential 2^-22.  Call the sum e, with the largest |q * c| and |s|: the rms of a weight's
relative error.  Numerator and denominator of the output have it, the sum over n tokens adds
sqrt(n) 2^-24, the output's rounding U / sqrt(3) (uniform), a weight's rounding to bf16 as much:
    f32:   rms(out - ref) <= (2 e + sqrt(n) 2^-24 + U) rms(ref)
    bf16:  rms(out - ref) <= (2 e + sqrt(n) 2^-24 + sqrt(2 / 3) U 1.2) rms(ref)
(1.2: the spread of an estimate from the few hundred weights that count in the smallest case).
On tensor cores the D products are added 16 at a time and may be cut off, always downwards: e gets
D / 16 2^-23 scale |q * c|.  The log-sum is a mean of the scores' errors over the weights: four
times e at most, and 2^-22 (|lse| + 4) for its logarithms and sums.

Counting: with q = 0 every weight is equal and exact, and token j's only value is a one in column
j % rank, so that out[k] is the share of tokens with j % rank == k and lse the log of their number.

Finding: cached rows of +-1, q a large multiple of one of them: the result is that row."""
import math

import torch

from oracle import latent as ref


def rms_close(x, out, lse):
    q, scale = x["q"], x["scale"]
    B, T, H, D = q.shape
    o, z, _, _ = ref.attend(q, x["cache"], x["table"], x["lens"], x["rank"], scale, x["cu"])
    some = ~torch.isnan(z) & (z > -math.inf)
    rows = q.double().reshape(B * T, H, D)
    norm = big = 0.0
    for n, (first, cnt) in enumerate(ref.sequences(len(x["lens"]), T, B * T, x["cu"])):
        c = ref.cached(x["cache"], x["table"], n, int(x["lens"][n])).double()
        if cnt and len(c):
            r = rows[first:first + cnt].reshape(-1, D)
            norm = max(norm, scale * float((r.square() @ c.square().T).max().sqrt()))
            big = max(big, scale * float((r @ c.T).abs().max()))
    half = q.dtype == torch.bfloat16
    u = torch.finfo(q.dtype).eps / 2
    steps = math.sqrt(D) * 2.0 ** -24 + (D / 16 * 2.0 ** -23 if half else 0.0)
    e = steps * norm + 2.0 ** -23 * big + 2.0 ** -22
    tol = 2 * e + math.sqrt(int(x["lens"].max())) * 2.0 ** -24 + (math.sqrt(2 / 3) * 1.2 * u if half else u)
    out, lse = out.double().cpu(), lse.double().cpu()
    off = float((out - o)[some].square().mean().sqrt() / o[some].square().mean().sqrt())
    assert off <= tol, (off, tol)
    bad = (lse - z).abs() > 4 * e + 2.0 ** -22 * (z.abs() + 4)
    assert not bool(bad[some].any()), ((lse - z).abs()[some].max(), e)
    return off / tol


def counting(x):
    """x with q = 0 and a one in column (position in its sequence) % rank of every cached row (pages
    shared by sequences hold the same positions of each)."""
    page, rank = x["cache"].shape[1], x["rank"]
    cache = torch.zeros_like(x["cache"])
    for n, t in enumerate(x["lens"].tolist()):
        j = torch.arange(t)
        cache[x["table"][n, j // page].long(), j % page, j % rank] = 1.0
    return dict(x, q=torch.zeros_like(x["q"]), cache=cache)


def counts_right(x, out, lse):
    """out is off by its rounding and, where results are joined, by weights good to 2^-20; the log-sum
    by 2^-22 of the logarithms (a CTA's, the joined one, their differences' exponential)."""
    rank, T = x["rank"], x["q"].shape[1]
    u = torch.finfo(x["q"].dtype).eps / 2
    out, lse = out.double().cpu().reshape(-1, *out.shape[2:]), lse.double().cpu().reshape(-1, lse.shape[2])
    for n, (first, cnt) in enumerate(ref.sequences(len(x["lens"]), T, out.shape[0], x["cu"])):
        for i in range(cnt):
            sees = int(x["lens"][n]) - cnt + i + 1
            if sees <= 0:
                assert bool((out[first + i] == 0).all()) and bool((lse[first + i] == -math.inf).all())
                continue
            want = torch.bincount(torch.arange(sees) % rank, minlength=rank).double() / sees
            assert not bool(((out[first + i] - want).abs() > (u + 2.0 ** -20) * want).any()), (n, i)
            log = math.log(sees)
            assert not bool(((lse[first + i] - log).abs() > 2.0 ** -22 * (2 * log + 8)).any()), (n, i)


def finding(x, seed=0):
    """x with cached rows of +-1 (position values zero), all sequences over the first one's pages, and
    each row's q a multiple of a token that it sees: the tokens in turn over sequences and heads,
    the last token first.  Returns x and the tokens [N, H] (one new token a sequence)."""
    g = torch.Generator().manual_seed(seed)
    rank, page = x["rank"], x["cache"].shape[1]
    N, _, H, _ = x["q"].shape
    t = int(x["lens"][0])
    cache, q = torch.zeros_like(x["cache"]), torch.zeros_like(x["q"])
    sign = torch.randint(0, 2, (t, rank), generator=g).float() * 2 - 1
    j = torch.arange(t)
    cache[x["table"][0, j // page].long(), j % page, :rank] = sign.to(cache.dtype)
    at = t - 1 - torch.arange(N * H) % t
    q[..., :rank] = 4 * sign[at].reshape(N, 1, H, rank).to(q.dtype)
    # another token's product is below rank / 2 (six standard deviations at rank 128): its weight
    # below e^-64
    y = dict(x, cache=cache, q=q, table=x["table"][:1].repeat(N, 1),
             lens=torch.full_like(x["lens"], t), scale=32.0 / rank)
    return y, sign[at].reshape(N, H, rank)


def found(x, want, out):
    """The row itself, off by the rounding of its one weight and of the output."""
    u = torch.finfo(x["q"].dtype).eps / 2
    tol = 2 * u if x["q"].dtype == torch.bfloat16 else 2.0 ** -20
    bad = (out[:, 0].double().cpu() - want.double()).abs() > tol
    assert not bool(bad.any()), bad.any(-1).nonzero()[:5]
