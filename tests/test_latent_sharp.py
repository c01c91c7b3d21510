"""The checks of latent_sharp.py find what they are for: mistakes planted in an fp32 form of the
operator, on the CPU, are refused, and the form without one passes."""
import math

import pytest
import torch

from latent_sharp import counting, counts_right, finding, found, rms_close
from oracle import latent as ref
from test_gpu_latent import make


def tf32(t):
    """Rounded to 11 significant bits."""
    i = t.float().contiguous().view(torch.int32)
    return ((i + 0x1000) & ~0x1fff).view(torch.float32)


def form(x, inputs=lambda t: t, weights=lambda t: t, share=None, edge=0):
    """out, lse in fp32, rounded to the inputs' type; share: {token: its factor in both sums};
    edge: tokens that each row sees beyond its own."""
    q, rank = x["q"], x["rank"]
    B, T, H, D = q.shape
    out = torch.zeros((B * T, H, rank))
    lse = torch.full((B * T, H), -math.inf)
    rows = inputs(q.float()).reshape(B * T, H, D)
    for n, (first, cnt) in enumerate(ref.sequences(len(x["lens"]), T, B * T, x["cu"])):
        t = int(x["lens"][n])
        c = inputs(ref.cached(x["cache"], x["table"], n, t).float())
        times = torch.ones(t)
        for j, f in (share or {}).items():
            if j < t:
                times[j] = f
        for i in range(cnt):
            sees = min(t - cnt + i + 1 + edge, t)
            if sees <= 0:
                continue
            s = x["scale"] * (rows[first + i] @ c[:sees].T)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m) * times[:sees]
            total = p.sum(-1)
            out[first + i] = (weights(p) @ c[:sees, :rank]) / total[:, None]
            lse[first + i] = torch.log(total) + m[:, 0]
    return out.reshape(B, T, H, rank).to(q.dtype), lse.reshape(B, T, H)


SHAPES = [("f32", [130, 5, 64], 3, 12, 256, 64, 16), ("f32", [300, 200], 1, 16, 512, 64, 64),
          ("bf16", [300, 65], 2, 12, 512, 64, 64)]


@pytest.mark.parametrize("shape", SHAPES)
def test_rms_passes_the_fp32_form(shape):
    x = make(*shape)
    w = (lambda p: p.bfloat16().float()) if shape[0] == "bf16" else (lambda p: p)
    assert rms_close(x, *form(x, weights=w)) <= 1


@pytest.mark.parametrize("shape", SHAPES[:2])
@pytest.mark.parametrize("fault", [dict(inputs=tf32), dict(inputs=lambda t: t.bfloat16().float()),
                                   dict(weights=lambda p: p.bfloat16().float()), dict(weights=tf32),
                                   dict(share={40: 0}), dict(share={63: 2.0})])
def test_rms_refuses_fewer_bits_and_lost_tokens(shape, fault):
    x = make(*shape)
    with pytest.raises(AssertionError):
        rms_close(x, *form(x, **fault))


@pytest.mark.parametrize("dtype,lens,L", [("bf16", [1000, 64, 1, 0], 1), ("f32", [1000, 65], 1),
                                          ("bf16", [9000], 1), ("bf16", [40, 3], 5)])
def test_counting_refuses_a_lost_doubled_or_shifted_token(dtype, lens, L):
    x = counting(make(dtype, lens, L, 3, 512, 64, 64))
    counts_right(x, *form(x))
    for j in (0, lens[0] // 2, lens[0] - L):
        for f in (0.0, 2.0):
            with pytest.raises(AssertionError):
                counts_right(x, *form(x, share={j: f}))
    if L > 1:
        with pytest.raises(AssertionError):
            counts_right(x, *form(x, edge=1))
    y = dict(x, cache=x["cache"].roll(1, -1))            # a token in the place of its neighbour
    with pytest.raises(AssertionError):
        counts_right(x, *form(y))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_finding_refuses_an_unseen_token(dtype):
    x, want = finding(make(dtype, [100] * 9, 1, 12, 128, 64, 16))
    found(x, want, form(x)[0])
    for j in (0, 47, 48, 99):
        with pytest.raises(AssertionError):
            found(x, want, form(x, share={j: 0.0})[0])
