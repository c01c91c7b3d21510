"""Packed latent attention calls whose sequences are unlike: against the float64 reference of
oracle/latent.py, and against the same work given in another form."""
import statistics

import pytest
import torch

import gated_delta_rule_74_b200 as kda
from latent_sharp import counting, counts_right
from test_gpu_latent import call, close, make

pytestmark = pytest.mark.gpu


def device_us(fn, calls=6):
    """Median time of a call on the device, from replays of a graph of several."""
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(calls):
            fn()
    times = []
    for _ in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) / calls * 1e3)
    return statistics.median(times[3:])


@pytest.mark.parametrize("dtype,n,H,rank", [("bf16", 100, 1, 512), ("bf16", 60, 1, 512), ("f32", 40, 2, 128)])
def test_one_token_sequences_packed_as_uniform(dtype, n, H, rank):
    """One new token a sequence, packed or not: the same work (and join, so the same bits). The
    packed call's blocks are one a sequence too, not as many as the rows would fill (which spent
    55 us on the join of 100 sequences behind 500 tokens, for 22; twice the time is refused)."""
    x = make(dtype, [500] * n, 1, H, rank, 64, 64)
    out, lse = call(x)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    q = d["q"].reshape(1, n, H, rank + 64)
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    args = (d["cache"], d["table"], d["lens"])
    kw = dict(rank=rank, scale=x["scale"])
    po, pz = kda.kda_latent_attn(q, *args, cu_seqlens=cu, **kw)
    torch.cuda.synchronize()
    close(x, out, lse)
    assert torch.equal(po.reshape(out.shape), out) and torch.equal(pz.reshape(lse.shape), lse)
    uniform = device_us(lambda: kda.kda_latent_attn(d["q"], *args, **kw))
    packed = device_us(lambda: kda.kda_latent_attn(q, *args, cu_seqlens=cu, **kw))
    assert packed <= 2 * uniform, (packed, uniform)


@pytest.mark.parametrize("dtype,H", [("bf16", 12), ("bf16", 3), ("f32", 4)])
def test_one_long_chunk_among_empty_and_one_token_sequences(dtype, H):
    """Most rows in one sequence, in the middle, at the end and at the start of the batch."""
    for at, others in ((20, 0), (40, 1), (0, 1)):
        new = [others] * 41
        new[at] = 400
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        lens = [90 + 3 * n if c else 0 for n, c in enumerate(new)]
        lens[at] = 450
        x = make(dtype, lens, cu[-1], H, 128, 64, 64, cu=cu, seed=at + others)
        close(x, *call(x))


@pytest.mark.parametrize("slots,new,ctx,H", [(64, [8, 8], 30000, 2), (128, [17], 60000, 1), (128, [5], 30000, 12)])
def test_few_sequences_among_empty_slots(slots, new, ctx, H):
    """Empty slots add little to the time of the few sequences whose blocks many CTAs share (twice is
    refused; counted as if each token could be a sequence's only one, the first took 57 us for 23)."""
    times = []
    for empty in (0, slots - len(new)):
        k = new + [0] * empty
        cu = [0]
        for n in k:
            cu.append(cu[-1] + n)
        x = counting(make("bf16", [ctx if n else 0 for n in k], cu[-1], H, 512, 64, 64, cu=cu))
        counts_right(x, *call(x))
        d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
        times.append(device_us(lambda: kda.kda_latent_attn(
            d["q"], d["cache"], d["table"], d["lens"], rank=512, scale=x["scale"], cu_seqlens=d["cu"])))
    assert times[1] <= 2 * times[0], times
