"""Calls on a side stream: the outputs that a call makes come from that stream's memory, so that
work which the current stream still has queued on memory it has freed does not reach them."""
import pytest
import torch

import gated_delta_rule_74_b200 as kda
import kda_inputs as ki

pytestmark = pytest.mark.gpu


def _dev(x):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}


def _prefill(seed):
    return _dev(ki.make_prefill(ki.PrefillSpec("side", B=2, T=200, H=2, dk=128, dv=128, dtype="bf16",
                                               decay="alog", seed=seed, h0=True)))


def _tokens():
    d = ki.make_decode(ki.DecodeSpec("side", N=40, H=4, dk=128, dv=128, steps=3, dtype="bf16",
                                     decay="alog", seed=7))
    t = {n: d[n].transpose(0, 1).contiguous().cuda() for n in ("q", "k", "v", "g", "beta")}
    return t, d["S0"].cuda()


def _fwd(stream):
    x = _prefill(3)
    return lambda: kda.kda_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], h0=x["h0"], stream=stream)


def _fused(stream):
    x = _dev(ki.make_fused_prefill(ki.PrefillSpec("side", B=1, T=150, H=2, dk=128, dv=128, dtype="bf16",
                                                  decay="alog", seed=4, h0=True)))
    return lambda: kda.kda_chunk_fwd_fused(x["q_raw"], x["k_raw"], x["v"], x["g"], x["beta"],
                                           conv_q=x["conv_q"], conv_k=x["conv_k"], gate=x["gate"],
                                           h0=x["h0"], stream=stream)


def _bwd(stream):
    x = _prefill(5)
    dout, dhT = torch.randn_like(x["v"]), torch.randn_like(x["h0"])
    return lambda: tuple(kda.kda_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], dout, h0=x["h0"],
                                           dhT=dhT, stream=stream).values())


def _step(stream):
    t, S0 = _tokens()
    x = [t[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")]
    S = S0.clone()
    return lambda: (kda.kda_decode_step(*x, S, stream=stream),)


def _multi(fn):
    def make(stream):
        t, S0 = _tokens()
        S = S0.clone()
        return lambda: (fn(t["q"], t["k"], t["v"], t["g"], t["beta"], S, stream=stream),)
    return make


CALLS = {"chunk_fwd": _fwd, "chunk_fwd_fused": _fused, "chunk_bwd": _bwd, "decode_step": _step,
         "decode_tokens": _multi(kda.kda_decode_tokens), "decode_chunk": _multi(kda.kda_decode_chunk)}


@pytest.mark.parametrize("name", CALLS)
def test_outputs_on_a_side_stream_are_that_streams(name):
    torch.manual_seed(11)
    want = [t.clone() for t in CALLS[name](None)()]
    s = torch.cuda.Stream()
    torch.manual_seed(11)
    call = CALLS[name](s)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty_like(t) for t in want]
    places = {t.data_ptr() for t in old}
    torch.cuda._sleep(200_000_000)
    for t in old:
        t.fill_(7)
    del old, t
    got = call()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert a.data_ptr() not in places
        if name != "chunk_bwd":
            assert torch.equal(a, b)
        else:
            # dg and dbeta add up to 16 parts a value in shared memory in any order (two calls on one
            # stream differ, too): two orders are 2 * 16 * 2^-24 of the parts' magnitudes apart, which
            # are below 128 times the largest sum
            assert not bool(((a - b).abs() > 2.0 ** -12 * b.abs().max()).any())
