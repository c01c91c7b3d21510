"""One serving step over drafted tokens as a hybrid model runs it: the latent layer's append
and attention, the KDA layer's multi-token decode, the check of the drafts, the KDA state
rolled to the accepted prefix, and the next step behind it, in one captured graph too."""
import math

import pytest
import torch

import gated_delta_rule_74_b200 as kda
import kda_inputs as ki
from oracle import latent as ref
from test_gpu_latent import append_close, close, make_append

pytestmark = pytest.mark.gpu

N, L, H, RANK, ROPE, PAGE, V = 5, 4, 12, 512, 64, 16, 999


def _inputs(seed=5):
    x = make_append("bf16", [40, 4, 17, 130, 0], L, H, RANK, ROPE, PAGE, True, seed=seed)
    g = torch.Generator().manual_seed(seed)
    x["q"] = torch.randn((N, L, H, RANK + ROPE), generator=g).to(torch.bfloat16)
    x["scale"] = 2 / math.sqrt(RANK + ROPE)
    d = ki.make_decode(ki.DecodeSpec("step", N=N, H=H, dk=128, dv=128, steps=L, dtype="bf16",
                                     decay="alog", seed=seed))
    tok = {n: d[n].transpose(0, 1).contiguous() for n in ("q", "k", "v", "g", "beta")}
    target = torch.softmax(2 * torch.randn((N, L, V), generator=g), -1)      # L - 1 drafts
    draft = torch.softmax(target[:, :L - 1].log() + 0.7 * torch.randn((N, L - 1, V), generator=g), -1)
    ids = torch.multinomial(draft.reshape(-1, V), 1, generator=g).reshape(N, L - 1).to(torch.int32)
    u = torch.rand((N, L), generator=g)
    return x, tok, d["S0"], (target, draft, ids, u)


def _dev(x):
    if isinstance(x, torch.Tensor):
        return x.cuda()
    return {k: _dev(v) for k, v in x.items()} if isinstance(x, dict) else \
        tuple(_dev(v) for v in x) if isinstance(x, tuple) else x


def _step(x, tok, S0, ver, q):
    kda.kda_latent_append(x["kv"], x["cache"], x["table"], x["lens"], rank=RANK, norm_weight=x["w"],
                          inv_freq=x["f"], q_pe=x["qi"], q_pe_out=q[..., RANK:])
    out, lse = kda.kda_latent_attn(q, x["cache"], x["table"], x["lens"], rank=RANK, scale=x["scale"])
    S = S0.clone()
    o = kda.kda_decode_tokens(tok["q"], tok["k"], tok["v"], tok["g"], tok["beta"], S)
    ids, acc = kda.kda_verify_tokens(*ver)
    # the accepted drafts and the token before them stand: the rest gets no decay and no write
    keep = torch.arange(L, device="cuda") <= acc[:, None]
    kept = S0.clone()
    kda.kda_decode_tokens(tok["q"], tok["k"], tok["v"], tok["g"] * keep[..., None, None],
                          tok["beta"] * keep[..., None], kept)
    return out, lse, o, ids, acc, kept


def _check(x, tok, S0, ver, got, cache_after, q_after):
    out, lse, o, ids, acc, kept = got
    append_close(x, cache_after, q_after[..., RANK:], False, q_fill=5.0)
    y = dict(x, cache=cache_after.cpu(), q=q_after.cpu())
    close(y, out, lse)
    ri, ra = ref.verify(*ver)
    assert torch.equal(ids.cpu(), ri) and torch.equal(acc.cpu(), ra)
    for n in range(N):                                    # the prefix alone, from the same state
        S = S0[n:n + 1].cuda().clone()
        m = int(ra[n]) + 1
        kda.kda_decode_tokens(*[tok[k][n:n + 1, :m].contiguous().cuda()
                                for k in ("q", "k", "v", "g", "beta")], S)
        assert torch.equal(S, kept[n:n + 1])


def test_step_over_drafts_eager_and_captured():
    x, tok, S0, ver = _inputs()
    xd, td, Sd, vd = _dev(x), _dev(tok), S0.cuda(), _dev(ver)
    cache0 = xd["cache"].clone()
    q0 = xd["q"].clone()
    got = _step(xd, td, Sd, vd, xd["q"])
    torch.cuda.synchronize()
    _check(x, tok, S0, ver, got, xd["cache"], xd["q"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = _step(xd, td, Sd, vd, xd["q"])
    # other inputs in the same buffers
    x2, tok2, S2, ver2 = _inputs(seed=9)
    x2["cache"], x2["table"] = x["cache"], x["table"]
    xd["cache"].copy_(cache0)
    xd["q"].copy_(x2["q"])
    for n in ("kv", "w", "qi"):
        xd[n].copy_(x2[n])
    for n in td:
        td[n].copy_(tok2[n])
    Sd.copy_(S2)
    for a, b in zip(vd, ver2):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    _check(x2, tok2, S2, ver2, res, xd["cache"], xd["q"])
    assert kda.kda_device_status(reset=False) == kda.KDA_OK


def test_two_steps_over_a_growing_cache():
    """The second step overwrites the fallen drafts' slots: lengths go back to the accepted."""
    x, tok, S0, ver = _inputs(seed=3)
    xd, vd = _dev(x), _dev(ver)
    kda.kda_latent_append(xd["kv"], xd["cache"], xd["table"], xd["lens"], rank=RANK,
                          norm_weight=xd["w"], inv_freq=xd["f"])
    ids, acc = kda.kda_verify_tokens(*vd)
    torch.cuda.synchronize()
    mid = xd["cache"].cpu()
    lens2 = x["lens"] - L + acc.cpu() + 1 + 1             # the accepted prefix and one more token
    lens2 = torch.where(x["lens"] > 0, lens2, x["lens"]).clamp(max=x["table"].shape[1] * PAGE)
    y = dict(x, cache=mid, kv=x["kv"][:, :1].contiguous(), q=x["q"][:, :1].contiguous(), qi=None,
             lens=lens2.to(torch.int32))
    # pages that the growth needs
    for n in range(N):
        need = -(-int(lens2[n]) // PAGE)
        y["table"] = y["table"].clone()
        y["table"][n, :max(need, 1)] = torch.where(y["table"][n, :max(need, 1)] < 0, mid.shape[0] - 1,
                                                   y["table"][n, :max(need, 1)])
    yd = _dev(y)
    kda.kda_latent_append(yd["kv"], yd["cache"], yd["table"], yd["lens"], rank=RANK,
                          norm_weight=yd["w"], inv_freq=yd["f"])
    out, lse = kda.kda_latent_attn(yd["q"], yd["cache"], yd["table"], yd["lens"], rank=RANK,
                                   scale=x["scale"])
    torch.cuda.synchronize()
    append_close(y, yd["cache"], None, False)
    close(dict(y, cache=yd["cache"].cpu()), out, lse)
