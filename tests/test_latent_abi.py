"""Refusals of the latent-cache operators and of the draft verification, on the host:
every call carries an invalid argument, so nothing reaches CUDA."""
import ctypes

import pytest
import torch

import gated_delta_rule_74_b200 as kda

P = 0x10000   # a 16-byte aligned fake address; never dereferenced by these calls


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_74_b200 import build
    build.build()
    return kda.lib()


def _append(L_, kv=P, w=None, f=None, qi=None, qo=None, cache=P, table=P, lens=P, cu=None, N=2,
            Lt=1, H=1, rank=512, rope=64, pages=4, page=64, most=2, ps=64 * 576, rs=576, ks=576,
            qt=64, qh=64, qot=64, qoh=64, eps=1e-6, inter=0, dt=0):
    return L_.kda_latent_append(kv, w, f, qi, qo, cache, table, lens, cu, N, Lt, H, rank, rope,
                                pages, page, most, ps, rs, ks, qt, qh, qot, qoh, eps, inter, dt,
                                None)


def _attn(L_, q=P, cache=P, table=P, lens=P, cu=None, out=P, lse=None, N=2, Lt=1, H=1, rank=512,
          rope=64, pages=4, page=64, most=2, ps=64 * 576, rs=576, scale=0.1, dt=0):
    return L_.kda_latent_attn(q, cache, table, lens, cu, out, lse, N, Lt, H, rank, rope, pages,
                              page, most, ps, rs, scale, dt, None)


SHAPE = [dict(N=0), dict(Lt=-1), dict(H=0), dict(dt=2), dict(pages=0), dict(page=0), dict(most=0),
         dict(rs=575), dict(rs=572), dict(ps=100), dict(ps=-576 * 64), dict(cache=None),
         dict(table=None), dict(lens=None), dict(cache=P + 4), dict(lens=P + 8), dict(cu=P + 4),
         dict(Lt=1 << 30, H=4), dict(N=1 << 25)]


@pytest.mark.parametrize("bad", SHAPE + [dict(q=None), dict(out=None), dict(out=P + 2),
                                         dict(lse=P + 4), dict(scale=0.0),
                                         dict(scale=float("nan")), dict(scale=float("inf"))])
def test_attn_rejects_invalid(L, bad):
    assert _attn(L, **bad) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", SHAPE + [dict(kv=None), dict(kv=P + 8), dict(w=P + 4),
                                         dict(f=P + 4), dict(qi=P), dict(qo=P),
                                         dict(qi=P, qo=P, qt=63), dict(qi=P, qo=P, qoh=0),
                                         dict(qi=P, qo=P, rope=0), dict(ks=572), dict(ks=577),
                                         dict(eps=-1.0), dict(eps=float("nan"))])
def test_append_rejects_invalid(L, bad):
    assert _append(L, **bad) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(rank=64), dict(rank=500), dict(rank=640), dict(rope=32),
                                 dict(rope=128)])
def test_sizes_that_are_not_supported(L, bad):
    assert _attn(L, **bad) == kda.KDA_ERR_UNSUPPORTED
    assert _append(L, **bad) == kda.KDA_ERR_UNSUPPORTED


def test_no_tokens_launch_nothing(L):
    before = kda.kda_launch_count()
    assert _attn(L, Lt=0, q=None, out=None) == kda.KDA_OK
    assert _append(L, Lt=0, kv=None) == kda.KDA_OK
    assert kda.kda_launch_count() == before


def _verify(L_, p=P, q=P, x=P, u=P, lens=None, tok=P, acc=P, N=1, Lt=4, V=100):
    return L_.kda_verify_tokens(p, q, x, u, lens, tok, acc, N, Lt, V, None)


@pytest.mark.parametrize("bad", [dict(p=None), dict(x=None), dict(u=None), dict(tok=None),
                                 dict(acc=None), dict(q=P + 4), dict(lens=P + 8), dict(N=0),
                                 dict(Lt=-1), dict(V=0), dict(V=(1 << 30) + 1), dict(N=1 << 25),
                                 dict(N=1 << 22, Lt=1 << 10)])
def test_verify_rejects_invalid(L, bad):
    assert _verify(L, **bad) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("args,status", [
    ((0, 1, 12, 512, 64, 64), kda.KDA_ERR_INVALID_ARG), ((1, -1, 12, 512, 64, 64), kda.KDA_ERR_INVALID_ARG),
    ((1, 1, 12, 512, 64, 0), kda.KDA_ERR_INVALID_ARG), ((1, 1, 12, 100, 64, 64), kda.KDA_ERR_UNSUPPORTED)])
def test_workspace_size_rejects(L, args, status):
    with pytest.raises(kda.KdaError) as e:
        kda.kda_latent_attn_workspace_size(*args, sms=148)
    assert e.value.status == status


def test_workspace_size_null(L):
    assert L.kda_latent_attn_workspace_size(1, 1, 1, 512, 64, 64, 0, 0, 148, None) == \
        kda.KDA_ERR_INVALID_ARG
    n = ctypes.c_size_t(0)
    assert L.kda_latent_attn_workspace_size(1, 1, 1, 512, 64, 64, 0, 0, 148,
                                            ctypes.byref(n)) == kda.KDA_OK and n.value > 0


def test_binding_rejects_cpu_tensors_and_shapes(L):
    q = torch.zeros(2, 1, 3, 576)
    cache = torch.zeros(4, 16, 576)
    table = torch.zeros(2, 2, dtype=torch.int32)
    lens = torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_latent_attn(q, cache, table, lens, rank=512, scale=0.1)
    with pytest.raises(ValueError):
        kda.kda_latent_append(q[:, :, 0], cache, table, lens, rank=512)
    with pytest.raises(ValueError):
        kda.kda_latent_append(q, cache, table, lens, rank=512)
    with pytest.raises(ValueError):
        kda.kda_verify_tokens(torch.zeros(1, 2, 5), None, torch.zeros(1, 1, dtype=torch.int32),
                              torch.zeros(1, 2))
