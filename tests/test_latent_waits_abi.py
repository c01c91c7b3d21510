"""Refusals of the latent attention's wait self-test, on the host."""
import pytest

import gated_delta_rule_74_b200 as kda

P = 0x10000   # a 16-byte aligned fake address; never dereferenced by these calls


def _call(polls=0, q=P, rank=512, page=64, scale=0.1):
    from gated_delta_rule_74_b200 import build
    build.build()
    return kda.lib().kda_selftest_latent_waits(polls, q, P, P, P, None, P, None, 1, 1, 1, rank, 64, 4,
                                               page, 2, 64 * 576, 576, scale, None)


@pytest.mark.parametrize("bad", [dict(polls=(1 << 20) + 1), dict(page=12), dict(q=None), dict(q=P + 8),
                                 dict(scale=0.0)])
def test_rejects_invalid(bad):
    assert _call(**bad) == kda.KDA_ERR_INVALID_ARG


def test_rejects_unsupported():
    assert _call(rank=100) == kda.KDA_ERR_UNSUPPORTED
