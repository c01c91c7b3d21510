"""Rows of a block of the latent attention, as the workspace that a call asks for shows them
(partial results of that many rows for each of the device's multiprocessors; host only)."""
import pytest

import gated_delta_rule_74_b200 as kda


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_74_b200 import build
    build.build()


def size(N, L, H, packed=False, rank=512, **kw):
    return kda.kda_latent_attn_workspace_size(N, L, H, rank, 64, 64, packed=packed, sms=148, **kw)


def rows(N, L, H, packed=False):
    """Block rows from the size: that of uniform calls of one token and r heads has r."""
    known = {size(100, 1, r): r for r in (16, 32, 48, 64, 80, 96)}
    assert len(known) == 6
    return known[size(N, L, H, packed)]


@pytest.mark.parametrize("N,T,H", [(512, 1024, 12), (300, 1324, 4), (2000, 3200, 1)])
def test_packed_rows_that_one_sequence_may_hold(N, T, H):
    """Few rows a sequence on average, many in all: one of the sequences may have most of them."""
    assert rows(N, T, H, packed=True) >= 48


@pytest.mark.parametrize("N,T,H,want", [(256, 256, 12, 16), (256, 200, 12, 16), (8, 16, 12, 32),
                                        (4, 40, 1, 16), (1, 1, 1, 16), (3, 1024, 12, 64)])
def test_packed_rows_of_like_sequences(N, T, H, want):
    assert rows(N, T, H, packed=True) == want
