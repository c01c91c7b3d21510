"""The latent attention's tensor-core kernel when its waits give up: its roles load, multiply and
wait for one another, and whichever stops first, what the others have in flight is waited for, the
flag is raised, and the next call is right.  (No wait is left out and no address is bad: a wait
that gives up leaves its role, which reads and writes nothing from then on.)"""
import pytest
import torch

import gated_delta_rule_74_b200 as kda
from test_gpu_latent import call, make

pytestmark = pytest.mark.gpu

# blocks of 16 to 96 rows, whole blocks and shared ones, few and many tiles
CASES = {"one": ([40], 1, 12, 512, 64), "ragged": ([3000, 40, 0, 700] * 25, 1, 12, 512, 64),
         "split": ([20000], 1, 24, 512, 64), "drafts": ([700, 33, 900] * 30, 4, 12, 512, 16),
         "heads80": ([2000] * 20, 1, 80, 256, 64), "heads96": ([3000, 200] * 20, 1, 96, 512, 64),
         "chunk": ([4000, 1500], 300, 12, 128, 64)}


def limited(x, polls, out, lse):
    c = lambda t: None if t is None else t.cuda()
    q, cache, table, lens, cu = c(x["q"]), c(x["cache"]), c(x["table"]), c(x["lens"]), c(x["cu"])
    L, H, D = q.shape[1:]
    rc = kda.lib().kda_selftest_latent_waits(
        polls, q.data_ptr(), cache.data_ptr(), table.data_ptr(), lens.data_ptr(),
        None if cu is None else cu.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), len(lens), L, H, x["rank"], D - x["rank"], cache.shape[0], cache.shape[1], table.shape[1],
        cache.stride(0), cache.stride(1), x["scale"], torch.cuda.current_stream().cuda_stream)
    assert rc == kda.KDA_OK
    torch.cuda.synchronize()


def outputs(x):
    B, L, H, _ = x["q"].shape
    return (torch.full((B, L, H, x["rank"]), 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((B, L, H), 7.0, device="cuda"))


@pytest.mark.parametrize("name", CASES)
def test_waits_that_give_up_are_reported_and_leave_the_device_usable(name):
    lens, L, H, rank, page = CASES[name]
    x = make("bf16", lens, L, H, rank, 64, page, seed=3)
    want = call(x)
    assert kda.kda_device_status(reset=True) == kda.KDA_OK
    for polls in (0, 1, 2, 3, 5, 8, 1 << 20):
        out, lse = outputs(x)
        limited(x, polls, out, lse)
        status = kda.kda_device_status(reset=True)
        assert polls > 0 or status == kda.KDA_ERR_TIMEOUT
        if polls == 1 << 20 or status == kda.KDA_OK:
            assert status == kda.KDA_OK
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        again = call(x)
        assert kda.kda_device_status(reset=False) == kda.KDA_OK
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def nan_or(got, want):
    """Rows that are NaN as a whole; of the others none differs."""
    bad = torch.isnan(got).reshape(*want.shape[:3], -1)
    assert torch.equal(bad.any(-1), bad.all(-1))
    bad = bad.any(-1)
    assert torch.equal(got[~bad], want[~bad])
    return bad


@pytest.mark.parametrize("name", CASES)
def test_rows_that_were_not_finished_are_nan(name):
    """Nothing that the buffers held before, and no part of a row: it is whole and right, or NaN."""
    lens, L, H, rank, page = CASES[name]
    x = make("bf16", lens, L, H, rank, 64, page, seed=4)
    want = call(x)
    for polls in (0, 1, 2, 3, 5, 8, 13):
        out, lse = outputs(x)
        limited(x, polls, out, lse)
        status = kda.kda_device_status(reset=True)
        bad = nan_or(out, want[0])
        assert torch.equal(bad, nan_or(lse, want[1]))
        assert bool(bad.any()) <= (status == kda.KDA_ERR_TIMEOUT)
        assert polls > 0 or bool(bad.all())
        alone = torch.full_like(out, 7.0)
        limited(x, polls, alone, None)
        kda.kda_device_status(reset=True)
        nan_or(alone, want[0])
    for t in call(x):
        assert not bool(torch.isnan(t).any())


def test_rows_of_no_sequence_stay_when_waits_give_up():
    x = make("bf16", [100, 70, 1, 5059], 107, 12, 256, 64, 64, cu=[0, 40, 40, 41, 100])
    out = torch.full((1, 107, 12, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 107, 12), 7.0, device="cuda")
    limited(x, 0, out, lse)
    assert kda.kda_device_status(reset=True) == kda.KDA_ERR_TIMEOUT
    assert bool(torch.isnan(out[:, :100]).all()) and bool(torch.isnan(lse[:, :100]).all())
    assert bool((out[:, 100:] == 7.0).all()) and bool((lse[:, 100:] == 7.0).all())
