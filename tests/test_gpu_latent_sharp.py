"""The latent attention under the checks of latent_sharp.py: the error's root mean square at every
size, and inputs that show a single token lost, doubled, misplaced or seen too early."""
import pytest
import torch

import gated_delta_rule_74_b200 as kda
from latent_sharp import counting, counts_right, finding, found, rms_close
from test_gpu_latent import CASES, call, close, make

pytestmark = pytest.mark.gpu

# every block height of the tensor-core kernel at the ranks where some of its warps have no columns
# (128) or one more than others (384), and sequences that many CTAs share
MORE = [("bf16", [300, 77, 64], 1, 48, 128, 64, 64), ("bf16", [300, 77], 2, 32, 128, 0, 16),
        ("bf16", [130, 40] * 10, 1, 80, 128, 64, 64), ("bf16", [150, 64] * 10, 1, 96, 128, 64, 32),
        ("bf16", [300, 77, 64], 1, 48, 384, 64, 64), ("bf16", [300, 77], 2, 32, 384, 64, 8),
        ("bf16", [130, 40] * 10, 1, 80, 384, 0, 64), ("bf16", [150, 64] * 10, 1, 96, 384, 64, 48),
        ("bf16", [200], 40, 12, 128, 64, 64), ("bf16", [200], 40, 12, 384, 64, 64),
        ("bf16", [9000], 1, 12, 512, 64, 64), ("bf16", [9500], 1, 96, 512, 64, 64),
        ("bf16", [700] * 26, 1, 96, 256, 64, 64), ("bf16", [2500, 40, 900], 4, 12, 512, 64, 16),
        ("f32", [5000], 1, 12, 256, 64, 64), ("f32", [900, 30], 1, 32, 512, 64, 64),
        ("f32", [700, 3] * 4, 1, 60, 256, 64, 24), ("f32", [300], 60, 5, 512, 64, 64)]


@pytest.mark.parametrize("dtype,lens,L,H,rank,rope,page", CASES + MORE)
def test_attn_rms(dtype, lens, L, H, rank, rope, page):
    x = make(dtype, lens, L, H, rank, rope, page, seed=7 + H)
    out, lse = call(x)
    close(x, out, lse)
    rms_close(x, out, lse)


@pytest.mark.parametrize("dtype,lens,L,H,rank,page", [
    ("bf16", [1, 2, 15, 16, 17, 47, 48, 49, 63, 64, 65, 0, 95, 96, 97, 127, 128, 129], 1, 12, 512, 64),
    ("bf16", [1000, 64, 300], 1, 1, 512, 16), ("bf16", [9000], 1, 12, 512, 64),
    ("bf16", [40001], 1, 40, 512, 64), ("bf16", [9500, 333], 1, 96, 512, 64),
    ("bf16", [1500, 700] * 12, 1, 96, 256, 64), ("bf16", [1501, 64, 3], 7, 12, 512, 24),
    ("bf16", [2000, 350], 300, 12, 384, 64), ("bf16", [777, 1], 3, 17, 128, 8),
    ("bf16", [1000, 65], 2, 12, 512, 12), ("bf16", [500], 40, 3, 256, 1),
    ("f32", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 0], 1, 12, 256, 32),
    ("f32", [9000], 1, 12, 512, 64), ("f32", [1000, 64, 300], 1, 1, 128, 7),
    ("f32", [1500, 333], 2, 32, 512, 64), ("f32", [1200], 100, 5, 384, 48)])
def test_attn_counts_every_token_once(dtype, lens, L, H, rank, page):
    x = counting(make(dtype, lens, L, H, rank, 64, page))
    counts_right(x, *call(x))


@pytest.mark.parametrize("dtype,t,N,H,rank,page", [
    ("bf16", 1000, 84, 12, 512, 64), ("bf16", 500, 500, 1, 256, 16), ("bf16", 1000, 11, 96, 512, 64),
    ("bf16", 1900, 20, 96, 128, 32), ("bf16", 700, 24, 30, 384, 8), ("bf16", 900, 20, 48, 512, 64),
    ("bf16", 1500, 24, 64, 512, 24), ("bf16", 1500, 19, 80, 512, 64), ("bf16", 300, 25, 12, 256, 7),
    ("bf16", 20000, 2, 96, 256, 64), ("f32", 1000, 84, 12, 512, 64), ("f32", 600, 20, 32, 256, 16),
    ("f32", 300, 100, 3, 128, 5), ("f32", 9000, 3, 16, 384, 64)])
def test_attn_finds_every_token(dtype, t, N, H, rank, page):
    """Each row looks for one token and gets it: every token of the shared pages is looked for, or,
    of long sequences, the last ones."""
    x, want = finding(make(dtype, [t] + [1] * (N - 1), 1, H, rank, 64, page), seed=t)
    found(x, want, call(x)[0])


@pytest.mark.parametrize("dtype,page", [("bf16", 64), ("bf16", 12), ("f32", 64)])
def test_attn_packed_prompts_without_context(dtype, page):
    """Whole prompts of unlike lengths, with nothing cached before them."""
    new = [900, 0, 1, 64, 333, 65]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    x = make(dtype, new, cu[-1], 4, 256, 64, page, cu=cu)
    out, lse = call(x)
    close(x, out, lse)
    rms_close(x, out, lse)
    y = counting(make(dtype, [4 * n for n in new], 4 * cu[-1], 3, 128, 64, page, cu=[4 * c for c in cu]))
    counts_right(y, *call(y))


@pytest.mark.parametrize("dtype,lens,H,page", [("bf16", [300, 64, 0], 12, 64), ("bf16", [9000, 3], 40, 64),
                                               ("bf16", [300, 5], 12, 12), ("f32", [5000, 40], 12, 16)])
def test_attn_without_log_sums(dtype, lens, H, page):
    """lse NULL at the C entry: the same output, by blocks that one CTA has and by the join."""
    x = make(dtype, lens, 1, H, 256, 64, page)
    want, _ = call(x)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    out = torch.full_like(want, 7.0)
    c, t = d["cache"], d["table"]
    rc = kda.lib().kda_latent_attn(
        d["q"].data_ptr(), c.data_ptr(), t.data_ptr(), d["lens"].data_ptr(), None, out.data_ptr(), None,
        len(lens), 1, H, 256, 64, c.shape[0], page, t.shape[1], c.stride(0), c.stride(1), x["scale"],
        kda.KDA_BF16 if dtype == "bf16" else kda.KDA_F32, torch.cuda.current_stream().cuda_stream)
    assert rc == kda.KDA_OK
    torch.cuda.synchronize()
    assert torch.equal(out, want)
