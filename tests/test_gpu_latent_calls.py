"""Calls of the serving operators that their documentation allows, at its ends: other orders of the
cache's memory, one page for all, very many sequences and heads, rows beyond 32 bits, two captured
graphs at once."""
import pytest
import torch

import gated_delta_rule_74_b200 as kda
from latent_sharp import counting, counts_right
from test_gpu_latent import DT, append_close, call, close, make, make_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("bf16", 12), ("f32", 16)])
def test_cache_with_a_pages_rows_apart(dtype, page):
    """Row r of all pages before row r + 1 of any: the page stride is the smaller one."""
    x = make(dtype, [100, 37], 2, 12, 256, 64, page)
    apart = x["cache"].transpose(0, 1).contiguous().cuda().transpose(0, 1)
    assert apart.stride(0) < apart.stride(1)
    close(x, *call(x, cache=apart))
    y = make_append(dtype, [30, 9], 3, 5, 128, 64, page, True)
    cache = y["cache"].transpose(0, 1).contiguous().cuda().transpose(0, 1)
    c = lambda t: t.cuda()
    q = kda.kda_latent_append(c(y["kv"]), cache, c(y["table"]), c(y["lens"]), rank=128, norm_weight=c(y["w"]),
                              inv_freq=c(y["f"]), q_pe=c(y["qi"]))
    torch.cuda.synchronize()
    append_close(y, cache, q, False)


@pytest.mark.parametrize("dtype,page", [("bf16", 5000), ("bf16", 4999), ("f32", 4999)])
def test_one_page_a_sequence(dtype, page):
    x = make(dtype, [4990, 1, 700], 1, 12, 128, 64, page, extra_pages=0)
    close(x, *call(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,L,H,lens", [(5000, 1, 1, None), (1, 1, 65535, [3]), (2, 3, 5000, [70, 2])])
def test_many_sequences_and_many_heads(dtype, N, L, H, lens):
    x = counting(make(dtype, lens or [n % 7 for n in range(N)], L, H, 128, 0, 8))
    counts_right(x, *call(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_batch_of_empty_slots(dtype):
    """100,000 sequences of which three have tokens."""
    N = 100_000
    at = {0: 2, 40_001: 70, N - 1: 5}
    cu, lens = [0], []
    for n in range(N):
        k = at.get(n, 0)
        cu.append(cu[-1] + k)
        lens.append(k + 30 if k else 0)
    g = torch.Generator().manual_seed(1)
    table = torch.zeros((N, 7), dtype=torch.int32)
    for i, n in enumerate(at):
        table[n] = torch.randperm(21, generator=g)[:7].to(torch.int32)
    x = dict(q=torch.randn((1, cu[-1], 12, 192), generator=g).to(DT[dtype]),
             cache=torch.randn((21, 16, 192), generator=g).to(DT[dtype]), table=table,
             lens=torch.tensor(lens, dtype=torch.int32), cu=torch.tensor(cu, dtype=torch.int32),
             scale=0.1, rank=128)
    out, lse = call(x)
    keep = torch.tensor(list(at))
    y = dict(x, table=table[keep], lens=x["lens"][keep], cu=torch.tensor([0, 2, 72, 77], dtype=torch.int32))
    close(y, out, lse)
    assert kda.kda_device_status(reset=False) == kda.KDA_OK


def test_two_captured_graphs_at_once():
    """Two graphs, each with a pool allocation of its own, replayed together on two streams."""
    xs = [make("bf16", [5000, 100], 1, 12, 512, 64, 64, seed=s) for s in (1, 2)]
    dev = [{k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()} for x in xs]
    run = lambda d: kda.kda_latent_attn(d["q"], d["cache"], d["table"], d["lens"], rank=512, scale=d["scale"])
    want = [run(d) for d in dev]
    torch.cuda.synchronize()
    graphs, got = [], []
    for d in dev:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append([run(d) for _ in range(5)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in dev]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for res, (o, z) in zip(got, want):
        for a, b in res:
            assert torch.equal(a, o) and torch.equal(b, z)


@pytest.mark.parametrize("drafts", [True, False])
def test_verify_rows_beyond_32_bits(drafts):
    """Rows whose elements lie beyond 2^31: all weight on single tokens near the rows' ends."""
    N, L, V = 3, 1, 400_000_001
    target = torch.zeros((N, L + 1, V), device="cuda")
    draft = torch.zeros((N, L, V), device="cuda") if drafts else None
    x = torch.tensor([[V - 1], [V - 2], [V - 3]], dtype=torch.int32, device="cuda")
    u = torch.full((N, L + 1), 0.5, device="cuda")
    for n in range(N):
        target[n, 0, V - 1 - n] = 1.0 if n != 2 else 0.25          # the third falls
        target[n, 0, V - 10] += 0.0 if n != 2 else 0.75
        target[n, 1, V - 20 - n] = 1.0
        if drafts:
            draft[n, 0, V - 1 - n] = 1.0
    t, a = kda.kda_verify_tokens(target, draft, x, u)
    torch.cuda.synchronize()
    assert a.tolist() == [1, 1, 0]
    assert t.tolist() == [[V - 1, V - 20], [V - 2, V - 21], [V - 10, -1]]
    del target, draft
    torch.cuda.empty_cache()


def test_verify_largest_vocabulary():
    V = 1 << 30
    target = torch.zeros((1, 1, V), device="cuda")
    target[0, 0, V - 1], target[0, 0, 5] = 0.75, 0.25
    none = torch.zeros((1, 0), dtype=torch.int32, device="cuda")
    for u, want in ((0.0, 5), (0.24, 5), (0.25, V - 1), (0.9, V - 1)):
        t, a = kda.kda_verify_tokens(target, None, none, torch.full((1, 1), u, device="cuda"))
        assert t.tolist() == [[want]] and a.tolist() == [0]
    del target
    torch.cuda.empty_cache()
