"""Latent attention over a paged cache and the appending to it, against the float64
references of oracle/latent.py, at the sizes and masks where they can go wrong.

Tolerances, elementwise.  U is half a step of the type (finfo.eps / 2).  A score is an fp32
sum of D products: off by at most D 2^-23 (a tensor core may truncate, a step a product) of
scale sum |q| |c|, to which come the rounding of the scaled score and of the exponential,
2^-21 (|s| + 4) together.  Call that d; a weight p_j / sum p is then off by 2 d, and its
bf16 rounding adds U.  A sum of n weighted rows adds n 2^-23, the final rounding U |out|:
    |out - ref| <= (2 d + U_p + n 2^-23) sum p |c| + U |ref|,   |lse - ref| <= d + n 2^-23
"""
import math

import pytest
import torch

import gated_delta_rule_74_b200 as kda
from oracle import latent as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(dtype, lens, L, H, rank, rope, page, seed=0, cu=None, spread=1.0, extra_pages=2):
    g = torch.Generator().manual_seed(seed)
    N, D, dt = len(lens), rank + rope, DT[dtype]
    need = [max(1, -(-t // page)) for t in lens]
    P = max(need) + 1
    ids = torch.randperm(sum(need) + extra_pages, generator=g)
    table = torch.full((N, P), -7, dtype=torch.int32)         # unused entries: no page at all
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = ids[at:at + k].to(torch.int32)
        at += k
    cache = torch.randn((sum(need) + extra_pages, page, D), generator=g).to(dt)
    B, T = (1, L) if cu is not None else (N, L)
    q = (spread * torch.randn((B, T, H, D), generator=g)).to(dt)
    return dict(q=q, cache=cache, table=table, lens=torch.tensor(lens, dtype=torch.int32),
                cu=None if cu is None else torch.tensor(cu, dtype=torch.int32),
                scale=2.0 / math.sqrt(D), rank=rank)


def call(x, **kw):
    c = lambda t: None if t is None else t.cuda()
    out, lse = kda.kda_latent_attn(c(x["q"]), kw.pop("cache", None) if "cache" in kw else c(x["cache"]),
                                   c(x["table"]), c(x["lens"]), rank=x["rank"], scale=x["scale"],
                                   cu_seqlens=c(x["cu"]), **kw)
    torch.cuda.synchronize()
    return out, lse


def close(x, out, lse, expect=None):
    o, z, mag, size = expect or ref.attend(x["q"], x["cache"], x["table"], x["lens"], x["rank"],
                                           x["scale"], x["cu"])
    u = torch.finfo(x["q"].dtype).eps / 2
    D = x["q"].shape[-1]
    n = int(x["lens"].max())
    some = ~torch.isnan(z)
    empty = z == -math.inf
    zf = torch.where(empty | ~some, torch.zeros_like(z), z)
    d = D * 2.0 ** -23 * size + 2.0 ** -21 * (size + zf.abs() + 4)
    up = u if x["q"].dtype == torch.bfloat16 else 0.0
    tol = (2 * d + up + n * 2.0 ** -23)[..., None] * mag + u * o.abs()
    out, lse = out.double().cpu(), lse.double().cpu()
    bad = (out - o).abs() > tol
    assert not bool(bad[some].any()), (out - o).abs()[some].max()
    assert bool(torch.isfinite(out[some]).all())
    assert bool((lse[some] == -math.inf).eq(empty[some]).all())
    assert not bool(((lse - zf).abs() > d + n * 2.0 ** -23)[some & ~empty].any())


# lengths of zero and one, tile edges, ragged; heads from one to more than a block holds
CASES = [
    ("bf16", [1], 1, 1, 512, 64, 64), ("bf16", [64, 65, 63, 0, 1, 300], 1, 12, 512, 64, 64),
    ("bf16", [1000], 1, 12, 512, 64, 16), ("bf16", [5, 130, 257], 4, 12, 512, 64, 48),
    ("bf16", [700, 33], 1, 96, 512, 64, 64), ("bf16", [90, 200], 3, 40, 512, 0, 24),
    ("bf16", [150, 2], 5, 5, 384, 64, 8), ("bf16", [129], 2, 100, 256, 0, 128),
    ("bf16", [77, 1, 128], 1, 17, 128, 64, 32), ("bf16", [40, 19], 2, 3, 128, 0, 7),
    ("bf16", [33, 64], 1, 16, 512, 64, 1), ("bf16", [200], 37, 7, 256, 64, 256),
    ("f32", [1], 1, 1, 512, 64, 64), ("f32", [64, 65, 31, 0, 1, 300], 1, 12, 256, 0, 32),
    ("f32", [5, 130], 4, 12, 512, 64, 48), ("f32", [90, 33], 3, 40, 384, 64, 7),
    ("f32", [77, 20], 21, 3, 128, 64, 16), ("f32", [70, 0, 33], 5, 32, 512, 64, 48),
    ("f32", [200, 16], 2, 16, 256, 64, 5), ("f32", [15, 16, 17, 1], 1, 30, 512, 0, 16),
    ("f32", [129], 37, 7, 384, 0, 64),
]


@pytest.mark.parametrize("dtype,lens,L,H,rank,rope,page", CASES)
def test_attn_matches_reference(dtype, lens, L, H, rank, rope, page):
    x = make(dtype, lens, L, H, rank, rope, page, seed=len(lens) + H)
    close(x, *call(x))


@pytest.mark.parametrize("dtype,H,page", [("bf16", 12, 64), ("bf16", 4, 16), ("f32", 3, 20)])
def test_attn_packed(dtype, H, page):
    """Ragged packed chunks, an empty one among them; rows behind the last sequence stay."""
    cu = [0, 40, 40, 41, 100]
    x = make(dtype, [100, 70, 1, 59], 107, H, 256, 64, page, cu=cu)
    D = x["q"].shape[-1]
    out = torch.full((1, 107, H, 256), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((1, 107, H), 7.0, device="cuda")
    call(x, out=out, lse=lse)
    close(x, out, lse)
    assert bool((out[:, 100:] == 7.0).all()) and bool((lse[:, 100:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,L", [([2, 0, 5], 4), ([0], 1), ([3], 130)])
def test_attn_rows_that_see_nothing(dtype, lens, L):
    x = make(dtype, lens, L, 12, 512, 64, 16)
    out, lse = call(x)
    close(x, out, lse)
    for n, t in enumerate(lens):
        assert bool((out[n, :max(L - t, 0)] == 0).all())
        assert bool((lse[n, :max(L - t, 0)] == -math.inf).all())


@pytest.mark.parametrize("dtype,L,H,more", [("bf16", 6, 12, 0), ("bf16", 6, 12, 23), ("bf16", 3, 4, 0),
                                            ("bf16", 4, 40, 0), ("bf16", 3, 32, 25), ("bf16", 4, 16, 0),
                                            ("f32", 6, 12, 0), ("f32", 6, 32, 0)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attn_hidden_rows_have_no_effect(dtype, L, H, more, bad):
    """NaN and infinities behind the length, in unused pages and in later new tokens."""
    page = 16
    x = make(dtype, [70, 6, 33] + [9] * more, L, H, 512, 64, page)
    good = ref.attend(x["q"], x["cache"], x["table"], x["lens"], x["rank"], x["scale"])
    seen = torch.zeros(x["cache"].shape[:2], dtype=torch.bool)
    for n, t in enumerate(x["lens"].tolist()):
        for j in range(t - 2):                           # the last two new tokens turn bad
            seen[x["table"][n, j // page], j % page] = True
    x["cache"][~seen] = bad
    out, lse = call(x)
    for n in range(3):                                   # the tokens before them are untouched
        y = dict(x, q=x["q"][n:n + 1, :L - 2], lens=x["lens"][n:n + 1])
        close(y, out[n:n + 1, :L - 2], lse[n:n + 1, :L - 2], tuple(t[n:n + 1, :L - 2] for t in good))


@pytest.mark.parametrize("dtype,H,more", [("bf16", 5, 0), ("bf16", 12, 0), ("bf16", 30, 0), ("bf16", 48, 0),
                                          ("bf16", 60, 0), ("bf16", 37, 23), ("bf16", 48, 23), ("f32", 12, 0),
                                          ("f32", 16, 0)])
def test_attn_large_scores_and_far_maximum(dtype, H, more):
    """Scores of hundreds, the largest one late: the running maximum has to move."""
    x = make(dtype, [500, 257] + [3] * more, 2, H, 256, 64, 64, spread=20.0)
    pos = x["table"][0, 480 // 64], 480 % 64
    x["cache"][pos] = x["q"][0, 0, 0] / 4
    close(x, *call(x))


@pytest.mark.parametrize("dtype,page", [("bf16", 64), ("bf16", 12), ("f32", 16)])
def test_attn_strided_cache(dtype, page):
    """One layer's slice of a pool that holds several, with padded rows."""
    x = make(dtype, [100, 37], 2, 12, 512, 64, page)
    P = x["cache"].shape[0]
    pool = torch.full((P, 3, page, 584), math.nan, dtype=DT[dtype], device="cuda")
    view = pool[:, 1, :, :576]
    view.copy_(x["cache"])
    out, lse = call(x, cache=view)
    close(x, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_lengths_and_pages_out_of_range_stay_inside(dtype):
    """A length beyond the table, negative lengths and page ids outside the cache: the other
    sequences are right."""
    x = make(dtype, [100, 37, 64, 50], 1, 12, 256, 64, 16)
    y = dict(x, lens=x["lens"].clone(), table=x["table"].clone())
    y["lens"][0] = 2 ** 31 - 1
    y["lens"][1] = -5
    y["table"][2, :2] = torch.tensor([2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    out, lse = call(y)
    z = dict(x, q=x["q"][3:], lens=x["lens"][3:], table=x["table"][3:])
    close(z, out[3:], lse[3:])
    assert bool((out[1] == 0).all())


@pytest.mark.parametrize("dtype,lens,H,rank,page", [
    ("bf16", [9000], 12, 512, 64), ("bf16", [9500], 96, 512, 64), ("bf16", [700] * 26, 96, 256, 64),
    ("bf16", [5000, 40, 7000], 30, 384, 16),
    ("bf16", [900] * 9 + [1], 12, 128, 64), ("bf16", [9000, 100, 200, 300, 50, 60], 96, 256, 64),
    ("f32", [5000], 12, 256, 64), ("f32", [300] * 20, 3, 128, 64), ("f32", [5000, 30], 32, 512, 64),
    ("f32", [700, 3] * 4, 60, 256, 24)])
def test_attn_long_sequence_is_split_and_joined(dtype, lens, H, rank, page):
    """One sequence or a few over all SMs, by few, some and many CTAs; and the same bits again."""
    x = make(dtype, lens, 1, H, rank, 64, page)
    out, lse = call(x)
    close(x, out, lse)
    again = call(x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("bf16", 9), ("f32", 16)])
def test_attn_shared_pages(dtype, page):
    """Sequences that share their first pages, and one that is another's twin."""
    x = make(dtype, [100, 90, 100, 33], 2, 12, 256, 64, page)
    share = 32 // page
    x["table"][1, :share] = x["table"][0, :share]
    x["table"][2] = x["table"][0]
    x["q"][2] = x["q"][0]
    out, lse = call(x)
    close(x, out, lse)
    assert torch.equal(lse[0], lse[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_packed_without_tokens(dtype):
    x = make(dtype, [10, 0], 6, 3, 128, 64, 16, cu=[0, 0, 0])
    out = torch.full((1, 6, 3, 128), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((1, 6, 3), 7.0, device="cuda")
    call(x, out=out, lse=lse)
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


@pytest.mark.parametrize("dtype,page", [("bf16", 64), ("bf16", 60), ("f32", 64)])
def test_offsets_beyond_32_bits(dtype, page):
    """The last pages of a cache of more than 2^31 elements (and 2^32 bytes)."""
    x = make(dtype, [150, 20], 2, 12, 512, 64, page)
    P = x["cache"].shape[0]
    total = 2 ** 31 // (page * 576) + P + 1
    big = torch.empty((total, page, 576), dtype=DT[dtype], device="cuda")
    big[total - P:] = x["cache"].cuda()
    y = dict(x, table=torch.where(x["table"] >= 0, x["table"] + (total - P), x["table"]))
    out, lse = call(y, cache=big)
    close(x, out, lse)
    kv = torch.randn((2, 2, 576)).to(DT[dtype])
    kda.kda_latent_append(kv.cuda(), big, y["table"].cuda(), y["lens"].cuda(), rank=512)
    for n, t in enumerate((150, 20)):
        for i in (1, 2):
            pos = t - i
            assert torch.equal(big[int(y["table"][n, pos // page]), pos % page].cpu(), kv[n, 2 - i])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_workspace_and_stream(dtype):
    x = make(dtype, [900, 70], 2, 12, 512, 64, 64)
    expect = call(x)
    need = kda.kda_latent_attn_workspace_size(2, 2, 12, 512, 64, 64,
                                              dtype=kda.KDA_BF16 if dtype == "bf16" else kda.KDA_F32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out, lse = call(x, workspace=ws)
    assert torch.equal(out, expect[0]) and torch.equal(lse, expect[1])
    s = torch.cuda.Stream()
    out, lse = call(x, stream=s)
    s.synchronize()
    assert torch.equal(out, expect[0]) and torch.equal(lse, expect[1])
    with pytest.raises(kda.KdaError):
        call(x, workspace=ws[:need - 256])


def test_outputs_on_a_side_stream_are_that_streams():
    """Work that the current stream still has queued on freed memory does not reach them."""
    x = make("bf16", [300, 70], 2, 12, 512, 64, 64)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    want = call(x)
    target, u = torch.softmax(torch.randn((40, 5, 900), device="cuda"), -1), torch.rand((40, 5), device="cuda")
    ids = target[:, :4].argmax(-1).to(torch.int32)
    tok, acc = kda.kda_verify_tokens(target, None, ids, u)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty_like(t) for t in (*want, tok, acc)]
    places = {t.data_ptr() for t in old}
    torch.cuda._sleep(200_000_000)
    for t in old:
        t.fill_(7)
    del old, t
    got = (*kda.kda_latent_attn(d["q"], d["cache"], d["table"], d["lens"], rank=512, scale=x["scale"], stream=s),
           *kda.kda_verify_tokens(target, None, ids, u, stream=s))
    torch.cuda.synchronize()
    for a, b in zip(got, (*want, tok, acc)):
        assert torch.equal(a, b)
        assert a.data_ptr() not in places


def test_attn_two_streams_at_once():
    xs = [make("bf16", [3000, 100], 1, 12, 512, 64, 64, seed=s) for s in (1, 2)]
    want = [call(x) for x in xs]
    dev = [{k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()} for x in xs]
    st = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [kda.kda_latent_attn(x["q"], x["cache"], x["table"], x["lens"], rank=512,
                                   scale=x["scale"], stream=s) for x, s in zip(dev, st)]
        torch.cuda.synchronize()
        for (o, z), (a, b) in zip(got, want):
            assert torch.equal(o, a) and torch.equal(z, b)


def test_attn_graph_replays_new_lengths():
    """One captured call serves a growing sequence; two graphs share one workspace in turn."""
    x = make("bf16", [200, 10], 1, 12, 512, 64, 64)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    ws = torch.empty(kda.kda_latent_attn_workspace_size(2, 1, 12, 512, 64, 64), dtype=torch.uint8,
                     device="cuda")
    graphs = []
    for kw in ({}, {"workspace": ws}, {"workspace": ws}):
        kda.kda_latent_attn(d["q"], d["cache"], d["table"], d["lens"], rank=512, scale=x["scale"])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = kda.kda_latent_attn(d["q"], d["cache"], d["table"], d["lens"], rank=512,
                                      scale=x["scale"], **kw)
        graphs.append((g, res))
    for lens in ([200, 10], [1, 64], [150, 0]):
        d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        for g, res in graphs:
            g.replay()
        torch.cuda.synchronize()
        y = dict(x, lens=torch.tensor(lens, dtype=torch.int32))
        for g, res in graphs:
            close(y, *res)


# ------------------------------------------------------------------------- append

def make_append(dtype, lens, L, H, rank, rope, page, norm, seed=0, cu=None):
    x = make(dtype, [max(t, 0) for t in lens], L, 1, rank, rope, page, seed=seed, cu=cu)
    g = torch.Generator().manual_seed(seed + 1)
    x["lens"] = torch.tensor(lens, dtype=torch.int32)
    B, T = x["q"].shape[:2]
    x["kv"] = (3 * torch.randn((B, T, rank + rope), generator=g)).to(DT[dtype])
    x["w"] = 1 + 0.1 * torch.randn(rank, generator=g) if norm else None
    x["f"] = x["qi"] = None
    if rope:
        x["f"] = (10000.0 ** (-torch.arange(0, rope, 2).double() / rope)).float()
        x["qi"] = torch.randn((B, T, H, rope), generator=g).to(DT[dtype])
    return x


def run_append(x, inter, q_fill=5.0, **kw):
    c = lambda t: None if t is None else t.cuda()
    cache = c(x["cache"]).clone()
    qo = None if x["qi"] is None else torch.full(x["qi"].shape, q_fill, dtype=x["kv"].dtype, device="cuda")
    got = kda.kda_latent_append(c(x["kv"]), cache, c(x["table"]), c(x["lens"]), rank=x["rank"],
                                cu_seqlens=c(x["cu"]), norm_weight=c(x["w"]), inv_freq=c(x["f"]),
                                interleaved=inter, q_pe=c(x["qi"]), q_pe_out=qo, **kw)
    torch.cuda.synchronize()
    assert got is qo
    return cache, qo


def append_close(x, cache, qo, inter, q_fill=5.0):
    """fp32 work on each value: the norm is a sum of rank squares (rank 2^-24), a root, a
    quotient and two products; a turn two products of a cosine good to 2^-21."""
    ro, rq = ref.append(x["kv"], x["cache"], x["table"], x["lens"], x["rank"], x["cu"], x["w"],
                        1e-6, x["f"], inter, x["qi"],
                        None if x["qi"] is None else torch.full(x["qi"].shape, q_fill))
    u = torch.finfo(x["kv"].dtype).eps / 2
    tol = (u + x["rank"] * 2.0 ** -24 + 2.0 ** -21) * ro.abs()
    tol[..., x["rank"]:] += 2.0 ** -20 * x["kv"].double().abs().max()
    got = cache.double().cpu()
    assert not bool(((got - ro).abs() > tol).any()), (got - ro).abs().max()
    if rq is not None:
        tol = u * rq.abs() + 2.0 ** -20 * x["qi"].double().abs().max()
        assert not bool(((qo.double().cpu() - rq).abs() > tol).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("lens,L,H,rank,rope,page,norm", [
    ([1], 1, 1, 512, 64, 64, True), ([64, 65, 0, 1, 200], 1, 12, 512, 64, 64, True),
    ([9, 3, 30], 5, 96, 512, 64, 16, False), ([40, 17], 9, 17, 384, 64, 7, True),
    ([33, 20], 3, 1, 128, 0, 1, True), ([100], 100, 33, 256, 64, 48, False)])
def test_append_matches_reference(dtype, inter, lens, L, H, rank, rope, page, norm):
    x = make_append(dtype, lens, L, H, rank, rope, page, norm)
    append_close(x, *run_append(x, inter), inter)


@pytest.mark.parametrize("N", [1, 3, 40, 1100])
def test_append_packed(N):
    """Many ragged sequences, empty ones among them, and tokens of no sequence at the end."""
    g = torch.Generator().manual_seed(N)
    new = torch.randint(0, 4, (N,), generator=g).tolist()
    new[0] = 2
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    lens = [n + int(e) for n, e in zip(new, torch.randint(0, 20, (N,), generator=g))]
    x = make_append("bf16", lens, cu[-1] + 3, 2, 128, 64, 16, True, cu=cu)
    append_close(x, *run_append(x, False), False)


@pytest.mark.parametrize("dtype,inter,H", [("bf16", False, 12), ("bf16", True, 9), ("f32", False, 5),
                                           ("f32", True, 33)])
def test_append_many_tokens(dtype, inter, H):
    """Enough tokens that a warp takes a whole one."""
    cu = [0, 1000, 1001, 1001, 2700]
    x = make_append(dtype, [1300, 90, 5, 1699], 2705, H, 128, 64, 64, True, cu=cu)
    append_close(x, *run_append(x, inter), inter)


def test_append_far_positions():
    """Angles of positions in the millions: a 32-bit product would be off by a tenth."""
    lens = [5_000_003, 2 ** 30 + 7]
    x = make_append("f32", [2, 2], 2, 3, 128, 64, 16, False)
    x["lens"] = torch.tensor(lens, dtype=torch.int32)        # beyond the table: queries only
    cache, qo = run_append(x, False)
    assert torch.equal(cache.cpu(), x["cache"])
    append_close(x, cache, qo, False)


def test_append_without_rotation_copies_bits():
    x = make_append("bf16", [30, 9], 3, 2, 512, 64, 16, False)
    x["kv"][0, 0, 3], x["kv"][0, 0, 515], x["kv"][0, 1, 530] = math.inf, -math.inf, math.nan
    x["f"] = None
    cache, qo = run_append(x, False)
    rows = torch.stack([ref.cached(cache.cpu(), x["table"], n, t)[-3:] for n, t in ((0, 30), (1, 9))])
    assert torch.equal(rows.view(torch.int16), x["kv"].view(torch.int16))
    assert torch.equal(qo.cpu(), x["qi"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_strided_inputs_and_cache(dtype):
    """kv a slice of a wider projection, the queries' parts inside of whole queries, one
    layer's pages; nothing around them changes."""
    x = make_append(dtype, [30, 9], 3, 5, 512, 64, 24, True)
    wide = torch.full((2, 3, 704), 2.0, dtype=DT[dtype], device="cuda")
    wide[..., 64:640] = x["kv"].cuda()
    qw = torch.full((2, 3, 5, 192), 2.0, dtype=DT[dtype], device="cuda")
    qw[..., 128:] = x["qi"].cuda()
    q = torch.full((2, 3, 5, 576), 5.0, dtype=DT[dtype], device="cuda")
    pool = torch.full((x["cache"].shape[0], 2, 24, 576), 3.0, dtype=DT[dtype], device="cuda")
    pool[:, 1] = x["cache"].cuda()
    kda.kda_latent_append(wide[..., 64:640], pool[:, 1], x["table"].cuda(), x["lens"].cuda(), rank=512,
                          norm_weight=x["w"].cuda(), inv_freq=x["f"].cuda(), q_pe=qw[..., 128:],
                          q_pe_out=q[..., 512:])
    torch.cuda.synchronize()
    append_close(x, pool[:, 1], q[..., 512:], False)
    assert bool((pool[:, 0] == 3.0).all()) and bool((q[..., :512] == 5.0).all())
    # in place, too
    kda.kda_latent_append(wide[..., 64:640], pool[:, 1], x["table"].cuda(), x["lens"].cuda(), rank=512,
                          norm_weight=x["w"].cuda(), inv_freq=x["f"].cuda(), q_pe=qw[..., 128:],
                          q_pe_out=qw[..., 128:])
    assert torch.equal(qw[..., 128:], q[..., 512:])


def test_append_pages_out_of_range_are_dropped():
    x = make_append("bf16", [30, 9], 3, 2, 128, 64, 16, True)
    x["table"][0] = torch.tensor([-1, 2 ** 31 - 1, -7], dtype=torch.int32)
    append_close(x, *run_append(x, False), False)
