"""kda_verify_tokens against the definition in 64 bits: whole numbers, equal."""
import math

import pytest
import torch

import gated_delta_rule_74_b200 as kda
from oracle import latent as ref

pytestmark = pytest.mark.gpu


def make(N, L, V, drafts=True, seed=0, near=0.8):
    g = torch.Generator().manual_seed(seed)
    logits = 2 * torch.randn((N, L + 1, V), generator=g)
    target = torch.softmax(logits, -1)
    draft = torch.softmax(near * logits[:, :L] + 0.5 * torch.randn((N, L, V), generator=g), -1)
    if drafts and L:
        tok = torch.multinomial(draft.reshape(N * L, V), 1, generator=g).reshape(N, L)
    else:
        tok = target[:, :L].argmax(-1)
    return target, draft if drafts else None, tok.to(torch.int32), torch.rand((N, L + 1), generator=g)


def check(target, draft, tok, u, lens=None, **kw):
    c = lambda t: None if t is None else t.cuda()
    t, a = kda.kda_verify_tokens(c(target), c(draft), c(tok), c(u), draft_lens=c(lens), **kw)
    torch.cuda.synchronize()
    rt, ra = ref.verify(target, draft, tok, u, lens)
    assert torch.equal(a.cpu(), ra)
    assert torch.equal(t.cpu(), rt)
    return t.cpu(), a.cpu()


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("N,L,V", [(1, 1, 1), (1, 4, 2), (3, 2, 31), (5, 3, 129), (2, 5, 1000),
                                   (40, 4, 4097), (1, 4, 32000), (2, 1, 100277), (300, 2, 513),
                                   (2, 40, 300), (700, 1, 65)])
def test_matches_definition(N, L, V, drafts):
    check(*make(N, L, V, drafts, seed=N + L + V))


@pytest.mark.parametrize("N,V", [(1, 50000), (9, 333)])
def test_no_drafts_samples_the_target(N, V):
    target, _, tok, u = make(N, 0, V, False)
    t, a = check(target, None, tok, u)
    assert t.shape == (N, 1) and bool((a == 0).all())


def test_ragged_drafts():
    x = make(8, 5, 777)
    check(*x, lens=torch.tensor([0, 1, 2, 3, 4, 5, 9, -3], dtype=torch.int32))


@pytest.mark.parametrize("u", [0.0, 1.0 - 2.0 ** -24])
@pytest.mark.parametrize("drafts", [True, False])
def test_random_numbers_at_their_ends(u, drafts):
    target, draft, tok, _ = make(6, 3, 5000, drafts)
    check(target, draft, tok, torch.full((6, 4), u))


@pytest.mark.parametrize("drafts", [True, False])
def test_tokens_outside_the_vocabulary_fall(drafts):
    target, draft, tok, u = make(4, 3, 100, drafts)
    tok[0, 0], tok[1, 1], tok[2, 2] = 100, -1, 2 ** 31 - 1
    t, a = check(target, draft, tok, u)
    assert int(a[0]) == 0 and bool(((t < 100) & (t >= -1)).all())


def test_rows_without_weight():
    """Equal rows (nothing to resample), rows of zeros, and a certain token with all weight."""
    target, draft, tok, u = make(4, 2, 600)
    draft[0, 0] = target[0, 0]
    u[0, 0] = 1.0                                        # falls although the rows are equal
    target[1] = 0.0
    target[2, 0] = 0.0
    target[2, 0, 599] = 1.0
    t, a = check(target, draft, tok, u)
    assert int(t[0, 0]) == int(tok[0, 0])
    hot = torch.zeros((1, 3, 50))
    hot[0, :, 7] = 1.0
    x = torch.tensor([[7, 7]], dtype=torch.int32)
    t, a = check(hot, None, x, torch.tensor([[0.5, 1.0, 0.3]]))
    assert t.tolist() == [[7, 7, -1]] and int(a[0]) == 1
    t, a = check(torch.zeros((1, 1, 9)), None, torch.zeros((1, 0), dtype=torch.int32), torch.rand((1, 1)))
    assert t.tolist() == [[-1]]


def test_not_finite_weights_are_bounded():
    """A NaN counts as no weight; the answer stays a token of the vocabulary or -1."""
    target, draft, tok, u = make(4, 2, 700)
    target[0, 0, 5], draft[1, 0, 9], target[2, 0] = math.nan, math.nan, math.nan
    target[3, 1, 3] = math.inf
    t, a = kda.kda_verify_tokens(target.cuda(), draft.cuda(), tok.cuda(), u.cuda())
    torch.cuda.synchronize()
    assert bool(((t >= -1) & (t < 700)).all()) and bool(((a >= 0) & (a <= 2)).all())


def test_distribution_is_the_targets():
    """Many draws of one position: the first token follows the target within five standard
    deviations of a count, whatever the draft."""
    N, V = 40000, 8
    g = torch.Generator().manual_seed(3)
    p = torch.softmax(torch.randn(V, generator=g), 0)
    q = torch.softmax(torch.randn(V, generator=g), 0)
    tok = torch.multinomial(q, N, replacement=True, generator=g).reshape(N, 1).to(torch.int32)
    u = torch.rand((N, 2), generator=g)
    t, a = kda.kda_verify_tokens(p.expand(N, 2, V).contiguous().cuda(), q.expand(N, 1, V).contiguous().cuda(),
                                 tok.cuda(), u.cuda())
    count = torch.bincount(t[:, 0].long().cpu(), minlength=V).double()
    sd = (N * p.double() * (1 - p.double())).sqrt()
    assert bool(((count - N * p.double()).abs() <= 5 * sd).all())


def test_graph_and_stream():
    x = [None if t is None else t.cuda() for t in make(5, 3, 3001)]
    want = kda.kda_verify_tokens(*x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.kda_verify_tokens(*x, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = kda.kda_verify_tokens(*x)
    x[3].copy_(torch.rand(5, 4))
    g.replay()
    torch.cuda.synchronize()
    rt, ra = ref.verify(*[t.cpu() for t in x])
    assert torch.equal(res[0].cpu(), rt) and torch.equal(res[1].cpu(), ra)
