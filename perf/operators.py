"""The serving operators beside Kimi Delta Attention: cases, plain forms and 64-bit values.

Three operators of one serving step of a model that mixes KDA layers with latent attention:

  append   the new tokens' latent rows, normed and rotated, written to a paged cache, with
           the queries' rotated parts in the same call (kda_latent_append)
  attn     absorbed latent attention of each sequence's new tokens over its cache pages
           (kda_latent_attn)
  verify   drafted tokens against the target's probabilities, from given random numbers
           (kda_verify_tokens)

`own` False computes them in elementary torch operations, `own` True through the package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one user's decode step with a short context: latency
        dict(name="attn_token_one", op="attn", dtype="bf16", N=1, L=1, H=12, rank=512, rope=64,
             page=64, ctx_lo=1000, ctx_hi=1000, packed=False),
        # a full decode batch, one token each, heads split over eight GPUs, ragged contexts
        dict(name="attn_token_pool", op="attn", dtype="bf16", N=256, L=1, H=12, rank=512, rope=64,
             page=64, ctx_lo=0, ctx_hi=8192, packed=False),
        # all 96 heads on one GPU at the concurrency its state pool allows
        dict(name="attn_token_96_heads", op="attn", dtype="bf16", N=43, L=1, H=96, rank=512,
             rope=64, page=64, ctx_lo=100, ctx_hi=16384, packed=False),
        # checking four drafted tokens a sequence, small pages
        dict(name="attn_drafts", op="attn", dtype="bf16", N=64, L=4, H=12, rank=512, rope=64,
             page=16, ctx_lo=4, ctx_hi=8192, packed=False),
        # a prefill chunk of ragged packed sequences behind long contexts: bound by the products
        dict(name="attn_chunk", op="attn", dtype="bf16", N=3, L=1024, H=12, rank=512, rope=64,
             page=64, ctx_lo=8192, ctx_hi=32768, packed=True),
        # single precision, smaller latent without a rotated part
        dict(name="attn_token_f32", op="attn", dtype="f32", N=16, L=1, H=12, rank=256, rope=0,
             page=32, ctx_lo=1, ctx_hi=4096, packed=False),
        # one new token of each sequence of a decode batch
        dict(name="append_token_pool", op="append", dtype="bf16", N=256, L=1, H=12, rank=512,
             rope=64, page=64, ctx_lo=1, ctx_hi=8192, packed=False, norm=True, interleaved=False),
        # a prefill chunk of ragged packed sequences
        dict(name="append_chunk", op="append", dtype="bf16", N=5, L=16384, H=12, rank=512, rope=64,
             page=64, ctx_lo=0, ctx_hi=65536, packed=True, norm=True, interleaved=False),
        # single precision, interleaved pairs, odd sizes
        dict(name="append_f32", op="append", dtype="f32", N=7, L=1001, H=5, rank=256, rope=64,
             page=48, ctx_lo=0, ctx_hi=131072, packed=True, norm=False, interleaved=True),
        # one user's drafted tokens: latency
        dict(name="verify_one", op="verify", dtype="f32", N=1, L=4, V=32000, drafts=True),
        # a batch of drafted sequences, odd vocabulary
        dict(name="verify_pool", op="verify", dtype="f32", N=256, L=4, V=100277, drafts=True),
        # drafts without probabilities (a lookup in the text), more tokens a sequence
        dict(name="verify_lookup", op="verify", dtype="f32", N=43, L=8, V=131072, drafts=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "verify"])
    if op == "verify":
        V = _log_int(rng, 1000, 160000)
        L = rng.randint(1, 8)
        N = _log_int(rng, 1, max(1, min(256, 130_000_000 // (V * (L + 1)))))
        return dict(op="verify", dtype="f32", N=N, L=L, V=V, drafts=rng.random() < 0.7)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    H = rng.choice([1, 4, 5, 8, 12, 16, 24, 32, 48, 96])
    rank = rng.choice([512, 512, 512, 256, 128, 384])
    rope = rng.choice([64, 64, 0])
    page = rng.choice([16, 32, 48, 64, 64, 128, 24])
    if op == "append":
        packed = rng.random() < 0.5
        N = _log_int(rng, 1, 16 if packed else 256)
        L = _log_int(rng, 1, 16384 if packed else 16)
        return dict(op="append", dtype=dtype, N=N, L=L, H=H, rank=rank, rope=rope, page=page,
                    ctx_lo=rng.randint(0, 40), ctx_hi=_log_int(rng, 64, 16384), packed=packed,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.5)
    packed = rng.random() < 0.3
    most = 8.0e9 if dtype == "f32" else 2.2e11             # products of one call
    if packed:
        N, L = _log_int(rng, 1, 8), _log_int(rng, 8, 1024)
        rows = L * H
    else:
        N, L = _log_int(rng, 1, 256), rng.choice([1, 1, 1, 2, 3, 4, 8, 16])
        rows = N * L * H
    hi = int(min(32768, most / (rows * (2 * rank + rope)), 4_000_000_000 / (N * (rank + rope) * 4)))
    if hi < 64:
        N, L, packed, hi = 1, 1, False, 4096
    return dict(op="attn", dtype=dtype, N=N, L=L, H=H, rank=rank, rope=rope, page=page,
                ctx_lo=rng.randint(0, 64), ctx_hi=_log_int(rng, 64, hi), packed=packed)


# --------------------------------------------------------------------------- inputs

def _lengths(case):
    """New tokens and cached tokens (the new ones included) of each sequence: a fixed
    spread over the case's range, so that every seed asks for the same work."""
    N, L = case["N"], case["L"]
    lo, hi = case["ctx_lo"], case["ctx_hi"]
    gen = torch.Generator().manual_seed(1234 + N)
    if case["packed"]:                      # L tokens in all, cut at N - 1 places
        cuts = sorted(torch.randint(0, L + 1, (N - 1,), generator=gen).tolist())
        ends = [0] + cuts + [L]
        new = [b - a for a, b in zip(ends, ends[1:])]
    else:
        new = [L] * N
    share = torch.rand(N, generator=gen).tolist()
    total = []
    for n in range(N):
        c = lo + int(round((hi - lo) * share[n]))
        # a sequence that has no cached token is a padding slot of the batch
        total.append(0 if c == 0 and not case["packed"] else max(c, new[n]))
    return new, total


def _pages(case, total, gen):
    """A shuffled page table, as an allocator leaves it after many sequences came and went."""
    page = case["page"]
    need = [max(1, -(-t // page)) for t in total]
    P = max(need)
    ids = torch.randperm(sum(need) + 3, generator=gen)[: sum(need)].to(torch.int32)
    table = torch.zeros((case["N"], P), dtype=torch.int32)
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = ids[at:at + k]
        at += k
    return sum(need) + 3, table


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    if case["op"] == "verify":
        N, L, V = case["N"], case["L"], case["V"]
        logits = torch.randn((N, L + 1, V), generator=g, device=dev).mul_(2.0)
        target = torch.softmax(logits, -1)
        st = {"case": case, "target": target}
        u = torch.rand((N, L + 1), generator=g, device=dev)
        if case["drafts"]:
            draft = logits[:, :L].mul_(0.8)
            draft.add_(torch.randn((N, L, V), generator=g, device=dev), alpha=0.8)
            draft = torch.softmax(draft, -1)
            tokens = torch.multinomial(draft.reshape(N * L, V), 1, generator=g).reshape(N, L)
        else:
            # a lookup that is right more often than not
            draft = None
            tokens = torch.where(torch.rand((N, L), generator=g, device=dev) < 0.7,
                                 target[:, :L].argmax(-1),
                                 torch.randint(0, V, (N, L), generator=g, device=dev))
        st.update(draft=draft, tokens=tokens.to(torch.int32), u=u)
        return st
    dt = DTYPES[case["dtype"]]
    N, L, H, rank, rope = case["N"], case["L"], case["H"], case["rank"], case["rope"]
    D = rank + rope
    new, total = _lengths(case)
    pages, table = _pages(case, total, cpu)
    # cached latents come out of a norm: of the order of one
    cache = torch.randn((pages, case["page"], D), generator=g, device=dev, dtype=dt)
    shape = (1, L) if case["packed"] else (N, L)
    st = {"case": case, "cache": cache, "table": table.to(dev), "new": new, "total": total,
          "lens": torch.tensor(total, dtype=torch.int32, device=dev),
          "cu": None}
    if case["packed"]:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["op"] == "attn":
        st["q"] = torch.randn((*shape, H, D), generator=g, device=dev).to(dt)
        # scores of a few units, with some tokens well ahead, as trained heads have
        st["scale"] = 2.0 / math.sqrt(D)
        return st
    st["kv"] = (3.0 * torch.randn((*shape, D), generator=g, device=dev)).to(dt)
    st["weight"] = (1.0 + 0.1 * torch.randn(rank, generator=g, device=dev)) if case["norm"] else None
    st["freq"] = st["q_pe"] = st["q"] = None
    if rope:
        st["freq"] = (10000.0 ** (-torch.arange(0, rope, 2, device=dev).double() / rope)).float()
        st["q_pe"] = torch.randn((*shape, H, rope), generator=g, device=dev).to(dt)
        # the absorbed queries, whose last columns take the rotated part
        st["q"] = torch.zeros((*shape, H, D), device=dev, dtype=dt)
    return st


# --------------------------------------------------------------------------- plain forms

def _keys(st, n):
    page, t = st["case"]["page"], st["total"][n]
    ids = st["table"][n, : -(-t // page)].long()
    return st["cache"][ids].reshape(-1, st["cache"].shape[-1])[:t]


def _attn_plain(st):
    c, q = st["case"], st["q"]
    rank, H = c["rank"], c["H"]
    rows = q.reshape(-1, H, q.shape[-1])
    out = torch.zeros((rows.shape[0], H, rank), dtype=q.dtype, device=q.device)
    lse = torch.full((rows.shape[0], H), -math.inf, device=q.device)
    at = 0
    for n, new in enumerate(st["new"]):
        t, a, at = st["total"][n], at, at + new
        if new == 0 or t == 0:
            continue
        k = _keys(st, n).float()
        qs = rows[a:at].reshape(new * H, -1).float()
        s = (qs @ k.T).reshape(new, H, t) * st["scale"]
        if new > 1:
            last = torch.arange(t - new, t, device=q.device)
            s.masked_fill_(torch.arange(t, device=q.device) > last[:, None, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = s.sub_(m).exp_()
        z = p.sum(-1, keepdim=True)
        o = (p.reshape(new * H, t) @ k[:, :rank]).reshape(new, H, rank)
        out[a:at] = torch.where(z > 0, o / z, torch.zeros_like(o)).to(q.dtype)
        lse[a:at] = (m + z.log()).squeeze(-1)
    return (out.reshape(*q.shape[:-1], rank), lse.reshape(q.shape[:-1]))


def _positions(st):
    pos, seq = [], []
    for n, (new, t) in enumerate(zip(st["new"], st["total"])):
        pos += [torch.arange(t - new, t)]
        seq += [torch.full((new,), n)]
    return torch.cat(pos).to(st["kv"].device), torch.cat(seq).to(st["kv"].device)


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _append_plain(st):
    c, kv = st["case"], st["kv"]
    rank = c["rank"]
    pos, seq = _positions(st)
    x = kv.reshape(-1, kv.shape[-1]).float()
    y = x[:, :rank]
    if c["norm"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * st["weight"]
    if c["rope"]:
        angle = pos.double()[:, None] * st["freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()
        y = torch.cat((y, _rotate(x[:, rank:], cos, sin, c["interleaved"])), -1)
        qp = st["q_pe"].reshape(len(pos), c["H"], -1).float()
        qr = _rotate(qp, cos[:, None], sin[:, None], c["interleaved"])
        st["q"][..., rank:] = qr.to(kv.dtype).reshape(st["q_pe"].shape)
    keep = pos >= 0
    pos, seq, y = pos[keep], seq[keep], y[keep]
    ids = st["table"][seq, pos // c["page"]].long()
    st["cache"][ids, pos % c["page"]] = y.to(kv.dtype)
    return [st["cache"]] if st["q"] is None else [st["cache"], st["q"]]


def _verify_plain(st):
    p, q, x, u = st["target"], st["draft"], st["tokens"].long(), st["u"].double()
    N, L = x.shape
    px = p[:, :L].gather(2, x[..., None])[..., 0].double()
    qx = torch.ones_like(px) if q is None else q.gather(2, x[..., None])[..., 0].double()
    acc = (u[:, :L] * qx < px).long().cumprod(1).sum(1)
    n = torch.arange(N, device=p.device)
    r = p[n, acc].double()
    j = acc.clamp(max=L - 1)
    if q is None:
        minus = torch.zeros_like(r).scatter_(1, x[n, j][:, None], math.inf)
    else:
        minus = q[n, j].double()
    r = torch.where((acc < L)[:, None], (r - minus).clamp(min=0), r)
    cum = r.cumsum(1)
    last = (cum > u[:, L, None] * cum[:, -1:]).long().argmax(1)
    place = torch.arange(L + 1, device=p.device)
    toks = torch.cat((x, x[:, :1]), 1)
    toks = torch.where(place == acc[:, None], last[:, None], toks)
    toks = torch.where(place > acc[:, None], torch.full_like(toks, -1), toks)
    return toks.to(torch.int32), acc.to(torch.int32)


def run(state):
    case = state["case"]
    if own:
        import gated_delta_rule_74_b200 as kda
        if case["op"] == "attn":
            return kda.kda_latent_attn(state["q"], state["cache"], state["table"], state["lens"],
                                       rank=case["rank"], scale=state["scale"],
                                       cu_seqlens=state["cu"])
        if case["op"] == "append":
            rank, q = case["rank"], state["q"]
            kda.kda_latent_append(state["kv"], state["cache"], state["table"], state["lens"],
                                  rank=rank, cu_seqlens=state["cu"], norm_weight=state["weight"],
                                  eps=1e-6, inv_freq=state["freq"],
                                  interleaved=case["interleaved"], q_pe=state["q_pe"],
                                  q_pe_out=None if q is None else q[..., rank:])
            return [state["cache"]] if q is None else [state["cache"], q]
        return kda.kda_verify_tokens(state["target"], state["draft"], state["tokens"], state["u"])
    return {"attn": _attn_plain, "append": _append_plain, "verify": _verify_plain}[case["op"]](state)


# --------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "verify":
        # the row that the last token is drawn from, of the target and, after a rejection, of
        # the draft (about three drafts in four stand)
        N, L, V = case["N"], case["L"], case["V"]
        rejected = 1.0 - 0.75 ** L if case["drafts"] else 0.0
        return {"bytes": 4.0 * N * (V * (1.0 + rejected) + 4 * L + 2 * (L + 1)),
                "flops": 2.0 * N * V}
    e = 2 if case["dtype"] == "bf16" else 4
    new, total = _lengths(case)
    D, H = case["rank"] + case["rope"], case["H"]
    toks = sum(new)
    if case["op"] == "append":
        q = 2 * toks * H * case["rope"]
        return {"bytes": float(e * (2 * toks * D + q)), "flops": float(toks * (4 * D + 3 * H * case["rope"]))}
    keys = sum(t for n, t in zip(new, total) if n)
    pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, total) if t)
    return {"bytes": float(e * (keys * D + toks * H * (D + case["rank"])) + 4 * toks * H),
            "flops": 2.0 * pairs * H * (2 * case["rank"] + case["rope"])}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "verify":
        return _verify_exact(st)
    if case["op"] == "append":
        return _append_exact(st)
    if work(case)["flops"] > 1e12:
        return None
    q, H, rank = st["q"].double(), case["H"], case["rank"]
    B, T = q.shape[:2]
    out = torch.zeros((B * T, H, rank), dtype=torch.float64, device=q.device)
    lse = torch.full((B * T, H), -math.inf, dtype=torch.float64, device=q.device)
    q = q.reshape(B * T, H, -1)
    first = 0
    for n, (new, t) in enumerate(zip(st["new"], st["total"])):
        if t:
            slot = torch.arange(t, device=q.device)
            page = st["table"][n].long()[slot // case["page"]]
            c = st["cache"][page, slot % case["page"]].double()
            for a in range(0, new, 256):            # the formula, a run of tokens at a time
                b = min(new, a + 256)
                sc = torch.einsum("ihd,jd->ihj", q[first + a:first + b], c) * st["scale"]
                sees = slot[None] <= torch.arange(t - new + a, t - new + b, device=q.device)[:, None]
                sc = torch.where(sees[:, None], sc, torch.full((), -math.inf, dtype=sc.dtype, device=sc.device))
                z = torch.logsumexp(sc, -1)
                w = torch.where(sees[:, None], (sc - z[..., None]).exp(), torch.zeros((), dtype=sc.dtype, device=sc.device))
                out[first + a:first + b] = torch.einsum("ihj,jd->ihd", w, c[:, :rank])
                lse[first + a:first + b] = z
        first += new
    return (out.reshape(B, T, H, rank), lse.reshape(B, T, H))


def _append_exact(st):
    case, rank, rope = st["case"], st["case"]["rank"], st["case"]["rope"]
    cache = st["cache"].double()
    kv = st["kv"].double().reshape(-1, rank + rope)
    where = [(n, t - new + i) for n, (new, t) in enumerate(zip(st["new"], st["total"])) for i in range(new)]
    seq = torch.tensor([w[0] for w in where], device=kv.device)
    pos = torch.tensor([w[1] for w in where], device=kv.device)
    lat = kv[:, :rank]
    if case["norm"]:
        lat = lat / torch.sqrt((lat * lat).sum(-1, keepdim=True) / rank + 1e-6) * st["weight"].double()
    row = lat
    q = None
    if rope:
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=kv.device),
                           torch.outer(pos.double(), st["freq"].double()))

        def turned(x, by):
            if case["interleaved"]:
                z = torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2).contiguous()) * by
                return torch.view_as_real(z).reshape(x.shape)
            z = torch.complex(x[..., : rope // 2].contiguous(), x[..., rope // 2:].contiguous()) * by
            return torch.cat((z.real, z.imag), -1)

        row = torch.cat((lat, turned(kv[:, rank:], turn)), -1)
        qp = st["q_pe"].double().reshape(len(where), case["H"], rope)
        q = st["q"].double()
        q[..., rank:] = turned(qp, turn[:, None]).reshape(st["q_pe"].shape)
    ok = pos >= 0
    slot = st["table"][seq[ok], pos[ok] // case["page"]].long() * case["page"] + pos[ok] % case["page"]
    cache.view(-1, rank + rope)[slot] = row[ok]
    return [cache] if q is None else [cache, q]


def _verify_exact(st):
    p, q, u = st["target"], st["draft"], st["u"].double().cpu()
    x = st["tokens"].cpu()
    N, L = x.shape
    toks = torch.full((N, L + 1), -1, dtype=torch.int32)
    count = torch.zeros(N, dtype=torch.int32)
    for n in range(N):
        i = 0
        while i < L:
            t = int(x[n, i])
            qx = 1.0 if q is None else float(q[n, i, t])
            if not float(u[n, i]) * qx < float(p[n, i, t]):
                break
            toks[n, i] = t
            i += 1
        left = p[n, i].double().cpu()
        if i < L:
            if q is None:
                left[int(x[n, i])] = 0.0
            else:
                left = torch.relu(left - q[n, i].double().cpu())
        cum = torch.cumsum(left, 0)
        toks[n, i] = int(torch.searchsorted(cum, float(u[n, L]) * float(cum[-1]), right=True))
        count[n] = i
    return toks.cuda(), count.cuda()
