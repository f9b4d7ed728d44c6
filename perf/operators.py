"""The speculative-decoding operators around the verification attention, as
measured cases: attention of a batch that shares a prefix, verification of
drafted tokens, compaction of a KV cache, and page bookkeeping (fork, grow,
release).  `run` computes them in a plain form of elementary torch operations,
or, where `own` is true, through the library's entry points."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # Attention of sequences forked from one prompt.
        # A short prompt, two sequences, small heads: launch latency.
        dict(name="prefix_tiny", op="prefix", b=2, groups=1, hq=4, hkv=2, d=64, w=4,
             n_prefix=256, n_own=32, page=0, ragged=False, window=True),
        # One decoding token per sequence over a paged pool, a wide batch of
        # ragged continuations of one system prompt.
        dict(name="prefix_decode_b64", op="prefix", b=64, groups=1, hq=64, hkv=8, d=128, w=1,
             n_prefix=8192, n_own=1024, page=16, ragged=True, window=False),
        # A verification step of eight samples of one prompt, 7B-shaped, paged.
        dict(name="prefix_verify_7b", op="prefix", b=8, groups=1, hq=28, hkv=4, d=128, w=4,
             n_prefix=8192, n_own=512, page=16, ragged=True, window=True),
        # Several prompts with eight samples each, ragged prompts, 32B-shaped.
        dict(name="prefix_groups_32b", op="prefix", b=32, groups=4, hq=40, hkv=8, d=128, w=5,
             n_prefix=16384, n_own=700, page=64, ragged=True, window=True),
        # The 72B-shaped verification step over one long document, contiguous.
        dict(name="prefix_verify_72b", op="prefix", b=16, groups=1, hq=64, hkv=8, d=128, w=5,
             n_prefix=32768, n_own=2048, page=0, ragged=True, window=True),
        # Accepting or rejecting drafted tokens.
        # One sequence, a small vocabulary: latency.
        dict(name="tokens_one", op="tokens", b=1, w=4, vocab=32000, dtype="fp32", drafted=True,
             ragged=False),
        # An odd vocabulary in bf16, ragged draft lengths, a wide batch.
        dict(name="tokens_odd_bf16", op="tokens", b=64, w=8, vocab=50257, dtype="bf16",
             drafted=True, ragged=True),
        # The 72B-shaped step's batch over a large vocabulary.
        dict(name="tokens_152k", op="tokens", b=16, w=5, vocab=152064, dtype="fp32", drafted=True,
             ragged=False),
        # Keeping the selected positions of a cache only.
        # A 7B-shaped budget, in place, paged.
        dict(name="compact_7b_in_place", op="compact", layers=4, b=4, hkv=4, d=128, n=8192, k=512,
             page=16, in_place=True, ragged=True),
        # The 72B-shaped budget into another cache, contiguous.
        dict(name="compact_72b", op="compact", layers=4, b=16, hkv=8, d=128, n=32768, k=2048,
             page=0, in_place=False, ragged=False),
        # One turn of a serving loop's page bookkeeping: release the finished
        # continuations, fork new ones from the prompts, grow them by a window.
        dict(name="pages_small", op="pages", layers=2, parents=1, children=4, hkv=4, d=128,
             page=16, n=2051, grow=5, pool=1024),
        dict(name="pages_large", op="pages", layers=4, parents=4, children=64, hkv=8, d=128,
             page=16, n=32749, grow=5, pool=12288),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "tokens", "compact", "pages"])
    if op == "prefix":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 4, 5, 7, 8])
        groups = rng.choice([1, 1, 1, 2, 4])
        per = _log(rng, 1, 64 // groups)
        w, b = rng.choice([1, 2, 4, 5, 8]), groups * per
        longest = min(32768 // groups, 160000000 // (b * hq * w))
        return dict(op=op, b=b, groups=groups, hq=hq, hkv=hkv, d=rng.choice([64, 128]), w=w,
                    n_prefix=_log(rng, 100, longest), n_own=_log(rng, 1, 32768 // max(16, b)),
                    page=rng.choice([0, 16, 48, 64]), ragged=rng.random() < 0.7,
                    window=rng.random() < 0.6)
    if op == "tokens":
        return dict(op=op, b=_log(rng, 1, 64), w=rng.randint(1, 8), vocab=_log(rng, 1000, 152064),
                    dtype=rng.choice(["fp32", "bf16"]), drafted=rng.random() < 0.8,
                    ragged=rng.random() < 0.5)
    if op == "compact":
        n = _log(rng, 200, 16384)
        return dict(op=op, layers=rng.randint(1, 4), b=_log(rng, 1, 16),
                    hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), n=n,
                    k=rng.randint(1, max(1, n // 8)), page=rng.choice([0, 16, 48, 64]),
                    in_place=rng.random() < 0.5, ragged=rng.random() < 0.5)
    n, parents, children = _log(rng, 40, 8192), rng.randint(1, 4), _log(rng, 1, 64)
    page = rng.choice([16, 32, 64])
    need = parents * -(-n // page) + children * 3
    return dict(op=op, layers=rng.randint(1, 4), parents=parents, children=children,
                hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), page=page, n=n,
                grow=rng.randint(1, 20), pool=need + _log(rng, 8, 2048))


# ------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    return {"prefix": _prepare_prefix, "tokens": _prepare_tokens, "compact": _prepare_compact,
            "pages": _prepare_pages}[case["op"]](case, g)


def _prepare_prefix(c, g):
    b, groups, hq, hkv, d, w = (c[k] for k in ("b", "groups", "hq", "hkv", "d", "w"))
    n_p, n_o, page = c["n_prefix"], c["n_own"], c["page"]
    s = dict(c, scale=d ** -0.5, ws=None, q=_randn(g, b, hq, w, d), prefix_table=None,
             own_table=None, prefix_len=None, own_len=None)
    # Peaked attention, as long contexts show it: the first positions (sinks)
    # and a few heavy hitters lean towards the queries' mean direction.
    lean = s["q"].float().view(groups, b // groups, hkv, hq // hkv, w, d).mean((1, 3, 4))
    lean = (lean / lean.norm(dim=-1, keepdim=True)).view(groups, hkv, 1, d)
    hot = torch.rand((groups, 1, n_p, 1), generator=g, device=DEV) < 0.01
    push = 3.0 * hot.float()
    push[:, :, :4] = 6.0
    k = (_randn(g, groups, hkv, n_p, d).float() + push * lean).to(torch.bfloat16)
    v = _randn(g, groups, hkv, n_p, d)
    if page:
        pp, po = -(-n_p // page), -(-n_o // page)
        perm = torch.randperm(groups * pp + b * po, generator=g, device=DEV).to(torch.int32)
        s["prefix_table"] = perm[:groups * pp].view(groups, pp).contiguous()
        s["own_table"] = perm[groups * pp:].view(b, po).contiguous()
        s["k"] = _randn(g, groups * pp + b * po, hkv, page, d)
        s["v"] = _randn(g, groups * pp + b * po, hkv, page, d)
        at = torch.arange(n_p, device=DEV)
        pages = s["prefix_table"][:, at // page].long()                  # [groups][n_p]
        s["k"][pages, :, at % page] = k.transpose(1, 2)
        s["v"][pages, :, at % page] = v.transpose(1, 2)
    else:
        s["k"], s["v"] = k, v
        s["ko"], s["vo"] = _randn(g, b, hkv, n_o, d), _randn(g, b, hkv, n_o, d)
    if c["ragged"]:
        s["own_len"] = _randint(g, 0, n_o + 1, b)
        if groups > 1:
            s["prefix_len"] = _randint(g, (n_p + 1) // 2, n_p + 1, groups)
    s["kw"] = s["vw"] = None
    if c["window"]:
        s["kw"], s["vw"] = _randn(g, b, hkv, w, d), _randn(g, b, hkv, w, d)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((b, hq, w), device=DEV)
    return s


def _prepare_tokens(c, g):
    b, w, vocab = c["b"], c["w"], c["vocab"]
    logits = 2.5 * torch.randn((b, w, vocab), generator=g, device=DEV)
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits[:, :w - 1] + 0.7 * torch.randn((b, w - 1, vocab), generator=g,
                                                            device=DEV), -1)
    draft = torch.zeros((b, w - 1), dtype=torch.int32, device=DEV)
    if w > 1:
        draft = torch.multinomial(q.view(-1, vocab), 1, generator=g).view(b, w - 1).to(torch.int32)
    t = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    return dict(c, p=p.to(t), q=q.to(t) if c["drafted"] else None, draft=draft,
                n_draft=_randint(g, 0, w, b) if c["ragged"] else None,
                u=torch.rand((b, w - 1), generator=g, device=DEV),
                us=torch.rand((b,), generator=g, device=DEV),
                tokens=torch.empty((b, w), dtype=torch.int32, device=DEV),
                accepted=torch.empty((b,), dtype=torch.int32, device=DEV))


def _prepare_compact(c, g):
    b, hkv, d, n, k, page = (c[x] for x in ("b", "hkv", "d", "n", "k", "page"))
    s = dict(c, table=None, to_table=None, k_len=None)
    score = torch.rand((b, n), generator=g, device=DEV)
    score[:, :4] = 2.0                                                   # sinks stay
    s["idx"] = torch.sort(torch.topk(score, k).indices, -1).values.to(torch.int32)
    if c["ragged"]:
        s["k_len"] = _randint(g, 0, k + 1, b)
    rows, to_rows = (b, n), (b, k)
    if page:
        pn, pk = -(-n // page), -(-k // page)
        s["table"] = torch.randperm(b * pn, generator=g, device=DEV).to(torch.int32).view(b, pn)
        s["to_table"] = torch.randperm(b * pk, generator=g, device=DEV).to(torch.int32).view(b, pk)
        rows, to_rows = (b * pn, page), (b * pk, page)
    s["k_"] = [_randn(g, rows[0], hkv, rows[1], d) for _ in range(c["layers"])]
    s["v_"] = [_randn(g, rows[0], hkv, rows[1], d) for _ in range(c["layers"])]
    if c["in_place"]:
        s["to_k"], s["to_v"], s["to_table"] = s["k_"], s["v_"], s["table"]
    else:
        s["to_k"] = [torch.zeros((to_rows[0], hkv, to_rows[1], d), dtype=torch.bfloat16,
                                 device=DEV) for _ in range(c["layers"])]
        s["to_v"] = [torch.zeros_like(x) for x in s["to_k"]]
    return s


def _prepare_pages(c, g):
    page, n, np_, nc = c["page"], c["n"], c["parents"], c["children"]
    per = -(-(n + c["grow"]) // page)
    lens = _randint(g, max(1, n - n // 8), n + 1, np_)
    lens[0] = n
    perm = torch.randperm(c["pool"], generator=g, device=DEV).to(torch.int32)
    table = torch.full((np_ + nc, per), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(per, device=DEV)[None] * page < lens[:, None]
    table[:np_] = torch.where(held, perm[:np_ * per].view(np_, per), -1)
    seq_len = torch.cat([lens, torch.zeros(nc, dtype=torch.int32, device=DEV)])
    refcount = torch.zeros(c["pool"] + 1, dtype=torch.int32, device=DEV)
    refcount.index_add_(0, torch.where(held, table[:np_], c["pool"]).view(-1).long(),
                        torch.ones(np_ * per, dtype=torch.int32, device=DEV))
    child = torch.randperm(nc, generator=g, device=DEV).to(torch.int32) + np_
    parent = (torch.arange(nc, device=DEV) % np_).to(torch.int32)
    pools = [[_randn(g, c["pool"], c["hkv"], page, c["d"]) for _ in range(c["layers"])]
             for _ in range(2)]
    s = dict(c, table=table, seq_len=seq_len, refcount=refcount[:-1].contiguous(), parent=parent,
             child=child, zeros=torch.zeros_like(child),
             new_len=lens[parent.long()] + c["grow"], k_=pools[0], v_=pools[1],
             copies=torch.empty((nc, 2), dtype=torch.int32, device=DEV))
    _plain_pages(s)                                                      # a loop that already turns
    return s


# -------------------------------------------------------------- the plain forms

def run(state):
    op = state["op"]
    if own:
        return {"prefix": _own_prefix, "tokens": _own_tokens, "compact": _own_compact,
                "pages": _own_pages}[op](state)
    return {"prefix": _plain_prefix, "tokens": _plain_tokens, "compact": _plain_compact,
            "pages": _plain_pages}[op](state)


def _from_pages(pool, table, n):
    """[rows][h_kv][n][d] of a pool [pages][h_kv][page][d] through a table."""
    got = pool[table.long()].transpose(1, 2).flatten(2, 3)
    return got[:, :, :n]


def _plain_prefix(s):
    b, groups, hq, hkv, d, w = (s[k] for k in ("b", "groups", "hq", "hkv", "d", "w"))
    n_p, n_o, per, gw = s["n_prefix"], s["n_own"], b // groups, hq // hkv * w
    if s["page"]:
        kp, vp = (_from_pages(s[x], s["prefix_table"], n_p) for x in ("k", "v"))
        ko, vo = (_from_pages(s[x], s["own_table"], n_o) for x in ("k", "v"))
    else:
        kp, vp, ko, vo = s["k"], s["v"], s["ko"], s["vo"]
    q = s["q"].float().view(groups, per, hkv, gw, d) * s["scale"]
    shared = q.transpose(1, 2).reshape(groups, hkv, per * gw, d)
    rows = q.reshape(b, hkv, gw, d)

    def part(rows, k, v, seen):
        """Scores of one part, and its values, with unseen positions out."""
        sc = rows @ k.float().transpose(-1, -2)
        return torch.where(seen, sc, -math.inf), v.float()

    def seen(lens, n, count):
        at = torch.arange(n, device=DEV).view(1, 1, 1, n)
        return at < (lens.view(count, 1, 1, 1) if lens is not None else n)

    parts = [part(shared, kp, vp, seen(s["prefix_len"], n_p, groups)),
             part(rows, ko, vo, seen(s["own_len"], n_o, b))]
    if s["kw"] is not None:
        t = torch.arange(gw, device=DEV) % w
        causal = torch.arange(w, device=DEV)[None] <= t[:, None]
        parts.append(part(rows, s["kw"], s["vw"], causal))

    def by_row(x):
        """[groups][hkv][per * gw][..] or [b][hkv][gw][..] as [b][hkv][gw][..]."""
        if x.shape[2] == gw and x.shape[0] == b:
            return x
        return x.view(groups, hkv, per, gw, -1).transpose(1, 2).reshape(b, hkv, gw, -1)

    m = torch.cat([by_row(sc.amax(-1, keepdim=True)) for sc, _ in parts], -1).amax(-1, keepdim=True)
    safe = torch.where(torch.isinf(m), 0.0, m)
    to_shared = safe.view(groups, per, hkv, gw, 1).transpose(1, 2).reshape(groups, hkv, -1, 1)
    es = [torch.exp(parts[0][0] - to_shared)] + [torch.exp(sc - safe) for sc, _ in parts[1:]]
    total = sum(by_row(e.sum(-1, keepdim=True)) for e in es)
    out = sum(by_row(e @ v) for e, (_, v) in zip(es, parts))
    out = torch.where(total > 0, out / torch.where(total > 0, total, 1.0), 0.0)
    lse = torch.where(total > 0, safe + torch.log(total), -math.inf)
    return out.reshape(b, hq, w, d).to(torch.bfloat16), lse.reshape(b, hq, w)


def _plain_tokens(s):
    b, w = s["b"], s["w"]
    p, draft = s["p"], s["draft"].long()
    last = torch.full((b,), w - 1, device=DEV) if s["n_draft"] is None else s["n_draft"].long()
    row = torch.arange(b, device=DEV)
    n_acc = torch.zeros(b, dtype=torch.long, device=DEV)
    if w > 1:
        px = p[:, :w - 1].gather(-1, draft[..., None])[..., 0].double()
        qx = torch.ones_like(px) if s["q"] is None else \
            s["q"].gather(-1, draft[..., None])[..., 0].double()
        ok = (s["u"].double() * qx < px) & (torch.arange(w - 1, device=DEV) < last[:, None])
        n_acc = ok.long().cumprod(-1).sum(-1)
    mass = p[row, n_acc].double()
    rejected = (n_acc < last)[:, None]
    if w > 1:
        at = n_acc.clamp(max=w - 2)
        if s["q"] is None:
            gone = torch.zeros_like(mass).scatter_(1, draft[row, at][:, None], 1.0) * mass
        else:
            gone = s["q"][row, at].double()
        rest = torch.where(rejected, (mass - gone).clamp(min=0), mass)
        mass = torch.where(rest.sum(-1, keepdim=True) > 0, rest, mass)
    run_sum = mass.cumsum(-1)
    to = (run_sum <= s["us"].double()[:, None] * run_sum[:, -1:]).sum(-1)
    at = torch.arange(w, device=DEV)[None]
    padded = torch.cat([draft, torch.zeros((b, 1), dtype=torch.long, device=DEV)], 1)
    tokens = torch.where(at < n_acc[:, None], padded, torch.where(at == n_acc[:, None],
                                                                  to[:, None], -1))
    return tokens.to(torch.int32), n_acc.to(torch.int32)


def _plain_compact(s):
    b, k, page = s["b"], s["k"], s["page"]
    idx, at = s["idx"].long(), torch.arange(k, device=DEV)
    keep = torch.ones((b, k), dtype=torch.bool, device=DEV) if s["k_len"] is None else \
        at[None] < s["k_len"][:, None]
    row = torch.arange(b, device=DEV)[:, None].expand(b, k)
    if page:
        src = (s["table"].long().gather(1, idx // page), idx % page)
        dst = (s["to_table"].long()[:, at // page], (at % page).expand(b, k))
    else:
        src, dst = (row, idx), (row, at.expand(b, k))

    def moved(x, to):
        to[dst[0], :, dst[1]] = torch.where(keep[..., None, None], x[src[0], :, src[1]],
                                            to[dst[0], :, dst[1]])
        return to

    return [moved(x, to) for x, to in zip(s["k_"] + s["v_"], s["to_k"] + s["to_v"])]


def _plain_resize(s, seqs, new):
    table, seq_len, refcount, page = s["table"], s["seq_len"], s["refcount"], s["page"]
    pool, per = s["pool"], table.shape[1]
    old = seq_len[seqs].long()
    at = torch.arange(per, device=DEV)[None]
    had, have = -(-old // page), -(-new // page)
    spare = torch.cat([refcount, torch.zeros(1, dtype=torch.int32, device=DEV)])

    def count(where, pages, by):
        spare.index_add_(0, torch.where(where, pages.long(), pool).reshape(-1),
                         torch.full((where.numel(),), by, dtype=torch.int32, device=DEV))

    rows = table[seqs]
    dropped = (at >= have[:, None]) & (at < had[:, None])
    count(dropped, rows, -1)
    rows = torch.where(dropped, -1, rows)
    # A partly full last page that others hold too is copied before it grows.
    last = rows.gather(1, (had - 1).clamp(min=0)[:, None])[:, 0].long()
    cow = (new > old) & (old % page > 0) & (spare[torch.where(last < 0, pool, last)] > 1)
    need = cow.long() + (have - had).clamp(min=0)
    before = need.cumsum(0) - need
    order = torch.sort((spare[:pool] != 0).to(torch.uint8), stable=True).indices
    fresh = (at >= had[:, None]) & (at < have[:, None])
    rank = before[:, None] + cow[:, None] + at - had[:, None]
    rows = torch.where(fresh, order[rank.clamp(0, pool - 1)].to(torch.int32), rows)
    copy = order[before.clamp(max=pool - 1)]
    rows = torch.where(cow[:, None] & (at == had[:, None] - 1), copy[:, None].to(torch.int32), rows)
    count(fresh, rows, 1)
    count(cow, copy, 1)
    count(cow, last, -1)
    refcount.copy_(spare[:pool])
    table[seqs] = rows
    seq_len[seqs] = new.to(torch.int32)
    src, dst = torch.where(cow, last, -1), torch.where(cow, copy, -1)
    s["copies"].copy_(torch.stack([src, dst], 1))
    kept = rows[:, 0].clamp(min=0).long()                # the others copy a page onto itself
    src, dst = torch.where(cow, src, kept), torch.where(cow, dst, kept)
    return src, dst


def _plain_pages(s):
    parent, child = s["parent"].long(), s["child"].long()
    _plain_resize(s, child, torch.zeros_like(child))
    rows = s["table"][parent]
    s["table"][child] = rows
    s["seq_len"][child] = s["seq_len"][parent]
    spare = torch.cat([s["refcount"], torch.zeros(1, dtype=torch.int32, device=DEV)])
    spare.index_add_(0, torch.where(rows < 0, s["pool"], rows).view(-1).long(),
                     torch.ones(rows.numel(), dtype=torch.int32, device=DEV))
    s["refcount"].copy_(spare[:-1])
    src, dst = _plain_resize(s, child, s["new_len"].long())

    def copied(x):
        x[dst] = x[src]
        return x

    pools = [copied(x) for x in s["k_"] + s["v_"]]
    return [s["table"], s["seq_len"], s["refcount"], s["copies"]] + pools


# ----------------------------------------------------- through the entry points

def _native():
    from sparse_kv_verification_gb300 import native
    return native


def _own_prefix(s):
    N = _native()
    b, groups, hq, hkv, d, w = (s[k] for k in ("b", "groups", "hq", "hkv", "d", "w"))
    if s["ws"] is None:                                  # kept by the program, as its q and o
        s["ws"] = N.workspace(N.dustin_prefix_verify_attn_workspace_size(
            b, groups, hq, hkv, d, w, s["n_prefix"], s["n_own"]), DEV)
    prefix = N.kv_desc(s["k"], s["v"], s["prefix_table"])
    mine = N.kv_desc(s["k"], s["v"], s["own_table"]) if s["page"] else N.kv_desc(s["ko"], s["vo"])
    win = None if s["kw"] is None else N.kv_desc(s["kw"], s["vw"])
    N.dustin_prefix_verify_attn(s["q"], prefix, mine, hkv, groups, s["n_prefix"], s["n_own"],
                                s["scale"], s["o"], s["lse"], s["ws"], win=win,
                                prefix_len=s["prefix_len"], own_len=s["own_len"])
    return s["o"], s["lse"]


def _own_tokens(s):
    N = _native()
    N.dustin_verify_tokens(s["p"], s["q"], s["draft"], s["u"], s["us"], s["tokens"], s["accepted"],
                           n_draft=s["n_draft"])
    return s["tokens"], s["accepted"]


def _own_compact(s):
    N = _native()
    src = [N.kv_desc(k, v, s["table"]) for k, v in zip(s["k_"], s["v_"])]
    dst = src if s["in_place"] else [N.kv_desc(k, v, s["to_table"])
                                     for k, v in zip(s["to_k"], s["to_v"])]
    N.dustin_kv_compact(src, dst, s["hkv"], s["d"], s["n"], s["idx"], k_len=s["k_len"])
    return s["to_k"] + s["to_v"]


def _own_pages(s):
    N = _native()
    kvs = [N.kv_desc(k, v, s["table"]) for k, v in zip(s["k_"], s["v_"])]
    book = (s["table"], s["seq_len"], s["refcount"], s["page"])
    N.dustin_kv_resize(*book, s["child"], s["zeros"], s["copies"])
    N.dustin_kv_fork(*book, s["parent"], s["child"])
    N.dustin_kv_resize(*book, s["child"], s["new_len"], s["copies"], kvs=kvs, h_kv=s["hkv"],
                       d=s["d"])
    return [s["table"], s["seq_len"], s["refcount"], s["copies"]] + s["k_"] + s["v_"]


# ------------------------------------------------------------------ their work

def work(c):
    if c["op"] == "prefix":
        # Ragged lengths count with their mean.
        n_o = c["n_own"] / 2 if c["ragged"] else c["n_own"]
        n_p = c["n_prefix"] * (0.75 if c["ragged"] and c["groups"] > 1 else 1.0)
        n_w = c["w"] if c["window"] else 0
        rows = c["b"] * c["hq"] * c["w"]
        kv = c["hkv"] * c["d"] * 4
        return {"bytes": kv * (c["groups"] * n_p + c["b"] * (n_o + n_w))
                + rows * (4 * c["d"] + 4),
                "flops": 4.0 * rows * c["d"] * (n_p + n_o + ((c["w"] + 1) / 2 if n_w else 0))}
    if c["op"] == "tokens":
        size = 4 if c["dtype"] == "fp32" else 2
        rows = 2 if c["drafted"] and c["w"] > 1 else 1
        return {"bytes": c["b"] * (rows * c["vocab"] * size + c["w"] * 16),
                "flops": 2.0 * c["b"] * rows * c["vocab"]}
    if c["op"] == "compact":
        k = c["k"] / 2 if c["ragged"] else c["k"]
        return {"bytes": c["b"] * k * (c["layers"] * c["hkv"] * c["d"] * 8 + 4), "flops": 0}
    entries = c["children"] * -(-c["n"] // c["page"])
    page = c["hkv"] * c["page"] * c["d"] * 2
    return {"bytes": entries * 2 * 16 + 4 * c["pool"] + c["children"] * c["layers"] * page * 4,
            "flops": 0}


# ------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    if case["op"] == "prefix":
        return _exact_prefix(prepare(case, seed))
    if case["op"] == "tokens":
        return _exact_tokens(prepare(case, seed))
    return None                                          # moved values, nothing computed


def _exact_prefix(s):
    """Sequence by sequence and kv head by kv head: all the keys a sequence
    sees laid one after another, then the softmax's definition in 64 bits."""
    b, hq, hkv, d, w = (s[k] for k in ("b", "hq", "hkv", "d", "w"))
    o = torch.zeros((b, hq, w, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((b, hq, w), dtype=torch.float64, device=DEV)
    per, gr = b // s["groups"], hq // hkv

    def rows(pool, own_pool, table, i, h, n):
        """The first n rows of kv head h of cache row i."""
        if table is None:
            return own_pool[i, h, :n]
        j = torch.arange(n, device=DEV)
        return pool[table[i][j // s["page"]].long(), h, j % s["page"]]

    for i in range(b):
        n_p = s["n_prefix"] if s["prefix_len"] is None else int(s["prefix_len"][i // per])
        n_o = s["n_own"] if s["own_len"] is None else int(s["own_len"][i])
        for h in range(hkv):
            ks, vs = ([rows(s[x], s[x], s["prefix_table"], i // per, h, n_p),
                       rows(s[x], s.get(x + "o"), s["own_table"], i, h, n_o)] for x in ("k", "v"))
            if s["kw"] is not None:
                ks.append(s["kw"][i, h])
                vs.append(s["vw"][i, h])
            k, v = torch.cat(ks).double(), torch.cat(vs).double()
            q = s["q"][i, h * gr:(h + 1) * gr].double()                  # [group][w][d]
            x = torch.einsum("gtd,nd->gtn", q, k) * s["scale"]
            if s["kw"] is not None:
                later = torch.ones((w, w), dtype=torch.bool, device=DEV).triu(1)
                x[:, :, n_p + n_o:].masked_fill_(later, -math.inf)
            z = torch.logsumexp(x, -1)
            weights = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[..., None])
            o[i, h * gr:(h + 1) * gr] = torch.einsum("gtn,nd->gtd", weights, v)
            lse[i, h * gr:(h + 1) * gr] = z
    return o, lse


def _exact_tokens(s):
    b, w = s["b"], s["w"]
    p, draft = s["p"].double().cpu().numpy(), s["draft"].cpu().numpy()
    q = None if s["q"] is None else s["q"].double().cpu().numpy()
    u, us = s["u"].double().cpu().numpy(), s["us"].double().cpu().numpy()
    lens = np.full(b, w - 1) if s["n_draft"] is None else s["n_draft"].cpu().numpy()
    tokens, accepted = np.full((b, w), -1, np.int32), np.zeros(b, np.int32)
    for i in range(b):
        a = 0
        while a < lens[i]:
            x = draft[i, a]
            if not u[i, a] * (1.0 if q is None else q[i, a, x]) < p[i, a, x]:
                break
            tokens[i, a] = x
            a += 1
        mass = p[i, a]
        if a < lens[i]:
            less = mass.copy()
            if q is None:
                less[draft[i, a]] = 0.0
            else:
                less = np.maximum(less - q[i, a], 0.0)
            mass = less if less.sum() > 0 else mass
        run_sum = np.cumsum(mass)
        tokens[i, a] = np.searchsorted(run_sum, us[i] * run_sum[-1], side="right")
        accepted[i] = a
    return tokens, accepted
