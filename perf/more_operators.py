"""The operators of a cache held in 4 bits (rows quantised as they are written,
rows read back, verification attention over it) and the log probabilities of
given tokens, as measured cases.  `run` computes them in a plain form of
elementary torch operations, or, where `own` is true, through the library's
entry points.

A 4-bit cache holds one record per (position, kv head): the codes of K (two
channels to a byte, the lower one in the lower bits), those of V, one scale per
16 channels of K, then of V, zeros up to a multiple of 16 bytes.  A value is
e2m1(code) * e4m3(scale) * 2^exponent."""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # Rows quantised into the cache and read back.
        # One new token of one layer, one sequence: launch latency.
        dict(name="write_one", op="write", layers=1, b=1, hkv=4, d=128, n=2048, w=1, page=16,
             ragged=False, k_exp=0, v_exp=0),
        # The accepted rows of a verification step's window, 16 layers at once,
        # behind caches of different lengths, 72B-shaped.
        dict(name="write_accepted", op="write", layers=16, b=16, hkv=8, d=128, n=2048, w=5,
             page=16, ragged=True, k_exp=0, v_exp=-4),
        # A long prompt of an odd length after its prefill.
        dict(name="write_prompt", op="write", layers=4, b=1, hkv=8, d=128, n=32749, w=32749,
             page=0, ragged=False, k_exp=0, v_exp=0),
        # Rows read back as bf16.
        # The budget of one short sequence, small heads: latency.
        dict(name="read_small", op="read", layers=1, b=1, hkv=2, d=64, n=1000, k=128, page=16,
             sparse=True, ragged=False, k_exp=2, v_exp=0),
        # The selected positions of 72B-shaped caches.
        dict(name="read_selected", op="read", layers=2, b=16, hkv=8, d=128, n=16384, k=2048,
             page=0, sparse=True, ragged=True, k_exp=0, v_exp=0),
        # Attention over the cache.
        # One token of one short sequence, small heads: launch latency.
        dict(name="attn_one", op="attn", b=1, hq=4, hkv=2, d=64, w=1, n=300, k=300, page=16,
             sparse=False, ragged=False, window=True),
        # One decoding token per sequence, a wide batch of ragged lengths in pages.
        dict(name="attn_decode_b64", op="attn", b=64, hq=64, hkv=8, d=128, w=1, n=8192, k=8192,
             page=16, sparse=False, ragged=True, window=False),
        # The 72B-shaped verification step over its selected positions.
        dict(name="attn_sparse_72b", op="attn", b=16, hq=64, hkv=8, d=128, w=5, n=32768, k=2048,
             page=0, sparse=True, ragged=False, window=True),
        # The same over the whole cache.
        dict(name="attn_dense_72b", op="attn", b=16, hq=64, hkv=8, d=128, w=5, n=32768, k=32768,
             page=0, sparse=False, ragged=False, window=True),
        # Log probabilities, entropy and the most likely alternatives.
        # One sequence's drafts, a small vocabulary: latency.
        dict(name="logprobs_one", op="logprobs", b=1, w=4, vocab=32000, dtype="fp32", m=1, top=5,
             ragged=False, banned=False),
        # An odd vocabulary in bf16, ragged windows, banned tokens, a wide batch.
        dict(name="logprobs_odd_bf16", op="logprobs", b=64, w=8, vocab=50257, dtype="bf16", m=2,
             top=20, ragged=True, banned=True),
        # A prompt's tokens over a large vocabulary.
        dict(name="logprobs_prompt", op="logprobs", b=2, w=1024, vocab=152064, dtype="bf16", m=1,
             top=1, ragged=False, banned=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn", "logprobs", "logprobs"])
    d, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    page = rng.choice([0, 16, 48, 64])
    exps = dict(k_exp=rng.randint(-6, 3), v_exp=rng.randint(-6, 3))
    if op == "write":
        layers, b = _log(rng, 1, 16), _log(rng, 1, 32)
        w = _log(rng, 1, max(2, 60000 // (layers * b)))
        return dict(op=op, layers=layers, b=b, hkv=hkv, d=d, n=w + rng.randint(0, 1000), w=w,
                    page=page, ragged=rng.random() < 0.5, **exps)
    if op == "read":
        layers, b = rng.randint(1, 4), _log(rng, 1, 16)
        n = _log(rng, 100, 16384)
        return dict(op=op, layers=layers, b=b, hkv=hkv, d=d, n=n,
                    k=_log(rng, 1, max(2, min(n, 65536 // (layers * b)))), page=page,
                    sparse=rng.random() < 0.6, ragged=rng.random() < 0.5, **exps)
    if op == "attn":
        hq = hkv * rng.choice([1, 4, 5, 7, 8])
        b, w = _log(rng, 1, 64), rng.choice([1, 1, 2, 4, 5, 8])
        n = _log(rng, 1, min(32768, 524288 // b, 160000000 // (b * hq * w)))
        sparse = rng.random() < 0.4
        return dict(op=op, b=b, hq=hq, hkv=hkv, d=d, w=w, n=n,
                    k=_log(rng, 1, n) if sparse else n, page=page, sparse=sparse,
                    ragged=rng.random() < 0.5, window=rng.random() < 0.5)
    b, vocab = _log(rng, 1, 128), _log(rng, 500, 152064)
    return dict(op=op, b=b, w=_log(rng, 1, max(2, min(64, 150000000 // (b * vocab)))), vocab=vocab,
                dtype=rng.choice(["fp32", "bf16"]), m=rng.randint(0, 4),
                top=rng.choice([0, 1, 5, 20, 64]), ragged=rng.random() < 0.5,
                banned=rng.random() < 0.5)


# ------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _record(d):
    return -(-(d + d // 8) // 16) * 16


def prepare(case, seed):
    g = _gen(seed)
    return {"write": _prepare_write, "read": _prepare_read, "attn": _prepare_attn,
            "logprobs": _prepare_logprobs}[case["op"]](case, g)


def _keys(g, *shape):
    """Keys as models have them: a few channels much larger than the others."""
    big = torch.rand((shape[1], 1, shape[3]), generator=g, device=DEV) < 0.04
    return _randn(g, *shape) * torch.where(big, 6.0, 1.0).to(torch.bfloat16)


def _cache(c, b, n, g):
    """An empty cache for n positions, and its page table."""
    rec, page = _record(c["d"]), c["page"]
    if not page:
        return torch.zeros((b, c["hkv"], n, rec), dtype=torch.uint8, device=DEV), None
    per = -(-n // page)
    table = torch.randperm(b * per, generator=g, device=DEV).to(torch.int32).view(b, per)
    return torch.zeros((b * per, c["hkv"], page, rec), dtype=torch.uint8, device=DEV), table


def _prepare_write(c, g):
    b, hkv, d, n, w = (c[k] for k in ("b", "hkv", "d", "n", "w"))
    s = dict(c, start=None, w_len=None, idx=None)
    _, s["table"] = _cache(c, b, n, g)
    s["caches"] = [_cache(dict(c), b, n, g)[0] for _ in range(c["layers"])]
    s["k_"] = [_keys(g, b, hkv, w, d) for _ in range(c["layers"])]
    s["v_"] = [_randn(g, b, hkv, w, d) * 2.0 ** c["v_exp"] for _ in range(c["layers"])]
    if n > w:
        s["start"] = _randint(g, 0, n - w + 1, b)
        s["idx"] = s["start"][:, None] + torch.arange(w, device=DEV, dtype=torch.int32)
    if c["ragged"]:
        s["w_len"] = _randint(g, 0, w + 1, b)
    s["back"] = [torch.zeros((b, hkv, w, d), dtype=torch.bfloat16, device=DEV)
                 for _ in range(2 * c["layers"])]
    return s


def _filled(c, s, k, v, cache, g):
    """The cache with rows [0, n) of k and v."""
    at = torch.arange(k.shape[2], device=DEV)
    # One sequence at a time: the temporaries of a long batch are large.
    for i in range(k.shape[0]):
        rows = _quantised(k[i], v[i], c["d"], s["k_exp"], s["v_exp"])
        if s["table"] is None:
            cache[i] = rows
        else:
            cache[s["table"][i][at // c["page"]].long(), :, at % c["page"]] = rows.transpose(0, 1)
    return cache


def _prepare_read(c, g):
    b, hkv, d, n, k = (c[x] for x in ("b", "hkv", "d", "n", "k"))
    s = dict(c, idx=None, k_len=None)
    _, s["table"] = _cache(c, b, n, g)
    s["caches"] = [_filled(c, s, _keys(g, b, hkv, n, d), _randn(g, b, hkv, n, d) * 2.0 ** c["v_exp"],
                           _cache(c, b, n, g)[0], g) for _ in range(c["layers"])]
    if c["sparse"]:
        s["idx"] = _selected(g, b, n, k)
    if c["ragged"]:
        s["k_len"] = _randint(g, 0, k + 1, b)
    s["back"] = [torch.zeros((b, hkv, k, d), dtype=torch.bfloat16, device=DEV)
                 for _ in range(2 * c["layers"])]
    return s


def _selected(g, b, n, k):
    score = torch.rand((b, n), generator=g, device=DEV)
    score[:, :4] = 2.0                                                   # sinks stay
    return torch.sort(torch.topk(score, k).indices, -1).values.to(torch.int32)


def _prepare_attn(c, g):
    b, hq, hkv, d, w, n = (c[k] for k in ("b", "hq", "hkv", "d", "w", "n"))
    s = dict(c, scale=d ** -0.5, ws=None, q=_randn(g, b, hq, w, d), idx=None, k_len=None,
             k_exp=0, v_exp=0, kw=None, vw=None)
    # Peaked attention, as long contexts show it: the first positions (sinks)
    # and a few heavy hitters lean towards the queries' mean direction.
    lean = s["q"].float().view(b, hkv, hq // hkv, w, d).mean((2, 3))
    lean = (lean / lean.norm(dim=-1, keepdim=True)).view(b, hkv, 1, d)
    push = 3.0 * (torch.rand((b, 1, n, 1), generator=g, device=DEV) < 0.01)
    push[:, :, :4] = 6.0
    k = _randn(g, b, hkv, n, d)
    k += (push * lean).to(torch.bfloat16)
    cache, s["table"] = _cache(c, b, n, g)
    s["cache"] = _filled(c, s, k, _randn(g, b, hkv, n, d), cache, g)
    if c["sparse"]:
        s["idx"] = _selected(g, b, n, c["k"])
    if c["ragged"]:
        s["k_len"] = _randint(g, 0, c["k"] + 1, b)
    if c["window"]:
        s["kw"], s["vw"] = _randn(g, b, hkv, w, d), _randn(g, b, hkv, w, d)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((b, hq, w), device=DEV)
    return s


def _prepare_logprobs(c, g):
    b, w, vocab, top = c["b"], c["w"], c["vocab"], c["top"]
    t = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    x = torch.randn((b, w, vocab), generator=g, device=DEV, dtype=t) * 2.5
    if c["banned"]:
        x.masked_fill_(torch.rand((1, 1, vocab), generator=g, device=DEV) < 0.02, -math.inf)
    s = dict(c, x=x, scale=1.25, tokens=_randint(g, 0, vocab, b, w, c["m"]), n_rows=None)
    if c["m"]:                                           # the first ones are likely tokens
        s["tokens"][..., 0] = torch.argmax(x, -1).to(torch.int32)
        s["tokens"][:, w // 2:, 0] = _randint(g, 0, vocab, b, w - w // 2)
    if c["ragged"]:
        s["n_rows"] = _randint(g, 0, w + 1, b)
    s["logprobs"] = torch.zeros((b, w, c["m"]), device=DEV)
    s["entropy"], s["lse"] = torch.zeros((b, w), device=DEV), torch.zeros((b, w), device=DEV)
    s["top_ids"] = torch.zeros((b, w, top), dtype=torch.int32, device=DEV)
    s["top_logprobs"] = torch.zeros((b, w, top), device=DEV)
    return s


# -------------------------------------------------------------- the plain forms

def run(state):
    op = state["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "attn": _own_attn,
                "logprobs": _own_logprobs}[op](state)
    return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn,
            "logprobs": _plain_logprobs}[op](state)


def _codes(x, exp):
    """Codes [..][d / 2] and scales [..][d / 16] of x [..][d]."""
    x = x.float().unflatten(-1, (-1, 16)) * 2.0 ** -exp
    top = x.abs().amax(-1)
    # A sixth in 64 bits: a quotient on the border of two scales stays there.
    scale = (top.double() / 6).float().clamp(max=448.0).to(torch.float8_e4m3fn)
    step, size = scale.float()[..., None], x.abs()
    code = sum((size > m * step if i % 2 == 0 else size >= m * step).to(torch.uint8)
               for i, m in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    code = torch.where(step > 0, code, 0) + 8 * torch.signbit(x).to(torch.uint8)
    good = torch.isfinite(top)
    code = torch.where(good[..., None], code, 0).flatten(-2)
    return code[..., ::2] + 16 * code[..., 1::2], torch.where(good, scale.view(torch.uint8), 0x7f)


def _quantised(k, v, d, k_exp, v_exp):
    (ck, sk), (cv, sv) = _codes(k, k_exp), _codes(v, v_exp)
    pad = torch.zeros((*ck.shape[:-1], _record(d) - d - d // 8), dtype=torch.uint8, device=DEV)
    return torch.cat([ck, cv, sk, sv, pad], -1)


def _values(codes, scales, exp):
    """fp32 [..][d] of codes [..][d / 2] and scales [..][d / 16]."""
    table = torch.tensor(E2M1, device=DEV)
    nibbles = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    x = table[nibbles & 7] * torch.where(nibbles >= 8, -1.0, 1.0)
    scale = scales.contiguous().view(torch.float8_e4m3fn).float() * 2.0 ** exp
    return (x.unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2)


def _dequantised(rec, d, k_exp, v_exp):
    h, sc = d // 2, d // 16
    return (_values(rec[..., :h], rec[..., d:d + sc], k_exp),
            _values(rec[..., h:d], rec[..., d + sc:d + 2 * sc], v_exp))


def _places(s, at):
    """Where positions at [b][k] of the sequences lie: (first, third) index."""
    if s["table"] is None:
        return torch.arange(s["b"], device=DEV)[:, None].expand_as(at), at
    return s["table"].long().gather(1, at // s["page"]), at % s["page"]


def _counted(lens, b, k):
    at = torch.arange(k, device=DEV)[None]
    return at < (lens[:, None] if lens is not None else torch.full((b, 1), k, device=DEV))


def _plain_back(s, cache, at, keep, k, v):
    i, j = _places(s, at)
    x, y = _dequantised(cache[i, :, j].transpose(1, 2), s["d"], s["k_exp"], s["v_exp"])
    keep = keep[:, None, :, None]
    k.copy_(torch.where(keep, x.to(torch.bfloat16), k))
    v.copy_(torch.where(keep, y.to(torch.bfloat16), v))


def _plain_write(s):
    b, w = s["b"], s["w"]
    at = torch.arange(w, device=DEV)[None].expand(b, w) if s["idx"] is None else s["idx"].long()
    keep = _counted(s["w_len"], b, w)
    i, j = _places(s, at)

    def layer(cache, k, v, to_k, to_v):
        rows = _quantised(k, v, s["d"], s["k_exp"], s["v_exp"]).transpose(1, 2)
        cache[i, :, j] = torch.where(keep[..., None, None], rows, cache[i, :, j])
        _plain_back(s, cache, at, keep, to_k, to_v)

    [layer(*x) for x in zip(s["caches"], s["k_"], s["v_"], s["back"][::2], s["back"][1::2])]
    return s["back"]


def _plain_read(s):
    b, k = s["b"], s["k"]
    at = torch.arange(k, device=DEV)[None].expand(b, k) if s["idx"] is None else s["idx"].long()
    keep = _counted(s["k_len"], b, k)
    [_plain_back(s, cache, at, keep, x, y)
     for cache, x, y in zip(s["caches"], s["back"][::2], s["back"][1::2])]
    return s["back"]


def _plain_attn(s):
    b, hq, hkv, d, w, k = (s[x] for x in ("b", "hq", "hkv", "d", "w", "k"))
    gw = hq // hkv * w
    at = torch.arange(k, device=DEV)[None].expand(b, k) if s["idx"] is None else s["idx"].long()
    i, j = _places(s, at)
    rec = s["cache"] if s["table"] is None and s["idx"] is None else \
        s["cache"][i, :, j].transpose(1, 2)
    keys, values = _dequantised(rec, d, s["k_exp"], s["v_exp"])
    q = s["q"].float().view(b, hkv, gw, d) * s["scale"]
    x = q @ keys.transpose(-1, -2)
    x = torch.where(_counted(s["k_len"], b, k)[:, None, None], x, -math.inf)
    if s["kw"] is not None:
        own_x = q @ s["kw"].float().transpose(-1, -2)
        causal = torch.arange(w, device=DEV)[None] <= (torch.arange(gw, device=DEV) % w)[:, None]
        x = torch.cat([x, torch.where(causal, own_x, -math.inf)], -1)
        values = torch.cat([values, s["vw"].float()], 2)
    m = x.amax(-1, keepdim=True)
    safe = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(x - safe)
    total = e.sum(-1, keepdim=True)
    out = torch.where(total > 0, (e @ values) / torch.where(total > 0, total, 1.0), 0.0)
    lse = torch.where(total > 0, safe + torch.log(total), -math.inf)
    return out.reshape(b, hq, w, d).to(torch.bfloat16), lse.reshape(b, hq, w)


def _plain_logprobs(s):
    b, w, top = s["b"], s["w"], s["top"]
    t = s["x"].float() * s["scale"]
    m = t.amax(-1, keepdim=True)
    e = torch.exp(t - m)
    total = e.sum(-1, keepdim=True, dtype=torch.float64)
    lse = m.double() + torch.log(total)
    mean = torch.where(e > 0, e * (m - t), 0.0).sum(-1, keepdim=True, dtype=torch.float64) / total
    given = t.gather(-1, s["tokens"].long()).double() - lse
    ids = torch.sort(s["x"], dim=-1, descending=True, stable=True).indices[..., :top]
    best = t.gather(-1, ids).double() - lse
    keep = _counted(s["n_rows"], b, w)

    def put(to, x):
        where = keep.view(b, w, *[1] * (to.dim() - 2))
        return to.copy_(torch.where(where, x.to(to.dtype), to))

    return (put(s["logprobs"], given), put(s["entropy"], (torch.log(total) + mean)[..., 0]),
            put(s["lse"], lse[..., 0]), put(s["top_ids"], ids), put(s["top_logprobs"], best))


# ----------------------------------------------------- through the entry points

def _native():
    from sparse_kv_verification_gb300 import native
    return native


def _descs(N, s):
    return [N.kv4_desc(x, s["table"], s["k_exp"], s["v_exp"]) for x in s["caches"]]


def _own_write(s):
    N = _native()
    caches = _descs(N, s)
    rows = [N.kv_desc(k, v) for k, v in zip(s["k_"], s["v_"])]
    back = [N.kv_desc(k, v) for k, v in zip(s["back"][::2], s["back"][1::2])]
    b, hkv, d, n, w = (s[k] for k in ("b", "hkv", "d", "n", "w"))
    N.dustin_kv4_write(rows, caches, b, hkv, d, n, w, start=s["start"], w_len=s["w_len"])
    N.dustin_kv4_read(caches, back, b, hkv, d, n, w, idx=s["idx"], k_len=s["w_len"])
    return s["back"]


def _own_read(s):
    N = _native()
    back = [N.kv_desc(k, v) for k, v in zip(s["back"][::2], s["back"][1::2])]
    N.dustin_kv4_read(_descs(N, s), back, s["b"], s["hkv"], s["d"], s["n"], s["k"], idx=s["idx"],
                      k_len=s["k_len"])
    return s["back"]


def _own_attn(s):
    N = _native()
    b, hq, hkv, d, w, n, k = (s[x] for x in ("b", "hq", "hkv", "d", "w", "n", "k"))
    if s["ws"] is None:                                  # kept by the program, as its q and o
        s["ws"] = N.workspace(N.dustin_kv4_verify_attn_workspace_size(b, hq, hkv, d, w, k), DEV)
    win = None if s["kw"] is None else N.kv_desc(s["kw"], s["vw"])
    N.dustin_kv4_verify_attn(s["q"], N.kv4_desc(s["cache"], s["table"], s["k_exp"], s["v_exp"]),
                             hkv, n, k, s["scale"], s["o"], s["lse"], s["ws"], idx=s["idx"],
                             k_len=s["k_len"], win=win)
    return s["o"], s["lse"]


def _own_logprobs(s):
    N = _native()
    N.dustin_token_logprobs(s["x"], s["tokens"], s["logprobs"], s["entropy"], s["lse"],
                            s["top_ids"], s["top_logprobs"], scale=s["scale"], n_rows=s["n_rows"])
    return s["logprobs"], s["entropy"], s["lse"], s["top_ids"], s["top_logprobs"]


# ------------------------------------------------------------------ their work

def work(c):
    if c["op"] == "logprobs":
        # Ragged counts count with their mean.
        rows = c["b"] * c["w"] * (0.5 if c["ragged"] else 1.0)
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": rows * (c["vocab"] * size + 8 * c["m"] + 8 * c["top"] + 8),
                "flops": 6.0 * rows * c["vocab"]}
    rec, half = _record(c["d"]), 0.5 if c["ragged"] else 1.0
    if c["op"] == "attn":
        n_w, rows, k = c["w"] if c["window"] else 0, c["b"] * c["hq"] * c["w"], c["k"] * half
        return {"bytes": c["b"] * (c["hkv"] * (k * rec + n_w * c["d"] * 4)
                                   + (k * 4 if c["sparse"] else 0)) + rows * (4 * c["d"] + 4),
                "flops": 4.0 * rows * c["d"] * (k + ((c["w"] + 1) / 2 if n_w else 0))}
    rows = c["layers"] * c["b"] * c["hkv"] * half * (c["w"] if c["op"] == "write" else c["k"])
    # A written row is read, stored, and for what it stands for read back.
    return {"bytes": rows * (rec + 4 * c["d"]) * (2 if c["op"] == "write" else 1), "flops": 0}


# ------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    return {"write": _exact_write, "read": _exact_read, "attn": _exact_attn,
            "logprobs": _exact_logprobs}[case["op"]](prepare(case, seed))


def _exact_scales():
    """The 127 numbers a scale can be, in ascending order of their bytes."""
    v = [(i % 8 / 8 if i < 8 else 1 + i % 8 / 8) * 2.0 ** (max(i // 8, 1) - 7) for i in range(127)]
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _nearest(x, values):
    """The nearest of ascending values to each x, of two equally near ones the
    one of even index."""
    hi = torch.searchsorted(values, x).clamp(1, len(values) - 1)
    lo = hi - 1
    down, up = x - values[lo], values[hi] - x
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def _exact_rounded(x, exp):
    """What rows x become in the cache (64 bits)."""
    x = x.double().unflatten(-1, (-1, 16)) * 2.0 ** -exp
    scales = _exact_scales()
    steps = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    # Six times the scales: nothing is divided before it is compared.
    s = scales[_nearest(x.abs().amax(-1), 6 * scales)][..., None]
    y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    # A quotient next to a border is the border if the product says so.
    y = torch.where((y * 4).round() / 4 * s == x.abs(), (y * 4).round() / 4, y)
    return (steps[_nearest(y, steps)] * s * torch.sign(x) * 2.0 ** exp).flatten(-2)


def _exact_write(s):
    lens = [s["w"]] * s["b"] if s["w_len"] is None else s["w_len"].tolist()
    back = []
    for k, v in zip(s["k_"], s["v_"]):
        for x, exp in ((k, s["k_exp"]), (v, s["v_exp"])):
            y = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
            for i, n in enumerate(lens):
                y[i, :, :n] = _exact_rounded(x[i, :, :n], exp)
            back.append(y)
    return back


def _exact_values(rec, d):
    """K and V of records [..][record] in 64 bits, without the exponents."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)
    scales, out = _exact_scales(), []
    for part in range(2):
        codes = rec[..., part * d // 2:(part + 1) * d // 2].long()
        x = torch.empty((*codes.shape[:-1], d), dtype=torch.float64, device=DEV)
        x[..., 0::2], x[..., 1::2] = table[codes % 16], table[codes // 16]
        at = d + part * d // 16
        scale = scales[rec[..., at:at + d // 16].long()]
        out.append(x * scale.repeat_interleave(16, -1))
    return out


def _exact_rows(s, cache, i, h, at):
    """Records of positions at of sequence i and kv head h."""
    if s["table"] is None:
        return cache[i, h, at]
    return cache[s["table"][i][at // s["page"]].long(), h, at % s["page"]]


def _exact_read(s):
    back = []
    for cache in s["caches"]:
        k = torch.zeros((s["b"], s["hkv"], s["k"], s["d"]), dtype=torch.float64, device=DEV)
        v = torch.zeros_like(k)
        for i in range(s["b"]):
            n = s["k"] if s["k_len"] is None else int(s["k_len"][i])
            at = torch.arange(n, device=DEV) if s["idx"] is None else s["idx"][i, :n].long()
            for h in range(s["hkv"]):
                x, y = _exact_values(_exact_rows(s, cache, i, h, at), s["d"])
                k[i, h, :n], v[i, h, :n] = x * 2.0 ** s["k_exp"], y * 2.0 ** s["v_exp"]
        back += [k, v]
    return back


def _exact_attn(s):
    """Sequence by sequence and kv head by kv head: all the keys a sequence
    sees laid one after another, then the softmax's definition in 64 bits."""
    b, hq, hkv, d, w = (s[k] for k in ("b", "hq", "hkv", "d", "w"))
    o = torch.zeros((b, hq, w, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((b, hq, w), dtype=torch.float64, device=DEV)
    gr = hq // hkv
    for i in range(b):
        n = s["k"] if s["k_len"] is None else int(s["k_len"][i])
        at = torch.arange(n, device=DEV) if s["idx"] is None else s["idx"][i, :n].long()
        for h in range(hkv):
            k, v = _exact_values(_exact_rows(s, s["cache"], i, h, at), d)
            if s["kw"] is not None:
                k, v = torch.cat([k, s["kw"][i, h].double()]), torch.cat([v, s["vw"][i, h].double()])
            q = s["q"][i, h * gr:(h + 1) * gr].double()                  # [group][w][d]
            x = torch.einsum("gtd,nd->gtn", q, k) * s["scale"]
            if s["kw"] is not None:
                later = torch.ones((w, w), dtype=torch.bool, device=DEV).triu(1)
                x[:, :, n:].masked_fill_(later, -math.inf)
            z = torch.logsumexp(x, -1)
            weights = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[..., None])
            o[i, h * gr:(h + 1) * gr] = torch.einsum("gtn,nd->gtd", weights, v)
            lse[i, h * gr:(h + 1) * gr] = z
    return o, lse


def _exact_logprobs(s):
    b, w, m, top = s["b"], s["w"], s["m"], s["top"]
    given = torch.zeros((b, w, m), dtype=torch.float64, device=DEV)
    entropy, lse = (torch.zeros((b, w), dtype=torch.float64, device=DEV) for _ in range(2))
    ids = torch.zeros((b, w, top), dtype=torch.int32, device=DEV)
    best = torch.zeros((b, w, top), dtype=torch.float64, device=DEV)
    for i in range(b):
        n = w if s["n_rows"] is None else int(s["n_rows"][i])
        for j in range(0, n, 64):
            rows = slice(j, min(n, j + 64))
            lp = s["x"][i, rows].double() * s["scale"]
            z = torch.logsumexp(lp, -1)
            lp -= z[:, None]
            lse[i, rows] = z
            entropy[i, rows] = torch.special.entr(torch.exp(lp)).sum(-1)
            given[i, rows] = lp.gather(-1, s["tokens"][i, rows].long())
            left = torch.nan_to_num(s["x"][i, rows].double(), neginf=-1e300)
            order = torch.arange(left.shape[-1], 0, -1, device=DEV)
            for a in range(top):
                most = left.amax(-1, keepdim=True)
                at = ((left == most) * order).argmax(-1, keepdim=True)   # the first of equals
                ids[i, rows, a:a + 1] = at.to(torch.int32)
                best[i, rows, a:a + 1] = lp.gather(-1, at)
                left.scatter_(-1, at, -math.inf)
    return given, entropy, lse, ids, best
