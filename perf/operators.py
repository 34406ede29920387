"""What is measured of the operators of full-width layers: the 4-bit paged cache (write and read back), decode attention
over it, prompt attention, the attention weights of a prompt, and eviction by accumulated weight.

``run`` computes a case in plain torch operations, or, where ``own`` is true, through the calls that a program makes of
``rank_mixed_precision_b200``.  Head shapes, contexts and batch sizes are those of the workloads in ``harness/gen.py``
(32 query heads over 32 or 8 KV heads of width 128, 4 of width 64; contexts 256 to 32768; batches 1 to 32).

A page of the 4-bit cache holds 16 tokens of one KV head, as 32-bit words in four planes, token by token:
  K codes   channels 32 g + 8 c .. + 7 of token t at t * d/8 + c * NG + g      (NG = d / 32 groups, c < 4)
  V codes   channels 8 w .. + 7 of token t at t * d/8 + w
  K meta, V meta   group g of token t at t * NG + g: fp16 scale, fp16 zero
"""
import math

import torch

own = False

PAGE = 16
HEADS = [(4, 4, 64), (8, 2, 64), (5, 1, 64), (14, 2, 64), (32, 32, 128), (32, 8, 128), (12, 4, 128), (16, 1, 128)]


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def listed():
    gqa = {"H": 32, "h_kv": 8, "d": 128}
    mha = {"H": 32, "h_kv": 32, "d": 128}
    return [
        # one new token of each of 32 sequences enters the cache, and is read back: the write of a decode step
        {"name": "cache_step_b32", "op": "cache", **gqa, "batch": 32, "ctx_lo": 4096, "ctx_hi": 8192, "new_lo": 1, "new_hi": 1},
        # four prompts' chunks of 2048 tokens enter the cache, and are read back for the next chunk's attention
        {"name": "cache_chunk_b4", "op": "cache", **mha, "batch": 4, "ctx_lo": 0, "ctx_hi": 37, "new_lo": 2001, "new_hi": 2048},
        # the smallest decode: four heads of width 64, 256 tokens; latency is all
        {"name": "decode_small", "op": "decode", "H": 4, "h_kv": 4, "d": 64, "batch": 1, "lo": 256, "hi": 256, "weigh": False},
        # a batch of 32 ragged sequences with grouped heads, the weights kept for a later eviction
        {"name": "decode_gqa_b32", "op": "decode", **gqa, "batch": 32, "lo": 4096, "hi": 8192, "weigh": True},
        # one long sequence without grouping
        {"name": "decode_long_b1", "op": "decode", **mha, "batch": 1, "lo": 32768, "hi": 32768, "weigh": False},
        # the smallest prompt
        {"name": "prompt_small", "op": "prompt", "H": 4, "h_kv": 4, "d": 64, "batch": 1, "lo": 256, "hi": 256, "before": 0},
        # sixteen packed prompts from one token to 1999
        {"name": "prompt_packed_b16", "op": "prompt", **gqa, "batch": 16, "lo": 1, "hi": 1999, "before": 0},
        # a chunk of 2048 tokens behind 30720 others: the largest
        {"name": "prompt_chunk", "op": "prompt", **mha, "batch": 1, "lo": 2048, "hi": 2048, "before": 30720},
        # the last 64 queries of four long prompts say what eviction keeps
        {"name": "weights_last64_b4", "op": "weights", **gqa, "batch": 4, "lo": 64, "hi": 64, "before": 32704, "window": 64},
        # every query of a prompt does
        {"name": "weights_full", "op": "weights", **gqa, "batch": 1, "lo": 8001, "hi": 8001, "before": 0, "window": 8001},
        # a batch of ragged sequences goes down to 40% of its tokens
        {"name": "evict_b32", "op": "evict", **gqa, "batch": 32, "lo": 4096, "hi": 8192, "keep": 0.4, "recent": 128},
        # one long sequence does
        {"name": "evict_long_b1", "op": "evict", **mha, "batch": 1, "lo": 32768, "hi": 32768, "keep": 0.4, "recent": 1024},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    H, h_kv, d = rng.choice(HEADS)
    op = rng.choice(["cache", "decode", "prompt", "weights", "evict"])
    case = {"op": op, "H": H, "h_kv": h_kv, "d": d}
    if op == "cache":
        new = _log(rng, 1, 4096)
        case["batch"] = _log(rng, 1, max(1, min(64, 8192 // new)))
        case["ctx_lo"] = rng.randrange(0, 40)
        case["ctx_hi"] = case["ctx_lo"] + _log(rng, 1, 4096)
        case["new_hi"] = new
        case["new_lo"] = rng.randint(0, new) if case["batch"] > 1 else new
    elif op in ("decode", "evict"):
        hi = _log(rng, 1, 32768)
        case["batch"] = _log(rng, 1, max(1, min(64, 1 << 20, 32 * 8192 * 8 // (hi * h_kv))))
        case["hi"] = hi
        case["lo"] = rng.randint(0, hi) if case["batch"] > 1 else hi
        if op == "decode":
            case["weigh"] = rng.random() < 0.5
        else:
            case["keep"] = round(rng.uniform(0.02, 1.0), 3)
            case["recent"] = _log(rng, 1, 256)
    else:
        hi = _log(rng, 1, 4096)
        before = rng.choice([0, rng.randrange(1, 64), _log(rng, 64, 8192)])
        most = (1 << 31) // (2 * H * hi * (hi + before))
        case["batch"] = _log(rng, 1, max(1, min(8, most)))
        case["hi"] = hi
        case["lo"] = rng.randint(0, hi) if case["batch"] > 1 else hi
        case["before"] = before
        if op == "weights":
            case["window"] = rng.choice([hi, _log(rng, 1, hi)])
    return case


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, both among them where n > 1, in a mixed order."""
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, n) == 1)
    return [hi if n == 1 else lo + (hi - lo) * (i * step % n) // (n - 1) for i in range(n)]


def _keeps(case):
    return [max(1, int(x * case["keep"])) for x in _spread(case["lo"], case["hi"], case["batch"])]


def _pairs(n, before, window):
    """(query, key) pairs of the last `window` of n queries behind `before` keys."""
    w = min(n, window)
    return w * (before + n - w) + w * (w + 1) // 2


def work(case):
    H, h_kv, d, op = case["H"], case["h_kv"], case["d"], case["op"]
    token = d + d // 4  # bytes of a token's codes and metadata, K and V, in one KV head
    if op == "cache":
        n = sum(_spread(case["new_lo"], case["new_hi"], case["batch"]))
        return {"bytes": n * h_kv * (4 * d + token + 4 * d) + 8 * n, "flops": n * h_kv * 2 * d * 10}
    lens = _spread(case["lo"], case["hi"], case["batch"])
    n = sum(lens)
    if op == "decode":
        return {"bytes": n * h_kv * (token + (8 if case["weigh"] else 0)) + 4 * case["batch"] * H * d, "flops": 4 * n * H * d}
    if op == "evict":
        kept = sum(min(a, b) for a, b in zip(lens, _keeps(case)))
        return {"bytes": n * h_kv * 4 + kept * h_kv * (2 * (token + 4) + 4), "flops": 2 * n * h_kv}
    keys = n + case["before"] * case["batch"]
    if op == "prompt":
        pairs = sum(_pairs(x, case["before"], x) for x in lens)
        return {"bytes": 4 * n * H * d + 4 * keys * h_kv * d + 4 * n * H, "flops": 4 * d * H * pairs}
    pairs = sum(_pairs(x, case["before"], case["window"]) for x in lens)
    rows = sum(min(x, case["window"]) for x in lens)
    return {"bytes": rows * H * (2 * d + 4) + keys * h_kv * (2 * d + 4), "flops": 2 * d * H * pairs}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _keys(g, n, h_kv, d):
    """Keys as they enter the score: two channels of each head are wide, as those of trained models are."""
    k = torch.randn((n, h_kv, d), generator=g, device="cuda")
    k[..., 3] *= 4
    k[..., d // 2 + 5] *= 4
    return k.bfloat16()


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return _i32(out)


def _table(g, caps, extra=0):
    """Block table with room for `caps` tokens of each sequence, its pages in random order, and the ids of `extra` more."""
    cols = max(1, max((c + PAGE - 1) // PAGE for c in caps))
    used = [(c + PAGE - 1) // PAGE for c in caps]
    ids = torch.randperm(sum(used) + extra, generator=g, device="cuda").int()
    table = torch.zeros((len(caps), cols), dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    return table, ids[at:], sum(used) + extra


def _slots(table, starts, lens):
    """Slots (page * 16 + offset) of tokens starts[b] .. starts[b] + lens[b] - 1 of every sequence, back to back."""
    got = []
    for b, (s, n) in enumerate(zip(starts, lens)):
        t = torch.arange(s, s + n, device="cuda")
        got.append(table[b].long()[t // PAGE] * PAGE + t % PAGE)
    return torch.cat(got)


def prepare(case, seed):
    H, h_kv, d, op, batch = case["H"], case["h_kv"], case["d"], case["op"], case["batch"]
    g = _gen(seed)
    state = {"case": case}
    if op == "cache":
        new = _spread(case["new_lo"], case["new_hi"], batch)
        starts = _spread(case["ctx_lo"], case["ctx_hi"], batch)
        table, _, pages = _table(g, [s + n for s, n in zip(starts, new)])
        n = sum(new)
        state.update(k=_keys(g, n, h_kv, d), v=_rand(g, n, h_kv, d), table=table, starts=_i32(starts), cu=_cu(new), n=n,
                     slots=_slots(table, starts, new), pool=torch.zeros((pages, h_kv, _page_bytes(d)), dtype=torch.uint8, device="cuda"))
        return state
    lens = _spread(case["lo"], case["hi"], batch)
    if op in ("decode", "evict"):
        n = sum(lens)
        room = []
        if op == "evict":
            room = [(min(a, b) + PAGE - 1) // PAGE for a, b in zip(lens, _keeps(case))]
        table, ids, pages = _table(g, lens, sum(room))
        pages = max(pages, 1)
        pool = torch.zeros((pages, h_kv, _page_bytes(d)), dtype=torch.uint8, device="cuda")
        slots = _slots(table, [0] * batch, lens)
        _write(pool, _keys(g, n, h_kv, d), _rand(g, n, h_kv, d), slots)
        # what a prompt and some steps leave: few tokens hold most of the weight
        weights = torch.randn((pages, h_kv, PAGE), generator=g, device="cuda").mul_(1.5).exp_()
        state.update(pool=pool, weights=weights, table=table, lens=_i32(lens))
        if op == "decode":
            state["q"] = _rand(g, batch, H, d)
        else:
            dst = torch.zeros((batch, max(1, max(room))), dtype=torch.int32, device="cuda")
            at = 0
            for b, u in enumerate(room):
                dst[b, :u] = ids[at:at + u]
                at += u
            state.update(dst=dst, keeps=_i32(_keeps(case)))
        return state
    keys = [x + case["before"] for x in lens]
    state.update(q=_rand(g, sum(lens), H, d), k=_keys(g, sum(keys), h_kv, d), cu_q=_cu(lens), cu_k=_cu(keys), max_q=max(lens), max_k=max(keys))
    if op == "prompt":
        state["v"] = _rand(g, sum(keys), h_kv, d)
    else:
        state["lse"] = _lse(state["q"], state["k"], lens, keys)
    return state


def _lse(q, k, lens, keys):
    """ln sum exp of every query's scores, as prompt attention returns it."""
    H, d, h_kv = q.shape[1], q.shape[2], k.shape[1]
    out = torch.full((q.shape[0], H), -math.inf, device="cuda")
    q0 = k0 = 0
    for n, m in zip(lens, keys):
        kk = k[k0:k0 + m].float().transpose(0, 1)
        for i in range(0, n, 1024):
            rows = q[q0 + i:q0 + min(n, i + 1024)].float()
            r = rows.shape[0]
            s = torch.matmul(rows.reshape(r, h_kv, -1, d).permute(1, 2, 0, 3).reshape(h_kv, -1, d), kk.transpose(1, 2)) / math.sqrt(d)
            s = s.view(h_kv, H // h_kv, r, m)
            seen = torch.arange(m, device="cuda")[None] <= (m - n + i + torch.arange(r, device="cuda"))[:, None]
            s.masked_fill_(~seen, -math.inf)
            out[q0 + i:q0 + i + r] = torch.logsumexp(s, -1).reshape(H, r).t()
        q0, k0 = q0 + n, k0 + m
    return out


# ---------------------------------------------------------------------------------------------------------------------
# the 4-bit cache in plain operations
# ---------------------------------------------------------------------------------------------------------------------
def _page_bytes(d):
    return PAGE * d + 128 * (d // 32)


def _places(d, dev):
    """Word indices within a page: K codes [16][d/8], V codes [16][d/8], K meta [16][d/32], V meta [16][d/32]."""
    t = torch.arange(PAGE, device=dev)[:, None]
    w = torch.arange(d // 8, device=dev)[None]
    ng = d // 32
    kc = t * (d // 8) + (w % 4) * ng + w // 4
    vc = 2 * d + t * (d // 8) + w
    km = 4 * d + t * ng + torch.arange(ng, device=dev)[None]
    vm = km + 16 * ng
    return kc, vc, km, vm


def _quantize(x):
    """(codes [n, h, d] as integers, metadata words [n, h, d/32]) of rows x [n, h, d]."""
    n, h, d = x.shape
    z = x.float().view(n, h, d // 32, 32)
    lo, hi = z.amin(-1, keepdim=True), z.amax(-1, keepdim=True)
    scale = ((hi - lo) / 15.0).half()
    zero = lo.half()
    step = torch.where(scale == 0, torch.ones_like(scale), scale).float()
    code = ((z - zero.float()) / step).round().clamp(0, 15) * (scale != 0)
    meta = torch.stack([scale, zero], -1).view(n, h, d // 32, 2).view(torch.int32).view(n, h, d // 32)
    return code.view(n, h, d).int(), meta


def _pack(code):
    c = code.view(*code.shape[:-1], -1, 8).long()
    word = (c << (4 * torch.arange(8, device=c.device))).sum(-1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).int()


def _write(pool, k, v, slots):
    d = k.shape[2]
    words = pool.view(torch.int32)
    page, t = (slots // PAGE)[:, None, None], slots % PAGE
    head = torch.arange(k.shape[1], device=k.device)[None, :, None]
    kc, vc, km, vm = _places(d, k.device)
    for x, codes, metas in ((k, kc, km), (v, vc, vm)):
        code, meta = _quantize(x)
        words[page, head, codes[t][:, None]] = _pack(code)
        words[page, head, metas[t][:, None]] = meta


def _values(words, codes, metas):
    """Values [..., 16, d] of pages `words` [..., words of a page]."""
    w = words[..., codes]
    code = (w[..., None] >> (4 * torch.arange(8, device=w.device, dtype=torch.int32))) & 15
    meta = words[..., metas].contiguous().view(torch.float16).view(*w.shape[:-1], metas.shape[1], 2).float()
    code = code.view(*w.shape[:-1], metas.shape[1], 32).float()
    return (code * meta[..., :1] + meta[..., 1:]).flatten(-2)


def _cache_plain(s):
    pool, k, v, slots = s["pool"], s["k"], s["v"], s["slots"]
    _write(pool, k, v, slots)
    words, t = pool.view(torch.int32)[slots // PAGE], slots % PAGE  # the page of each token
    n = torch.arange(len(t), device=t.device)
    kc, vc, km, vm = _places(k.shape[2], k.device)
    return {"k": _values(words, kc, km)[n, :, t].bfloat16(), "v": _values(words, vc, vm)[n, :, t].bfloat16()}


def _decode_plain(s):
    q, pool, table, lens = s["q"], s["pool"], s["table"].long(), s["lens"]
    B, H, d = q.shape
    h = pool.shape[1]
    kc, vc, km, vm = _places(d, q.device)
    words = pool.view(torch.int32)[table]  # [B, P, h, words]
    T = table.shape[1] * PAGE
    key = _values(words, kc, km).transpose(1, 2).reshape(B, h, T, d)
    p = torch.matmul(q.float().view(B, h, H // h, d), key.transpose(2, 3)) / math.sqrt(d)
    del key
    held = (torch.arange(T, device=q.device)[None] < lens[:, None])[:, None, None]
    p = torch.where(held, p, -math.inf)
    p = torch.where(held, torch.exp(p - p.amax(-1, keepdim=True)), 0.0)
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    value = _values(words, vc, vm).transpose(1, 2).reshape(B, h, T, d)
    value = torch.where(held[:, 0, 0][:, None, :, None], value, 0.0)
    out = torch.matmul(p, value).view(B, H, d).bfloat16()
    if not s["case"]["weigh"]:
        return {"out": out}
    add = p.sum(2).view(B, h, table.shape[1], PAGE).transpose(1, 2)
    inside = (torch.arange(table.shape[1], device=q.device)[None] * PAGE < lens[:, None])[:, :, None, None]
    s["weights"].index_put_((table.reshape(-1),), torch.where(inside, add, 0.0).flatten(0, 1), accumulate=True)
    return {"out": out, "weights": s["weights"]}


def _padded(x, cu, most):
    """[B, most, ...] of packed rows, and which of them are rows."""
    start, n = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    i = torch.arange(most, device=x.device)[None]
    there = i < n[:, None]
    rows = torch.where(there, start[:, None] + i, 0)
    return torch.where(there.view(*there.shape, *[1] * (x.dim() - 1)), x[rows], 0), there


def _scores(q, k, there_q, there_k, n_q, n_k, first):
    """fp32 scores [B, h_kv, G, rows, keys] of padded queries and keys; -inf where a key is not seen. `first`: the rows' first query."""
    B, R, H, d = q.shape
    h = k.shape[2]
    qq = q.float().view(B, R, h, H // h, d).permute(0, 2, 3, 1, 4)
    s = torch.matmul(qq.reshape(B, h, -1, d), k.float().permute(0, 2, 3, 1)).view(B, h, H // h, R, k.shape[1])
    s.div_(math.sqrt(d))
    last = (n_k - n_q + first)[:, None] + torch.arange(R, device=q.device)[None]
    seen = torch.arange(k.shape[1], device=q.device)[None, None] <= last[:, :, None]
    seen = seen & there_q[:, :, None] & there_k[:, None, :]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    return s


def _prompt_plain(s):
    cu_q, cu_k = s["cu_q"], s["cu_k"]
    q, there_q = _padded(s["q"], cu_q, max(1, s["max_q"]))
    k, there_k = _padded(s["k"], cu_k, s["max_k"])
    v, _ = _padded(s["v"], cu_k, s["max_k"])
    n_q, n_k = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    p = _scores(q, k, there_q, there_k, n_q, n_k, torch.zeros_like(n_q))
    top = p.amax(-1, keepdim=True).clamp_min(-1e30)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    B, R, H, d = q.shape
    out = torch.matmul(p.flatten(2, 3), v.float().permute(0, 2, 1, 3)).view(*p.shape[:-1], d) / total.clamp_min(1e-30)
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(B, R, H, d)[there_q]
    return {"out": out.bfloat16(), "lse": lse.permute(0, 3, 1, 2).reshape(B, R, H)[there_q]}


def _weights_plain(s):
    cu_q, cu_k = s["cu_q"], s["cu_k"]
    n_q, n_k = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    R = min(s["case"]["window"], max(1, s["max_q"]))
    first = (n_q - R).clamp_min(0)
    cu = torch.stack([cu_q[:-1] + first, cu_q[1:]])
    i = torch.arange(R, device=cu.device)[None]
    there_q = cu[0][:, None] + i < cu[1][:, None]
    rows = torch.where(there_q, cu[0][:, None] + i, 0).long()
    q, lse = s["q"][rows], s["lse"][rows]
    k, there_k = _padded(s["k"], cu_k, s["max_k"])
    p = _scores(q, k, there_q, there_k, n_q, n_k, first)
    B, h, G = p.shape[:3]
    p.sub_(lse.view(B, R, h, G).permute(0, 2, 3, 1)[..., None].clamp_min(-1e30)).exp_()
    return {"weights": p.sum((2, 3)).transpose(1, 2)[there_k]}


def _evict_plain(s):
    pool, weights, table, dst = s["pool"], s["weights"], s["table"].long(), s["dst"].long()
    lens, keeps = s["lens"], torch.minimum(s["keeps"], s["lens"])
    B, P = table.shape
    h, T, cap = pool.shape[1], P * PAGE, dst.shape[1] * PAGE
    i = torch.arange(T, device=pool.device)[None]
    recent = torch.minimum(keeps, torch.full_like(keeps, s["case"]["recent"]))
    w = weights[table].transpose(1, 2).reshape(B, h, T)
    w = torch.where((i >= (lens - recent)[:, None])[:, None], math.inf, w)
    w = torch.where((i < lens[:, None])[:, None], w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, torch.arange(T, device=pool.device).expand_as(order).contiguous())
    stays = rank < keeps[:, None, None]
    b, head, token = stays.nonzero(as_tuple=True)
    place = (stays.cumsum(-1) - 1)[b, head, token]
    kept = torch.full((B, h, cap), -1, dtype=torch.int32, device=pool.device)
    kept[b, head, place] = token.int()
    src, to = table[b, token // PAGE], dst[b, place // PAGE]
    words, d = pool.view(torch.int32), s["case"]["d"]
    at, into = token % PAGE, place % PAGE
    for places in _places(d, pool.device):
        words[to[:, None], head[:, None], places[into]] = words[src[:, None], head[:, None], places[at]]
    weights[to, head, into] = weights[src, head, at]
    return {"kept": kept, "lens": keeps, "pool": words, "weights": weights}  # the pool's bytes are moved, not computed: they come as they are


# ---------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------------------------------
_handles = {}


def _handle(case):
    """The context that a program keeps for its head shape (the factors are a latent layer's, and small here)."""
    from rank_mixed_precision_b200 import starkv as S

    shape = (case["H"], case["h_kv"], case["d"])
    if shape not in _handles:
        H, h_kv, d = shape
        cfg = S.make_config(H, h_kv, d, 64, 16, 64, 16)
        zero = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        _handles[shape] = S.StarKV(cfg, zero(64, h_kv * 16), zero(64, 64), zero(h_kv, 16, d), zero(64, h_kv * d))
    return S, _handles[shape]


def _run_own(s):
    case = s["case"]
    S, kv = _handle(case)
    op = case["op"]
    if op == "cache":
        cache = S.KV4Cache(kv.cfg, pages=s["pool"])
        kv.kv4_append(cache, s["k"], s["v"], s["slots"])
        k, v = kv.kv4_read(cache, s["table"], s["cu"], s["n"], starts=s["starts"])
        return {"k": k, "v": v}
    if op == "decode":
        cache = S.KV4Cache(kv.cfg, pages=s["pool"], weights=s["weights"])
        out = kv.kv4_decode(cache, s["q"], s["table"], s["lens"], accumulate=case["weigh"])
        return {"out": out, "weights": s["weights"]} if case["weigh"] else {"out": out}
    if op == "prompt":
        out, lse = kv.prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"])
        return {"out": out, "lse": lse}
    if op == "weights":
        return {"weights": kv.prompt_weights(s["q"], s["k"], s["lse"], s["cu_q"], s["cu_k"], s["max_k"], case["window"])}
    cache = S.KV4Cache(kv.cfg, pages=s["pool"], weights=s["weights"])
    lens, kept = kv.kv4_evict(cache, s["table"], s["lens"], s["keeps"], case["recent"], s["dst"])
    return {"kept": kept, "lens": lens, "pool": s["pool"].view(torch.int32), "weights": s["weights"]}


def run(state):
    if own:
        return _run_own(state)
    return {"cache": _cache_plain, "decode": _decode_plain, "prompt": _prompt_plain, "weights": _weights_plain, "evict": _evict_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _nibbles(raw, d, value):
    """Channel values [tokens, d] in 64 bits of raw pages [P, page bytes] (uint8) of one KV head, byte by byte."""
    t = torch.arange(PAGE, device=raw.device)[:, None]
    c = torch.arange(d, device=raw.device)[None]
    ng = d // 32
    if value:
        byte = 8 * d + t * (d // 2) + c // 2
    else:
        byte = t * (d // 2) + (c % 32 // 8) * (d // 8) + (c // 32) * 4 + c % 8 // 2
    meta = 16 * d + (64 * ng if value else 0) + (t * ng + c // 32) * 4
    code = (raw[:, byte].int() >> (c % 2 * 4)) & 15
    half = lambda at: raw[:, torch.stack([at, at + 1], -1)].contiguous().view(torch.float16)[..., 0].double()  # noqa: E731
    return (code.double() * half(meta) + half(meta + 2)).reshape(-1, d)


def _exact_quantized(x):
    got = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[2], 32):
        z = x[..., c:c + 32].double()
        lo, hi = z.min(-1, keepdim=True).values, z.max(-1, keepdim=True).values
        scale, zero = ((hi - lo) / 15).float().half().double(), lo.half().double()
        code = torch.where(scale > 0, torch.round((z - zero) / scale), 0.0).clamp(0, 15)
        got[..., c:c + 32] = code * scale + zero
    return got


def exact(case, seed):
    s = prepare(case, seed)
    H, h_kv, d, op = case["H"], case["h_kv"], case["d"], case["op"]
    G, c = H // h_kv, 1 / math.sqrt(d)
    if op == "cache":
        return {"k": _exact_quantized(s["k"]), "v": _exact_quantized(s["v"])}
    if op == "decode":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        weights = s["weights"].double()
        for b, n in enumerate(s["lens"].tolist()):
            pages = s["table"][b, :(n + PAGE - 1) // PAGE].long()
            for h in range(h_kv if n else 0):
                raw = s["pool"][pages, h]
                p = torch.softmax(c * (s["q"][b, h * G:(h + 1) * G].double() @ _nibbles(raw, d, False)[:n].t()), -1)
                out[b, h * G:(h + 1) * G] = p @ _nibbles(raw, d, True)[:n]
                t = torch.arange(n, device="cuda")
                weights[pages[t // PAGE], h, t % PAGE] += p.sum(0)
        return {"out": out, "weights": weights} if case["weigh"] else {"out": out}
    if op == "evict":
        weights = s["weights"].double()
        for b, (n, keep) in enumerate(zip(s["lens"].tolist(), s["keeps"].tolist())):
            keep = min(n, keep)
            old = n - min(keep, case["recent"])
            t, i = torch.arange(n, device="cuda"), torch.arange(keep, device="cuda")
            src, to = s["table"][b].long(), s["dst"][b].long()
            for h in range(h_kv):
                w = s["weights"][src[t // PAGE], h, t % PAGE].double()
                heavy = torch.argsort(w[:old], descending=True, stable=True)[:keep - (n - old)]
                stays = torch.cat([heavy.sort().values, t[old:]])
                weights[to[i // PAGE], h, i % PAGE] = w[stays]
        return {"kept": None, "lens": None, "pool": None, "weights": weights}
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    weights = torch.zeros(s["k"].shape[:2], dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        first = max(q0, q1 - case["window"]) if op == "weights" else q0
        for h in range(H):
            key = s["k"][k0:k1, h // G].double()
            for r in range(first, q1, 4096):
                e = min(q1, r + 4096)
                z = c * (s["q"][r:e, h].double() @ key.t())
                last = (k1 - k0) - (q1 - q0) + torch.arange(r - q0, e - q0, device="cuda")
                z = torch.where(torch.arange(k1 - k0, device="cuda")[None] <= last[:, None], z, -math.inf)
                if op == "weights":
                    weights[k0:k1, h // G] += torch.exp(z - s["lse"][r:e, h].double()[:, None]).sum(0)
                else:
                    lse[r:e, h] = torch.logsumexp(z, -1)
                    out[r:e, h] = torch.exp(z - lse[r:e, h][:, None]) @ s["v"][k0:k1, h // G].double()
    return {"weights": weights} if op == "weights" else {"out": out, "lse": lse}
