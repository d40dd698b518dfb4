"""What is measured of the latent-attention operators: the store into the paged latent cache, the
read-back, the absorbed attention over ragged slots and over whole paged contexts, and the expanded
attention of a prefill.

Shapes come from the indexer's own workloads: pages of 64 tokens, 64 query heads, top-2048, batches of
32 to 128 sequences with contexts of 4096 to 131072 tokens, prefill chunks of 2048 rows on 8192 tokens.
A cached token is 512 latents and 64 rotated elements, held in bf16 or in e4m3 with one e8m0 scale
for each 64 latents (the rotated part stays bf16).
"""
import math
import random

import torch

own = False

LATENT, ROPE, GROUP = 512, 64, 64
TOKEN = LATENT + ROPE
NOPE, VDIM = 128, 128  # the expanded form's dimensions a head
EPS = 1e-6
SCALE = 1.0 / math.sqrt(NOPE + ROPE)


def listed():
    return [
        # one decode step's new tokens: 128 sequences, two rows each
        {"name": "store_fp8_step", "op": "store", "fmt": "fp8", "tokens": 256, "page": 64, "pad": 0},
        # a whole prompt written at once, a few of its tokens without a slot
        {"name": "store_fp8_prompt", "op": "store", "fmt": "fp8", "tokens": 8192, "page": 64, "pad": 0},
        # the cached context of a long prompt read back for the expanded form
        {"name": "gather_fp8_context", "op": "gather", "fmt": "fp8", "seqs": 2, "tokens": 131072, "page": 64},
        # several short contexts of odd lengths
        {"name": "gather_bf16_ragged", "op": "gather", "fmt": "bf16", "seqs": 5, "tokens": 10007, "page": 64},
        # one user's decode step on one of four devices' heads
        {"name": "sparse_bf16_single", "op": "sparse", "fmt": "bf16", "rows": 1, "heads": 16, "topk": 2048,
         "lo": 1777, "hi": 1777, "page": 64},
        # the paged decode workload's step
        {"name": "sparse_fp8_decode", "op": "sparse", "fmt": "fp8", "rows": 64, "heads": 64, "topk": 2048,
         "lo": 4096, "hi": 32768, "page": 64},
        # two rows a sequence, every head of a large model on this device
        {"name": "sparse_fp8_mtp", "op": "sparse", "fmt": "fp8", "rows": 256, "heads": 128, "topk": 2048,
         "lo": 1024, "hi": 16384, "page": 64},
        # a prefill chunk through the sparse path: 2048 rows on one 8192-token sequence
        {"name": "sparse_fp8_chunk", "op": "sparse", "fmt": "fp8", "rows": 2048, "heads": 64, "topk": 2048,
         "lo": 8192, "hi": 8192, "page": 64},
        # whole contexts, a batch of ordinary lengths
        {"name": "paged_fp8_decode", "op": "paged", "fmt": "fp8", "seqs": 32, "next_n": 1, "heads": 16,
         "lo": 4096, "hi": 32768, "page": 64},
        # whole contexts, few long ones with two rows each
        {"name": "paged_bf16_long", "op": "paged", "fmt": "bf16", "seqs": 4, "next_n": 2, "heads": 16,
         "lo": 100000, "hi": 131072, "page": 64},
        # a chunk of 2048 rows at the end of 8192 tokens
        {"name": "prefill_chunk", "op": "prefill", "seqs": 1, "heads": 64, "q_lo": 2048, "q_hi": 2048,
         "before_lo": 6144, "before_hi": 6144},
        # a pack of whole short prompts of odd lengths, none cached before
        {"name": "prefill_pack", "op": "prefill", "seqs": 7, "heads": 16, "q_lo": 65, "q_hi": 1500,
         "before_lo": 0, "before_hi": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "gather", "sparse", "sparse", "paged", "paged", "prefill", "prefill"])
    fmt, page = rng.choice(["fp8", "bf16"]), rng.choice([16, 64, 64, 128])
    if op == "store":
        return {"op": op, "fmt": fmt, "tokens": _log(rng, 1, 8192), "page": page, "pad": rng.choice([0, 64])}
    if op == "gather":
        return {"op": op, "fmt": fmt, "seqs": rng.randint(1, 16), "tokens": _log(rng, 16, 131072), "page": page}
    if op == "sparse":
        heads, topk = rng.choice([8, 16, 24, 32, 64, 128]), rng.choice([_log(rng, 1, 2048), 512, 1024, 2048])
        rows = _log(rng, 1, min(512, max(1, (1 << 26) // (heads * topk))))
        most = min(16384, (1 << 21) // rows)
        lo = _log(rng, 1, most)
        return {"op": op, "fmt": fmt, "rows": rows, "heads": heads, "topk": topk, "lo": lo,
                "hi": min(most, lo + _log(rng, 1, most)), "page": page}
    if op == "paged":
        seqs, next_n, heads = _log(rng, 1, 64), rng.randint(1, 4), rng.choice([8, 16, 24, 32, 64, 128])
        most = min(131072, (1 << 26) // (seqs * next_n * heads), (1 << 20) // seqs)
        lo = _log(rng, 1, max(2, most // 2))
        return {"op": op, "fmt": fmt, "seqs": seqs, "next_n": next_n, "heads": heads, "lo": lo,
                "hi": max(lo, _log(rng, max(1, lo), max(lo, most))), "page": page}
    seqs, heads = rng.randint(1, 8), rng.choice([1, 3, 8, 16, 32])
    q_hi = _log(rng, 1, 2048)
    return {"op": op, "seqs": seqs, "heads": heads, "q_lo": max(1, q_hi // rng.randint(1, 8)), "q_hi": q_hi,
            "before_lo": 0, "before_hi": rng.choice([0, _log(rng, 1, 2048)])}


# ------------------------------------------------------------------------- inputs


def _lengths(case, seed):
    """The lengths that the case's seed gives, as Python numbers (work() needs none of them exactly).
    A prefill's are the case's own: its outputs have a row for each query."""
    op = case["op"]
    rng = random.Random(case["q_hi"] + case["seqs"] if op == "prefill" else seed)
    if op == "sparse":
        return [rng.randint(case["lo"], case["hi"]) for _ in range(case["rows"])]
    if op == "paged":
        return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if op == "gather":
        cuts = sorted(rng.randint(0, case["tokens"]) for _ in range(case["seqs"] - 1))
        return [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    return list(zip(q, [rng.randint(case["before_lo"], case["before_hi"]) for _ in q]))


def _token_bytes(fmt):
    return LATENT + 2 * ROPE + LATENT // GROUP if fmt == "fp8" else 2 * TOKEN


def _page_bytes(fmt, page):
    return -(-page * _token_bytes(fmt) // 16) * 16


def _pool(fmt, pages, page, g):
    """A pool of cached tokens, normalised latents and rotated elements, as the store leaves them."""
    n = pages * page
    pool = torch.zeros(pages, _page_bytes(fmt, page), dtype=torch.uint8, device="cuda")
    x = torch.randn(n, TOKEN, generator=g, device="cuda")
    if fmt == "bf16":
        pool[:, :page * 2 * TOKEN] = x.bfloat16().view(torch.uint8).view(pages, -1)
        return pool
    y = x[:, :LATENT].reshape(n, LATENT // GROUP, GROUP)
    bits = torch.ceil(torch.log2(y.abs().amax(2, keepdim=True) / 448.0)) + 127
    codes = (y * torch.exp2(127 - bits)).to(torch.float8_e4m3fn).view(torch.uint8)
    a, b, c = page * LATENT, page * 2 * ROPE, page * (LATENT // GROUP)
    pool[:, :a] = codes.reshape(pages, a)
    pool[:, a:a + b] = x[:, LATENT:].bfloat16().view(torch.uint8).reshape(pages, b)
    pool[:, a + b:a + b + c] = bits.to(torch.uint8).reshape(pages, c)
    return pool


def _table(lengths, page, g):
    """A block table of randomly placed pages for contexts of these lengths, and the pages of the pool."""
    need = [-(-n // page) for n in lengths]
    pages = max(1, sum(need))
    order = torch.randperm(pages, generator=g, device="cuda").int()
    first = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    at = first[:, None] + torch.arange(max(1, max(need)), device="cuda")
    return order[at.clamp(max=pages - 1)].contiguous(), pages


def _cu(lengths):
    return torch.tensor([0] + list(lengths), device="cuda").cumsum(0).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    lengths = _lengths(case, seed) if op != "store" else None
    if op == "store":
        n, page = case["tokens"], case["page"]
        pages = -(-n // page) + 2
        s["pool"] = _pool(case["fmt"], pages, page, g)
        s["kv"] = torch.randn(n, TOKEN + case["pad"], generator=g, device="cuda").bfloat16()[:, :TOKEN]
        s["positions"] = torch.randint(0, 131072, (n,), generator=g, device="cuda").int()
        inv = 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda").double() / ROPE)
        angle = torch.arange(131072, device="cuda").double()[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["weight"] = 1 + 0.1 * torch.randn(LATENT, generator=g, device="cuda")
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:n]
        s["slots"] = torch.where(torch.rand(n, generator=g, device="cuda") < 0.01, -1, slots)
    elif op == "gather":
        start = [random.Random(seed + 1 + i).choice([0, 0, i * 7]) for i in range(len(lengths))]
        s["table"], pages = _table([a + b for a, b in zip(start, lengths)], case["page"], g)
        s["pool"] = _pool(case["fmt"], pages, case["page"], g)
        s["cu"], s["start"] = _cu(lengths), torch.tensor(start, device="cuda").int()
        s["out"] = torch.empty(case["tokens"], TOKEN, dtype=torch.bfloat16, device="cuda")
    elif op == "sparse":
        # the prefill chunk's rows share one context, decode rows have one each
        shared = case["lo"] == case["hi"] and case["rows"] > 1024
        table, pages = _table(lengths[:1] if shared else lengths, case["page"], g)
        s["pool"] = _pool(case["fmt"], pages, case["page"], g)
        ctx = torch.tensor(lengths, device="cuda")
        n = ctx.clamp(max=case["topk"])
        i = torch.arange(case["topk"], device="cuda")
        lo, hi = i * ctx[:, None] // n[:, None], (i + 1) * ctx[:, None] // n[:, None]
        u = torch.rand(lo.shape, generator=g, device="cuda")
        pos = torch.minimum(lo + (u * (hi - lo)).long(), (hi - 1).clamp(min=0))
        row = torch.zeros_like(ctx) if shared else torch.arange(len(lengths), device="cuda")
        block = (pos // case["page"]).clamp(max=table.shape[1] - 1)
        slot = table[row[:, None], block].long() * case["page"] + pos % case["page"]
        s["slots"] = slot[i < n[:, None]].int()
        s["indptr"] = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)]).int()
        s["q"] = torch.randn(case["rows"], case["heads"], TOKEN, generator=g, device="cuda").bfloat16()
    elif op == "paged":
        s["table"], pages = _table(lengths, case["page"], g)
        s["pool"] = _pool(case["fmt"], pages, case["page"], g)
        s["ctx"], s["longest"] = torch.tensor(lengths, device="cuda").int(), max(lengths)
        s["q"] = torch.randn(case["seqs"] * case["next_n"], case["heads"], TOKEN, generator=g,
                             device="cuda").bfloat16()
    else:
        q_len, before = [a for a, _ in lengths], [b for _, b in lengths]
        k_len = [a + b for a, b in lengths]
        nq, nk, h = sum(q_len), sum(k_len), case["heads"]
        s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = _cu(q_len), _cu(k_len), max(q_len), max(k_len)
        s["q"] = torch.randn(nq, h, NOPE + ROPE, generator=g, device="cuda").bfloat16()
        # keys and values as the up-projection leaves them, side by side for each head
        s["kv"] = torch.randn(nk, h, NOPE + VDIM, generator=g, device="cuda").bfloat16()
        # the rotated part as the read-back leaves it, behind the latents
        s["cached"] = torch.randn(nk, TOKEN, generator=g, device="cuda").bfloat16()
    return s


# --------------------------------------------------------------------- plain forms


def _decode(pool, fmt, page, slot):
    """The tokens of these slots in 32 bits, [..., 576]."""
    p, o = slot // page, slot % page
    if fmt == "bf16":
        return pool[:, :page * 2 * TOKEN].unflatten(1, (page, 2 * TOKEN))[p, o].view(torch.bfloat16).float()
    a, b, c = page * LATENT, page * 2 * ROPE, page * (LATENT // GROUP)
    codes = pool[:, :a].unflatten(1, (page, LATENT))[p, o].view(torch.float8_e4m3fn).float()
    rope = pool[:, a:a + b].unflatten(1, (page, 2 * ROPE))[p, o].view(torch.bfloat16).float()
    bits = pool[:, a + b:a + b + c].unflatten(1, (page, LATENT // GROUP))[p, o]
    scale = torch.exp2(bits.float() - 127).repeat_interleave(GROUP, -1)
    return torch.cat([codes * scale, rope], -1)


def _softmax_sum(score, value):
    """Values weighted by the softmax of the last dimension (nothing left there: zeros), and the log of its sum."""
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, value) / total.masked_fill(total == 0, 1.0)
    lse = (torch.log(total) + top.masked_fill(total == 0, 0.0)).squeeze(-1)
    return out.bfloat16(), lse


def _cached_views(pool, fmt, page):
    """The pool's parts as the values that they stand for (views)."""
    if fmt == "bf16":
        return {"token": pool[:, :page * 2 * TOKEN].view(torch.bfloat16)}
    a, b, c = page * LATENT, page * 2 * ROPE, page * (LATENT // GROUP)
    return {"latent": pool[:, :a].view(torch.float8_e4m3fn), "rope": pool[:, a:a + b].view(torch.bfloat16),
            "scale": pool[:, a + b:a + b + c].view(torch.float8_e8m0fnu)}


def _plain_store(s):
    pool, page = s["pool"], s["page"]
    # 64 bits: the rounding to a code, or a group's exponent, may stand next to a border
    x = s["kv"].double()
    y = x[:, :LATENT]
    y = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * s["weight"].double()
    cs = s["cos_sin"].double()[s["positions"].long()]
    c, d = cs[:, :ROPE // 2], cs[:, ROPE // 2:]
    even, odd = x[:, LATENT::2], x[:, LATENT + 1::2]
    rope = torch.stack([even * c - odd * d, odd * c + even * d], -1).flatten(1)
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    p, o = slot // page, slot % page
    if s["fmt"] == "bf16":
        token = torch.cat([y, rope], 1).bfloat16()[keep].view(torch.uint8)
        pool[:, :page * 2 * TOKEN].unflatten(1, (page, 2 * TOKEN))[p, o] = token
    else:
        y = y.unflatten(1, (LATENT // GROUP, GROUP))
        amax = y.abs().amax(2, keepdim=True).clamp(min=2.0 ** -126)
        bits = (torch.ceil(torch.log2(amax / 448.0)) + 127).clamp(0, 254)
        codes = (y * torch.exp2(127 - bits)).flatten(1).float().to(torch.float8_e4m3fn)[keep].view(torch.uint8)
        a, b, c = page * LATENT, page * 2 * ROPE, page * (LATENT // GROUP)
        pool[:, :a].unflatten(1, (page, LATENT))[p, o] = codes
        pool[:, a:a + b].unflatten(1, (page, 2 * ROPE))[p, o] = rope.bfloat16()[keep].view(torch.uint8)
        pool[:, a + b:a + b + c].unflatten(1, (page, LATENT // GROUP))[p, o] = bits[keep, :, 0].to(torch.uint8)
    return _cached_views(pool, s["fmt"], page)


def _plain_gather(s):
    row = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    pos = row - s["cu"][seq] + s["start"][seq]
    slot = s["table"][seq, pos // s["page"]].long() * s["page"] + pos % s["page"]
    s["out"].copy_(_decode(s["pool"], s["fmt"], s["page"], slot).bfloat16())
    return s["out"]


def _plain_sparse(s):
    i = torch.arange(s["topk"], device="cuda")
    first, n = s["indptr"][:-1, None].long(), (s["indptr"][1:] - s["indptr"][:-1])[:, None]
    slot = s["slots"][(first + i).clamp(max=s["slots"].numel() - 1)].long()
    token = _decode(s["pool"], s["fmt"], s["page"], slot)
    score = torch.matmul(s["q"].float(), token.mT) * SCALE
    return _softmax_sum(score.masked_fill((i >= n)[:, None], -math.inf), token[..., :LATENT])


def _plain_paged(s):
    b, n, h = s["seqs"], s["next_n"], s["heads"]
    pos = torch.arange(s["longest"], device="cuda")
    slot = s["table"][:, pos // s["page"]].long() * s["page"] + pos % s["page"]
    token = _decode(s["pool"], s["fmt"], s["page"], slot)
    score = torch.matmul(s["q"].float().view(b, n * h, TOKEN), token.mT).view(b, n, h, -1) * SCALE
    end = s["ctx"][:, None] - n + 1 + torch.arange(n, device="cuda")
    score = score.masked_fill((pos >= end[..., None])[:, :, None], -math.inf)
    out, lse = _softmax_sum(score.view(b, n * h, -1), token[..., :LATENT])
    return out.view(b * n, h, LATENT), lse.view(b * n, h)


def _plain_prefill(s):
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    nq, nk = s["cu_q"].diff()[:, None], s["cu_k"].diff()[:, None]
    at_q = (s["cu_q"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    at_k = (s["cu_k"][:-1, None] + j).clamp(max=s["kv"].shape[0] - 1).long()
    q, kv = s["q"][at_q].float().transpose(1, 2), s["kv"][at_k].float().transpose(1, 2)
    rope = s["cached"][at_k][..., LATENT:].float()
    score = torch.matmul(q[..., :NOPE], kv[..., :NOPE].mT) + torch.matmul(q[..., NOPE:], rope.mT[:, None])
    seen = (j <= (i + nk - nq)[..., None]) & (j < nk)[:, None]
    out, lse = _softmax_sum((score * SCALE).masked_fill(~seen[:, None], -math.inf), kv[..., NOPE:])
    live = i < nq
    return out.transpose(1, 2)[live], lse.transpose(1, 2)[live]


def run(s):
    op = s["op"]
    if not own:
        return {"store": _plain_store, "gather": _plain_gather, "sparse": _plain_sparse, "paged": _plain_paged,
                "prefill": _plain_prefill}[op](s)
    import sparse_attention_indexer_mxfp4_gb300 as idx
    if op == "prefill":
        return idx.idx_latent_prefill(s["q"], s["kv"][..., :NOPE], s["cached"][:, LATENT:], s["kv"][..., NOPE:],
                                      s["cu_q"], s["cu_k"], SCALE)
    fmt = idx.LATENT_FP8 if s["fmt"] == "fp8" else idx.LATENT_BF16
    if op == "store":
        idx.idx_latent_store(s["kv"], s["positions"], s["cos_sin"], s["weight"], EPS, s["pool"], s["page"],
                             s["slots"], fmt)
        return _cached_views(s["pool"], s["fmt"], s["page"])
    if op == "gather":
        return idx.idx_latent_gather(s["pool"], s["page"], fmt, s["table"], s["cu"], s["out"],
                                     seq_starts=s["start"])
    if op == "sparse":
        return idx.idx_latent_attention(s["q"], s["pool"], s["page"], fmt, s["slots"], s["indptr"], SCALE)
    return idx.idx_paged_latent_attention(s["q"], s["pool"], s["page"], fmt, s["table"], s["ctx"],
                                          s["next_n"], SCALE, s["longest"])


def work(case):
    op = case["op"]
    if op in ("store", "gather"):
        n, token = case["tokens"], _token_bytes(case["fmt"])
        if op == "store":
            return {"bytes": n * (2 * TOKEN + token + 4 * ROPE + 12) + 4 * LATENT, "flops": n * 8 * TOKEN}
        return {"bytes": n * (2 * TOKEN + token + 4 / case["page"]), "flops": n * LATENT}
    lengths = _lengths(case, 1)
    h = case["heads"]
    if op == "prefill":
        pairs = sum(a * b + a * (a + 1) / 2 for a, b in lengths)
        nq, nk = sum(a for a, _ in lengths), sum(a + b for a, b in lengths)
        moved = 2 * nq * h * (NOPE + ROPE + VDIM) + 4 * nq * h + 2 * nk * (h * (NOPE + VDIM) + ROPE)
        return {"bytes": moved, "flops": 2 * h * pairs * (NOPE + ROPE + VDIM)}
    if op == "sparse":
        rows, seen = case["rows"], sum(min(n, case["topk"]) for n in lengths)
        read, pairs, ids = (min(seen, lengths[0]) if rows > 1024 and case["lo"] == case["hi"] else seen), seen, seen
    else:
        rows, read = case["seqs"] * case["next_n"], sum(lengths)
        pairs = sum(max(0, n - j) for n in lengths for j in range(case["next_n"]))
        ids = read / case["page"]
    moved = rows * h * (2 * TOKEN + 2 * LATENT + 4) + read * _token_bytes(case["fmt"]) + 4 * ids
    return {"bytes": moved, "flops": 2 * h * pairs * (TOKEN + LATENT)}


# ------------------------------------------------------------------ the definition


def _token64(s, slot):
    """Tokens of these slots in 64 bits, read byte by byte from the page's definition."""
    page, pool = s["page"], s["pool"]
    line, at = pool[slot // page], (slot % page)[:, None]
    take = lambda first, size, n: line.gather(1, first + at * size * n + torch.arange(size * n, device="cuda"))  # noqa: E731
    if s["fmt"] == "bf16":
        return take(0, 2, TOKEN).view(torch.bfloat16).double()
    byte = take(0, 1, LATENT).long()
    e, m = byte >> 3 & 15, (byte & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7).double())
    mag = torch.where(byte >> 7 == 1, -mag, mag)
    ex = take(page * (LATENT + 2 * ROPE), 1, LATENT // GROUP).double() - 127
    mag = (mag.view(-1, LATENT // GROUP, GROUP) * 2.0 ** ex[..., None]).flatten(1)
    return torch.cat([mag, take(page * LATENT, 2, ROPE).view(torch.bfloat16).double()], 1)


def _attend64(q, k, v, seen):
    """q [h, n, d], k [.., m, d], v [.., m, e], seen [n, m] or None."""
    w = q @ k.mT * SCALE
    if seen is not None:
        w = torch.where(seen, w, -math.inf)
    lse = torch.logsumexp(w, -1)
    return torch.exp(w - lse[..., None]).nan_to_num(0.0) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gather":
        cu, rows = s["cu"].tolist(), []
        for b, first in enumerate(s["start"].tolist()):
            pos = torch.arange(first, first + cu[b + 1] - cu[b], device="cuda")
            rows.append(_token64(s, s["table"][b].long()[pos // s["page"]] * s["page"] + pos % s["page"]))
        return torch.cat(rows)
    if op == "store":
        # what the codes stand for is compared with the plain form's; in bf16 the tokens have a value before rounding
        if case["fmt"] != "bf16":
            return None
        x = s["kv"].double()
        lat = x[:, :LATENT]
        lat = lat * s["weight"].double() / (lat.square().sum(1, keepdim=True) / LATENT + EPS).sqrt()
        cs = s["cos_sin"].double()[s["positions"].long()]
        z = torch.view_as_complex(x[:, LATENT:].reshape(-1, ROPE // 2, 2).contiguous())
        z = torch.view_as_real(z * torch.complex(cs[:, :ROPE // 2], cs[:, ROPE // 2:])).flatten(1)
        keep = s["slots"] >= 0
        pool = s["pool"][:, :s["page"] * 2 * TOKEN].view(torch.bfloat16).double().view(-1, TOKEN)
        pool[s["slots"][keep]] = torch.cat([lat, z], 1)[keep]
        return {"token": pool.view(s["pool"].shape[0], -1)}
    outs, lses = [], []
    if op == "prefill":
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(case["seqs"]):
            q = s["q"][cq[b]:cq[b + 1]].double().transpose(0, 1)
            kv = s["kv"][ck[b]:ck[b + 1]].double().transpose(0, 1)
            rope = s["cached"][ck[b]:ck[b + 1], LATENT:].double()
            k = torch.cat([kv[..., :NOPE], rope.expand(kv.shape[0], -1, -1)], -1)
            n, m = q.shape[1], k.shape[1]
            seen = torch.ones(n, m, dtype=torch.bool, device="cuda").tril(m - n)
            parts = [_attend64(q[i:i + 4], k[i:i + 4], kv[i:i + 4, :, NOPE:], seen) for i in range(0, q.shape[0], 4)]
            outs.append(torch.cat([p[0] for p in parts]).transpose(0, 1))
            lses.append(torch.cat([p[1] for p in parts]).transpose(0, 1))
        return torch.cat(outs), torch.cat(lses)
    if op == "sparse":
        cut = s["indptr"].tolist()
        sets = [(r, s["slots"][cut[r]:cut[r + 1]].long()) for r in range(case["rows"])]
    else:
        sets = []
        for b, n in enumerate(s["ctx"].tolist()):
            pos = torch.arange(n, device="cuda")
            slot = s["table"][b].long()[pos // s["page"]] * s["page"] + pos % s["page"]
            sets += [(b * s["next_n"] + j, slot[:max(0, n - s["next_n"] + j + 1)]) for j in range(s["next_n"])]
    for r, slot in sets:
        token = _token64(s, slot)
        o, lse = _attend64(s["q"][r].double(), token, token[:, :LATENT], None)
        outs.append(o)
        lses.append(lse)
    return torch.stack(outs), torch.stack(lses)
