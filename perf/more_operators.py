"""What is measured of the grouped-head operators: attention over whole packed prompts, the 4-bit cache
(store with read-back), attention over it by slots and over whole contexts, the attention weights of its
tokens, and the eviction of the light ones.

Shapes come from the indexer's workloads: pages of 64 tokens, top-2048, batches of 32 to 128 sequences,
contexts of 4096 to 131072 tokens, prefill chunks of 2048 rows on 8192 tokens, heads of 128 elements.
A cached token of one key head is 128 key and 128 value elements in e2m1, one e8m0 scale for each 32.
"""
import math
import random

import torch

own = False

DIM, GROUP = 128, 32
SCALE = 1.0 / math.sqrt(DIM)


def listed():
    return [
        # a pack of whole short prompts of odd lengths, none cached before
        {"name": "prefill_pack", "op": "prefill", "seqs": 7, "kv": 4, "group": 4, "q_lo": 65, "q_hi": 1500,
         "before_lo": 0, "before_hi": 0},
        # a chunk of 2048 rows at the end of 8192 tokens
        {"name": "prefill_chunk", "op": "prefill", "seqs": 1, "kv": 8, "group": 8, "q_lo": 2048, "q_hi": 2048,
         "before_lo": 6144, "before_hi": 6144},
        # one decode step's new tokens, 128 sequences, and their read-back
        {"name": "store_step", "op": "store", "kv": 8, "seqs": 128, "tokens": 128, "page": 64, "pad": 0},
        # a prompt's tokens written at once and read back for its next chunk, in a projection's wider rows
        {"name": "store_prompt", "op": "store", "kv": 8, "seqs": 3, "tokens": 8191, "page": 64, "pad": 128},
        # one user's decode step on the slots that an indexer selected
        {"name": "sparse_single", "op": "sparse", "rows": 1, "kv": 2, "group": 8, "topk": 2048, "lo": 1777, "hi": 1777,
         "page": 64},
        # the paged decode workload's step
        {"name": "sparse_decode", "op": "sparse", "rows": 64, "kv": 8, "group": 8, "topk": 2048, "lo": 4096, "hi": 32768,
         "page": 64},
        # whole contexts, a batch of ordinary lengths
        {"name": "paged_decode", "op": "paged", "seqs": 32, "next_n": 1, "kv": 8, "group": 4, "lo": 4096, "hi": 32768,
         "page": 64},
        # whole contexts, few long ones, two rows each
        {"name": "paged_long", "op": "paged", "seqs": 4, "next_n": 2, "kv": 8, "group": 8, "lo": 100000, "hi": 131072,
         "page": 64},
        # the weights that a decode step gives the tokens of one long context
        {"name": "weights_single", "op": "weights", "seqs": 1, "next_n": 1, "kv": 8, "group": 4, "lo": 30011, "hi": 30011,
         "page": 64},
        # the same of a batch
        {"name": "weights_batch", "op": "weights", "seqs": 32, "next_n": 1, "kv": 8, "group": 8, "lo": 4096, "hi": 32768,
         "page": 64},
        # each head of a few sequences shrunk to its own 2048 tokens
        {"name": "evict_heads", "op": "evict", "seqs": 4, "kv": 8, "lo": 4096, "hi": 8192, "budget": 2048, "recent": 256,
         "whole": False, "page": 64},
        # whole tokens of a batch of longer contexts
        {"name": "evict_tokens", "op": "evict", "seqs": 32, "kv": 8, "lo": 8192, "hi": 32768, "budget": 8192, "recent": 1024,
         "whole": True, "page": 64},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "store", "sparse", "sparse", "paged", "paged", "weights", "evict"])
    kv, group, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([16, 64, 64, 128])
    if op == "prefill":
        seqs, group = rng.randint(1, 8), min(group, 8)
        q_hi, before = _log(rng, 1, 2048), rng.choice([0, _log(rng, 1, 2048)])
        while seqs > 1 and seqs * kv * group * q_hi * (q_hi // 2 + before) > 1 << 29:
            seqs -= 1
        return {"op": op, "seqs": seqs, "kv": kv, "group": group, "q_lo": max(1, q_hi // rng.randint(1, 8)),
                "q_hi": q_hi, "before_lo": 0, "before_hi": before}
    if op == "store":
        return {"op": op, "kv": kv, "seqs": rng.randint(1, 128), "tokens": _log(rng, 1, 8192), "page": page,
                "pad": rng.choice([0, 64])}
    if op == "sparse":
        topk = rng.choice([_log(rng, 1, 2048), 512, 1024, 2048])
        rows = _log(rng, 1, max(1, min(512, (1 << (20 if group <= 8 else 19)) // (kv * topk))))
        most = min(32768, (1 << 21) // rows)
        lo = _log(rng, 1, most)
        return {"op": op, "rows": rows, "kv": kv, "group": group, "topk": topk, "lo": lo,
                "hi": min(most, lo + _log(rng, 1, most)), "page": page}
    seqs, next_n, group = _log(rng, 1, 64), rng.randint(1, 4), min(group, 8)
    most = min(131072, (1 << (19 if next_n * group <= 16 else 18)) // seqs)
    lo = _log(rng, 1, max(2, most // 2))
    hi = max(lo, _log(rng, lo, max(lo, most)))
    if op == "evict":
        most = min(most, 32768)
        lo, hi = min(lo, most), min(hi, most)
        budget = _log(rng, 1, max(1, hi))
        return {"op": op, "seqs": seqs, "kv": kv, "lo": lo, "hi": hi, "budget": budget,
                "recent": rng.randint(0, budget), "whole": rng.random() < 0.5, "page": page}
    return {"op": op, "seqs": seqs, "next_n": next_n, "kv": kv, "group": group, "lo": lo, "hi": hi,
            "page": page}


# ------------------------------------------------------------------------- inputs


def _lengths(case, seed):
    """The lengths that the case's seed gives, as Python numbers.  A prefill's and the read-back's are the
    case's own: their outputs have a row for each token."""
    op = case["op"]
    if op == "store":
        rng, n, b = random.Random(case["tokens"]), case["tokens"], case["seqs"]
        cuts = [0] + sorted(rng.randint(0, n) for _ in range(b - 1)) + [n]
        return [b - a for a, b in zip(cuts, cuts[1:])]
    rng = random.Random(case["q_hi"] + case["seqs"] if op == "prefill" else seed)
    if op == "sparse":
        return [rng.randint(case["lo"], case["hi"]) for _ in range(case["rows"])]
    if op != "prefill":
        return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    return list(zip(q, [rng.randint(case["before_lo"], case["before_hi"]) for _ in q]))


def _page_bytes(page, kv):
    return -(-page * kv * 2 * (DIM // 2 + DIM // GROUP) // 16) * 16


def _pool(pages, page, kv, g):
    """A pool of cached tokens, normal values as the store leaves them: the codes of a page's keys, of its
    values, their scales, each [key heads, tokens, ...]."""
    pool = torch.zeros(pages, _page_bytes(page, kv), dtype=torch.uint8, device="cuda")
    at = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 27) // (page * kv * 2 * DIM))
    a, c = 2 * kv * page * DIM // 2, 2 * kv * page * DIM // GROUP
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn(n, a * 2 // GROUP, GROUP, generator=g, device="cuda")
        bits = torch.ceil(torch.log2(x.abs().amax(2, keepdim=True) / 6.0)) + 127
        x = x * torch.exp2(127 - bits)
        code = torch.bucketize(x.abs(), at, out_int32=True).to(torch.uint8) | (x < 0).to(torch.uint8) << 3
        code = code.view(n, a, 2)
        pool[i:i + n, :a] = code[..., 0] | code[..., 1] << 4
        pool[i:i + n, a:a + c] = bits.to(torch.uint8).view(n, c)
    return pool


def _table(lengths, page, g, longest=0, more=0):
    """A block table of randomly placed pages for contexts of these lengths, the pages of the pool (room for
    the longest of each, and `more` pages a sequence besides), and a table of those."""
    need = [-(-n // page) for n in lengths]
    used = max(1, sum(need), len(need) * -(-longest // page))
    pages = used + more * len(lengths)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    first = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    at = first[:, None] + torch.arange(max(1, max(need)), device="cuda")
    return order[at.clamp(max=used - 1)].contiguous(), pages, order[used:].view(len(lengths), more).contiguous()


def _cu(lengths):
    return torch.tensor([0] + list(lengths), device="cuda").cumsum(0).int()


def _rows(n, heads, pad, g):
    """bf16 [n, heads, DIM], a part of wider rows where there is a pad, as a joint projection leaves it."""
    return torch.randn(n, heads * DIM + pad, generator=g, device="cuda").bfloat16()[:, :heads * DIM].view(n, heads, DIM)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op, kv = case["op"], case["kv"]
    lengths = _lengths(case, seed)
    if op == "prefill":
        q_len, before = [a for a, _ in lengths], [b for _, b in lengths]
        k_len = [a + b for a, b in lengths]
        s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = _cu(q_len), _cu(k_len), max(q_len), max(k_len)
        s["q"] = _rows(sum(q_len), kv * case["group"], 0, g)
        s["k"], s["v"] = _rows(sum(k_len), kv, 0, g), _rows(sum(k_len), kv, 0, g)
        return s
    page = case["page"]
    if op == "store":
        # new tokens of several sequences, each at the start of its pages; a few keys' channels are larger
        s["table"], pages, _ = _table(lengths, page, g)
        s["pool"] = _pool(pages, page, kv, g)
        s["cu"] = _cu(lengths)
        wide = 1 + 7 * (torch.rand(DIM, generator=g, device="cuda") < 0.05).bfloat16()
        s["k"] = _rows(case["tokens"], kv, case["pad"], g)
        s["k"].mul_(wide)
        s["v"] = _rows(case["tokens"], kv, case["pad"], g)
        row = torch.arange(case["tokens"], device="cuda")
        seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
        pos = row - s["cu"][seq]
        s["slots"] = s["table"][seq, pos // page].long() * page + pos % page
        s["k_out"] = torch.empty(case["tokens"], kv, DIM, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    elif op == "sparse":
        s["table"], pages, _ = _table(lengths, page, g)
        s["pool"] = _pool(pages, page, kv, g)
        ctx = torch.tensor(lengths, device="cuda")
        n = ctx.clamp(max=case["topk"])
        i = torch.arange(case["topk"], device="cuda")
        lo, hi = i * ctx[:, None] // n[:, None], (i + 1) * ctx[:, None] // n[:, None]
        u = torch.rand(lo.shape, generator=g, device="cuda")
        pos = torch.minimum(lo + (u * (hi - lo)).long(), (hi - 1).clamp(min=0))
        block = (pos // page).clamp(max=s["table"].shape[1] - 1)
        slot = s["table"].gather(1, block).long() * page + pos % page
        s["slots"] = slot[i < n[:, None]].int()
        s["indptr"] = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)]).int()
        s["q"] = _rows(case["rows"], kv * case["group"], 0, g)
    else:
        new = -(-case["budget"] // page) if op == "evict" else 0
        s["table"], pages, s["new_table"] = _table(lengths, page, g, case["hi"] if new else 0, new)
        s["pool"] = _pool(pages, page, kv, g)
        s["ctx"], s["longest"] = torch.tensor(lengths, device="cuda").int(), max(lengths)
        # what earlier steps gave the tokens: a few heavy ones, many light ones; the columns are as many as
        # the longest context may have
        u = torch.rand(case["seqs"], kv, case["hi"], generator=g, device="cuda")
        s["mass"] = u.pow_(4).reciprocal_().clamp_(max=1e3).mul_(1e-3)
        if op != "evict":
            s["q"] = _rows(case["seqs"] * case["next_n"], kv * case["group"], 0, g)
        if op == "weights":
            s["out"] = torch.empty_like(s["mass"])
            # the logarithms that the step's attention left
            s["lse"] = _plain_paged(s)[1]
    return s


# --------------------------------------------------------------------- plain forms


def _parts(pool, page, kv):
    """Views of a pool: codes [pages, 2, kv, page, 64] and scales [pages, 2, kv, page, 4]."""
    a, c = 2 * kv * page * DIM // 2, 2 * kv * page * DIM // GROUP
    return pool[:, :a].unflatten(1, (2, kv, page, DIM // 2)), pool[:, a:a + c].unflatten(1, (2, kv, page, DIM // GROUP))


def _decode(pool, page, kv, slot):
    """Keys and values of these slots in 32 bits, each [kv, ..., DIM]."""
    codes, bits = _parts(pool, page, kv)
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=pool.device)
    value = torch.cat([value, -value])
    p, o = slot // page, slot % page
    got = []
    for side in range(2):
        c = codes[:, side].transpose(0, 1)[:, p, o]
        x = torch.stack([value[(c & 15).int()], value[(c >> 4).int()]], -1).flatten(-2)
        e = bits[:, side].transpose(0, 1)[:, p, o]
        got.append(x * torch.exp2(e.float() - 127).repeat_interleave(GROUP, -1))
    return got


def _softmax_sum(score, value):
    """Values weighted by the softmax of the last dimension (nothing left there: zeros), and the log of its sum."""
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, value) / total.masked_fill(total == 0, 1.0)
    lse = (torch.log(total) + top.masked_fill(total == 0, 0.0)).squeeze(-1)
    return out.bfloat16(), lse


def _plain_prefill(s):
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    nq, nk = s["cu_q"].diff()[:, None], s["cu_k"].diff()[:, None]
    at_q = (s["cu_q"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    at_k = (s["cu_k"][:-1, None] + j).clamp(max=s["k"].shape[0] - 1).long()
    q = s["q"][at_q].float().transpose(1, 2).unflatten(1, (s["kv"], s["group"]))
    k, v = (s[x][at_k].float().transpose(1, 2)[:, :, None] for x in ("k", "v"))
    seen = (j <= (i + nk - nq)[..., None]) & (j < nk)[:, None]
    score = (torch.matmul(q, k.mT) * SCALE).masked_fill(~seen[:, None, None], -math.inf)
    out, lse = _softmax_sum(score, v)
    live = i < nq
    return out.flatten(1, 2).transpose(1, 2)[live], lse.flatten(1, 2).transpose(1, 2)[live]


def _plain_store(s):
    kv, page, pool = s["kv"], s["page"], s["pool"]
    # 64 bits: the rounding to a code, or a group's exponent, may stand next to a border
    x = torch.stack([s["k"], s["v"]], 1).double().unflatten(-1, (DIM // GROUP, GROUP))
    amax = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -126)
    bits = (torch.ceil(torch.log2(amax / 6.0)) + 127).clamp(0, 254)
    x = (x * torch.exp2(127 - bits)).flatten(-2)
    y = x.abs()
    # steps of 1/2, 1 and 2 between codes below 2, 4 and 6; ties to even
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = torch.round(y / step) * step
    code = torch.where(y < 2, y * 2, torch.where(y < 4, y + 2, y / 2 + 4)).clamp(max=7).to(torch.uint8)
    code = code | torch.signbit(x).to(torch.uint8) << 3
    codes, scales = _parts(pool, page, kv)
    p, o = s["slots"] // page, s["slots"] % page
    codes[p, :, :, o] = code[..., ::2] | code[..., 1::2] << 4
    scales[p, :, :, o] = bits[..., 0].to(torch.uint8)
    row = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    pos = row - s["cu"][seq]
    k, v = _decode(pool, page, kv, s["table"][seq, pos // page].long() * page + pos % page)
    s["k_out"].copy_(k.transpose(0, 1).bfloat16())
    s["v_out"].copy_(v.transpose(0, 1).bfloat16())
    return s["k_out"], s["v_out"]


def _plain_sparse(s):
    i = torch.arange(s["topk"], device="cuda")
    first, n = s["indptr"][:-1, None].long(), (s["indptr"][1:] - s["indptr"][:-1])[:, None]
    slot = s["slots"][(first + i).clamp(max=s["slots"].numel() - 1)].long()
    k, v = _decode(s["pool"], s["page"], s["kv"], slot)  # [kv, rows, topk, DIM]
    q = s["q"].float().unflatten(1, (s["kv"], s["group"])).transpose(0, 1)
    score = (torch.matmul(q, k.mT) * SCALE).masked_fill((i >= n)[:, None], -math.inf)
    out, lse = _softmax_sum(score, v)
    return out.transpose(0, 1).flatten(1, 2), lse.transpose(0, 1).flatten(1, 2)


def _scores_paged(s):
    """Scores [kv, seqs, next_n, group, longest] and the values [kv, seqs, longest, DIM]."""
    b, n, kv, group = s["seqs"], s["next_n"], s["kv"], s["group"]
    pos = torch.arange(s["longest"], device="cuda")
    slot = s["table"][:, pos // s["page"]].long() * s["page"] + pos % s["page"]
    k, v = _decode(s["pool"], s["page"], kv, slot)
    q = s["q"].float().view(b, n, kv, group, DIM).permute(2, 0, 1, 3, 4).flatten(2, 3)
    score = (torch.matmul(q, k.mT) * SCALE).unflatten(2, (n, group))
    end = s["ctx"][:, None] - n + 1 + torch.arange(n, device="cuda")
    return score.masked_fill((pos >= end[..., None])[:, :, None], -math.inf), v


def _plain_paged(s):
    b, n, kv, group = s["seqs"], s["next_n"], s["kv"], s["group"]
    score, v = _scores_paged(s)
    out, lse = _softmax_sum(score.flatten(2, 3), v)
    out = out.unflatten(2, (n, group)).permute(1, 2, 0, 3, 4).reshape(b * n, kv * group, DIM)
    return out, lse.unflatten(2, (n, group)).permute(1, 2, 0, 3).reshape(b * n, kv * group)


def _plain_weights(s):
    score, _ = _scores_paged(s)
    lse = s["lse"].view(s["seqs"], s["next_n"], s["kv"], s["group"]).permute(2, 0, 1, 3)[..., None]
    # a row that sees nothing (its logarithm is -inf) gives nothing
    w = torch.exp(score - lse.masked_fill(lse == -math.inf, 0.0)).sum((2, 3)).transpose(0, 1)
    s["out"].copy_(s["mass"])
    s["out"][..., :s["longest"]] += w
    return s["out"]


def _plain_evict(s):
    b, kv, page, budget, recent = s["seqs"], s["kv"], s["page"], s["budget"], s["recent"]
    mass, ctx = s["mass"], s["ctx"].long()[:, None, None]
    # the sum of a token's heads in 64 bits, then rounded: its order is the selection's
    score = mass.double().sum(1, keepdim=True).float() if s["whole"] else mass
    t = torch.arange(score.shape[-1], device="cuda")
    score = torch.where(t >= ctx - recent, math.inf, score).masked_fill(t >= ctx, -math.inf)
    # the heaviest first, ties to the lowest index, then by position; places past the kept ones: -1
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.nn.functional.pad(order, (0, max(0, budget - order.shape[-1])), value=1 << 40)
    left = torch.arange(budget, device="cuda") < ctx
    order = torch.sort(order.masked_fill(~left, 1 << 40)).values
    keep = torch.where(left, order, -1)
    at = keep.clamp(min=0).expand(b, kv, budget)
    new_mass = mass.gather(2, at).masked_fill(~left, 0.0)
    codes, bits = _parts(s["pool"], page, kv)
    seq, head = torch.arange(b, device="cuda")[:, None, None], torch.arange(kv, device="cuda")[:, None]
    live = left.expand(b, kv, budget)
    p, o = s["table"].long()[seq, at // page], at % page
    j = torch.arange(budget, device="cuda")
    to_p, to_o = s["new_table"].long()[:, None, j // page].expand(b, kv, budget), (j % page).expand(b, kv, budget)
    head = head.expand(b, kv, budget)
    for x in (codes, bits):
        x.transpose(1, 2)[to_p[live], head[live], :, to_o[live]] = x.transpose(1, 2)[p[live], head[live], :, o[live]]
    return keep.int(), s["ctx"].clamp(max=budget), new_mass, s["pool"]


def run(s):
    op = s["op"]
    if not own:
        return {"prefill": _plain_prefill, "store": _plain_store, "sparse": _plain_sparse, "paged": _plain_paged,
                "weights": _plain_weights, "evict": _plain_evict}[op](s)
    import sparse_attention_indexer_mxfp4_gb300 as idx
    if op == "prefill":
        return idx.idx_grouped_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], SCALE)
    if op == "store":
        idx.idx_kv4_store(s["k"], s["v"], s["pool"], s["page"], s["slots"])
        return idx.idx_kv4_gather(s["pool"], s["page"], s["table"], s["cu"], s["k_out"], s["v_out"])
    if op == "sparse":
        return idx.idx_kv4_attention(s["q"], s["pool"], s["page"], s["kv"], s["slots"], s["indptr"], SCALE)
    if op == "paged":
        return idx.idx_paged_kv4_attention(s["q"], s["pool"], s["page"], s["kv"], s["table"], s["ctx"], s["next_n"],
                                           SCALE, s["longest"])
    if op == "weights":
        return idx.idx_paged_kv4_weights(s["q"], s["pool"], s["page"], s["kv"], s["table"], s["ctx"], s["next_n"],
                                         SCALE, s["longest"], s["lse"], s["mass"], s["out"])
    keep, lens, mass = idx.idx_kv4_evict(s["mass"], s["ctx"], s["budget"], s["recent"], s["pool"], s["page"],
                                         s["table"], s["new_table"], whole_tokens=s["whole"])
    return keep, lens, mass, s["pool"]


def work(case):
    op, kv = case["op"], case["kv"]
    token = 2 * (DIM // 2 + DIM // GROUP)  # of one key head
    lengths = _lengths(case, 1)
    if op == "prefill":
        h = kv * case["group"]
        pairs = sum(a * b + a * (a + 1) / 2 for a, b in lengths)
        nq, nk = sum(a for a, _ in lengths), sum(a + b for a, b in lengths)
        return {"bytes": nq * h * (4 * DIM + 4) + 4 * nk * kv * DIM, "flops": 4 * h * pairs * DIM}
    if op == "store":
        n = case["tokens"] * kv
        return {"bytes": n * (4 * DIM + token) + 8 * case["tokens"] + n * (token + 4 * DIM), "flops": n * 8 * DIM}
    if op == "evict":
        seen, kept = sum(lengths), sum(min(n, case["budget"]) for n in lengths)
        lists = kept * (1 if case["whole"] else kv)
        return {"bytes": seen * kv * 4 + kept * kv * (2 * token + 4) + 4 * lists, "flops": seen * kv}
    h = kv * case["group"]
    if op == "sparse":
        rows, read = case["rows"], sum(min(n, case["topk"]) for n in lengths)
        pairs, ids = read, read
    else:
        rows, read = case["seqs"] * case["next_n"], sum(lengths)
        pairs = sum(max(0, n - j) for n in lengths for j in range(case["next_n"]))
        ids = read / case["page"]
    if op == "weights":
        return {"bytes": rows * h * (2 * DIM + 4) + read * kv * (token / 2 + 8) + 4 * ids, "flops": 2 * h * pairs * DIM}
    return {"bytes": rows * h * (4 * DIM + 4) + read * kv * token + 4 * ids, "flops": 4 * h * pairs * DIM}


# ------------------------------------------------------------------ the definition


def _token64(s, slot, head, side):
    """Keys (side 0) or values (1) of one key head at these slots in 64 bits, byte by byte by the page's
    definition."""
    page, kv, half, groups = s["page"], s["kv"], DIM // 2, DIM // GROUP
    line, at = s["pool"][slot // page], (slot % page)[:, None]
    take = lambda first, n: line.gather(1, first + at * n + torch.arange(n, device="cuda")).long()  # noqa: E731
    byte = take((side * kv + head) * page * half, half)
    x = torch.empty(slot.numel(), DIM, dtype=torch.float64, device="cuda")
    for i, c in enumerate((byte & 15, byte >> 4)):
        e, m = c >> 1 & 3, (c & 1).double()
        mag = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1).double())
        x[:, i::2] = torch.where(c >> 3 == 1, -mag, mag)
    bits = take(2 * kv * page * half + (side * kv + head) * page * groups, groups)
    return (x.view(-1, groups, GROUP) * 2.0 ** (bits - 127).double()[..., None]).flatten(1)


def _nearest(x):
    """x rounded to e2m1 codes under the least power of two that keeps its group within 6 (ties to the even code)."""
    y = x.double().unflatten(-1, (DIM // GROUP, GROUP))
    m, e = torch.frexp(y.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -126) / 6.0)
    scale = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e).clamp(-127, 127))
    code = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    below = torch.searchsorted(code, (y / scale).abs().clamp(max=6).contiguous(), right=True) - 1
    above = (below + 1).clamp(max=7)
    down, up = (y / scale).abs() - code[below], code[above] - (y / scale).abs()
    pick = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    return (torch.where(pick == 7, 6.0, code[pick]) * scale).copysign(y).flatten(-2)


def _attend64(q, k, v, seen=None):
    """q [n, d], k [m, d], v [m, e], seen [n, m] or None."""
    w = q @ k.mT * SCALE
    if seen is not None:
        w = torch.where(seen, w, -math.inf)
    lse = torch.logsumexp(w, -1)
    return torch.exp(w - lse[..., None]).nan_to_num(0.0) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    op, kv = case["op"], case["kv"]
    if op == "store":
        # a token is read back from where it was written: its values, each the nearest code of its group
        return _nearest(s["k"]), _nearest(s["v"])
    if op == "evict":
        keep, lens, mass = [], [], []
        for b, n in enumerate(s["ctx"].tolist()):
            kept = min(n, case["budget"])
            lens.append(kept)
            last = min(case["recent"], kept)
            m = s["mass"][b, :, :n]
            score = sum(m.double()).float()[None] if case["whole"] else m
            for row in score.cpu().tolist():
                old = sorted(range(n - last), key=lambda i: (-row[i], i))[:kept - last]
                keep.append(sorted(old) + list(range(n - last, n)) + [-1] * (case["budget"] - kept))
        keep = torch.tensor(keep, device="cuda").view(case["seqs"], -1, case["budget"])
        for b in range(case["seqs"]):
            for h in range(kv):
                at = keep[b, h % keep.shape[1]]
                mass.append(torch.where(at >= 0, s["mass"][b, h][at.clamp(min=0)], 0.0).double())
        return keep.int(), torch.tensor(lens, device="cuda").int(), torch.stack(mass).view(case["seqs"], kv, -1), None
    group = case["group"]
    h = kv * group
    if op == "prefill":
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        out = torch.empty(cq[-1], h, DIM, dtype=torch.float64, device="cuda")
        lse = torch.empty(cq[-1], h, dtype=torch.float64, device="cuda")
        for b in range(case["seqs"]):
            n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
            seen = torch.ones(n, m, dtype=torch.bool, device="cuda").tril(m - n)
            for i in range(h):
                k, v = (s[x][ck[b]:ck[b + 1], i // group].double() for x in ("k", "v"))
                out[cq[b]:cq[b + 1], i], lse[cq[b]:cq[b + 1], i] = _attend64(s["q"][cq[b]:cq[b + 1], i].double(), k, v,
                                                                          seen)
        return out, lse
    if op == "sparse":
        cut = s["indptr"].tolist()
        sets = [([r], s["slots"][cut[r]:cut[r + 1]].long(), [cut[r + 1] - cut[r]]) for r in range(case["rows"])]
    else:
        sets, n = [], case["next_n"]
        for b, m in enumerate(s["ctx"].tolist()):
            pos = torch.arange(m, device="cuda")
            slot = s["table"][b].long()[pos // s["page"]] * s["page"] + pos % s["page"]
            sets.append(([b * n + j for j in range(n)], slot, [max(0, m - n + j + 1) for j in range(n)]))
    rows = s["q"].shape[0]
    out = torch.empty(rows, h, DIM, dtype=torch.float64, device="cuda")
    lse = torch.empty(rows, h, dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if op == "weights" else None
    for b, (at, slot, ends) in enumerate(sets):
        end = torch.tensor(ends, device="cuda").repeat_interleave(group)[:, None]
        seen = torch.arange(slot.numel(), device="cuda") < end
        for i in range(kv):
            q = s["q"][at, i * group:(i + 1) * group].double().flatten(0, 1)
            k = _token64(s, slot, i, 0)
            if op == "weights":
                w = torch.where(seen, q @ k.mT * SCALE, -math.inf)
                # relative to the logarithms that the call is given
                z = s["lse"][at, i * group:(i + 1) * group].double().flatten()[:, None]
                mass[b, i, :slot.numel()] += torch.where(seen, torch.exp(w - z.masked_fill(z == -math.inf, 0.0)), 0).sum(0)
                continue
            o, z = _attend64(q, k, _token64(s, slot, i, 1), seen)
            out[at, i * group:(i + 1) * group] = o.view(len(at), group, DIM)
            lse[at, i * group:(i + 1) * group] = z.view(len(at), group)
    return mass if op == "weights" else (out, lse)
