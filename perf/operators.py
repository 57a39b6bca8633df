"""Operators on a paged cache, as they are measured: attention over a 4-bit cache, writing new
tokens into a cache, and the life of its pages.

A case is a dict; `prepare` makes what a serving program holds before the call, `run` makes one
pass, in elementary torch operations or (`own`) through the framework's calls.

attention  one decode step of softmax attention: `drafts` query positions a row, `heads` query heads
           on `kv_heads` heads of K and V, both in FP4 pages (e2m1 codes, an e4m3 scale per 16
           elements); over every cached token (k = 0) or over a list of k tokens per position.
append     new tokens of every row are quantised and written to the last positions of their rows.
pages      the block tables and page counts of a batch: rows take over other rows' tokens (fork),
           shrink or grow (pages freed, taken, copied before they are written), the pool is compacted,
           pages are copied.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def attention(name, batch, drafts, heads, kv_heads, dim, page, lo, hi, k=0, type="bf16", lse=False):
    return {"name": name, "op": "attention", "batch": batch, "drafts": drafts, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "lo": lo, "hi": hi, "k": k, "type": type, "lse": lse}


def append(name, cache, batch, lo, hi, past, kv_heads, dim, page, type="bf16", values=False):
    return {"name": name, "op": "append", "cache": cache, "batch": batch, "lo": lo, "hi": hi, "past": past,
            "kv_heads": kv_heads, "dim": dim, "page": page, "type": type, "values": values}


def pages(name, work, batch, page, lo, hi, kv_heads, dim):
    return {"name": name, "op": "pages", "work": work, "batch": batch, "page": page, "lo": lo, "hi": hi,
            "kv_heads": kv_heads, "dim": dim}


def listed():
    return [
        # one user's next token over a short context: latency
        attention("one row", 1, 1, 32, 1, 128, 64, 1000, 1000),
        # a decode batch with grouped heads, ragged contexts
        attention("grouped heads", 64, 1, 64, 8, 128, 64, 1024, 8192, lse=True),
        # long contexts, two draft positions a row, every head on one K and V
        attention("long drafts", 32, 2, 64, 1, 128, 64, 32768, 131072),
        # the indexer's 2048 best tokens of each row
        attention("selected", 128, 1, 32, 1, 128, 64, 512, 16384, k=2048),
        # a few rows' selected tokens, three drafts, an odd number of heads and tokens, half precision
        attention("selected odd", 5, 3, 21, 3, 64, 16, 1, 9000, k=777, type="f16", lse=True),
        # the tokens of one decode step into the K and V of a 4-bit cache
        append("append step", "fp4", 128, 1, 1, 16384, 1, 128, 64),
        # prompts of many lengths into a 4-bit cache with grouped heads
        append("append prompts", "fp4", 24, 1, 4001, 0, 8, 128, 64, values=True),
        # prompts into the indexer's 8-bit cache
        append("append index", "fp8", 31, 0, 8191, 4096, 1, 128, 64, type="f16", values=True),
        # beam search: rows take over other rows, then every row grows by a token
        pages("beams", "beams", 64, 64, 1000, 8192, 1, 128),
        # a large batch's step: rows end, rows grow, rows begin
        pages("turnover", "turnover", 2048, 64, 0, 4096, 1, 64),
        # a pool with holes is packed to its front
        pages("compact", "compact", 300, 64, 512, 4096, 1, 128),
        # pages of shared prompts are copied for new rows
        pages("copy", "copy", 77, 16, 1, 20001, 2, 128),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attention", "attention", "append", "pages"])
    dim, page, type = rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), rng.choice(["bf16", "f16"])
    if op == "attention":
        drafts, kv_heads = rng.randint(1, 4), rng.choice([1, 1, 2, 4, 8])
        group = log(1, 128 // drafts)
        k = rng.choice([0, 0, log(1, 4096)])
        batch = log(1, 256)
        k = min(k, max(1, int(2e6 / (batch * drafts * kv_heads))))
        most = max(16, min(131072, int(4e6 / (batch * kv_heads)), int(4e6 * 64 / (batch * kv_heads * drafts * group))))
        hi = log(1, most)
        return {k_: v for k_, v in attention("", batch, drafts, kv_heads * group, kv_heads, dim, page, log(1, hi), hi, k, type,
                                             rng.random() < 0.5).items() if k_ != "name"}
    if op == "append":
        cache = rng.choice(["fp4", "fp4", "fp8"])
        kv_heads = 1 if cache == "fp8" else rng.choice([1, 2, 4, 8])
        batch = log(1, 512)
        hi = log(1, max(1, 400000 // (batch * kv_heads)))
        return {k_: v for k_, v in append("", cache, batch, rng.randint(0, hi), hi, rng.choice([0, log(1, 8192)]), kv_heads,
                                          dim, page, type, rng.random() < 0.5).items() if k_ != "name"}
    batch = log(1, 2048)
    hi = log(1, max(1, 1200000 // batch))
    return {k_: v for k_, v in pages("", rng.choice(["beams", "turnover", "compact", "copy"]), batch, page, rng.randint(0, hi),
                                     hi, rng.choice([1, 2]), dim).items() if k_ != "name"}


# ---------------------------------------------------------------- inputs
def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def whole(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int64)


def lengths(g, case):
    """From lo to hi in even steps, in any order: ragged rows, and the same sum for every seed."""
    B = case["batch"]
    n = case["hi"] - (case["hi"] - case["lo"]) * torch.arange(B, device=DEV) // max(1, B - 1)
    return n[torch.randperm(B, generator=g, device=DEV)]


def table_of(g, n, page, pool, width):
    """Block tables of rows with n tokens: pages of a shuffled pool, -1 behind a row's last."""
    counts = (n + page - 1) // page
    used = torch.arange(width, device=DEV)[None, :] < counts[:, None]
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full(used.shape, -1, dtype=torch.int32, device=DEV)
    table[used] = order[: int(counts.sum())]
    return table


def fp4_bytes(page, dim):
    return page * (dim // 2 + dim // 16)


def activations(g, shape, type=torch.float32):
    """What a projection gives: tokens of unequal size, a few large channels."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(shape[:-1], generator=g, device=DEV))[..., None]
    x[..., :: shape[-1] // 4] *= 4.0
    return x.to(type)


def to_e2m1(x):
    """The nearest e2m1 code of each value, ties to the even code, no negative zero."""
    a = x.abs()
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
    code += (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte()
    return code + 8 * ((x < 0) & (code > 0)).byte()


def to_fp4(x):
    """x [..., dim] fp32 as packed e2m1 codes [..., dim / 2] and e4m3 scales [..., dim / 16]."""
    b = x.unflatten(-1, (-1, 16))
    most = b.abs().amax(-1)
    s = (most / torch.full_like(most, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn).float()  # by a tensor: a quotient, not a product with 1/6
    least = torch.full_like(s, 2.0**-9)
    scale = torch.where(s == 0, least, s).to(torch.float8_e4m3fn)
    code = to_e2m1(b / scale.float()[..., None]).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def fp4_pool(g, count, heads, page, dim):
    code, scale = to_fp4(activations(g, (count, heads, page, dim)))
    both = torch.cat((code.flatten(2), scale.view(torch.uint8).flatten(2)), 2)
    return both.reshape(count, -1)


def prepare(case, seed):
    g = generator(seed)
    if case["op"] == "attention":
        return prepare_attention(case, g)
    if case["op"] == "append":
        return prepare_append(case, g)
    return prepare_pages(case, g)


def prepare_attention(case, g):
    B, n, H, D, page, k = case["batch"], case["drafts"], case["heads"], case["dim"], case["page"], case["k"]
    ctx = lengths(g, case)
    pool = int(((ctx + page - 1) // page).sum())
    s = {"op": "attention", "case": case, "table": table_of(g, ctx, page, pool, -(-case["hi"] // page)), "context": ctx.to(torch.int32)}
    s["q"] = (2.0 * torch.randn(B, n, H, D, generator=g, device=DEV)).to(TYPES[case["type"]])
    s["k_cache"] = fp4_pool(g, pool, case["kv_heads"], page, D)
    s["v_cache"] = fp4_pool(g, pool, case["kv_heads"], page, D)
    s["list"] = None
    if k:  # distinct tokens of each position in ascending order, -1 behind them
        last = (ctx[:, None] - n + 1 + torch.arange(n, device=DEV)).clamp(min=0)
        wide = max(k, case["hi"])
        rank = torch.rand(B, n, wide, generator=g, device=DEV)
        rank.masked_fill_(torch.arange(wide, device=DEV) >= last[..., None], 2.0)
        best, token = rank.topk(k, dim=-1, largest=False)
        token = torch.where(best < 2.0, token, wide).sort(-1).values
        s["list"] = torch.where(token < wide, token, -1).to(torch.int32)
    if own:  # the split of the rows over the GPU, kept for all layers of a step, and the partial results' memory, for all steps
        import paged_mqa_logits_b200 as mq

        s["plan"] = None if k else mq.mqa_logits_schedule(s["context"])
        s["work"] = mq.mqa_attention_workspace(s["q"], kv_heads=case["kv_heads"], topk=k)
    return s


def prepare_append(case, g):
    B, page, D, heads = case["batch"], case["page"], case["dim"], case["kv_heads"]
    new = lengths(g, case)
    ctx = new + whole(g, 0, case["past"], B)
    pool = int(((new + case["past"] + page - 1) // page).sum())
    offsets = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = new.cumsum(0)
    T = int(offsets[-1])
    s = {"op": "append", "case": case, "table": table_of(g, ctx, page, pool, -(-(case["hi"] + case["past"]) // page)), "context": ctx.to(torch.int32),
         "offsets": offsets.to(torch.int32)}
    if case["cache"] == "fp8":
        s["k"] = activations(g, (T, D), TYPES[case["type"]])
        s["k_cache"] = torch.zeros(pool, page * (D + 4), dtype=torch.uint8, device=DEV)
    else:  # K and V are parts of one projection's output
        kv = activations(g, (T, 2, heads, D), TYPES[case["type"]])
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["k_cache"], s["v_cache"] = torch.zeros(2, pool, heads * fp4_bytes(page, D), dtype=torch.uint8, device=DEV)
    return s


def prepare_pages(case, g):
    B, page, D, work = case["batch"], case["page"], case["dim"], case["work"]
    n = lengths(g, case)
    counts = (n + page - 1) // page
    live = int(counts.sum())
    spare = {"beams": 4 * B, "turnover": live // 4 + 8 * B, "compact": live, "copy": live + 1}[work]
    pool = live + spare
    grow = whole(g, 1, 4, B) if work == "turnover" else torch.ones_like(n)
    width = (case["hi"] + 4) // page + 1
    s = {"op": "pages", "case": case, "page": page, "table": table_of(g, n, page, pool, width), "lens": n.to(torch.int32)}
    refs = torch.zeros(pool + 1, dtype=torch.int32, device=DEV)
    refs.index_add_(0, torch.where(s["table"] < 0, pool, s["table"]).flatten().long(), torch.ones(B * width, dtype=torch.int32, device=DEV))
    s["refs"] = refs[:pool].contiguous()
    sizes = (page * (D + 4), case["kv_heads"] * fp4_bytes(page, D), case["kv_heads"] * fp4_bytes(page, D))
    s["caches"] = [torch.randint(0, 256, (pool, b), generator=g, device=DEV, dtype=torch.uint8) for b in sizes]
    rows = torch.arange(B, device=DEV)
    if work == "beams":  # four rows a prompt; each goes on from one of the four
        parents = torch.minimum(rows // 4 * 4 + whole(g, 0, 3, B), torch.tensor(B - 1, device=DEV))
        s["parents"], s["new"] = parents.to(torch.int32), (n[parents] + 1).to(torch.int32)
    elif work == "turnover":  # a tenth ends, a tenth of the places takes new prompts, the others grow
        fate = torch.rand(B, generator=g, device=DEV)
        s["parents"] = torch.where(fate < 0.2, -1, rows).to(torch.int32)
        new = torch.where(fate < 0.1, 0, torch.where(fate < 0.2, whole(g, case["lo"], case["hi"], B), n + grow))
        s["new"] = new.to(torch.int32)
    elif work == "copy":
        free = torch.nonzero(s["refs"] == 0)[:, 0]
        src = s["table"][s["table"] >= 0]
        order = torch.randperm(src.numel(), generator=g, device=DEV)
        s["src"] = src[order].contiguous()
        s["dst"] = free[torch.randperm(free.numel(), generator=g, device=DEV)][: src.numel()].to(torch.int32)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    if state["op"] == "attention":
        return (own_attention if own else plain_attention)(state)
    if state["op"] == "append":
        return (own_append if own else plain_append)(state)
    return (own_pages if own else plain_pages)(state)


def own_attention(s):
    import paged_mqa_logits_b200 as mq

    c = s["case"]
    return mq.paged_mqa_attention_fp4(s["q"], s["k_cache"], s["v_cache"], s["table"], s["context"], s["plan"],
                                      kv_heads=c["kv_heads"], page_size=c["page"], indices=s["list"], with_lse=c["lse"],
                                      workspace=s["work"])


def own_append(s):
    import paged_mqa_logits_b200 as mq

    c = s["case"]
    if c["cache"] == "fp8":
        values = mq.mqa_cache_append_fp8(s["k"], s["k_cache"], s["table"], s["context"], s["offsets"], page_size=c["page"],
                                         with_values=c["values"])
        return (s["k_cache"], values) if c["values"] else s["k_cache"]
    values = mq.mqa_cache_append_fp4(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["context"], s["offsets"],
                                     page_size=c["page"], with_values=c["values"])
    return (s["k_cache"], s["v_cache"], *(values if c["values"] else ()))


def own_pages(s):
    import paged_mqa_logits_b200 as mq

    work, page = s["case"]["work"], s["page"]
    if work == "copy":
        mq.mqa_pages_copy(s["caches"], s["src"], s["dst"])
        return s["caches"]
    refs = s["refs"].clone()
    if work == "compact":
        table = s["table"].clone()
        src, dst, count, places = mq.mqa_pages_compact(table, s["lens"], refs, page_size=page)
        mq.mqa_pages_copy(s["caches"], src, dst, count)
        return table, refs, src, dst, count, places, s["caches"]
    table, lens = mq.mqa_pages_fork(s["table"], s["lens"], s["parents"], refs, page_size=page)
    src, dst = mq.mqa_pages_resize(table, lens, s["new"], refs, page_size=page)
    mq.mqa_pages_copy(s["caches"], src, dst)
    return table, lens, refs, src, dst, s["caches"]


def fp4_values(cache, heads, page, dim):
    """Pages [..., bytes] as fp32 [..., heads, page, dim]."""
    c = cache.unflatten(-1, (heads, -1))
    code, scale = c[..., : page * dim // 2], c[..., page * dim // 2:]
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=cache.device)
    both = torch.stack((value[(code & 15).int()], value[(code >> 4).int()]), -1)
    both = both.reshape(*c.shape[:-1], page, dim // 16, 16)
    scale = scale.contiguous().view(torch.float8_e4m3fn).float().reshape(*c.shape[:-1], page, dim // 16, 1)
    return (both * scale).flatten(-2)


def plain_attention(s):
    c = s["case"]
    B, n, H, D, page, heads = c["batch"], c["drafts"], c["heads"], c["dim"], c["page"], c["kv_heads"]
    G = H // heads
    last = (s["context"].long()[:, None] - n + 1 + torch.arange(n, device=DEV)).clamp(min=0)
    q = s["q"].float().unflatten(2, (heads, G))
    if s["list"] is None:
        table = s["table"].clamp(min=0).long()
        T = table.shape[1] * page
        k, v = (fp4_values(x[table], heads, page, D).transpose(1, 2).reshape(B, heads, T, D) for x in (s["k_cache"], s["v_cache"]))
        ok = (torch.arange(T, device=DEV) < last[..., None])[:, None, :, None]  # [B, 1, n, 1, T]
        score = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, heads, n * G, D), k.transpose(2, 3)).view(B, heads, n, G, T)
    else:
        token = s["list"].long()
        ok = ((token >= 0) & (token < last[..., None]))
        token = torch.where(ok, token, 0)
        at = torch.gather(s["table"].long(), 1, (token // page).flatten(1)).view_as(token).clamp(min=0)
        slot = token % page
        code, scale = page * D // 2, page * (D // 2 + D // 16)
        take = torch.cat((slot[..., None] * (D // 2) + torch.arange(D // 2, device=DEV),
                          code + slot[..., None] * (D // 16) + torch.arange(D // 16, device=DEV)), -1)  # one token as a page of one
        take = torch.arange(heads, device=DEV)[:, None] * scale + take[..., None, :]
        k, v = (fp4_values(x[at[..., None, None], take].flatten(-2), heads, 1, D).squeeze(-2).transpose(2, 3) for x in (s["k_cache"], s["v_cache"]))
        ok = ok[:, None, :, None]
        k, v = k.transpose(1, 2), v.transpose(1, 2)  # [B, heads, n, k, D]
        score = torch.matmul(q.permute(0, 2, 1, 3, 4), k.transpose(3, 4))  # [B, heads, n, G, k]
    score = (score / math.sqrt(D)).masked_fill(~ok, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    if s["list"] is None:
        o = torch.matmul(p.view(B, heads, n * G, -1), v).view(B, heads, n, G, D)
    else:
        o = torch.matmul(p, v)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, n, H, D).to(s["q"].dtype)
    if not c["lse"]:
        return o
    return o, (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, n, H)


def new_slots(s):
    """Row, page and slot of each new token."""
    T, page = s["k"].shape[0], s["case"]["page"]
    i = torch.arange(T, device=DEV)
    row = torch.searchsorted(s["offsets"].long(), i, right=True) - 1
    at = s["context"].long()[row] - s["offsets"].long()[row + 1] + i
    return s["table"].long()[row, at // page], at % page


def plain_append(s):
    c = s["case"]
    page, D = c["page"], c["dim"]
    place, slot = new_slots(s)
    if c["cache"] == "fp8":
        x = s["k"].float()
        amax = x.abs().amax(-1)
        part, power = torch.frexp(amax)  # amax = part * 2^power, part in [0.5, 1); 448 = 0.875 * 2^9
        power = torch.where(amax > 0, power - 9 + (part > 0.875), 0).clamp(min=-126).to(torch.int32)
        scale = ((power + 127) << 23).view(torch.float32)  # 2^power
        code = (x / scale[:, None]).to(torch.float8_e4m3fn)
        s["k_cache"][:, : page * D].unflatten(-1, (page, D))[place, slot] = code.view(torch.uint8)
        s["k_cache"][:, page * D:].unflatten(-1, (page, 4))[place, slot] = scale[:, None].view(torch.uint8)
        return (s["k_cache"], (code.float() * scale[:, None]).to(s["k"].dtype)) if c["values"] else s["k_cache"]
    outs = []
    heads = torch.arange(c["kv_heads"], device=DEV)[None, :]
    for x, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        code, scale = to_fp4(x.float())
        view = cache.unflatten(-1, (c["kv_heads"], -1))
        view[..., : page * D // 2].unflatten(-1, (page, D // 2))[place[:, None], heads, slot[:, None]] = code
        view[..., page * D // 2:].unflatten(-1, (page, D // 16))[place[:, None], heads, slot[:, None]] = scale.view(torch.uint8)
        if c["values"]:
            token = torch.cat((code, scale.view(torch.uint8)), -1).flatten(-2)
            outs.append(fp4_values(token, c["kv_heads"], 1, D).squeeze(-2).to(x.dtype))
    return (s["k_cache"], s["v_cache"], *outs)


def plain_copy(caches, src, dst):
    keep = (src >= 0) & (dst >= 0)
    src, dst = src[keep].long(), dst[keep].long()
    for cache in caches:
        cache[dst] = cache[src]


def plain_pages(s):
    work, page, table, lens = s["case"]["work"], s["page"], s["table"], s["lens"].long()
    if work == "copy":
        plain_copy(s["caches"], s["src"], s["dst"])
        return s["caches"]
    refs = s["refs"].clone()
    P, width = refs.numel(), table.shape[1]
    col = torch.arange(width, device=DEV)[None, :]
    if work == "compact":
        live = refs > 0
        n_live, ids = live.sum(), torch.arange(P, device=DEV)
        mover, hole = live & (ids >= n_live), ~live & (ids < n_live)
        half = P // 2
        src = torch.full((half + 1,), -1, dtype=torch.int64, device=DEV)
        dst = src.clone()
        src[torch.where(mover, mover.cumsum(0) - 1, half)] = torch.where(mover, ids, -1)
        dst[torch.where(hole, hole.cumsum(0) - 1, half)] = torch.where(hole, ids, -1)
        places = torch.where(live, torch.where(mover, dst[(mover.cumsum(0) - 1).clamp(min=0)], ids), -1)
        src, dst = src[:half], dst[:half]
        moved = torch.zeros_like(refs).index_add_(0, places.clamp(min=0), torch.where(live, refs, 0))
        used = col < ((lens + page - 1) // page)[:, None]
        table = torch.where(used, places[table.clamp(min=0).long()], table.long()).to(torch.int32)
        plain_copy(s["caches"], src, dst)
        return table, moved, src.to(torch.int32), dst.to(torch.int32), mover.sum().to(torch.int32).reshape(1), places.to(torch.int32), s["caches"]

    def count(pages, keep, by):
        refs.index_add_(0, torch.where(keep, pages, 0).flatten().long(), (by * keep.int()).flatten().to(torch.int32))

    # fork: every row goes on from its parent's tokens
    count(table, col < ((lens + page - 1) // page)[:, None], -1)
    parents = s["parents"].long()
    lens = torch.where(parents >= 0, lens[parents.clamp(min=0)], 0)
    used = col < ((lens + page - 1) // page)[:, None]
    table = torch.where(used, table[parents.clamp(min=0)], -1)
    count(table, used, 1)
    # resize: pages behind the new end go, rows that grow take the lowest free pages, in order, and
    # get a page of their own in the place of a shared one that they would write to
    new = s["new"].long().clamp(0, width * page)
    had, has = (lens + page - 1) // page, (new + page - 1) // page
    end = table.gather(1, (had - 1).clamp(min=0)[:, None])[:, 0].long()
    grows = new > lens
    shared = grows & (lens % page != 0) & (refs[end.clamp(min=0)] > 1)
    need = torch.where(grows, has - had, 0) + shared
    upto = need.cumsum(0)
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)
    fits = (need == 0) | (upto <= (refs == 0).sum())
    new, grows, shared = torch.where(fits, new, lens), grows & fits, shared & fits
    has = torch.where(fits, has, had)
    first = (upto - need)[:, None]
    gone = (col >= has[:, None]) & (col < had[:, None])
    count(table, gone, -1)
    src = torch.where(shared, end, -1)
    count(end, shared, -1)
    take = (grows[:, None] & (col >= had[:, None]) & (col < has[:, None])) | (shared[:, None] & (col == had[:, None] - 1))
    at = first + shared[:, None] + col - had[:, None]
    fresh = free[at.clamp(0, P - 1)]
    dst = torch.where(shared, free[first[:, 0].clamp(0, P - 1)], -1)
    table = torch.where(take, fresh, torch.where(gone, -1, table.long()))
    count(table, take, 1)
    plain_copy(s["caches"], src, dst)
    return table.to(torch.int32), new.to(torch.int32), refs, src.to(torch.int32), dst.to(torch.int32), s["caches"]


# ---------------------------------------------------------------- cost and truth
def work(case):
    D, page, mean = case["dim"], case["page"], (case["lo"] + case["hi"]) / 2
    B = case["batch"]
    if case["op"] == "attention":
        rows = B * case["drafts"] * case["heads"]
        tokens = B * case["drafts"] * min(case["k"], mean) if case["k"] else B * mean
        data = 2 * tokens * case["kv_heads"] * (D // 2 + D // 16)
        lists = 4 * B * case["drafts"] * case["k"] if case["k"] else 4 * B * math.ceil(mean / page)
        return {"bytes": data + 4 * rows * D + lists + (4 * rows if case["lse"] else 0),
                "flops": 4 * D * case["heads"] * tokens * (1 if case["k"] else case["drafts"])}
    if case["op"] == "append":
        tokens = B * mean * case["kv_heads"] * (1 if case["cache"] == "fp8" else 2)
        held = D + 4 if case["cache"] == "fp8" else D // 2 + D // 16
        return {"bytes": max(1, tokens * (2 * D + held + (2 * D if case["values"] else 0))), "flops": 4 * tokens * D}
    one = page * (D + 4) + 2 * case["kv_heads"] * fp4_bytes(page, D)
    table = B * ((case["hi"] + 4) // page + 1) * 4
    used = B * math.ceil(mean / page)
    if case["work"] == "copy":
        return {"bytes": 2 * used * one + 8 * used, "flops": 0}
    if case["work"] == "compact":  # half the pool is live, half of that lies in the upper half
        return {"bytes": 2 * table + 2 * used * 8 + used * one, "flops": 0}
    copies = B * 0.65 * (page - 1) / page if case["work"] == "beams" else 0
    return {"bytes": 3 * table + 12 * B + 8 * used + 2 * copies * one, "flops": 0}


def fp4_numbers(code, scale):
    """Codes [..., dim / 2] and scale bytes [..., dim / 16] as numbers in 64 bits, from the formats' bits."""
    both = torch.stack((code % 16, code // 16), -1).flatten(-2).double()
    sign, both = torch.where(both >= 8, -1.0, 1.0).double(), both % 8
    power, odd = torch.floor(both / 2), both % 2
    number = sign * torch.where(power > 0, (1 + odd / 2) * 2.0 ** (power - 1), odd / 2)
    b = scale.double()
    b, minus = b % 128, b >= 128
    power, part = torch.floor(b / 8), b % 8
    by = torch.where(power > 0, (1 + part / 8) * 2.0 ** (power - 7), part / 8 * 2.0**-6) * torch.where(minus, -1.0, 1.0)
    return number * by.repeat_interleave(16, -1)


def exact(case, seed):
    if case["op"] == "pages":
        return None  # tables, counts and bytes: nothing is rounded
    s = prepare(case, seed)
    D, page, heads = case["dim"], case["page"], case["kv_heads"]
    if case["op"] == "append":
        return exact_append(s, case)
    n, G = case["drafts"], case["heads"] // heads
    outs = torch.zeros(case["batch"], n, case["heads"], D, dtype=torch.float64, device=DEV)
    logs = torch.full(outs.shape[:-1], -math.inf, dtype=torch.float64, device=DEV)
    context = s["context"].tolist()
    for b in range(case["batch"]):
        def tokens(cache, t):
            c = cache.view(cache.shape[0], heads, -1)
            at, slot = s["table"][b].long()[t // page], t % page
            code = c[:, :, : page * D // 2].view(-1, heads, page, D // 2) if heads == 1 else c[:, :, : page * D // 2].reshape(-1, heads, page, D // 2)
            scale = c[:, :, page * D // 2:].reshape(-1, heads, page, D // 16)
            return fp4_numbers(code[at, :, slot], scale[at, :, slot]).transpose(0, 1)  # [heads, T, D]

        whole_row = torch.arange(context[b], device=DEV)
        kv = None if s["list"] is not None else [tokens(x, whole_row) for x in (s["k_cache"], s["v_cache"])]
        for d in range(n):
            upto = max(0, context[b] - n + 1 + d)
            if s["list"] is None:
                k, v = kv[0][:, :upto], kv[1][:, :upto]
            else:
                t = s["list"][b, d].long()
                t = t[(t >= 0) & (t < upto)]
                k, v = tokens(s["k_cache"], t), tokens(s["v_cache"], t)
            if not k.shape[1]:
                continue
            a = torch.einsum("hgd,htd->hgt", s["q"][b, d].double().view(heads, G, D), k) * D**-0.5
            logs[b, d] = torch.logsumexp(a, -1).flatten()
            outs[b, d] = torch.einsum("hgt,htd->hgd", torch.softmax(a, -1), v).reshape(-1, D)
    return (outs, logs) if case["lse"] else outs


def exact_append(s, case):
    """The values that the cache holds for the new tokens; its bytes have no 64-bit value."""
    if not case["values"]:
        return None

    def below(a):  # the power of two at or below a, exactly: the exponent's bits alone
        return (a.view(torch.int64) >> 52 << 52).view(torch.float64)

    if case["cache"] == "fp8":
        x = s["k"].double()
        most = x.abs().amax(-1, keepdim=True) / 448
        scale = torch.where(below(most) == most, most, 2 * below(most)).clamp(min=2.0**-126)
        scale = torch.where(most > 0, scale, 1.0)
        a = (x / scale).abs()
        step = below(a.clamp(min=2.0**-6)) / 8
        return None, torch.sign(x) * torch.round(a / step) * step * scale
    outs = []
    for x in (s["k"], s["v"]):
        x = x.double().unflatten(-1, (-1, 16))
        sixth = (x.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0)
        step = below(sixth.clamp(min=2.0**-6)) / 8
        scale = torch.round(sixth / step) * step
        scale = torch.where(scale == 0, 2.0**-9, scale)
        a = (x / scale).abs().clamp(max=6.0)
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
        outs.append((torch.sign(x) * torch.round(a / step) * step * scale).flatten(-2))
    return (None, None, *outs)
