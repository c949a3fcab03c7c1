"""Cases of the paged-cache operators: what they compute, in plain torch and by the library.

Four operators that a serving loop runs in this order for every step:

  tables   block tables, slot map and lengths of a batch, built on the GPU from
           the requests' cached and new token counts and a stack of free pages
  append   the step's K/V rows into their slots of the paged cache, and the mean
           key of every page that the step completes
  decode   attention of one new token over each sequence's pages
  sparse   the pages whose mean keys promise most attention mass, chosen for each
           query and KV head, and attention over those pages alone

``own`` false: elementary torch operations in 32 bits (64 for the page scores,
whose order decides between near-equal pages).  ``own`` true: the calls that a
user makes of ``kv_cache_sparsity_b200.hylra``.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    heads = {"hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"}
    return [
        # one decode step of a 16-sequence batch: every request gets one token
        {"name": "tables_decode16", "op": "tables", "batch": 16, "lo": 8192, "hi": 131072,
         "new_lo": 1, "new_hi": 1, "page": 128, "short": False, "pad": 0, "mix": 1},
        # a full scheduler batch, small pages, more demand than free pages
        {"name": "tables_decode1024", "op": "tables", "batch": 1024, "lo": 0, "hi": 4096,
         "new_lo": 1, "new_hi": 1, "page": 16, "short": True, "pad": 0, "mix": 2},
        # chunked prefill: 64 prompts admitted at once, slot map padded to a captured size
        {"name": "tables_prefill64", "op": "tables", "batch": 64, "lo": 0, "hi": 2048,
         "new_lo": 1024, "new_hi": 8192, "page": 16, "short": False, "pad": 77, "mix": 3},
        # one token of each of 16 sequences
        {"name": "append_decode16", "op": "append", "batch": 16, "lo": 8192, "hi": 131072,
         "new_lo": 1, "new_hi": 1, "page": 128, "layout": "hnd", "fused": True, "mix": 4, **heads},
        # prefill of eight prompts that continue a cached prefix
        {"name": "append_prefill8", "op": "append", "batch": 8, "lo": 0, "hi": 1024,
         "new_lo": 4096, "new_hi": 12288, "page": 64, "layout": "nhd", "fused": True, "mix": 5,
         **heads},
        # a short context with few heads: latency
        {"name": "decode_1x4k", "op": "decode", "batch": 1, "idle": 0, "lo": 4001, "hi": 4001,
         "page": 16, "layout": "hnd", "mix": 6, "hq": 8, "hkv": 2, "d": 128, "dtype": "bf16"},
        # many short ragged sequences, some rows of the batch idle
        {"name": "decode_64x2k", "op": "decode", "batch": 64, "idle": 5, "lo": 1, "hi": 4096,
         "page": 16, "layout": "nhd", "mix": 7, "hq": 14, "hkv": 2, "d": 64, "dtype": "fp16"},
        # one long context
        {"name": "decode_1x32k", "op": "decode", "batch": 1, "idle": 0, "lo": 32768, "hi": 32768,
         "page": 128, "layout": "hnd", "mix": 8, **heads},
        # a ragged batch of long contexts: the largest
        {"name": "decode_16x128k", "op": "decode", "batch": 16, "idle": 0, "lo": 8192,
         "hi": 131072, "page": 64, "layout": "hnd", "mix": 9, **heads},
        # the same two kinds of context, attended through chosen pages
        {"name": "sparse_1x32k", "op": "sparse", "batch": 1, "idle": 0, "lo": 32768, "hi": 32768,
         "page": 128, "layout": "hnd", "topk": 16, "sink": 1, "recent": 2, "mix": 10, **heads},
        # small pages, a long list
        {"name": "sparse_4x64k_p16", "op": "sparse", "batch": 4, "idle": 1, "lo": 20000,
         "hi": 65536, "page": 16, "layout": "nhd", "topk": 256, "sink": 4, "recent": 8, "mix": 11,
         "hq": 32, "hkv": 8, "d": 128, "dtype": "fp16"},
        {"name": "sparse_16x128k", "op": "sparse", "batch": 16, "idle": 0, "lo": 8192,
         "hi": 131072, "page": 128, "layout": "hnd", "topk": 32, "sink": 1, "recent": 1,
         "mix": 12, **heads},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["tables", "append", "decode", "sparse"])
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 30)
    if op == "tables":
        batch = log(1, 1024)
        many = rng.random() < 0.5
        new_hi = log(2, max(2, min(8192, 260000 // batch))) if many else 1
        return {"op": op, "batch": batch, "lo": 0, "hi": log(1, 32768), "new_lo": 1,
                "new_hi": new_hi, "page": page, "short": rng.random() < 0.3,
                "pad": rng.choice([0, 0, log(1, 300)]), "mix": mix}
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    heads = {"hkv": hkv, "hq": hkv * rng.randint(1, 8), "d": d,
             "dtype": rng.choice(["bf16", "bf16", "fp16"]), "page": page,
             "layout": rng.choice(["hnd", "nhd"]), "mix": mix}
    if op == "append":
        batch = log(1, 256)
        many = rng.random() < 0.5
        new_hi = log(2, max(2, min(12288, 65536 // batch))) if many else 1
        # the cache held before the step stays within 2**20 rows
        hi = log(1, min(131072, max(1, (1 << 20) // batch)))
        return {"op": op, "batch": batch, "lo": 0, "hi": hi, "new_lo": 1, "new_hi": new_hi,
                "fused": rng.random() < 0.5, **heads}
    batch = log(1, 64)
    hi = log(1, min(131072, (1 << 21) * 8 // (batch * hkv)))
    lo = rng.choice([1, max(1, hi // 8), hi])
    case = {"op": op, "batch": batch, "idle": rng.choice([0, 0, batch // 4]), "lo": lo, "hi": hi,
            **heads}
    if op == "sparse":
        recent = rng.randint(1, 4)
        case.update(topk=log(1, 8192 // page), sink=rng.randint(0, 3), recent=recent)
    return case


# ------------------------------------------------------------------- inputs


def lengths(case):
    """Token counts held before the step (tables, append) or attended (decode, sparse)."""
    rng = random.Random(case["mix"])
    n = [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    for _ in range(case.get("idle", 0)):
        n[rng.randrange(case["batch"])] = 0
    return n


def new_lengths(case):
    rng = random.Random(case["mix"] + 1)
    return [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]


def pages_of(n, page):
    return -(-n // page)


def device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def prepare(case, seed):
    gen = torch.Generator(device=device()).manual_seed(seed * 1009 + case["mix"] % 1000003)
    host = torch.Generator().manual_seed(seed * 31 + 7)
    return {"tables": prepare_tables, "append": prepare_append, "decode": prepare_decode,
            "sparse": prepare_decode}[case["op"]](case, gen, host)


def tables_sizes(case):
    """(pages held, pages asked for, free pages, columns of the table, slots)."""
    page, held, new = case["page"], lengths(case), new_lengths(case)
    have = [pages_of(n, page) for n in held]
    need = [pages_of(n + w, page) - a for n, w, a in zip(held, new, have)]
    free = sum(need) * 3 // 4 if case["short"] else sum(need) + 64
    cols = max(a + w for a, w in zip(have, need))
    return have, need, free, cols, sum(new) + case["pad"]


def to_device(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).to(device())


def held_table(have, cols, order):
    """Rows of the block table, sequence after sequence from the page order; -1 past a row's pages."""
    have = torch.tensor(have)
    first = torch.cumsum(have, 0) - have
    j = torch.arange(cols)
    at = (first[:, None] + j).clamp(max=max(0, len(order) - 1))
    return torch.where(j < have[:, None], order[at], torch.tensor(-1)).to(torch.int32)


def prepare_tables(case, gen, host):
    have, need, free, cols, slots = tables_sizes(case)
    pool = sum(have) + free + 16
    order = torch.randperm(pool, generator=host)
    s = {"case": case, "cached": to_device(lengths(case)), "new": to_device(new_lengths(case)),
         "table": held_table(have, cols, order).to(device()),
         "free": order[sum(have):].to(torch.int32).to(device()),
         "free_count": to_device([free]), "seqlens": to_device([0] * case["batch"]),
         "cu": to_device([0] * (case["batch"] + 1)), "left": to_device([0]),
         "slots": torch.empty(slots, dtype=torch.int32, device=device())}
    if own:
        from kv_cache_sparsity_b200 import hylra as H
        s["shape"] = H.make_paged_shape(case["batch"], 32, 8, case["page"], pool, cols)
        s["ws"] = workspace(H, s["shape"])
    return s


def shape_of(H, case, keys, cols):
    return H.make_paged_shape(case["batch"], case["hq"], case["hkv"], case["page"], len(keys), cols,
                              dtype=H.BF16 if case["dtype"] == "bf16" else H.FP16,
                              head_dim=case["d"], pool=keys)


def workspace(H, shape):
    ws = torch.empty(H.paged_workspace_bytes(shape), dtype=torch.uint8, device=device())
    H.workspace_init(ws)
    return ws


def empty_pool(case, pages):
    """[pages][hkv][page][d]; "nhd" keeps a page's tokens, not its heads, apart in memory."""
    if case["layout"] == "nhd":
        return torch.empty(pages, case["page"], case["hkv"], case["d"], dtype=DTYPES[case["dtype"]],
                           device=device()).transpose(1, 2)
    return torch.empty(pages, case["hkv"], case["page"], case["d"], dtype=DTYPES[case["dtype"]],
                       device=device())


def page_means(keys):
    step = max(1, (1 << 27) // keys[0].numel())
    return torch.cat([k.float().mean(2).to(keys.dtype) for k in keys.split(step)])


def prepare_append(case, gen, host):
    page, held, new = case["page"], lengths(case), new_lengths(case)
    total = [n + w for n, w in zip(held, new)]
    have = [pages_of(n, page) for n in total]
    pool = sum(have) + 3
    order = torch.randperm(pool, generator=host)
    table = held_table(have, max(have), order)
    keys, vals = empty_pool(case, pool), empty_pool(case, pool)
    keys.normal_(generator=gen)
    vals.normal_(generator=gen)
    pos = torch.cat([torch.arange(n, t) for n, t in zip(held, total)])
    row = torch.repeat_interleave(torch.arange(case["batch"]), torch.tensor(new))
    slots = table[row, pos // page].long() * page + pos % page
    # a step's K and V are slices of the projection's rows, or arrays of their own
    tokens = len(slots)
    heads = (case["hq"] if case["fused"] else 0) + 2 * case["hkv"]
    rows = torch.randn(tokens, heads, case["d"], device=device(), generator=gen)
    rows = rows.to(DTYPES[case["dtype"]])
    k_new, v_new = rows[:, heads - 2 * case["hkv"]:heads - case["hkv"]], rows[:, heads - case["hkv"]:]
    if not case["fused"]:
        k_new, v_new = k_new.contiguous(), v_new.contiguous()
    done = slots[pos % page == page - 1] // page
    s = {"case": case, "k_new": k_new, "v_new": v_new, "keys": keys, "vals": vals,
         "means": page_means(keys), "slots": slots.to(torch.int32).to(device()),
         "done": done.to(device())}
    if own:
        from kv_cache_sparsity_b200 import hylra as H
        s["shape"] = shape_of(H, case, keys, max(have))
        s["ws"] = workspace(H, s["shape"])
    return s


def prepare_decode(case, gen, host):
    """Keys with some pages that a query attends to, as long contexts have them."""
    page, n, d, hkv = case["page"], lengths(case), case["d"], case["hkv"]
    batch, r = case["batch"], case["hq"] // case["hkv"]
    have = [pages_of(x, page) for x in n]
    pool = sum(have) + 5
    order = torch.randperm(pool, generator=host)
    table = held_table(have, max(1, max(have)), order)
    owner = torch.zeros(pool, dtype=torch.long)
    owner[order[:sum(have)]] = torch.repeat_interleave(torch.arange(batch), torch.tensor(have))
    owner = owner.to(device())
    u = torch.randn(batch, hkv, d, device=device(), generator=gen)
    u = u / u.norm(dim=-1, keepdim=True)
    keys, vals = empty_pool(case, pool), empty_pool(case, pool)
    keys.normal_(generator=gen).mul_(0.5)
    vals.normal_(generator=gen)
    # about 64 pages of a long sequence stand out, by 2 to 6 times a unit direction
    share = min(0.5, 64.0 / max(1, max(have)))
    amp = 2.0 + 4.0 * torch.rand(pool, hkv, 1, device=device(), generator=gen)
    amp = amp * (torch.rand(pool, hkv, 1, device=device(), generator=gen) < share)
    keys.add_((amp * u[owner]).to(keys.dtype)[:, :, None])
    q = torch.randn(batch, hkv, r, d, device=device(), generator=gen)
    q = (q + math.sqrt(d) * u[:, :, None]).reshape(batch, case["hq"], d).to(keys.dtype)
    s = {"case": case, "q": q, "keys": keys, "vals": vals, "table": table.to(device()),
         "seqlens": to_device(n), "out": torch.empty(batch, case["hq"], d, device=device()),
         "lse": torch.empty(batch, case["hq"], device=device())}
    if case["op"] == "sparse":
        s["means"] = page_means(keys)
        s["chosen"] = torch.empty(batch, hkv, case["topk"], dtype=torch.int32, device=device())
    if own:
        from kv_cache_sparsity_b200 import hylra as H
        s["shape"] = shape_of(H, case, keys, table.shape[1])
        s["ws"] = workspace(H, s["shape"])
    return s


# ---------------------------------------------------------------- operators


def run(s):
    if own:
        return run_own(s)
    return {"tables": plain_tables, "append": plain_append, "decode": plain_decode,
            "sparse": plain_sparse}[s["case"]["op"]](s)


def run_own(s):
    from kv_cache_sparsity_b200 import hylra as H
    op = s["case"]["op"]
    if op == "tables":
        H.paged_tables(s["shape"], s["cached"], s["new"], s["free"], s["free_count"], s["table"],
                       s["seqlens"], s["cu"], s["slots"], s["left"], s["ws"])
        return s["table"], s["slots"], s["seqlens"], s["cu"], s["left"]
    if op == "append":
        H.paged_append(s["shape"], s["k_new"], s["v_new"], s["slots"], s["keys"], s["vals"],
                       s["means"], s["ws"])
        return s["keys"], s["vals"], s["means"]
    if op == "decode":
        H.paged_decode(s["shape"], s["q"], s["keys"], s["vals"], s["table"], s["seqlens"],
                       s["out"], s["ws"], lse=s["lse"])
        return s["out"], s["lse"]
    H.paged_select(s["shape"], s["q"], s["means"], s["table"], s["seqlens"], s["chosen"], s["ws"],
                   sink=s["case"]["sink"], recent=s["case"]["recent"])
    H.paged_decode_topk(s["shape"], s["q"], s["keys"], s["vals"], s["table"], s["seqlens"],
                        s["chosen"], s["out"], s["ws"], lse=s["lse"])
    return s["chosen"], s["out"], s["lse"]


def plain_tables(s):
    page = s["case"]["page"]
    held, new, table = s["cached"].long(), s["new"].long(), s["table"].long()
    have = (held + page - 1) // page
    need = (held + new + page - 1) // page - have
    end = torch.cumsum(need, 0)
    count = s["free_count"].long()
    served = (need == 0) | (end <= count)
    # pages come off the end of the free list, request after request
    j = torch.arange(table.shape[1], device=table.device)
    nth = (end - need)[:, None] + j - have[:, None]
    fresh = served[:, None] & (j >= have[:, None]) & (j < (have + need)[:, None])
    popped = s["free"].long()[(count - 1 - nth).clamp(0, len(s["free"]) - 1)]
    table = torch.where(fresh, popped, table)
    cu = torch.cat([torch.zeros_like(end[:1]), torch.cumsum(new, 0)])
    t = torch.arange(len(s["slots"]), device=table.device)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=len(held) - 1)
    pos = held[b] + t - cu[b]
    at = table[b, (pos // page).clamp(max=table.shape[1] - 1)]
    slots = torch.where((t < cu[-1]) & served[b], at * page + pos % page, torch.tensor(-1, device=t.device))
    s["table"].copy_(table)
    return (s["table"], slots.to(torch.int32), torch.where(served, held + new, held).to(torch.int32),
            cu.to(torch.int32), (count - (need * served).sum()).to(torch.int32))


def plain_append(s):
    page = s["case"]["page"]
    at = s["slots"].long()
    s["keys"][at // page, :, at % page] = s["k_new"]
    s["vals"][at // page, :, at % page] = s["v_new"]
    s["means"][s["done"]] = s["keys"][s["done"]].float().mean(2).to(s["means"].dtype)
    return s["keys"], s["vals"], s["means"]


def attend(q, keys, vals, mask, d):
    """q [b, h, r, d], keys and vals [b, h, n, d], mask [b, h or 1, n] -> out [b, h, r, d], lse [b, h, r]."""
    x = torch.matmul(q.float(), keys.float().transpose(-1, -2)) * (1.0 / math.sqrt(d))
    x = x.masked_fill(~mask[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, torch.where(mask[..., None], vals.float(), torch.zeros((), device=x.device)))
    return out / torch.where(z == 0, torch.ones_like(z), z), (m + torch.log(z))[..., 0]


def plain_decode(s):
    c = s["case"]
    batch, r = c["batch"], c["hq"] // c["hkv"]
    at = s["table"].long().clamp(min=0)
    keys = s["keys"][at].transpose(1, 2).reshape(batch, c["hkv"], -1, c["d"])
    vals = s["vals"][at].transpose(1, 2).reshape(batch, c["hkv"], -1, c["d"])
    mask = torch.arange(keys.shape[2], device=at.device) < s["seqlens"].long()[:, None]
    out, lse = attend(s["q"].view(batch, c["hkv"], r, c["d"]), keys, vals, mask[:, None], c["d"])
    return out.reshape(batch, c["hq"], c["d"]), lse.reshape(batch, c["hq"])


def plain_choice(s):
    c = s["case"]
    batch, r = c["batch"], c["hq"] // c["hkv"]
    at = s["table"].long().clamp(min=0)
    count = (s["seqlens"].long()[:, None, None] + c["page"] - 1) // c["page"]
    j = torch.arange(at.shape[1], device=at.device)
    forced = ((j < c["sink"]) | (j >= count - c["recent"])) & (j < count)
    ranked = (j < count) & ~forced
    q = s["q"].view(batch, c["hkv"], r, c["d"]).double()
    x = torch.matmul(q, s["means"][at].double().permute(0, 2, 3, 1)) * (1.0 / math.sqrt(c["d"]))
    x = x.masked_fill(~ranked[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    score = (p / torch.where(z == 0, torch.ones_like(z), z)).sum(2).float()
    score = score.masked_fill(forced, math.inf).masked_fill(~(j < count), -1.0)
    score, order = torch.sort(score, dim=-1, descending=True, stable=True)
    order = torch.where(score >= 0, order, torch.full_like(order, -1))[..., : c["topk"]]
    short = c["topk"] - order.shape[-1]
    return torch.nn.functional.pad(order, (0, max(0, short)), value=-1)


def plain_sparse(s):
    c = s["case"]
    batch, hkv, r = c["batch"], c["hkv"], c["hq"] // c["hkv"]
    chosen = plain_choice(s)
    row = torch.arange(batch, device=chosen.device)[:, None, None]
    head = torch.arange(hkv, device=chosen.device)[:, None]
    at = s["table"].long()[row, chosen.clamp(min=0)].clamp(min=0)
    keys = s["keys"][at, head].reshape(batch, hkv, -1, c["d"])
    vals = s["vals"][at, head].reshape(batch, hkv, -1, c["d"])
    pos = chosen[..., None] * c["page"] + torch.arange(c["page"], device=at.device)
    mask = (pos < s["seqlens"].long()[:, None, None, None]) & (chosen >= 0)[..., None]
    out, lse = attend(s["q"].view(batch, hkv, r, c["d"]), keys, vals, mask.flatten(2), c["d"])
    return (chosen.to(torch.int32), out.reshape(batch, c["hq"], c["d"]), lse.reshape(batch, c["hq"]))


# ---------------------------------------------------------------------- work


def work(case):
    if case["op"] == "tables":
        have, need, free, cols, slots = tables_sizes(case)
        got = min(free, sum(need))
        return {"bytes": 4.0 * (4 * case["batch"] + 2 * got + slots), "flops": 0.0}
    row = case["hkv"] * case["d"] * 2  # bytes of one token's keys
    if case["op"] == "append":
        page, new = case["page"], new_lengths(case)
        tokens = sum(new)
        done, old = 0, 0
        for n, w in zip(lengths(case), new):
            pages = (n + w) // page - n // page
            done += pages
            old += n % page if pages else 0
        return {"bytes": float(4 * row * tokens + 4 * tokens + row * (done + old)),
                "flops": float(done * page * case["hkv"] * case["d"])}
    n, page = lengths(case), case["page"]
    small = case["batch"] * case["hq"] * (case["d"] * 6 + 4) + 4 * case["batch"]
    if case["op"] == "decode":
        tokens = sum(n)
        pages = sum(pages_of(x, page) for x in n)
        return {"bytes": float(2 * row * tokens + small + 4 * pages),
                "flops": 4.0 * tokens * case["hq"] * case["d"]}
    ranked, tokens = 0, 0
    for x in n:
        count = pages_of(x, page)
        ranked += max(0, count - case["sink"] - case["recent"])
        take = min(case["topk"], count)
        # the last page may be partly filled; it is taken unless the list ends before it
        full = min(case["sink"], max(0, count - case["recent"])) + case["recent"] <= case["topk"]
        tokens += min(x, (take - 1) * page + x - (count - 1) * page) if full and count else take * page
    return {"bytes": float(row * ranked + 2 * row * tokens + small + 4 * ranked
                           + 8 * case["batch"] * case["hkv"] * case["topk"]),
            "flops": (2.0 * ranked + 4.0 * tokens) * case["hq"] * case["d"]}


# --------------------------------------------------------------------- exact


def exact(case, seed):
    """The definitions in 64 bits, one sequence at a time."""
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None  # whole numbers alone: their plain form is already exact
    if case["op"] == "append":
        return None, None, exact_means(s)
    scale = 1.0 / math.sqrt(case["d"])
    r = case["hq"] // case["hkv"]
    outs, lses = [], []
    for b, n in enumerate(lengths(case)):
        q = s["q"][b].double().view(case["hkv"], r, case["d"])
        if n == 0:
            outs.append(torch.zeros_like(q))
            lses.append(torch.full_like(q[..., 0], -math.inf))
            continue
        pages = s["table"][b, : pages_of(n, case["page"])].long()
        heads = []
        for h in range(case["hkv"]):
            k = s["keys"][pages, h].reshape(-1, case["d"])[:n].double()
            v = s["vals"][pages, h].reshape(-1, case["d"])[:n].double()
            if case["op"] == "sparse":
                take = exact_tokens(s, b, h, q[h], pages, n)
                k, v = k[take], v[take]
            x = q[h] @ k.T * scale
            lse = torch.logsumexp(x, -1)
            heads.append((torch.exp(x - lse[:, None]) @ v, lse))
        outs.append(torch.stack([o for o, _ in heads]))
        lses.append(torch.stack([x for _, x in heads]))
    out = torch.stack(outs).reshape(case["batch"], case["hq"], case["d"])
    lse = torch.stack(lses).reshape(case["batch"], case["hq"])
    return (out, lse) if case["op"] == "decode" else (None, out, lse)


def exact_means(s):
    page, means = s["case"]["page"], s["means"].double()
    where = {int(x): t for t, x in enumerate(s["slots"].tolist())}
    fresh = s["k_new"].double()
    for p in s["done"].tolist():
        total = torch.zeros_like(means[p])
        at = [where.get(p * page + i, -1) for i in range(page)]
        new = [t for t in at if t >= 0]
        old = [i for i, t in enumerate(at) if t < 0]
        total = fresh[new].sum(0) + s["keys"][p][:, old].double().sum(1)
        means[p] = total / page
    return means


def exact_tokens(s, b, h, q, pages, n):
    """Positions of the tokens of the pages that sequence b, KV head h attends to."""
    c = s["case"]
    count, page = len(pages), c["page"]
    last = max(0, count - c["recent"])
    forced = sorted(set(range(min(c["sink"], count))) | set(range(last, count)))
    mid = torch.arange(min(c["sink"], last), last, device=q.device)
    rank = []
    if len(mid):
        x = q @ s["means"][pages[mid], h].double().T / math.sqrt(c["d"])
        score = torch.softmax(x, -1).sum(0).float()
        rank = (mid[torch.argsort(score, descending=True, stable=True)]).tolist()
    take = torch.tensor((forced + rank)[: c["topk"]], device=q.device)
    pos = (take[:, None] * page + torch.arange(page, device=q.device)).flatten()
    return pos[pos < n]
