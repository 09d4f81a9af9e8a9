"""More operators over the paged KV cache: what is measured, and their plain form.

* chunk: attention of a chunk of new tokens of each sequence (a prompt, a part of one,
  a drafted continuation) over its pages, causal, the chunk's own keys included; with a
  sliding window and first tokens that stay visible ("sinks") where `window` is not 0;
* window: decode attention of the newest Tq tokens with a window and sinks;
* fork: sequences that continue others: rows of the block table that share the parent's
  full pages, and a copy of its last, partly filled page;
* free: the ids of the pages that no sequence uses, in ascending order;
* compact: the pages in use moved to the front of the cache, and the block table that
  names them there.

Pages hold 16-bit elements or e4m3 with one float32 scale per page and KV head, as
[page, token, head, dim] ("thd") or [page, head, token, dim] ("htd").
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def attention(name, op, kv, dtype, B, Hq, Hkv, D, page, layout, lo, hi, new_lo, new_hi, window=0, sinks=0, lens=1):
    return dict(name=name, op=op, kv=kv, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, layout=layout, lo=lo, hi=hi,
                new_lo=new_lo, new_hi=new_hi, window=window, sinks=sinks, lens=lens)


def chunk(name, *sizes, **more):
    return attention(name, "chunk", *sizes, **more)


def window(name, kv, dtype, B, Tq, Hq, Hkv, D, page, layout, lo, hi, window, sinks, lens=1):
    return attention(name, "window", kv, dtype, B, Hq, Hkv, D, page, layout, lo, hi, Tq, Tq, window, sinks, lens)


def pages(name, op, kv, B, Hkv, D, page, layout, lo, hi, children=0, spare=3, lens=1):
    return dict(name=name, op=op, kv=kv, B=B, Hkv=Hkv, D=D, page=page, layout=layout, lo=lo, hi=hi, children=children,
                spare=spare, lens=lens)


def listed():
    return [
        # a short question in a conversation that is already cached: latency of one call
        chunk("chunk_one_user", "bf16", "bf16", 1, 32, 8, 128, 16, "thd", 1131, 1131, 107, 107),
        # prompts of unequal lengths, some of them the second part of one, beside sequences that only decode
        chunk("chunk_ragged", "f16", "f16", 24, 28, 4, 128, 64, "thd", 64, 6000, 1, 2048),
        # a part of a long document over an 8-bit cache
        chunk("chunk8_long", "e4m3", "bf16", 1, 32, 8, 128, 64, "htd", 32768, 32768, 4096, 4096),
        # prompts of a model with a sliding window
        chunk("chunk_window", "bf16", "bf16", 3, 16, 2, 64, 32, "thd", 16000, 24000, 4000, 8192, window=4096, sinks=4),
        # one decode step of a batch of long conversations that see their last 2000 tokens and the first four
        window("window_decode", "bf16", "bf16", 32, 1, 32, 8, 128, 64, "thd", 4096, 65536, 2000, 4),
        # drafted tokens verified over an 8-bit cache, one user
        window("window8_drafted", "e4m3", "bf16", 1, 4, 28, 4, 128, 64, "htd", 40961, 40961, 8192, 128),
        # four answers to each of two prompts
        pages("fork_answers", "fork", "bf16", 2, 8, 128, 16, "thd", 1000, 3000, children=8),
        # beams of a large batch, pages of 128 tokens
        pages("fork_beams", "fork", "bf16", 128, 8, 128, 128, "htd", 100, 900, children=512),
        # the pool of one small model
        pages("free_small", "free", "f16", 16, 4, 128, 64, "thd", 100, 4000, spare=500),
        # a large pool of small pages under long sequences
        pages("free_large", "free", "e4m3", 1000, 1, 64, 16, "thd", 1, 8192, spare=100000),
        # a small pool after a few sequences have ended
        pages("compact_small", "compact", "bf16", 7, 8, 128, 16, "thd", 100, 900, spare=80),
        # a large pool of 8-bit pages, half of it free
        pages("compact_large", "compact", "e4m3", 100, 8, 128, 64, "htd", 500, 4000, spare=2500),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    kv = rng.choice(["f16", "bf16", "e4m3", "e4m3"])
    dtype = kv if kv != "e4m3" else rng.choice(["f16", "bf16"])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 48, 64, 128])
    layout = rng.choice(["thd", "htd"])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 3, 4, 7, 8])
    seed = rng.randrange(1 << 30)
    op = rng.choice(["chunk", "chunk", "chunk", "window", "window", "fork", "free", "compact"])
    if op == "chunk":
        B = spread(rng, 1, 16)
        new_hi = max(1, spread(rng, 8, 4096) // B)
        new_lo = rng.choice([1, max(1, new_hi // 3), new_hi])
        hi = new_hi + spread(rng, 1, 16384) - 1
        lo = rng.choice([new_lo, hi])
        w, s = rng.choice([(0, 0), (0, 0), (spread(rng, 1, 4096), rng.choice([0, 4, spread(rng, 1, 300)]))])
        c = chunk("", kv, dtype, B, Hkv * G, Hkv, D, page, layout, lo, hi, new_lo, new_hi, window=w, sinks=s, lens=seed)
    elif op == "window":
        B = spread(rng, 1, 128)
        hi = spread(rng, 64, max(64, 524288 // B))
        lo = rng.choice([1, max(1, hi // 8), hi])
        Tq = rng.choice([1, 1, 1, 2, 4, 5])
        c = window("", kv, dtype, B, Tq, Hkv * G, Hkv, D, page, layout, lo, hi, spread(rng, 1, 8192),
                   rng.choice([0, 4, spread(rng, 1, 300)]), lens=seed)
    else:
        B = spread(rng, 1, 200)
        hi = spread(rng, 32, 131072 // B)
        lo = rng.choice([1, max(1, hi // 4)])
        total = sum(-(-n // page) for n in lengths(dict(lo=lo, hi=hi, B=B, lens=seed, op=op))[0])
        c = pages("", op, kv, B, Hkv, D, page, layout, lo, hi, children=spread(rng, 1, 400) if op == "fork" else 0,
                  spare=spread(rng, 1, 1 + total), lens=seed)
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes and inputs
def lengths(case):
    """(length of each sequence with its new tokens, new tokens of each), the case's own."""
    rng = random.Random(case["lens"])
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if case["op"] == "window":
        return lens, [case["new_lo"]] * case["B"]
    if case["op"] != "chunk":
        return lens, [0] * case["B"]
    return lens, [min(n, rng.randint(case["new_lo"], case["new_hi"])) for n in lens]


def family(case):
    """(parent of each child, whether it needs a page of its own): every parent's last child may go on writing
    where the parent did, the others need a copy of a page that is partly filled."""
    rng = random.Random(case["lens"] + 1)
    parents = [rng.randrange(case["B"]) for _ in range(case["children"])]
    last = {p: i for i, p in enumerate(parents)}
    lens, _ = lengths(case)
    return parents, [lens[p] % case["page"] != 0 and last[p] != i for i, p in enumerate(parents)]


def pages_of(case, lens):
    return [-(-n // case["page"]) for n in lens]


def made_pages(case, total, gen):
    """Keys or values as a model leaves them in its cache."""
    inner = (case["page"], case["Hkv"]) if case["layout"] == "thd" else (case["Hkv"], case["page"])
    shape = (total, *inner, case["D"])
    if case["kv"] != "e4m3":
        return torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[case["kv"]]), None
    # powers of two, as appending gives them, and elements that use the type's range
    scale = torch.exp2(torch.randint(-9, -5, (total, case["Hkv"]), generator=gen, device="cuda").float())
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(100.0)
    return x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens, new = lengths(case)
    need = pages_of(case, lens)
    used = sum(need)
    extra = case.get("spare", 3) + (sum(family(case)[1]) if case["op"] == "fork" else 0)
    total = used + extra
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(case["B"], max(need), dtype=torch.int32, device="cuda")
    filled = torch.arange(max(need))[None, :] < torch.tensor(need)[:, None]
    table[filled.cuda()] = order[:used]
    s = dict(case=case, lens=lens, new=new, table=table, total=total, filled=filled.cuda(),
             kv_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["op"] != "free":
        s["k"], s["k_scale"] = made_pages(case, total, gen)
        s["v"], s["v_scale"] = made_pages(case, total, gen)
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] in ("chunk", "window"):
        Hq, dt = case["Hq"], DTYPES[case["dtype"]]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu_new"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["q"] = torch.randn(cu[-1], Hq, D, generator=gen, device="cuda", dtype=dt)
        if case["op"] == "window":
            s["q"] = s["q"].view(case["B"], case["new_lo"], Hq, D)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:-1], device="cuda")
    elif case["op"] == "fork":
        parents, copies = family(case)
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
        fresh = torch.full((len(parents),), -1, dtype=torch.int32, device="cuda")
        fresh[torch.tensor(copies, device="cuda")] = order[used:used + sum(copies)]
        s["new_pages"] = fresh
        s["lens_out"] = torch.zeros(len(parents), dtype=torch.int32, device="cuda")
        s["table_out"] = torch.zeros(len(parents), max(need), dtype=torch.int32, device="cuda")
    elif case["op"] == "free":
        s["free"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        s["table_out"] = torch.zeros_like(table)
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import split_kv_decode_decoding_gb300 as da

        if case["op"] != "free":
            s["cache"] = da.PagedCache(s["k"], s["v"], s["k_scale"], s["v_scale"],
                                       layout=da.DA_LAYOUT_VARLEN if case["layout"] == "thd" else da.DA_LAYOUT_BHSD)
        if case["op"] == "chunk":
            s["workspace"] = da.alloc_paged_chunk_workspace(case["Hq"], Hkv, D)
        elif case["op"] == "window":
            s["workspace"] = da.alloc_paged_workspace(case["new_lo"], case["Hq"], Hkv, D)
        else:
            s["workspace"] = da.alloc_paged_pages_workspace(total)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return run_own(state, op)
    return {"chunk": plain_attention, "window": plain_attention, "fork": plain_fork, "free": plain_free,
            "compact": plain_compact}[op](state)


def run_own(s, op):
    import split_kv_decode_decoding_gb300 as da

    c, ws = s["case"], s["workspace"]
    if op == "chunk":
        da.decode_attn_paged_chunk(s["q"], s["cache"], s["cu_new"], s["kv_lens"], s["table"], s["out"], ws, window=c["window"],
                                   sinks=c["sinks"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "window":
        da.decode_attn_paged_window(s["q"], s["cache"], s["kv_lens"], s["table"], s["out"], ws, window=c["window"],
                                    sinks=c["sinks"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "fork":
        da.decode_attn_paged_fork(s["cache"], s["kv_lens"], s["table"], s["parents"], s["new_pages"], s["lens_out"],
                                  s["table_out"], ws)
        return forked(s)
    if op == "free":
        da.decode_attn_paged_free_pages(s["kv_lens"], s["table"], s["free"], s["count"], ws, page_size=c["page"])
        return {"free": s["free"], "count": s["count"]}
    da.decode_attn_paged_compact(s["cache"], s["kv_lens"], s["table"], s["table_out"], s["count"], ws)
    return compacted(s)


def cache_of(s):
    got = {"k": s["k"], "v": s["v"]}
    if s["k_scale"] is not None:
        got |= {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return got


def forked(s):
    return {"lens": s["lens_out"], "table": s["table_out"], **cache_of(s)}


def compacted(s):
    return {"table": s["table_out"], "count": s["count"], **cache_of(s)}


def bits(x):
    """An integer view of pages: torch indexes 8-bit floats only so."""
    return x.view(torch.uint8 if x.element_size() == 1 else torch.int16)


def keys_at(pages, scale, row, position, case, head):
    """[positions, D] in float32 of one head of a sequence's pages."""
    page, slot = row[position // case["page"]].long(), position % case["page"]
    raw = bits(pages)
    x = raw[page, slot, head] if case["layout"] == "thd" else raw[page, head, slot]
    x = x.view(pages.dtype).float()
    return x if scale is None else x * scale[page, head][:, None]


def visible(position, key, case):
    """[positions, keys]: whether a token at a position sees a key."""
    seen = key[None, :] <= position[:, None]
    if case["window"]:
        seen &= (key[None, :] > position[:, None] - case["window"]) | (key[None, :] < case["sinks"])
    return seen


def key_range(first, last, case):
    """Positions that a token between `first` and `last` may see."""
    low = max(0, first - case["window"] + 1) if case["window"] else 0
    sinks = torch.arange(min(case["sinks"], low), device="cuda")
    return torch.cat([sinks, torch.arange(low, last + 1, device="cuda")])


def plain_attention(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    q, out, lse = s["q"].view(-1, Hkv, G, D), s["out"].view(-1, Hkv, G, D), s["lse"].view(-1, Hkv, G)
    row0 = 0
    for b, (n, m) in enumerate(zip(s["lens"], s["new"])):
        # tokens at a time: what a few GB of scores hold
        step = max(1, min(m, (1 << 29) // (G * n)))
        for t0 in range(0, m, step):
            t1 = min(m, t0 + step)
            position = torch.arange(n - m + t0, n - m + t1, device="cuda")
            if n - m + t1 - 1 < 0:
                out[row0 + t0:row0 + t1] = 0
                lse[row0 + t0:row0 + t1] = -math.inf
                continue
            key = key_range(max(0, n - m + t0), n - m + t1 - 1, c)
            hidden = ~visible(position, key, c)
            for h in range(Hkv):
                k = keys_at(s["k"], s["k_scale"], s["table"][b], key, c, h)
                x = q[row0 + t0:row0 + t1, h].float().reshape(-1, D) @ k.T
                x = x.mul_(1.0 / math.sqrt(D)).view(t1 - t0, G, -1).masked_fill_(hidden[:, None], -math.inf)
                top = x.amax(-1, keepdim=True)
                none = top == -math.inf
                e = x.sub_(top.masked_fill(none, 0.0)).exp_()
                total = e.sum(-1, keepdim=True)
                v = keys_at(s["v"], s["v_scale"], s["table"][b], key, c, h)
                o = (e.view(-1, key.numel()) @ v).view(t1 - t0, G, D) / total.masked_fill(none, 1.0)
                out[row0 + t0:row0 + t1, h] = o.to(out.dtype)
                lse[row0 + t0:row0 + t1, h] = torch.where(none, top, top + total.log())[..., 0]
        row0 += m
    return {"out": s["out"], "lse": s["lse"]}


def plain_fork(s):
    c = s["case"]
    parents, fresh = s["parents"].long(), s["new_pages"]
    lens = s["kv_lens"][parents]
    need = (lens + c["page"] - 1) // c["page"]
    rows = s["table"][parents]
    entry = torch.arange(rows.shape[1], device="cuda")[None, :]
    own_page = (fresh >= 0) & (lens % c["page"] != 0)
    replaced = own_page[:, None] & (entry == need[:, None] - 1)
    s["lens_out"].copy_(lens)
    s["table_out"].copy_(torch.where(entry < need[:, None], torch.where(replaced, fresh[:, None], rows), s["table_out"]))
    child = torch.nonzero(own_page)[:, 0]
    old = rows[child, need[child].long() - 1].long()
    new = fresh[child].long()
    slot = torch.arange(c["page"], device="cuda")[None, :] < (lens[child] % c["page"])[:, None]
    slot = slot[:, :, None, None] if c["layout"] == "thd" else slot[:, None, :, None]
    for name in ("k", "v"):
        raw = bits(s[name])
        raw[new] = torch.where(slot, raw[old], raw[new])
        if s["k_scale"] is not None:
            s[name + "_scale"][new] = s[name + "_scale"][old]
    return forked(s)


def in_use(s):
    used = torch.zeros(s["total"], dtype=torch.bool, device="cuda")
    entry = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    live = entry < (s["kv_lens"][:, None] + s["case"]["page"] - 1) // s["case"]["page"]
    used[s["table"][live].long()] = True
    return used, live


def plain_free(s):
    used, _ = in_use(s)
    free = torch.nonzero(~used)[:, 0]
    s["free"][:free.numel()] = free.to(torch.int32)
    s["count"].fill_(free.numel())
    return {"free": s["free"], "count": s["count"]}


def plain_compact(s):
    used, live = in_use(s)
    n = int(used.sum())
    holes, movers = torch.nonzero(~used[:n])[:, 0], n + torch.nonzero(used[n:])[:, 0]
    for x in cache_of(s).values():
        raw = bits(x) if x.dim() == 4 else x
        raw[holes] = raw[movers]
    at = torch.arange(s["total"], dtype=torch.int32, device="cuda")
    at[movers] = holes.to(torch.int32)
    s["table_out"].copy_(torch.where(live, at[s["table"].long()], s["table_out"]))
    s["count"].fill_(n)
    return compacted(s)


# ------------------------------------------------------------------ what a pass cannot do without
def seen_keys(first, last, case):
    """(keys that some token at first..last sees, pairs of a token and a key that it sees)"""
    w, sinks = case["window"], case["sinks"]
    pairs = 0
    if not w:
        count = last - first + 1
        return last + 1, count * (first + 1 + last + 1) // 2
    for p in range(first, last + 1):
        low = max(0, p - w + 1)
        pairs += p + 1 - low + min(sinks, low)
    low = max(0, first - w + 1)
    return last + 1 - low + min(sinks, low), pairs


def page_bytes(case):
    wide = 1 if case["kv"] == "e4m3" else 2
    return 2 * case["page"] * case["Hkv"] * case["D"] * wide + (8 * case["Hkv"] if wide == 1 else 0)


def work(case):
    lens, new = lengths(case)
    need = pages_of(case, lens)
    if case["op"] in ("chunk", "window"):
        wide = 1 if case["kv"] == "e4m3" else 2
        keys = pairs = 0
        for n, m in zip(lens, new):
            first = max(0, n - m)
            if n > 0 and m > 0:
                k, p = seen_keys(first, n - 1, case)
                keys, pairs = keys + k, pairs + p
        scales = 8 * case["Hkv"] * (keys // case["page"]) if wide == 1 else 0
        rows = sum(new) * case["Hq"]
        return {"bytes": 2 * keys * case["Hkv"] * case["D"] * wide + scales + 4 * (keys // case["page"]) + 8 * case["B"]
                + rows * (4 * case["D"] + 4), "flops": 4 * pairs * case["Hq"] * case["D"]}
    if case["op"] == "fork":
        parents, copies = family(case)
        part = sum(lens[p] % case["page"] for p, c in zip(parents, copies) if c)
        entries = sum(need[p] for p in set(parents)) + sum(need[p] for p in parents)
        return {"bytes": 2 * part * (page_bytes(case) // case["page"]) + 4 * entries + 16 * len(parents), "flops": 0}
    if case["op"] == "free":
        return {"bytes": 4 * sum(need) + 4 * case["B"] + 4 * case["spare"], "flops": 0}
    # half the pages behind the last one in use are holes in front of it: as many pages move as free ones lie there
    used, total = sum(need), sum(need) + case["spare"]
    moved = used * case["spare"] // total
    return {"bytes": 2 * moved * page_bytes(case) + 8 * used + 4 * case["B"], "flops": 0}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("chunk", "window"):
        # a few seconds of 64-bit products at most
        return exact_attention(case, s) if work(case)["flops"] < 4e12 else None
    return {"fork": exact_fork, "free": exact_free, "compact": exact_compact}[case["op"]](case, s)


def sequence64(pages, scale, row, n, case):
    """[n, Hkv, D] of one sequence's first n keys."""
    at = torch.tensor(row[:max(1, -(-n // case["page"]))], device="cuda")
    x = bits(pages).index_select(0, at).view(pages.dtype).double()
    if case["layout"] == "htd":
        x = x.transpose(1, 2)
    if scale is not None:
        x = x * scale.index_select(0, at).double()[:, None, :, None]
    return x.reshape(-1, case["Hkv"], case["D"])[:n]


def exact_attention(case, s):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G, W, sinks = Hq // Hkv, case["window"], case["sinks"]
    q = s["q"].view(-1, Hq, D)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    table, done = s["table"].cpu().tolist(), 0
    for b, (n, m) in enumerate(zip(s["lens"], s["new"])):
        k = sequence64(s["k"], s["k_scale"], table[b], n, case)
        v = sequence64(s["v"], s["v_scale"], table[b], n, case)
        for t0 in range(0, m, 256):
            count = min(256, m - t0)
            p = torch.arange(n - m + t0, n - m + t0 + count, device="cuda").view(-1, 1)
            lo = max(0, n - m + t0 - W + 1) if W else 0
            hi = n - m + t0 + count
            if hi <= 0:
                continue
            pick = torch.arange(n, device="cuda")
            pick = pick[((pick >= lo) | (pick < sinks)) & (pick < hi)]
            bad = pick[None] > p
            if W:
                bad |= (p - pick[None] >= W) & (pick[None] >= sinks)
            rows = slice(done + t0, done + t0 + count)
            for h in range(Hkv):
                heads = slice(h * G, (h + 1) * G)
                x = torch.einsum("tgd,kd->gtk", q[rows, heads].double(), k[pick, h]) / math.sqrt(D)
                x[:, bad] = -math.inf
                z = torch.logsumexp(x, -1)
                weight = torch.exp(x - z.masked_fill(z == -math.inf, 0.0)[..., None])
                out[rows, heads] = torch.einsum("gtk,kd->tgd", weight, v[pick, h])
                lse[rows, heads] = z.T
        done += m
    return {"out": out.view(s["q"].shape), "lse": lse.view(s["lse"].shape)}


def exact_fork(case, s):
    P, thd = case["page"], case["layout"] == "thd"
    table, fresh = s["table"].cpu().tolist(), s["new_pages"].cpu().tolist()
    parents = s["parents"].cpu().tolist()
    lens = [s["lens"][p] for p in parents]
    rows = s["table_out"].cpu().tolist()
    old, new, first = [], [], []
    for i, (p, n) in enumerate(zip(parents, lens)):
        full, part = divmod(n, P)
        rows[i][:full] = table[p][:full]
        if part:
            rows[i][full] = table[p][full] if fresh[i] < 0 else fresh[i]
            if fresh[i] >= 0:
                old.append(table[p][full]), new.append(fresh[i]), first.append(part)
    got = {"lens": torch.tensor(lens, dtype=torch.int32), "table": torch.tensor(rows, dtype=torch.int32)}
    for name in ("k", "v"):
        pages = bits(s[name]).clone()
        view = pages if thd else pages.transpose(1, 2)
        for a, b, n in zip(old, new, first):
            view[b, :n] = view[a, :n]
        got[name] = pages.view(s[name].dtype)
        if s["k_scale"] is not None:
            scale = s[name + "_scale"].clone()
            for a, b in zip(old, new):
                scale[b] = scale[a]
            got[name + "_scale"] = scale
    return got


def uses(case, s):
    table = s["table"].cpu().tolist()
    rows = [table[b][:-(-n // case["page"])] for b, n in enumerate(s["lens"])]
    return rows, sorted({page for row in rows for page in row})


def exact_free(case, s):
    _, used = uses(case, s)
    used = set(used)
    ids = [i for i in range(s["total"]) if i not in used]
    return {"free": torch.tensor(ids + [-1] * (s["total"] - len(ids)), dtype=torch.int32),
            "count": torch.tensor([len(ids)], dtype=torch.int32)}


def exact_compact(case, s):
    rows, used = uses(case, s)
    n, taken = len(used), set(used)
    moves = dict(zip([i for i in used if i >= n], [i for i in range(n) if i not in taken]))
    table = s["table_out"].cpu().tolist()
    for b, row in enumerate(rows):
        table[b][:len(row)] = [moves.get(i, i) for i in row]
    got = {"table": torch.tensor(table, dtype=torch.int32), "count": torch.tensor([n], dtype=torch.int32)}
    for name, x in cache_of(s).items():
        raw = (bits(x) if x.dim() == 4 else x).clone()
        for a, b in moves.items():
            raw[b] = raw[a]
        got[name] = raw.view(x.dtype)
    return got
