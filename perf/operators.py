"""Paged KV cache operators: what is measured, and their plain form.

Two operations over a key/value cache kept in pages, each for pages of 16-bit
elements and for pages of 8-bit (e4m3) elements with one float32 scale per page
and KV head:

* attend: decode attention of the newest T_q query tokens of each sequence over
  its pages, causal among those tokens;
* append: rotate the new tokens' queries and keys by their positions and write
  their keys and values into the sequences' pages. An 8-bit page's scale is the
  smallest power of two that holds the largest element it has met; where a new
  token raises it, the page's earlier elements are rounded again to it.

Pages are [page, token, head, dim] ("thd") or [page, head, token, dim] ("htd").
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
LEAST_EXPONENT = -126


def attend(name, kv, dtype, B, Tq, Hq, Hkv, D, page, layout, lo, hi, lens=1):
    return dict(name=name, op="attend", kv=kv, dtype=dtype, B=B, Tq=Tq, Hq=Hq, Hkv=Hkv, D=D, page=page, layout=layout,
                lo=lo, hi=hi, lens=lens)


def append(name, kv, dtype, B, Hq, Hkv, D, page, layout, lo, hi, new_lo, new_hi, rope="half", rot=None, lens=1):
    return dict(name=name, op="append", kv=kv, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, layout=layout, lo=lo, hi=hi,
                new_lo=new_lo, new_hi=new_hi, rope=rope, rot=D if rot is None else rot, lens=lens)


def listed():
    return [
        # one user, a short conversation: latency of a single call
        attend("attend_one_sequence", "bf16", "bf16", 1, 1, 32, 8, 128, 16, "thd", 1024, 1024),
        # a serving batch of unequal lengths
        attend("attend_ragged", "f16", "f16", 64, 1, 28, 4, 128, 64, "thd", 512, 8192),
        # one KV head per query head, pages with the heads outside the tokens
        attend("attend_heads_first", "f16", "f16", 8, 1, 32, 32, 128, 64, "htd", 4096, 4096),
        # long documents, the largest cache
        attend("attend_long", "bf16", "bf16", 16, 1, 32, 8, 128, 64, "thd", 131072, 131072),
        # one user over an 8-bit cache
        attend("attend8_one_sequence", "e4m3", "bf16", 1, 1, 32, 8, 128, 64, "htd", 8192, 8192),
        # the serving batch over an 8-bit cache
        attend("attend8_ragged", "e4m3", "f16", 64, 1, 28, 4, 128, 64, "htd", 512, 8192),
        # four drafted tokens verified at once over long 8-bit caches
        attend("attend8_drafted", "e4m3", "bf16", 16, 4, 32, 8, 128, 128, "htd", 32768, 32768),
        # small heads, odd lengths from one token on, small pages
        attend("attend8_small_heads", "e4m3", "f16", 33, 1, 16, 2, 64, 32, "thd", 1, 5001),
        # one decode step's new tokens
        append("append_decode", "f16", "f16", 64, 28, 4, 128, 64, "thd", 512, 8192, 1, 1),
        # prompts of unequal lengths in one batch
        append("append_prompts", "bf16", "bf16", 5, 32, 8, 128, 64, "thd", 1500, 4000, 1021, 2500),
        # one decode step's new tokens into 8-bit pages
        append("append8_decode", "e4m3", "bf16", 256, 16, 2, 128, 64, "htd", 1, 4096, 1, 1),
        # prompts into 8-bit pages, rotation of half of each head in adjacent pairs
        append("append8_prompts", "e4m3", "bf16", 5, 32, 8, 128, 64, "htd", 1500, 4000, 1021, 2500, "interleaved", 64),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    Hkv = rng.choice([1, 2, 4, 5, 8, 32])
    G = rng.choice([1, 4, 7, 8]) if Hkv < 32 else 1
    D = rng.choice([64, 128, 128])
    kv = rng.choice(["f16", "bf16", "e4m3", "e4m3"])
    dtype = kv if kv != "e4m3" else rng.choice(["f16", "bf16"])
    page = rng.choice([16, 32, 64, 64, 128])
    layout = rng.choice(["thd", "htd"])
    B = spread(rng, 1, 256)
    seed = rng.randrange(1 << 30)
    if rng.random() < 0.6:
        Tq = rng.choice([1, 1, 1, 2, 4, 5])
        # at most a quarter of the largest listed cache: B sequences of up to `hi` keys
        most = max(64, min(131072, (1 << 21) // (4 * B) * 8 // max(8, Hkv)))
        hi = spread(rng, 64, most)
        lo = rng.choice([1, max(1, hi // 16), hi])
        return {k: v for k, v in attend("", kv, dtype, B, Tq, Hkv * G, Hkv, D, page, layout, lo, hi, seed).items() if k != "name"}
    if rng.random() < 0.5:
        new_lo, new_hi = 1, rng.choice([1, 1, 4])
        hi = spread(rng, 64, 4096)
        lo = rng.choice([4, max(4, hi // 8)])
    else:
        B = min(B, 16)
        new_hi = spread(rng, 17, 8192 // B)
        new_lo = max(1, new_hi // rng.choice([1, 3]))
        lo, hi = new_hi, new_hi + spread(rng, 1, 2000)
    rot = rng.choice([D, D, D // 2, 32])
    c = append("", kv, dtype, B, Hkv * G, Hkv, D, page, layout, lo, hi, new_lo, new_hi, rng.choice(["half", "interleaved"]), rot, seed)
    return {k: v for k, v in c.items() if k != "name"}


# ------------------------------------------------------------------ sizes and inputs
def lengths(case):
    """(length of each sequence with its new tokens, new tokens of each), the case's own."""
    rng = random.Random(case["lens"])
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if case["op"] == "attend":
        return lens, [case["Tq"]] * case["B"]
    return lens, [min(n, rng.randint(case["new_lo"], case["new_hi"])) for n in lens]


def pages_of(case, lens):
    return [max(1, -(-n // case["page"])) for n in lens]


def page_shape(case, pages):
    inner = (case["page"], case["Hkv"]) if case["layout"] == "thd" else (case["Hkv"], case["page"])
    return (pages, *inner, case["D"])


def scale_exponent(amax):
    """The least e with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    f, k = torch.frexp(amax)
    return torch.where(amax > 0, (k - 9 + (f > 0.875).to(k.dtype)).clamp(min=LEAST_EXPONENT), LEAST_EXPONENT)


def made_pages(case, pages, gen):
    """Keys or values as a model leaves them in its cache: normal, heads of unequal size."""
    dev = "cuda"
    shape = page_shape(case, pages)
    if case["kv"] != "e4m3":
        return torch.randn(shape, generator=gen, device=dev, dtype=DTYPES[case["kv"]]), None
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
    size = torch.exp2(torch.randint(-2, 3, (pages, case["Hkv"]), generator=gen, device=dev).float())
    over = (1, 3) if case["layout"] == "thd" else (2, 3)
    at = (slice(None), None, slice(None), None) if case["layout"] == "thd" else (slice(None), slice(None), None, None)
    x *= size[at]
    scale = torch.exp2(scale_exponent(x.abs().amax(over)).float())
    x /= scale[at]
    return x.to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lens, new = lengths(case)
    need = pages_of(case, lens)
    total, spare = sum(need), 3
    order = torch.randperm(total + spare, generator=gen, device=dev).to(torch.int32)
    rows = torch.zeros(case["B"], max(need), dtype=torch.int32)
    filled = torch.arange(max(need))[None, :] < torch.tensor(need)[:, None]
    table = rows.to(dev)
    table[filled.to(dev)] = order[:total]
    k, k_scale = made_pages(case, total + spare, gen)
    v, v_scale = made_pages(case, total + spare, gen)
    s = dict(case=case, k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=table,
             kv_lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    B, Hq, Hkv, D, dt = case["B"], case["Hq"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    if case["op"] == "attend":
        s["q"] = torch.randn(B, case["Tq"], Hq, D, generator=gen, device=dev, dtype=dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, case["Tq"], Hq, device=dev)
    else:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu_new"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        # one projection's output: queries, keys and values of a token side by side
        qkv = torch.randn(cu[-1], Hq + 2 * Hkv, D, generator=gen, device=dev, dtype=dt)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_out"] = torch.empty(cu[-1], Hq, D, device=dev, dtype=dt)
        half = case["rot"] // 2
        angle = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * torch.pow(
            500000.0, -torch.arange(half, dtype=torch.float64, device=dev) / half)[None, :]
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if own:
        import split_kv_decode_decoding_gb300 as da

        s["cache"] = da.PagedCache(k, v, k_scale, v_scale,
                                   layout=da.DA_LAYOUT_VARLEN if case["layout"] == "thd" else da.DA_LAYOUT_BHSD)
        s["workspace"] = da.alloc_paged_workspace(case.get("Tq", 1), Hq, Hkv, D)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        import split_kv_decode_decoding_gb300 as da

        if case["op"] == "attend":
            da.decode_attn_paged(state["q"], state["cache"], state["kv_lens"], state["table"], state["out"], state["workspace"],
                                 lse=state["lse"])
            return {"out": state["out"], "lse": state["lse"]}
        da.decode_attn_paged_append(state["q"], state["k_new"], state["v_new"], state["cache"], state["cu_new"], state["kv_lens"],
                                    state["table"], state["workspace"], cos_sin=state["cos_sin"],
                                    rope=da.DA_ROPE_HALF if case["rope"] == "half" else da.DA_ROPE_INTERLEAVED,
                                    q_out=state["q_out"])
        return written(state)
    return plain_attend(state) if case["op"] == "attend" else plain_append(state)


def written(s):
    got = {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if s["k_scale"] is not None:
        got |= {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return got


def gathered(pages, scale, table, layout):
    """[B, Hkv, keys, D] in float32 of a table's pages."""
    i = table.long()
    if scale is None:
        x = pages[i].float()
    else:
        x = pages.view(torch.uint8)[i].view(torch.float8_e4m3fn).float()
        by = scale[i]
        x *= by[:, :, None, :, None] if layout == "thd" else by[:, :, :, None, None]
    x = x.permute(0, 3, 1, 2, 4) if layout == "thd" else x.permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], x.shape[2] * x.shape[3], x.shape[4])


def plain_attend(s):
    c = s["case"]
    B, Tq, Hq, Hkv, D = c["B"], c["Tq"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    k = gathered(s["k"], s["k_scale"], s["table"], c["layout"])
    n = k.shape[2]
    q = s["q"].float().view(B, Tq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Tq, D)
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    del k
    key = torch.arange(n, device="cuda")
    last = s["kv_lens"].long()[:, None] - Tq + torch.arange(Tq, device="cuda")[None, :]   # [B, Tq]
    seen = key[None, None, :] <= last[:, :, None]
    x = x.view(B, Hkv, G, Tq, n).masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    none = top == -math.inf
    e = torch.exp(x - top.masked_fill(none, 0.0))
    total = e.sum(-1, keepdim=True)
    lse = torch.where(none, top, top + torch.log(total))
    e = e / total.masked_fill(none, 1.0)
    del x
    v = gathered(s["v"], s["v_scale"], s["table"], c["layout"])
    # a page's unused tokens hold whatever was there: they weigh nothing
    v = v * (key[None, :] < s["kv_lens"].long()[:, None])[:, None, :, None]
    o = (e.view(B, Hkv, G * Tq, n) @ v).view(B, Hkv, G, Tq, D).permute(0, 3, 1, 2, 4).reshape(B, Tq, Hq, D)
    return {"out": o.to(s["q"].dtype), "lse": lse.squeeze(-1).permute(0, 3, 1, 2).reshape(B, Tq, Hq)}


def rotated(x, cos_sin, position, rope):
    """float32 of x [rows, heads, D], its first dims rotated by the rows' positions."""
    x = x.float()
    rot = cos_sin.shape[1]
    cs = cos_sin[position]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if rope == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    p, r = a * c - b * s, b * c + a * s
    turned = torch.cat([p, r], -1) if rope == "half" else torch.stack([p, r], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def plain_append(s):
    c = s["case"]
    P, thd = c["page"], c["layout"] == "thd"
    cu, lens, table = s["cu_new"].long(), s["kv_lens"].long(), s["table"].long()
    T = s["q"].shape[0]
    row = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, row, right=True) - 1
    position = lens[b] - cu[b + 1] + row
    s["q_out"].copy_(rotated(s["q"], s["cos_sin"], position, c["rope"]))
    page, at = table[b, position // P], position % P
    new = {"k": rotated(s["k_new"], s["cos_sin"], position, c["rope"]), "v": s["v_new"].float()}
    if s["k_scale"] is None:
        for_k, for_v = new["k"].to(s["k"].dtype), new["v"].to(s["v"].dtype)
        if thd:
            s["k"][page, at] = for_k
            s["v"][page, at] = for_v
        else:
            s["k"][page, :, at] = for_k
            s["v"][page, :, at] = for_v
        return written(s)
    append8(s["k"], s["k_scale"], new["k"], page, at, thd, cu, lens, table, P)
    append8(s["v"], s["v_scale"], new["v"], page, at, thd, cu, lens, table, P)
    return written(s)


def append8(pages, scale, x, page, at, thd, cu, lens, table, P):
    """Writes rows x [rows, heads, D] at (page, at) of 8-bit pages, their scales raised where they have to be."""
    n, heads = scale.shape
    most = torch.zeros(n, heads, device="cuda").index_reduce_(0, page, x.abs().amax(-1), "amax")
    begun = torch.zeros(n, dtype=torch.bool, device="cuda")
    begun[page] = True
    fresh = torch.zeros(n, dtype=torch.bool, device="cuda")
    fresh[torch.where(at == 0, page, n - 1)] = True
    fresh[n - 1] = ((page == n - 1) & (at == 0)).any()
    need = torch.exp2(scale_exponent(most).float())
    old = scale.clone()
    wanted = torch.where(fresh[:, None], need, torch.maximum(old, need))
    scale.copy_(torch.where(begun[:, None], wanted, old))
    # the earlier tokens of the page in which a sequence's new tokens start
    start = lens - (cu[1:] - cu[:-1])
    first = table.gather(1, (start // P).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    raw = pages.view(torch.uint8)
    was = raw[first]
    by = (old / scale)[first]
    by = by[:, None, :, None] if thd else by[:, :, None, None]
    again = (was.view(torch.float8_e4m3fn).float() * by).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    slot = torch.arange(P, device="cuda")
    earlier = (slot[None, :] < (start % P)[:, None]) & (cu[1:] > cu[:-1])[:, None]
    earlier = earlier[:, :, None, None] if thd else earlier[:, None, :, None]
    raw[first] = torch.where(earlier, again, was)
    code = (x / scale[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    if thd:
        raw[page, at] = code
    else:
        raw[page, :, at] = code


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    lens, new = lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    wide = 1 if case["kv"] == "e4m3" else 2
    pages = sum(pages_of(case, lens))
    scales = 8 * Hkv * pages if case["kv"] == "e4m3" else 0
    if case["op"] == "attend":
        Tq, keys = case["Tq"], sum(lens)
        rows = case["B"] * Tq * Hq
        return {"bytes": 2 * keys * Hkv * D * wide + scales + 4 * pages + 4 * case["B"] + rows * (4 * D + 4),
                "flops": 4 * keys * Hq * Tq * D}
    T = sum(new)
    touched = sum(-(-n // case["page"]) - (n - m) // case["page"] for n, m in zip(lens, new))
    scales = 16 * Hkv * touched if case["kv"] == "e4m3" else 0
    return {"bytes": T * D * (4 * Hq + 2 * Hkv * (2 + wide)) + 4 * T * case["rot"] + scales + 4 * touched + 8 * case["B"],
            "flops": T * (Hq + Hkv) * case["rot"] * 3}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    lens, new = lengths(case)
    table = s["table"].cpu().tolist()
    return exact_attend(case, s, lens, table) if case["op"] == "attend" else exact_append(case, s, lens, new, table)


def sequence64(pages, scale, row, n, case):
    """[keys, Hkv, D] of one sequence's first n keys."""
    P = case["page"]
    at = torch.tensor(row[:max(1, -(-n // P))], device="cuda")
    x = pages.view(torch.uint8 if scale is not None else torch.int16).index_select(0, at).view(pages.dtype).double()
    if case["layout"] == "htd":
        x = x.transpose(1, 2)
    if scale is not None:
        x = x * scale.index_select(0, at).double()[:, None, :, None]
    return x.reshape(-1, case["Hkv"], case["D"])[:n]


def exact_attend(case, s, lens, table):
    Tq, Hq, Hkv, D = case["Tq"], case["Hq"], case["Hkv"], case["D"]
    out, lse = torch.zeros(case["B"], Tq, Hq, D, dtype=torch.float64), torch.full((case["B"], Tq, Hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(lens):
        k = sequence64(s["k"], s["k_scale"], table[b], n, case)
        v = sequence64(s["v"], s["v_scale"], table[b], n, case)
        for t in range(Tq):
            m = n - Tq + t + 1
            if m <= 0:
                continue
            q = s["q"][b, t].double().view(Hkv, Hq // Hkv, D)
            x = torch.einsum("hgd,khd->hgk", q, k[:m]) / math.sqrt(D)
            z = torch.logsumexp(x, -1)
            out[b, t] = torch.einsum("hgk,khd->hgd", torch.exp(x - z[..., None]), v[:m]).reshape(Hq, D).cpu()
            lse[b, t] = z.reshape(Hq).cpu()
    return {"out": out, "lse": lse}


def e4m3_64(x):
    """The nearest e4m3 value, ties to even, of float64 x (|x| <= 448)."""
    _, e = torch.frexp(x)
    step = torch.exp2((e.double() - 4).clamp(min=-9))
    return torch.round(x / step) * step


def exact_append(case, s, lens, new, table):
    P, Hkv, D, rot, thd = case["page"], case["Hkv"], case["D"], case["rot"], case["layout"] == "thd"
    position = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).cuda()
    page = torch.tensor([table[b][p // P] for b, (n, m) in enumerate(zip(lens, new)) for p in range(n - m, n)], device="cuda")
    cs = s["cos_sin"].double()[position]

    def turn(x):
        x = x.double().clone()
        i = torch.arange(rot // 2, device="cuda")
        i, j = (i, i + rot // 2) if case["rope"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., i], x[..., j]) * torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]
        x[..., i], x[..., j] = z.real, z.imag
        return x

    got = {"q": turn(s["q"])}
    for name, x in (("k", turn(s["k_new"])), ("v", s["v_new"].double())):
        pages, scale = s[name].double(), s[name + "_scale"]
        view = pages if thd else pages.transpose(1, 2)          # [page, token, head, dim]
        if scale is None:
            view[page, position % P] = x
            got[name] = pages
            continue
        scale = scale.double().clone()
        done = 0
        for b, (n, m) in enumerate(zip(lens, new)):
            p = n - m
            while p < n:
                here, first = table[b][p // P], p % P
                stop = min(n, p - first + P)
                rows = x[done:done + stop - p]
                amax = rows.abs().amax((0, 2))
                e = torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(min=LEAST_EXPONENT)
                need = torch.exp2(e)
                if first:
                    up = torch.maximum(scale[here], need)
                    view[here, :first] = e4m3_64(view[here, :first] * (scale[here] / up)[None, :, None])
                    need = up
                scale[here] = need
                view[here, first:first + stop - p] = e4m3_64(rows / need[None, :, None])
                done, p = done + stop - p, stop
        got[name], got[name + "_scale"] = pages, scale
    return got
