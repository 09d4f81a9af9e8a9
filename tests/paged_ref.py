"""Plain references of the paged-cache operators in 64 bits, inputs for their tests, and the
tolerances that follow from the arithmetic. Everything here runs on the CPU."""
import math
import random

import numpy as np
import torch

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
VARLEN, BHSD = 0, 1
LEAST_EXPONENT = -126


def token_view(pages, layout):
    """[page, token, head, ...] view of pages in either layout."""
    return pages if layout == VARLEN else pages.transpose(1, 2)


class Paged:
    """Pages on the CPU, a block table over them, and the lengths of its sequences.

    Pages of a sequence are scattered; every slot behind a sequence's end, and every page that
    belongs to none, holds NaN (scales of such pages: NaN too)."""

    def __init__(self, lens, Hkv, D, kv, page, layout, seed=0, extra_pages=0, width=None, scale_spread=0, mean=0.0):
        rng = random.Random(seed)
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.D, self.kv, self.page, self.layout = list(lens), Hkv, D, kv, page, layout
        need = [-(-n // page) for n in lens]
        total = sum(need) + 2 + extra_pages
        order = list(range(total))
        rng.shuffle(order)
        width = max([1] + need) if width is None else width
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)   # unused entries: never read
        for b, n in enumerate(need):
            for i in range(n):
                self.table[b, i] = order.pop()
        inner = (page, Hkv) if layout == VARLEN else (Hkv, page)
        self.k, self.k_scale = self._make((total, *inner, D), gen, scale_spread, mean)
        self.v, self.v_scale = self._make((total, *inner, D), gen, scale_spread, mean)
        used = torch.zeros(total, page, dtype=torch.bool)
        for b, n in enumerate(self.lens):
            for p in range(n):
                used[int(self.table[b, p // page]), p % page] = True
        self.used = used
        for x in (self.k, self.v):
            raw = x.view(torch.uint8 if kv == "e4m3" else torch.int16)
            token_view(raw, layout)[~used] = 0x7F if kv == "e4m3" else 0x7FFF
        for s in (self.k_scale, self.v_scale):
            if s is not None:
                s[~used.any(1)] = math.nan

    def _make(self, shape, gen, scale_spread, mean):
        x = torch.randn(shape, generator=gen) + mean
        if self.kv != "e4m3":
            return x.to(DTYPES[self.kv]), None
        scale = torch.exp2(torch.randint(-scale_spread, scale_spread + 1, (shape[0], self.Hkv), generator=gen).float() - 6)
        return (x * 64).clamp(-448, 448).to(torch.float8_e4m3fn), scale

    def sequence(self, b):
        """Keys and values of sequence b in 64 bits: [L, Hkv, D] each."""
        got = []
        n = self.lens[b]
        at = self.table[b, : -(-n // self.page)].long()
        for x, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
            y = token_view(x.view(torch.uint8)[at].view(x.dtype) if s is not None else x[at], self.layout).double()
            if s is not None:
                y = y * s[at].double()[:, None, :, None]
            got.append(y.reshape(-1, self.Hkv, self.D)[:n])
        return got


def attend64(q, paged, scale=None):
    """(out [B, T, Hq, D], lse [B, T, Hq], tolerance of out without its last rounding, of lse), q [B, T, Hq, D]."""
    B, T, Hq, D = q.shape
    G = Hq // paged.Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    # a weight is rounded to the 16-bit type it is multiplied in (fp16 for 8-bit pages)
    u = 2.0 ** -8 if paged.kv == "bf16" else 2.0 ** -11
    out, lse = np.zeros((B, T, Hq, D)), np.full((B, T, Hq), -np.inf)
    tol_o, tol_l = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq))
    for b in range(B):
        k, v = (x.numpy() for x in paged.sequence(b))
        for t in range(T):
            n = paged.lens[b] - T + t + 1
            if n <= 0:
                continue
            for h in range(Hq):
                qh, kh, vh = q[b, t, h].double().numpy(), k[:n, h // G], v[:n, h // G]
                x = kh @ qh * scale
                m = x.max()
                w = np.exp(x - m)
                z = w.sum()
                out[b, t, h] = w @ vh / z
                lse[b, t, h] = m + math.log(z)
                # float32: a dot product of D terms, times two factors; exp2 within 2^-22; sums over n keys
                dot = (D + 4) * 2.0 ** -24 * abs(scale) * np.linalg.norm(qh) * np.linalg.norm(kh, axis=1).max()
                wt = dot + 2.0 ** -22 * (1 + np.abs(x).max() * 2)
                tol_l[b, t, h] = wt + n * 2.0 ** -24 + 2.0 ** -21 * abs(lse[b, t, h])
                tol_o[b, t, h] = (u + 2 * wt + 2 * n * 2.0 ** -24) * np.abs(vh).max() + 1e-30
    return out, lse, tol_o, tol_l


def half_step(ref, dtype):
    """Half a unit in the last place of float64 ref in a 16-bit torch dtype."""
    bits = 11 if dtype == torch.float16 else 8
    least = -14 if dtype == torch.float16 else -126
    a = np.abs(np.asarray(ref, dtype=np.float64))
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 2.0 ** least))), least)
    return np.exp2(e - bits)


# ------------------------------------------------------------------ append
def table_of(max_pos, rot, theta=10000.0):
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * torch.pow(
        theta, -torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def turned(x, cos_sin, position, rope, dtype=torch.float64):
    """x [T, heads, D] rotated at the rows' positions in `dtype` arithmetic (rope 0: none)."""
    x = x.to(dtype)
    if rope == 0:
        return x
    rot = cos_sin.shape[1]
    c, s = (y[:, None].to(dtype) for y in cos_sin[position].split(rot // 2, 1))
    i = torch.arange(rot // 2)
    i, j = (i, i + rot // 2) if rope == 1 else (2 * i, 2 * i + 1)
    a, b = x[..., i], x[..., j]
    y = x.clone()
    y[..., i] = a * c - b * s
    y[..., j] = b * c + a * s
    return y


def needed(amax):
    """Least power of two 2^e, e >= -126, with amax <= 448 * 2^e (a loop, on purpose)."""
    e = LEAST_EXPONENT
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def to_e4m3(x):
    """float32 to e4m3, nearest even, saturating; NaN stays."""
    return x.float().clamp(-448, 448).to(torch.float8_e4m3fn)


def append32(paged, q, k, v, lens, new, cos_sin, rope):
    """The append as documented, evaluated step by step in float32, in place on `paged` (16-bit or
    e4m3 pages); returns the rotated queries. `paged.table` must cover lens."""
    P, layout = paged.page, paged.layout
    position = torch.tensor([p for n, m in zip(lens, new) for p in range(n - m, n)], dtype=torch.long)
    T = position.numel()
    rows = {"k": turned(k[:T], cos_sin, position, rope, torch.float32), "v": v[:T].float()}
    q_out = None if q is None else turned(q[:T], cos_sin, position, rope, torch.float32).to(q.dtype)
    for name, x in rows.items():
        pages, scale = getattr(paged, name), getattr(paged, name + "_scale")
        raw = pages.view(torch.uint8 if scale is not None else torch.int16)
        at = token_view(raw, layout)
        done = 0
        for b, (n, m) in enumerate(zip(lens, new)):
            p = n - m
            while p < n:
                page, slot = int(paged.table[b, p // P]), p % P
                stop = min(n, p - slot + P)
                part = x[done:done + stop - p]
                if scale is None:
                    at[page, slot:slot + stop - p] = part.to(pages.dtype).view(torch.int16)
                else:
                    for h in range(paged.Hkv):
                        y = part[:, h]
                        fine = y[torch.isfinite(y)].abs()
                        s = needed(float(fine.max()) if fine.numel() else 0.0)
                        if slot:
                            old = float(scale[page, h])
                            s = max(s, old)
                            if s > old:
                                by = torch.tensor(old) / torch.tensor(s)
                                was = at[page, :slot, h].contiguous().view(torch.float8_e4m3fn).float()
                                at[page, :slot, h] = to_e4m3(was * by).view(torch.uint8)
                        scale[page, h] = s
                        at[page, slot:slot + stop - p, h] = to_e4m3(y / torch.tensor(s)).view(torch.uint8)
                done, p = done + stop - p, stop
    return q_out
