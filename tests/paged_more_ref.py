"""Plain references in 64 bits of chunk and windowed attention over a paged cache, and the
tolerances that follow from the arithmetic. Everything here runs on the CPU."""
import math

import torch


def sees(position, key, window, sinks):
    """[positions, keys]: whether a token at a position sees a key."""
    seen = key[None, :] <= position[:, None]
    if window:
        seen &= (key[None, :] > position[:, None] - window) | (key[None, :] < sinks)
    return seen


def chunk64(q, paged, new, scale=None, window=0, sinks=0):
    """(out [T, Hq, D], lse [T, Hq], tolerance of out without its last rounding, of lse), all float64; q [T, Hq, D]
    holds new[b] rows of each sequence, one after the other."""
    T, Hq, D = q.shape
    G = Hq // paged.Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    # a weight is rounded once to the 16-bit type that it is multiplied in (fp16 for 8-bit pages), half a step at most
    u = 2.0 ** -8 if paged.kv == "bf16" else 2.0 ** -11
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    row = 0
    for b, m in enumerate(new):
        n = paged.lens[b]
        k, v = paged.sequence(b)
        position, key = torch.arange(n - m, n), torch.arange(n)
        seen = sees(position, key, window, sinks)
        any_seen = seen.any(1)
        for h in range(Hq if m and n else 0):
            qh, kh, vh = q[row:row + m, h].double(), k[:, h // G], v[:, h // G]
            x = ((qh @ kh.T) * scale).masked_fill(~seen, -math.inf)
            top = torch.where(any_seen, x.amax(1), torch.zeros(m, dtype=torch.float64))
            w = torch.exp(x - top[:, None])
            z = w.sum(1)
            some = any_seen.clone()
            one = torch.where(some, z, torch.ones_like(z))
            value = torch.where(seen.any(0)[:, None], vh, torch.zeros_like(vh))   # (a value that no row sees counts for none)
            finite = torch.isfinite(value).all()
            if finite:
                o = (w @ value) / one[:, None]
            else:
                o = torch.zeros(m, D, dtype=torch.float64)
                for t in range(m):
                    if some[t]:
                        o[t] = w[t, seen[t]] @ vh[seen[t]] / z[t]
            out[row:row + m, h] = torch.where(some[:, None], o, torch.zeros_like(o))
            lse[row:row + m, h] = torch.where(some, top + one.log(), torch.full_like(z, -math.inf))
            # float32: a dot product of D terms (the tensor cores' sums may drop a bit more), times two or three factors;
            # exp2 within 2^-22; sums over n keys
            big = kh[torch.isfinite(kh).all(1)].norm(dim=1)
            big = big.max() if big.numel() else torch.tensor(0.0, dtype=torch.float64)
            dot = 2 * (D + 4) * 2.0 ** -24 * abs(scale) * qh.nan_to_num(0, 0, 0).norm(dim=1) * big
            most = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(1)
            wt = dot + 2.0 ** -22 * (1 + 2 * most)
            tol_l[row:row + m, h] = wt + n * 2.0 ** -24 + 2.0 ** -21 * (1 + lse[row:row + m, h].abs().nan_to_num(0, 0, 0))
            size = value.nan_to_num(0, 0, 0).abs()
            mean = (w.nan_to_num(0) @ size) / one[:, None]     # a weight's relative error moves its own value
            # weights count down to 2^-36 of the largest: n of them at most go missing
            tol_o[row:row + m, h] = (u + 2 * wt[:, None] + 2 * n * 2.0 ** -24) * mean + n * 2.0 ** -36 * size.amax(0)[None] + 1e-30
        row += m
    return out, lse, tol_o, tol_l


def rounding(ref, dtype):
    """Half a step of a 16-bit type at float64 ref."""
    bits, least = (11, -14) if dtype == torch.float16 else (8, -126)
    a = ref.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.full_like(a, 2.0 ** least)))).clamp(min=least)
    return torch.exp2(e - bits)


def check(out, lse, want, dtype):
    """Compare a kernel's outputs with chunk64's; None, or what differs."""
    ref, ref_l, tol_o, tol_l = want
    out, lse = out.double().cpu().view(ref.shape), lse.double().cpu().view(ref_l.shape)
    fine = torch.isfinite(ref)
    if not torch.equal(torch.isnan(out), torch.isnan(ref)):
        return "NaN in other places: %s" % torch.nonzero(torch.isnan(out) != torch.isnan(ref))[:5].tolist()
    inf = torch.isinf(ref)
    if not torch.equal(out[inf], ref[inf]):
        return "infinities differ"
    over = ((out - ref).abs() - rounding(ref, dtype) * 1.001 - tol_o)[fine]
    if over.numel() and over.max() > 0:
        i = torch.nonzero(((out - ref).abs() - rounding(ref, dtype) * 1.001 - tol_o > 0) & fine)
        return "out off by %g beyond its tolerance, at %s (%d elements)" % (over.max(), i[:4].tolist(), len(i))
    none = torch.isinf(ref_l)
    if not torch.equal(lse[none], ref_l[none]):
        return "lse of rows without keys"
    off = ((lse - ref_l).abs() - tol_l)[torch.isfinite(ref_l)]
    if off.numel() and off.max() > 0:
        return "lse off by %g beyond its tolerance" % off.max()
    return None
