"""fp64 oracle of the full-width entries (include/starkv_full.h), in numpy: the 4-bit cache's bytes, decode attention over
it, eviction, attention of packed prompts and its weights.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

PAGE, GROUP = 16, 32


def page_bytes(d: int) -> int:
    return PAGE * d + 2 * PAGE * 4 * (d // GROUP)


def quantize(x):
    """x fp32 [..., 32]: (codes uint8, scale fp16, zero fp16, overflowed)."""
    x = np.asarray(x, np.float32)
    lo, hi = x.min(-1), x.max(-1)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        s = ((hi - lo) / np.float32(15)).astype(np.float32).astype(np.float16)
        z = lo.astype(np.float16)
        sf, zf = s.astype(np.float32), z.astype(np.float32)
        top = (np.float64(15) * sf + zf).astype(np.float32).astype(np.float16)
        bad = ~(np.isfinite(x).all(-1) & np.isfinite(sf) & np.isfinite(zf) & np.isfinite(top))
        c = np.rint((x - zf[..., None]) / sf[..., None])
    c = np.where((sf == 0)[..., None] | bad[..., None], 0, np.clip(c, 0, 15))
    return c.astype(np.uint8), np.where(bad, np.float16(0), s), np.where(bad, np.float16(0), z), bad


def write(pages, k, v, slots):
    """Token rows k, v fp32 [n, h, d] into pages uint8 [P, h, page_bytes(d)]; True where a group overflowed."""
    n, h, d = k.shape
    ng = d // GROUP
    any_bad = False
    for x, is_v in ((k, False), (v, True)):
        code, s, z, bad = quantize(x.reshape(n, h, ng, GROUP))
        for i, slot in enumerate(slots):
            if slot < 0:
                continue
            any_bad |= bool(bad[i].any())
            p, t = divmod(int(slot), PAGE)
            for g in range(ng):
                for c in range(4):  # words of a group: channels 32 g + 8 c .. + 7
                    w = c * ng + g if not is_v else 4 * g + c
                    at = (PAGE * d // 2 if is_v else 0) + t * d // 2 + 4 * w
                    nib = code[i, :, g, 8 * c:8 * c + 8]
                    pages[p, :, at:at + 4] = nib[:, 0::2] | (nib[:, 1::2] << 4)
                at = PAGE * d + (PAGE * 4 * ng if is_v else 0) + (t * ng + g) * 4
                pages[p, :, at:at + 2] = s[i, :, g].astype("<f2").reshape(h, 1).view(np.uint8)
                pages[p, :, at + 2:at + 4] = z[i, :, g].astype("<f2").reshape(h, 1).view(np.uint8)
    return any_bad


def values(pages, slots, d):
    """(k, v) fp64 [n, h, d] of the tokens at `slots`."""
    h, ng = pages.shape[1], d // GROUP
    out = []
    for is_v in (False, True):
        y = np.empty((len(slots), h, d))
        for i, slot in enumerate(slots):
            p, t = divmod(int(slot), PAGE)
            for g in range(ng):
                at = PAGE * d + (PAGE * 4 * ng if is_v else 0) + (t * ng + g) * 4
                s = np.ascontiguousarray(pages[p, :, at:at + 2]).view("<f2").astype(np.float64)
                z = np.ascontiguousarray(pages[p, :, at + 2:at + 4]).view("<f2").astype(np.float64)
                for c in range(4):
                    w = c * ng + g if not is_v else 4 * g + c
                    at = (PAGE * d // 2 if is_v else 0) + t * d // 2 + 4 * w
                    b = pages[p, :, at:at + 4]
                    nib = np.stack([b & 15, b >> 4], -1).reshape(h, 8).astype(np.float64)
                    y[i, :, 32 * g + 8 * c:32 * g + 8 * c + 8] = nib * s + z
        out.append(y)
    return out


def slots_of(table_row, n, start=0):
    t = np.arange(start, start + n)
    return table_row[t // PAGE].astype(np.int64) * PAGE + t % PAGE


def attend(q, k, v, seen):
    """q fp64 [n, H, d] over k, v fp64 [m, h, d]; row i sees its first seen[i] keys.  Returns out [n, H, d], lse [n, H],
    p [n, H, m], and sum_j p_j |v_j| [n, H, d] (what a relative error of p or v can move)."""
    n, H, d = q.shape
    m, h = k.shape[:2]
    G = H // h
    out, mag = np.zeros((n, H, d)), np.zeros((n, H, d))
    lse, p = np.full((n, H), -np.inf), np.zeros((n, H, m))
    for head in range(H):
        z = q[:, head] @ k[:, head // G].T / np.sqrt(d)
        for i in range(n):
            if seen[i] <= 0:
                continue
            zi = z[i, :seen[i]]
            top = zi.max()
            e = np.exp(zi - top)
            lse[i, head] = top + np.log(e.sum())
            p[i, head, :seen[i]] = e / e.sum()
            vv = v[:seen[i], head // G]
            out[i, head] = p[i, head, :seen[i]] @ vv
            mag[i, head] = p[i, head, :seen[i]] @ np.abs(vv)
    return out, lse, p, mag


def kept_tokens(weights, n, keep, recent):
    """The kept tokens' indices of one KV head, in rising order (weights fp32 [n])."""
    keep = min(n, keep)
    old = n - min(keep, recent)
    w = np.where(np.isnan(weights[:old]), -np.inf, weights[:old].astype(np.float64))
    nan = np.isnan(weights[:old])
    order = sorted(range(old), key=lambda i: (nan[i], -w[i], i))  # heaviest first, NaN last, then the lowest index
    return np.array(sorted(order[:keep - (n - old)]) + list(range(old, n)), np.int64)
