"""Shared builders of the full-width tests."""
import numpy as np
import torch

from oracle import full_oracle as F

SHAPES = [(4, 4, 64), (8, 2, 64), (5, 1, 64), (14, 2, 64), (8, 8, 128), (16, 2, 128), (12, 4, 128), (20, 1, 128)]


def skv():
    from rank_mixed_precision_b200 import starkv
    return starkv


def context(H, h_kv, d, device="cuda"):
    """A context of the head shape (its latent factors play no part)."""
    S = skv()
    cfg = S.make_config(H, h_kv, d, 64, 16, 64, 16)
    zero = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device=device)  # noqa: E731
    return S.StarKV(cfg, zero(64, h_kv * 16), zero(64, 64), zero(h_kv, 16, d), zero(64, h_kv * d))


def bf16(rng, *shape, scale=1.0):
    """bf16 tensor on the GPU and the same values in fp32 on the CPU."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16()
    return t.cuda(), t.float().numpy()


def keys(rng, n, h, d):
    x = rng.standard_normal((n, h, d)).astype(np.float32)
    x[..., 3] *= 4
    x[..., d // 2 + 5] *= 4
    t = torch.from_numpy(x).bfloat16()
    return t.cuda(), t.float().numpy()


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32).cuda()


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def tables(rng, caps, extra=0):
    """Block table of random pages with room for `caps` tokens, the ids of `extra` further pages, and the page count."""
    used = [-(-c // F.PAGE) for c in caps]
    ids = rng.permutation(sum(used) + extra + 1).astype(np.int32)  # one page that nothing uses
    t = np.zeros((len(caps), max(1, max(used, default=1))), np.int32)
    at = 0
    for b, u in enumerate(used):
        t[b, :u] = ids[at:at + u]
        at += u
    return t, ids[at:at + extra], sum(used) + extra + 1


def fill(rng, lens, h, d, extra=0):
    """An oracle-written cache of sequences of `lens` tokens: (pages uint8, block table, spare page ids)."""
    t, spare, n_pages = tables(rng, lens, extra)
    pages = rng.integers(0, 256, (n_pages, h, F.page_bytes(d)), dtype=np.uint8)  # free slots hold anything
    for b, n in enumerate(lens):
        _, k = keys_cpu(rng, n, h, d)
        _, v = keys_cpu(rng, n, h, d)
        F.write(pages, k, v, F.slots_of(t[b], n))
    return pages, t, spare


def keys_cpu(rng, n, h, d):
    x = rng.standard_normal((n, h, d)).astype(np.float32)
    x[..., 3] *= 4
    t = torch.from_numpy(x).bfloat16()
    return t, t.float().numpy()


def score_error(q, k):
    """Bound on a score's fp32 error, per (query, head): 2^-20 of the largest sum of |q| |k| / sqrt(d).  A sum of
    d <= 128 exact products in fp32, in blocks of 16 (tensor cores) and however truncated, is off by less than
    16 * 2^-24 = 2^-20 of the sum of their magnitudes."""
    n, H, d = q.shape
    h = k.shape[1]
    if len(k) == 0:
        return np.zeros((n, H))
    top = np.stack([np.abs(q[:, i]) @ np.abs(k[:, i // (H // h)]).T for i in range(H)], 1).max(-1)
    return top * 2.0**-20 / np.sqrt(d)
