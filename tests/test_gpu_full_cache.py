"""GPU tests of the 4-bit cache of full-width layers: append, read back, decode attention, eviction."""
import numpy as np
import pytest
import torch

from oracle import full_oracle as F

from _full import SHAPES, bf16, context, cu_of, fill, i32, keys, score_error, skv, tables

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("new", [[1], [0, 17, 1], [40, 33]])
def test_append_writes_the_oracles_bytes_and_no_others(shape, new):
    H, h, d = shape
    rng = np.random.default_rng(len(new) + H)
    kv = context(*shape)
    starts = [5 + 3 * b for b in range(len(new))]
    t, _, n_pages = tables(rng, [s + n for s, n in zip(starts, new)])
    pages = rng.integers(0, 256, (n_pages, h, F.page_bytes(d)), dtype=np.uint8)
    n = sum(new)
    kd, k = keys(rng, n, h, d)
    vd, v = bf16(rng, n, h, d)
    slots = np.concatenate([F.slots_of(t[b], m, s) for b, (s, m) in enumerate(zip(starts, new))])
    slots[-1:] = -1 if n > 1 else slots[-1:]  # a token that is skipped
    w0 = rng.standard_normal((n_pages, h, 16)).astype(np.float32)
    first = rng.standard_normal((n, h)).astype(np.float32)
    for given in (None, first):
        want, ww = pages.copy(), w0.copy()
        F.write(want, k, v, slots)
        for i, s in enumerate(slots):
            if s >= 0:
                ww[s // 16, :, s % 16] = 0 if given is None else given[i]
        cache = skv().KV4Cache(kv.cfg, pages=torch.from_numpy(pages.copy()).cuda(), weights=torch.from_numpy(w0.copy()).cuda())
        kv.kv4_append(cache, kd, vd, torch.from_numpy(slots).cuda(), None if given is None else torch.from_numpy(given).cuda())
        assert kv.status() == 0
        np.testing.assert_array_equal(cache.pages.cpu().numpy(), want)
        np.testing.assert_array_equal(cache.weights.cpu().numpy(), ww)


def test_append_of_rows_that_are_parts_of_one_projection():
    H, h, d = 8, 2, 64
    rng = np.random.default_rng(3)
    kv = context(H, h, d)
    qkvd, qkv = bf16(rng, 21, H + 2 * h, d)
    t, _, n_pages = tables(rng, [21])
    slots = F.slots_of(t[0], 21)
    want = np.zeros((n_pages, h, F.page_bytes(d)), np.uint8)
    F.write(want, qkv[:, H:H + h], qkv[:, H + h:], slots)
    cache = kv.new_kv4_cache(n_pages)
    kv.kv4_append(cache, qkvd[:, H:H + h], qkvd[:, H + h:], torch.from_numpy(slots).cuda())
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), want)


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e30, -1e6])
def test_append_of_a_group_that_fp16_cannot_hold(value):
    S = skv()
    H, h, d = 4, 2, 128
    rng = np.random.default_rng(4)
    kv = context(H, h, d)
    kd, _ = keys(rng, 3, h, d)
    vd, _ = bf16(rng, 3, h, d)
    kd[1, 0, 40] = value
    k, v = kd.float().cpu().numpy(), vd.float().cpu().numpy()
    want = np.zeros((1, h, F.page_bytes(d)), np.uint8)
    assert F.write(want, k, v, [3, 4, 5])
    cache = kv.new_kv4_cache(1)
    kv.kv4_append(cache, kd, vd, torch.tensor([3, 4, 5], device="cuda"))
    assert kv.status() == S.DEV_QUANT_OVERFLOW
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), want)


def test_append_of_equal_channels_and_bad_slots():
    S = skv()
    H, h, d = 4, 4, 64
    rng = np.random.default_rng(5)
    kv = context(H, h, d)
    kd, k = keys(rng, 4, h, d)
    vd = torch.full((4, h, d), 0.3, device="cuda").bfloat16()  # no spread: code 0, scale 0
    slots = [7, 32, 1 << 40, -5]                                # two pages: slot 32 is beyond them
    want = np.zeros((2, h, F.page_bytes(d)), np.uint8)
    F.write(want, k, vd.float().cpu().numpy(), [7, -1, -1, -1])
    cache = kv.new_kv4_cache(2)
    kv.kv4_append(cache, kd, vd, torch.tensor(slots, device="cuda"))
    assert kv.status() == S.DEV_BAD_SLOT
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), want)


@pytest.mark.parametrize("shape", SHAPES)
def test_read_returns_the_stored_values_in_bf16(shape):
    H, h, d = shape
    rng = np.random.default_rng(H)
    kv = context(*shape)
    lens, starts = [35, 0, 1, 20], [3, 0, 0, 7]
    pages, t, _ = fill(rng, [n + s for n, s in zip(lens, starts)], h, d)
    cache = skv().KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda())
    got = kv.kv4_read(cache, i32(t), i32(cu_of(lens)), sum(lens), starts=i32(starts))
    assert kv.status() == 0
    slots = np.concatenate([F.slots_of(t[b], n, s) for b, (n, s) in enumerate(zip(lens, starts))])
    for x, y in zip(got, F.values(pages, slots, d)):
        # code * s + z is one fp32 rounding from the 64-bit value, and bf16 another
        want = torch.from_numpy(y.astype(np.float32)).bfloat16().float().numpy()
        np.testing.assert_array_equal(x.float().cpu().numpy(), want)


def test_read_of_bad_pages_lengths_and_spans():
    S = skv()
    H, h, d = 4, 2, 64
    rng = np.random.default_rng(6)
    kv = context(H, h, d)
    pages, t, _ = fill(rng, [40, 40], h, d)
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda())
    good = F.values(pages, F.slots_of(t[0], 40), d)[0]
    bad = t.copy()
    bad[0, 1] = len(pages)
    k, _ = kv.kv4_read(cache, i32(bad), i32([0, 40, 40]), 40)
    assert kv.status() == S.DEV_BAD_PAGE
    assert (k[16:32] == 0).all() and np.abs(k[:16].float().cpu().numpy() - good[:16]).max() < 0.1
    k, _ = kv.kv4_read(cache, i32(t), i32([0, 50, 50]), 50)  # three pages hold 48
    assert kv.status() == S.DEV_BAD_SEQ_LEN and (k[48:] == 0).all()
    k, _ = kv.kv4_read(cache, i32(t), i32([0, 9, 4]), 9)     # the last bound is not the row count
    assert kv.status() == S.DEV_BAD_QUERY_SPAN and (k == 0).all()


# ---------------------------------------------------------------------------------------------------------------------
# decode attention
# ---------------------------------------------------------------------------------------------------------------------
def check_decode(shape, lens, accumulate, seed=0, q_scale=1.0, kv=None, stream=None):
    H, h, d = shape
    rng = np.random.default_rng(seed)
    kv = kv or context(*shape)
    pages, t, _ = fill(rng, lens, h, d)
    qd, q = bf16(rng, len(lens), H, d, scale=q_scale)
    w0 = rng.random((len(pages), h, 16)).astype(np.float32)
    cache = skv().KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda(), weights=torch.from_numpy(w0).cuda())
    torch.cuda.synchronize()
    out = kv.kv4_decode(cache, qd, i32(t), i32(lens), accumulate=accumulate, stream=stream)
    assert kv.status(stream) == 0
    out = out.double().cpu().numpy()
    want_w, tol_w = w0.astype(np.float64), np.zeros(w0.shape)
    for b, n in enumerate(lens):
        slots = F.slots_of(t[b], n)
        k, v = F.values(pages, slots, d)
        o, _, p, mag = F.attend(q[b:b + 1].astype(np.float64), k, v, [n])
        es = score_error(q[b:b + 1], k)[0] if n else np.zeros(H)
        # v: fp16, 2^-11 of its magnitude (code * s + z may cancel: 2^-11 of the group's largest value instead);
        # p: fp16 against a maximum whose p is 1, 2^-11 and 2^-25 a token; the score's error twice (numerator, sum)
        vmax = np.abs(v).max() if n else 0.0
        tol = 2.0**-8 * np.abs(o[0]) + mag[0] * (2.0**-11 + 2 * es[:, None] + 2.0**-20) + 2.0**-11 * vmax + n * 2.0**-25 * vmax
        assert (np.abs(out[b] - o[0]) <= tol).all(), (b, n, np.abs(out[b] - o[0]).max())
        if n:
            add = p[0].reshape(h, H // h, n).sum(1)
            err = (p[0] * (2 * es[:, None] + 2.0**-19)).reshape(h, H // h, n).sum(1)  # ex2, 1 / sum, G additions
            want_w[slots // 16, :, slots % 16] += add.T
            tol_w[slots // 16, :, slots % 16] += err.T
    if accumulate:
        got = cache.weights.double().cpu().numpy()
        assert (np.abs(got - want_w) <= tol_w + 2.0**-23 * np.abs(want_w)).all()
    else:
        np.testing.assert_array_equal(cache.weights.cpu().numpy(), w0)
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), pages)


@pytest.mark.parametrize("shape", SHAPES + [(24, 1, 64), (80, 2, 64)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_decode_small(shape, accumulate):
    check_decode(shape, [1, 16, 0, 17, 100], accumulate, seed=sum(shape))


@pytest.mark.parametrize("shape", [(4, 4, 64), (14, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("lens", [[1500], [333, 0, 1027]])
def test_decode_of_several_splits(shape, lens):
    check_decode(shape, lens, True, seed=len(lens))


@pytest.mark.parametrize("shape,lens", [((14, 2, 64), [9000, 5003]), ((20, 1, 128), [12001]), ((8, 1, 64), [7000, 0, 40])])
def test_decode_of_long_sequences_of_few_heads(shape, lens):
    """A unit of many parts: their heads are joined in several blocks."""
    check_decode(shape, lens, True, seed=lens[0])
    check_decode(shape, lens, False, seed=lens[0])


def test_decode_of_short_sequences_in_wide_tables():
    """A table with room for far more pages than its sequences hold: fewer pages than the work is cut into."""
    S = skv()
    shape = H, h, d = 8, 2, 64
    for lens in ([40, 3, 0, 100], [17], [0, 1]):
        rng = np.random.default_rng(sum(lens))
        kv = context(*shape)
        pages, t, _ = fill(rng, lens, h, d)
        wide = np.full((len(lens), 700), 1 << 30, np.int32)  # what lies behind a sequence's pages is not read
        wide[:, :t.shape[1]] = t
        qd, q = bf16(rng, len(lens), H, d)
        cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda(), weights=torch.zeros((len(pages), h, 16), device="cuda"))
        for accumulate in (False, True):
            out = kv.kv4_decode(cache, qd, i32(wide), i32(lens), accumulate=accumulate).double().cpu().numpy()
            assert kv.status() == 0
            for b, n in enumerate(lens):
                k, v = F.values(pages, F.slots_of(t[b], n), d)
                o, _, _, mag = F.attend(q[b:b + 1].astype(np.float64), k, v, [n])
                assert (np.abs(out[b] - o[0]) <= 2.0**-8 * np.abs(o[0]) + 2.0**-10 * (mag[0] + np.abs(v).max(initial=0))).all()
        w = cache.weights.double().cpu().numpy()
        assert abs(w.sum() - H * sum(n > 0 for n in lens)) < 1e-4


def test_decode_with_scores_far_apart():
    check_decode((8, 2, 128), [400, 90], True, seed=2, q_scale=30.0)
    check_decode((8, 2, 128), [400, 90], True, seed=2, q_scale=1e-3)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [2.0**90, 2.0**112])
def test_decode_with_queries_of_large_magnitude(d, scale):
    """Scores of either sign and up to 2^118: a single token takes all of its heads' weight, however low its score."""
    S = skv()
    H, h = 8, 2
    rng = np.random.default_rng(d)
    kv = context(H, h, d)
    lens = [1] * 12 + [40]
    pages, t, _ = fill(rng, lens, h, d)
    qd, q = bf16(rng, len(lens), H, d, scale=scale)
    assert np.abs(q).max() < 2.0**115
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda(), weights=torch.zeros((len(pages), h, 16), device="cuda"))
    out = kv.kv4_decode(cache, qd, i32(t), i32(lens), accumulate=True).double().cpu().numpy()
    assert kv.status() == 0
    w = cache.weights.double().cpu().numpy()
    seen = set()
    for b, n in enumerate(lens):
        k, v = F.values(pages, F.slots_of(t[b], n), d)
        if n == 1:
            want = np.repeat(v[0], H // h, 0)
            seen |= set(np.sign((q[b].reshape(h, -1, d) * k[0][:, None]).sum(-1)).ravel())
            # p = 1 exactly; v in fp16 and the output in bf16, half a step each
            assert (np.abs(out[b] - want) <= 2.0**-8 * np.abs(want) + 2.0**-10 * np.abs(v).max()).all(), b
            assert (w[t[b, 0], :, 0] == H // h).all()
        else:
            assert np.isfinite(out[b]).all() and (np.abs(out[b]) <= 1.01 * np.abs(v).max()).all()
            assert abs(w[t[b, :3]].sum() - H) < 1e-4
    assert seen == {-1.0, 1.0}


def test_decode_of_empty_sequences_only():
    check_decode((8, 2, 64), [0, 0, 0], True)


def test_decode_leaves_out_bad_pages_and_lengths():
    S = skv()
    H, h, d = 8, 2, 64
    rng = np.random.default_rng(8)
    kv = context(H, h, d)
    pages, t, _ = fill(rng, [40, 30, 20], h, d)
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda(), weights=torch.zeros((len(pages), h, 16), device="cuda"))
    qd, q = bf16(rng, 3, H, d)
    bad = t.copy()
    bad[1, 0] = -3
    out = kv.kv4_decode(cache, qd, i32(bad), i32([40, 30, 99]), accumulate=True).double().cpu().numpy()
    assert kv.status() == S.DEV_BAD_PAGE | S.DEV_BAD_SEQ_LEN
    k, v = F.values(pages, F.slots_of(t[1], 30)[16:], d)
    want = F.attend(q[1:2].astype(np.float64), k, v, [14])[0][0]
    assert np.abs(out[1] - want).max() < 2.0**-7 * max(1, np.abs(want).max()) + 2.0**-9 * np.abs(v).max()
    assert (out[2] == 0).all()
    w = cache.weights.double().cpu().numpy()
    assert abs(w[t[0, :3]].sum() - H) < 1e-4 and abs(w[t[1, 1]].sum() - H) < 1e-4 and w.sum() < 2 * H + 1e-3


def test_decode_is_the_same_each_time_and_on_another_stream():
    S = skv()
    H, h, d = 14, 2, 64
    rng = np.random.default_rng(9)
    kv = context(H, h, d)
    pages, t, _ = fill(rng, [700, 300], h, d)
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda())
    qd, _ = bf16(rng, 2, H, d)
    td, ld = i32(t), i32([700, 300])
    first = kv.kv4_decode(cache, qd, td, ld)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        other = kv.kv4_decode(cache, qd, td, ld, stream=side)
        again = kv.kv4_decode(cache, qd, td, ld)  # two calls at once
        torch.cuda.synchronize()
        assert torch.equal(first, again) and torch.equal(first, other)


# ---------------------------------------------------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------------------------------------------------
def check_evict(shape, lens, keeps, recent, seed=0, weights=None, alias=False):
    S = skv()
    H, h, d = shape
    rng = np.random.default_rng(seed)
    kv = context(*shape)
    room = [-(-min(n, k) // 16) for n, k in zip(lens, keeps)]
    pages, t, spare = fill(rng, lens, h, d, extra=sum(room))
    dst = np.zeros((len(lens), max(1, max(room))), np.int32)
    at = 0
    for b, r in enumerate(room):
        dst[b, :r] = spare[at:at + r]
        at += r
    w0 = np.exp(1.5 * rng.standard_normal((len(pages), h, 16))).astype(np.float32) if weights is None else weights(rng, (len(pages), h, 16))
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages.copy()).cuda(), weights=torch.from_numpy(w0.copy()).cuda())
    ld, kd = i32(lens), i32(keeps)
    if alias:
        kept = torch.empty((len(lens), h, dst.shape[1] * 16), dtype=torch.int32, device="cuda")
        S.starkv_kv4_evict(kv.ctx, kv.cfg, cache.struct, i32(t), ld, kd, recent, i32(dst), ld, kept)
        new = ld
    else:
        new, kept = kv.kv4_evict(cache, i32(t), ld, kd, recent, i32(dst))
    assert kv.status() == 0
    np.testing.assert_array_equal(new.cpu().numpy(), np.minimum(lens, keeps))
    want_p, want_w = pages.copy(), w0.copy()
    want_kept = np.full((len(lens), h, dst.shape[1] * 16), -1, np.int32)
    ng = d // 32
    planes = [(0, d // 2), (8 * d, d // 2), (16 * d, 4 * ng), (16 * d + 64 * ng, 4 * ng)]
    for b, (n, keep) in enumerate(zip(lens, keeps)):
        src = F.slots_of(t[b], n)
        for head in range(h):
            stay = F.kept_tokens(w0[src // 16, head, src % 16], n, keep, recent)
            want_kept[b, head, :len(stay)] = stay
            for i, j in enumerate(stay):
                s, o = src[j], F.slots_of(dst[b], 1, i)[0]
                for base, row in planes:
                    want_p[o // 16, head, base + o % 16 * row:base + (o % 16 + 1) * row] = \
                        pages[s // 16, head, base + s % 16 * row:base + (s % 16 + 1) * row]
                want_w[o // 16, head, o % 16] = w0[s // 16, head, s % 16]
    np.testing.assert_array_equal(kept.cpu().numpy(), want_kept)
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), want_p)
    np.testing.assert_array_equal(cache.weights.cpu().numpy().view(np.int32), want_w.view(np.int32))


@pytest.mark.parametrize("shape", [(4, 4, 64), (8, 2, 128)])
@pytest.mark.parametrize("recent", [0, 1, 8, 10**6])
def test_evict(shape, recent):
    check_evict(shape, [100, 0, 1, 33, 16], [40, 5, 1, 33, 0], recent, seed=recent % 7)


def test_evict_with_lengths_written_in_place():
    check_evict((8, 2, 64), [70, 20, 50], [10, 30, 49], 4, alias=True)


@pytest.mark.parametrize("n", [1025, 4000])
def test_evict_longer(n):
    check_evict((2, 1, 64), [n], [n // 3], 17, seed=n)


def check_selection(h, lens, keeps, recent, weights):
    """The kept tokens of long sequences in scattered pages against a stable sort."""
    S = skv()
    kv = context(h, h, 64)
    rng = np.random.default_rng(len(lens) + lens[0])
    room = [-(-min(n, k) // 16) for n, k in zip(lens, keeps)]
    t, spare, n_pages = tables(rng, lens, extra=sum(room))
    dst = np.zeros((len(lens), max(room)), np.int32)
    at = 0
    for b, r in enumerate(room):
        dst[b, :r] = spare[at:at + r]
        at += r
    w = weights(rng, (n_pages, h, 16)).astype(np.float32)
    cache = S.KV4Cache(kv.cfg, n_pages, weights=torch.from_numpy(w).cuda())
    new, kept = kv.kv4_evict(cache, i32(t), i32(lens), i32(keeps), recent, i32(dst))
    assert kv.status() == 0
    kept = kept.cpu().numpy()
    for b, (n, keep) in enumerate(zip(lens, keeps)):
        src = F.slots_of(t[b], n)
        keep = min(n, keep)
        for head in range(h):
            x = w[src // 16, head, src % 16].copy()
            x[n - min(keep, recent):] = np.inf
            stay = np.sort(np.argsort(-x, kind="stable")[:keep])
            np.testing.assert_array_equal(kept[b, head, :keep], stay)
            assert (kept[b, head, keep:] == -1).all()


@pytest.mark.parametrize("h,lens", [(1, [20000]), (3, [9000, 300]), (2, [70001]), (1, [140000]), (160, [5000])])
def test_evict_selects_from_long_sequences(h, lens):
    """On one CTA a list and on clusters of two, four and eight; more tokens than registers hold."""
    keeps = [max(1, n * 2 // 5) for n in lens]
    check_selection(h, lens, keeps, 33, lambda rng, s: np.exp(1.5 * rng.standard_normal(s)))
    if h < 100:
        check_selection(h, lens, [n - 1 for n in lens], 1, lambda rng, s: rng.integers(0, 3, s))   # ties across CTAs
        check_selection(h, lens, [5] * len(lens), 0, lambda rng, s: rng.standard_normal(s))


def test_evict_of_equal_weights_takes_the_lowest_index():
    check_evict((4, 2, 64), [90, 50], [30, 20], 4, weights=lambda rng, s: np.zeros(s, np.float32))
    check_evict((4, 2, 64), [90, 50], [30, 20], 4, weights=lambda rng, s: rng.integers(0, 3, s).astype(np.float32))
    check_evict((4, 2, 64), [90], [30], 4, weights=lambda rng, s: np.where(rng.random(s) < 0.5, -0.0, 0.0).astype(np.float32))


def test_evict_of_weights_that_are_not_finite():
    def weights(rng, s):
        w = rng.standard_normal(s).astype(np.float32)
        kind = rng.integers(0, 4, s)
        return np.where(kind == 0, np.float32("nan"), np.where(kind == 1, np.float32("inf"), np.where(kind == 2, np.float32("-inf"), w))).astype(np.float32)
    for keep in (10, 60, 85):
        check_evict((4, 2, 64), [90], [keep], 3, weights=weights)


def test_evict_skips_bad_lengths_and_pages():
    S = skv()
    H, h, d = 4, 2, 64
    rng = np.random.default_rng(11)
    kv = context(H, h, d)
    pages, t, spare = fill(rng, [40, 40, 40, 40], h, d, extra=4)
    w0 = rng.random((len(pages), h, 16)).astype(np.float32)
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages.copy()).cuda(), weights=torch.from_numpy(w0).cuda())
    bad = t.copy()
    bad[1, 2] = len(pages)
    new, kept = kv.kv4_evict(cache, i32(bad), i32([49, 40, -1, 40]), i32([8, 8, 8, 17]), 2, i32(spare.reshape(4, 1)))
    assert kv.status() == S.DEV_BAD_PAGE | S.DEV_BAD_SEQ_LEN
    assert new.tolist() == [0, 0, 0, 0] and (kept == -1).all()
    np.testing.assert_array_equal(cache.pages.cpu().numpy(), pages)


# ---------------------------------------------------------------------------------------------------------------------
# captured
# ---------------------------------------------------------------------------------------------------------------------
def test_steps_captured_into_graphs_that_run_in_turn():
    """Append, decode and evict in two graphs of one context, replayed with other inputs: the same as plain calls."""
    S = skv()
    H, h, d = 8, 2, 64
    rng = np.random.default_rng(12)
    kv = context(H, h, d)
    pages, t, spare = fill(rng, [90, 70], h, d, extra=8)
    td, dst = i32(t), i32(spare.reshape(2, 4))
    lens, keeps = i32([90, 70]), i32([60, 33])
    qs = [bf16(rng, 2, H, d)[0] for _ in range(3)]
    ks = [bf16(rng, 2, h, d)[0] for _ in range(3)]
    slots = torch.tensor([F.slots_of(t[0], 1, 89)[0], F.slots_of(t[1], 1, 69)[0]], device="cuda")

    def fresh():
        return S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages.copy()).cuda(), keep_weights=True)

    def step(cache, q, k):
        kv.kv4_append(cache, k, k, slots)
        out = kv.kv4_decode(cache, q, td, lens, accumulate=True)
        return out, *kv.kv4_evict(cache, td, lens, keeps, 5, dst)

    plain, want = fresh(), []
    for q, k in zip(qs, ks):
        want.append([x.clone() for x in step(plain, q, k)])
    graphs = []
    for _ in range(2):
        cache, q, k = fresh(), qs[0].clone(), ks[0].clone()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(cache, q, k)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(cache, q, k)
        cache.pages.copy_(torch.from_numpy(pages))
        cache.weights.zero_()
        graphs.append((g, cache, q, k, out))
    for i in range(3):
        for g, cache, q, k, out in graphs:
            q.copy_(qs[i])
            k.copy_(ks[i])
            g.replay()
        for g, cache, q, k, out in graphs:
            for x, y in zip(out, want[i]):
                assert torch.equal(x, y)
    for g, cache, *_ in graphs:
        assert torch.equal(cache.pages, plain.pages) and torch.equal(cache.weights, plain.weights)
    assert kv.status() == 0


# ---------------------------------------------------------------------------------------------------------------------
# refusals: from the host's checks, before anything is launched
# ---------------------------------------------------------------------------------------------------------------------
def test_calls_that_are_refused():
    S = skv()
    H, h, d = 8, 2, 64
    kv = context(H, h, d)
    L = S.lib()
    cache = kv.new_kv4_cache(4, keep_weights=True)
    bare = kv.new_kv4_cache(4)
    no_pages = S.starkv_kv4_cache(None, None, 0)
    big = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    p = big.data_ptr()
    import ctypes
    ref, width = ctypes.byref, h * d

    def append(c=cache.struct, k=p, v=p, ks=width, vs=width, slots=p, n=1):
        return L.starkv_kv4_append(kv.ctx, ref(c), k, v, ks, vs, slots, None, n, None)

    def decode(c=cache.struct, q=p, table=p, lens=p, batch=1, pages=40, acc=0, out=p, ws=p, size=1 << 20):
        return L.starkv_kv4_decode_attn(kv.ctx, ref(c), q, table, lens, batch, pages, acc, out, ws, size, None)

    def evict(c=cache.struct, recent=1, batch=1, pages=1, dst=1, kept=p):
        return L.starkv_kv4_evict(kv.ctx, ref(c), p, p, p, recent, batch, pages, p, dst, p, kept, None)

    def read(batch=1, pages=1, total=1, out=p, cu=p):
        return L.starkv_kv4_read(kv.ctx, ref(cache.struct), p, None, cu, batch, pages, total, out, p, None)

    def prompt(q=p, k=p, v=p, qs=H * d, ks=width, vs=width, batch=1, nq=1, nk=1, most=1, out=p, lse=p, ws=p, size=1 << 20):
        return L.starkv_prompt_attn(kv.ctx, q, k, v, qs, ks, vs, p, p, batch, nq, nk, most, out, lse, ws, size, None)

    def weigh(lse=p, batch=1, nq=1, nk=1, most=1, window=1, out=p, ks=width):
        return L.starkv_prompt_weights(kv.ctx, p, p, H * d, ks, lse, p, p, batch, nq, nk, most, window, out, None)

    bad, shape, small = S.ERR_INVALID_ARG, S.ERR_UNSUPPORTED_SHAPE, S.ERR_WORKSPACE_TOO_SMALL
    refused = [
        (append(n=-1), bad), (append(k=None), bad), (append(v=p + 2), bad), (append(ks=width - 8), bad), (append(vs=width + 4), bad),
        (append(slots=None), bad), (append(c=no_pages), bad), (append(n=1 << 40), shape),
        (append(c=S.starkv_kv4_cache(p + 8, None, 1)), bad), (append(c=S.starkv_kv4_cache(p, p + 4, 1)), bad),
        (append(c=S.starkv_kv4_cache(None, None, 1)), bad), (append(c=S.starkv_kv4_cache(p, None, -1)), bad),
        (decode(batch=-1), bad), (decode(pages=0), bad), (decode(batch=65536), shape), (decode(pages=(1 << 26) + 1), shape),
        (decode(q=None), bad), (decode(out=p + 4), bad), (decode(c=bare.struct, acc=1), bad), (decode(size=16), small),
        (decode(ws=None), small), (decode(ws=p + 16), bad),
        (evict(recent=-1), bad), (evict(dst=0), bad), (evict(kept=None), bad), (evict(c=bare.struct), bad), (evict(batch=1 << 17), shape),
        (read(total=-1), bad), (read(batch=0), bad), (read(out=p + 2), bad), (read(cu=None), bad), (read(total=1 << 40), shape),
        (prompt(nq=-1), bad), (prompt(most=0), bad), (prompt(batch=0), bad), (prompt(batch=1 << 16), shape), (prompt(nk=1 << 31), shape),
        (prompt(q=p + 8), bad), (prompt(qs=H * d - 8), bad), (prompt(ks=0), bad), (prompt(vs=width + 1), bad), (prompt(out=None), bad),
        (prompt(lse=p + 2), bad), (prompt(nk=4096, ws=None), small), (prompt(nk=4096, size=64), small),
        (prompt(nk=4096, ws=p + 64), small),  # 32 parts of 256 rows take 4 MB, and 1 MB is given
        (prompt(nk=4096, ws=p + 64, size=1 << 23), bad),
        (weigh(window=-1), bad), (weigh(most=0), bad), (weigh(lse=None), bad), (weigh(out=p + 2), bad), (weigh(ks=8), bad),
        (weigh(batch=1 << 16), shape), (weigh(nk=1 << 31, most=1 << 30), shape),
    ]
    for i, (got, want) in enumerate(refused):
        assert got == want, (i, got, want, S.starkv_last_error())
    # nothing to do is not an error
    assert append(n=0, k=None, v=None, slots=None) == 0 and decode(batch=0, pages=0) == 0 and evict(batch=0, pages=0, dst=0) == 0
    assert read(total=0) == 0 and prompt(nq=0, batch=0) == 0 and weigh(nk=0, batch=0) == 0
    assert kv.status() == 0
    q = torch.zeros((2, H, d), dtype=torch.bfloat16, device="cuda")
    table, lens = i32(np.zeros((2, 1))), i32([0, 0])
    for call in (lambda: kv.kv4_decode(cache, q[:1], table, lens), lambda: kv.kv4_decode(cache, q[:, :4], table, lens),
                 lambda: kv.kv4_decode(cache, q, table, lens, out=q[:1]), lambda: kv.kv4_read(cache, table, lens, 2),
                 lambda: kv.prompt(q, q[:, :2], q[:1, :2], lens, lens, 1), lambda: kv.prompt(q[:, :, :32], q, q, lens, lens, 1),
                 lambda: kv.kv4_append(cache, q[:, :2], q[:, :2], torch.zeros(3, dtype=torch.int64, device="cuda")),
                 lambda: kv.kv4_decode(cache, q.cpu(), table, lens), lambda: kv.kv4_evict(cache, table, lens, lens, 0, table[:1])):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_pages_whose_offsets_pass_32_bits():
    """A pool of more than 4 GB, its last pages in use: write, read, decode with weights, evict."""
    S = skv()
    shape = H, h, d = 16, 8, 128
    rng = np.random.default_rng(15)
    kv = context(*shape)
    n_pages = (1 << 32) // (h * F.page_bytes(d)) + 40
    cache = kv.new_kv4_cache(n_pages, keep_weights=True)
    n, keep = 70, 40
    t = np.arange(n_pages - 5, n_pages, dtype=np.int32)[None]
    dst = np.arange(n_pages - 20, n_pages - 17, dtype=np.int32)[None]
    slots = F.slots_of(t[0], n)
    kd, k = keys(rng, n, h, d)
    vd, v = bf16(rng, n, h, d)
    kv.kv4_append(cache, kd, vd, torch.from_numpy(slots).cuda())
    small = np.zeros((5, h, F.page_bytes(d)), np.uint8)
    F.write(small, k, v, slots - int(t[0, 0]) * 16)
    np.testing.assert_array_equal(cache.pages[n_pages - 5:].cpu().numpy(), small)
    kk, vv = F.values(small, slots - int(t[0, 0]) * 16, d)
    got, _ = kv.kv4_read(cache, i32(t), i32([0, n]), n)
    np.testing.assert_array_equal(got.float().cpu().numpy(), torch.from_numpy(kk.astype(np.float32)).bfloat16().float().numpy())
    qd, q = bf16(rng, 1, H, d)
    out = kv.kv4_decode(cache, qd, i32(t), i32([n]), accumulate=True).double().cpu().numpy()
    o, _, p, mag = F.attend(q.astype(np.float64), kk, vv, [n])
    assert (np.abs(out - o) <= 2.0**-8 * np.abs(o) + 2.0**-10 * (mag + np.abs(vv).max())).all()
    w = cache.weights[n_pages - 5:].cpu().numpy()
    _, kept = kv.kv4_evict(cache, i32(t), i32([n]), i32([keep]), 4, i32(dst))
    assert kv.status() == 0
    local = slots - int(t[0, 0]) * 16
    moved = cache.pages[n_pages - 20:n_pages - 17].cpu().numpy()
    for head in range(h):
        stay = F.kept_tokens(w[local // 16, head, local % 16], n, keep, 4)
        np.testing.assert_array_equal(kept[0, head, :keep].cpu().numpy(), stay)
        km, vm = F.values(moved[:, head:head + 1], np.arange(keep), d)
        np.testing.assert_array_equal(km[:, 0], kk[stay, head])
        np.testing.assert_array_equal(vm[:, 0], vv[stay, head])


def test_calls_behind_close_are_refused():
    S = skv()
    kv = context(8, 2, 64)
    cache = kv.new_kv4_cache(4)
    q, one = torch.zeros((1, 8, 64), dtype=torch.bfloat16, device="cuda"), i32([1])
    k = q[:, :2].contiguous()
    kv.kv4_decode(cache, q, i32([[0]]), one)
    kv.close()
    for call in (lambda: kv.kv4_decode(cache, q, i32([[0]]), one), lambda: kv.prompt(q, k, k, i32([0, 1]), i32([0, 1]), 1),
                 lambda: kv.kv4_append(cache, k, k, torch.zeros(1, dtype=torch.int64, device="cuda"))):
        with pytest.raises(S.StarKVError) as e:
            call()
        assert e.value.code == S.ERR_INVALID_ARG


def test_decode_of_scores_one_step_of_fp32_apart():
    """Scores of 2^27 to 2^28 (log2), where fp32 numbers are 16 apart, that rise by one such step at a time: as far as the
    running maximum lets a score pass it, and no farther (a probability of 2^16 is infinite in fp16)."""
    S = skv()
    shape = H, h, d = 64, 8, 64
    rng = np.random.default_rng(27)
    kv = context(*shape)
    B, n = 8, 2048  # 64 units of 128 pages: each by one CTA, whose warps take 32 tokens of every 128 in turn
    k = np.zeros((n, h, d), np.float32)
    k[:, :, :32] = 1024
    k[:, :, 32:] = (np.arange(n) // 128)[:, None, None]
    v = rng.standard_normal((n, h, d)).astype(np.float32)
    pages = np.zeros((n // 16, h, F.page_bytes(d)), np.uint8)
    slots = np.arange(n)
    F.write(pages, k, v, slots)
    q = np.zeros((B, H, d), np.float32)
    q[:, :, 0] = 2.0**20 * (0.75 + rng.integers(0, 28, (B, H)) / 128)  # bf16 numbers: products of 0.75 to 0.97 of 2^30
    q[:, :, 32] = 64                                                   # the step of fp32 there
    scale = np.float32(1.4426950408889634 / 8)
    dots = q[:, :, :1].astype(np.float64) * 1024 + 64 * (np.arange(n) // 128)  # [B, H, n], exact in fp32
    z = (dots.astype(np.float32) * scale).astype(np.float32)
    assert (z >= 2.0**27).all() and (z < 2.0**28).all()
    steps = z[:, :, ::128]
    up, even = steps[:, :, 1:] == steps[:, :, :-1] + np.float32(16), steps[:, :, :-1] % 32 == 0
    assert (up & ~even).sum() > 100 and (up & even).sum() > 100  # the sum of an odd multiple of 16 and 8 rounds up
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda(), weights=torch.zeros((n // 16, h, 16), device="cuda"))
    t = np.tile(np.arange(n // 16, dtype=np.int32), (B, 1))
    kk, vv = F.values(pages, slots, d)
    np.testing.assert_array_equal(kk, k)
    for accumulate in (False, True):
        out = kv.kv4_decode(cache, torch.from_numpy(q).bfloat16().cuda(), i32(t), i32([n] * B), accumulate=accumulate)
        assert kv.status() == 0 and torch.isfinite(out).all()
        x = z.astype(np.float64)
        p = np.exp2(x - x.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        for head in range(H):
            o, mag = p[:, head] @ vv[:, head // 8], p[:, head] @ np.abs(vv[:, head // 8])
            # the output in bf16, v and p in fp16, ex2 and fp32 sums
            tol = 2.0**-8 * np.abs(o) + 2.0**-10 * (mag + np.abs(vv).max()) + 2.0**-18 * mag
            assert (np.abs(out[:, head].double().cpu().numpy() - o) <= tol).all()
    want = p.reshape(B, h, 8, n).sum((0, 2))  # [h, n]
    got = cache.weights.double().cpu().numpy().transpose(1, 0, 2).reshape(h, n)
    assert (np.abs(got - want) <= 2.0**-17 * want + 2.0**-30).all()


@pytest.mark.parametrize("shape,n,batch", [((8, 2, 64), 2000, 1), ((16, 2, 128), 2000, 1), ((14, 2, 64), 300, 3), ((64, 32, 128), 700, 3)])
def test_decode_keeps_a_long_light_tail(shape, n, batch):
    """One token in 32 takes nearly all of the weight, the others 2^-25 to 2^-30 of it each, and their values alone count."""
    S = skv()
    H, h, d = shape
    kv = context(*shape)
    tail = np.arange(n) % 32 != 5
    k, v = np.zeros((n, h, d), np.float32), np.zeros((n, h, d), np.float32)
    k[tail] = -32
    v[tail] = 1
    pages = np.zeros((-(-n // 16), h, F.page_bytes(d)), np.uint8)
    F.write(pages, k, v, np.arange(n))
    q = np.zeros((batch, H, d), np.float32)
    q[:, :, 7] = 4.5 * (d / 64) ** 0.5 * (1 + np.arange(batch * H).reshape(batch, H) % 5 / 32)
    qd = torch.from_numpy(q).bfloat16().cuda()
    z = -32 * qd.double().cpu().numpy()[:, :, 7] / d**0.5 / np.log(2.0)
    assert (z < -25).all() and (z > -30).all()
    t = np.tile(np.arange(-(-n // 16), dtype=np.int32), (batch, 1))
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda())
    out = kv.kv4_decode(cache, qd, i32(t), i32([n] * batch)).double().cpu().numpy()
    assert kv.status() == 0
    p = np.exp2(z) * tail.sum()
    want = (p / (p + (~tail).sum()))[..., None]
    # the output in bf16; a probability's half step in fp16 against a maximum of 2^7 or more, 2^-32, each; score, ex2, sums
    lost = tail.sum() / (~tail).sum() * 2.0**-32
    assert (np.abs(out - want) <= want * (2.0**-8 + 2.0**-16) + lost).all()
    assert (lost < want / 4).all()


@pytest.mark.parametrize("batch,many", [(3, 1), (400, 100)])
def test_read_reports_bounds_that_fall(batch, many):
    """cu = 0 .. 5, 3 .. 9: every row lies in some sequence, but one sequence ends before it begins."""
    S = skv()
    H, h, d = 4, 2, 64
    kv = context(H, h, d)
    pages, t, _ = fill(np.random.default_rng(16), [40] * 4, h, d)
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda())
    table = i32(np.tile(t[:1], (batch, 1)))
    good = np.zeros(batch + 1, np.int32)
    good[batch - 2:batch], good[batch] = 5 * many, 9 * many
    cu = good.copy()
    cu[batch - 1] = 3 * many
    starts = i32(np.zeros(batch))
    if many > 1:
        table = i32(np.tile(np.resize(t[0], (1, 64)), (batch, 1)))
    kv.kv4_read(cache, table, i32(good), 9 * many, starts=starts)
    assert kv.status() == 0
    kv.kv4_read(cache, table, i32(cu), 9 * many, starts=starts)
    assert kv.status() == S.DEV_BAD_QUERY_SPAN


@pytest.mark.parametrize("shape", [(1, 1, 64), (2, 1, 128), (3, 1, 64), (1024, 8, 64), (256, 256, 64)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_decode_of_the_fewest_and_the_most_heads(shape, accumulate):
    check_decode(shape, [37, 0, 600], accumulate, seed=shape[0])


def test_evict_of_one_head_and_of_many():
    check_evict((1, 1, 128), [70, 33], [30, 33], 5)
    check_evict((300, 300, 64), [40], [17], 3)


@pytest.mark.parametrize("accumulate", [False, True])
def test_decode_of_more_sequences_than_a_block_has_threads(accumulate):
    """Short sequences, empty ones and bad lengths in wide tables, whose pages are cut evenly: where a sequence begins is
    summed over several rounds of a block's threads."""
    S = skv()
    shape = H, h, d = 8, 2, 64
    rng = np.random.default_rng(41)
    kv = context(*shape)
    lens = rng.integers(0, 60, 301)
    lens[rng.integers(0, 301, 60)] = 0
    pages, t, _ = fill(rng, lens, h, d)
    wide = np.full((301, 200), -1, np.int32)
    wide[:, :t.shape[1]] = t
    given = lens.copy()
    given[[0, 150, 300]] = -1, 200 * 16 + 1, 1 << 30
    qd, q = bf16(rng, 301, H, d)
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda(), weights=torch.zeros((len(pages), h, 16), device="cuda"))
    out = kv.kv4_decode(cache, qd, i32(wide), i32(given), accumulate=accumulate).double().cpu().numpy()
    assert kv.status() == S.DEV_BAD_SEQ_LEN
    w = cache.weights.double().cpu().numpy()
    for b, n in enumerate(lens):
        if given[b] != n or n == 0:
            assert (out[b] == 0).all()
            continue
        slots = F.slots_of(t[b], n)
        k, v = F.values(pages, slots, d)
        o, _, p, mag = F.attend(q[b:b + 1].astype(np.float64), k, v, [n])
        assert (np.abs(out[b] - o[0]) <= 2.0**-8 * np.abs(o[0]) + 2.0**-10 * (mag[0] + np.abs(v).max())).all(), b
        if accumulate:
            add = p[0].reshape(h, H // h, n).sum(1).T
            es = score_error(q[b:b + 1], k)[0].max()
            assert (np.abs(w[slots // 16, :, slots % 16] - add) <= add * (2 * es + 2.0**-18) + 2.0**-30).all(), b
    if not accumulate:
        assert (w == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_decode_of_sequences_that_share_pages(d):
    """A common beginning in the tables of all sequences, and a page that stands twice in one: each use adds its share."""
    S = skv()
    H, h = 8, 2
    rng = np.random.default_rng(43)
    kv = context(H, h, d)
    pages, t, _ = fill(rng, [64, 80], h, d)
    table = np.stack([t[0], t[0], np.concatenate([t[0, :4], t[1, 4:5]]), t[1, [0, 1, 0, 1, 2]]])  # [4, 5]
    table[:, 4] = t[1, 4]
    lens = [64, 50, 80, 70]
    qd, q = bf16(rng, 4, H, d)
    w0 = rng.random((len(pages), h, 16)).astype(np.float32)
    cache = S.KV4Cache(kv.cfg, pages=torch.from_numpy(pages).cuda(), weights=torch.from_numpy(w0).cuda())
    out = kv.kv4_decode(cache, qd, i32(table), i32(lens), accumulate=True).double().cpu().numpy()
    assert kv.status() == 0
    want, tol = w0.astype(np.float64), np.zeros(w0.shape)
    for b, n in enumerate(lens):
        slots = F.slots_of(table[b], n)
        k, v = F.values(pages, slots, d)
        o, _, p, mag = F.attend(q[b:b + 1].astype(np.float64), k, v, [n])
        assert (np.abs(out[b] - o[0]) <= 2.0**-8 * np.abs(o[0]) + 2.0**-10 * (mag[0] + np.abs(v).max())).all(), b
        add = p[0].reshape(h, H // h, n).sum(1).T
        es = score_error(q[b:b + 1], k)[0].max()
        np.add.at(want, (slots // 16, slice(None), slots % 16), add)
        np.add.at(tol, (slots // 16, slice(None), slots % 16), add * (2 * es + 2.0**-18) + 2.0**-24)
    assert (np.abs(cache.weights.double().cpu().numpy() - want) <= tol + 2.0**-22 * want).all()


def all_values(pages, d):
    """(k, v) fp64 [tokens, d] on the GPU of every slot of pages [P, 1, page bytes], in order."""
    P, ng = pages.shape[0], d // 32
    w = pages[:, 0].contiguous().view(torch.int32)
    shift = 4 * torch.arange(8, device=pages.device, dtype=torch.int32)
    out = []
    for x, order, at in ((w[:, :2 * d].reshape(P, 16, 4, ng), (0, 1, 3, 2, 4), 4 * d), (w[:, 2 * d:4 * d].reshape(P, 16, ng, 4), (0, 1, 2, 3, 4), 4 * d + 16 * ng)):
        code = ((x[..., None] >> shift) & 15).permute(order).reshape(P, 16, ng, 32).double()
        meta = w[:, at:at + 16 * ng].contiguous().view(torch.float16).view(P, 16, ng, 2).double()
        out.append((code * meta[..., :1] + meta[..., 1:]).reshape(P * 16, d))
    return out


def test_a_sequence_of_a_million_tokens():
    """Written, decoded with its weights, evicted: 8 heads over one, one sequence of 2^20 + 12345 tokens in pages in order."""
    S = skv()
    H, h, d = 8, 1, 64
    kv = context(H, h, d)
    n, keep, recent = (1 << 20) + 12345, 300001, 1000
    used, room = -(-n // 16), -(-keep // 16)
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = kv.new_kv4_cache(used + room, keep_weights=True)
    k, v = (torch.randn((n, h, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    w0 = torch.rand((n, h), generator=g, device="cuda")
    kv.kv4_append(cache, k, v, torch.arange(n, device="cuda"), w0)
    q = (2 * torch.randn((1, H, d), generator=g, device="cuda")).bfloat16()
    table, lens = torch.arange(used, device="cuda", dtype=torch.int32)[None], i32([n])
    out = kv.kv4_decode(cache, q, table, lens, accumulate=True)
    assert kv.status() == 0
    kk, vv = (x[:n] for x in all_values(cache.pages[:used], d))
    z = q[0].double() @ kk.t() / 8
    es = (q[0].double().abs() @ kk.abs().t()).amax(-1) * 2.0**-20 / 8
    p = torch.softmax(z, -1)
    o, mag = p @ vv, p @ vv.abs()
    # the output in bf16, v in fp16, p in fp16 (2^-11, and 2^-32 of the largest a token), the score's error, ex2 and sums
    lost = (p.amax(-1) * n * 2.0**-32)[:, None] * vv.abs().max()
    tol = 2.0**-8 * o.abs() + (mag + vv.abs().max()) * 2.0**-11 + mag * (2.0**-11 + 2 * es[:, None] + 2.0**-17) + lost
    assert ((out[0].double() - o).abs() <= tol).all()
    w = cache.weights[:used].reshape(-1)[:n]
    add = p.sum(0)
    assert ((w.double() - (w0[:, 0].double() + add)).abs() <= (p * (2 * es[:, None] + 2.0**-17)).sum(0) + 2.0**-23).all()
    dst = torch.arange(used, used + room, device="cuda", dtype=torch.int32)[None]
    new, kept = kv.kv4_evict(cache, table, lens, i32([keep]), recent, dst)
    assert kv.status() == 0 and new.tolist() == [keep]
    heavy = torch.sort(w[:n - recent], descending=True, stable=True).indices[:keep - recent].sort().values
    stay = torch.cat([heavy, torch.arange(n - recent, n, device="cuda")])
    assert torch.equal(kept[0, 0, :keep].long(), stay) and (kept[0, 0, keep:] == -1).all()
    moved = all_values(cache.pages[used:], d)
    assert torch.equal(moved[0][:keep], kk[stay]) and torch.equal(moved[1][:keep], vv[stay])
    assert torch.equal(cache.weights[used:].reshape(-1)[:keep], w[stay])


def test_every_call_on_another_stream():
    """Append, read, decode into a given output and eviction on a stream of their own: as on the current one."""
    S = skv()
    H, h, d = 8, 2, 128
    rng = np.random.default_rng(51)
    kv = context(H, h, d)
    n = [700, 90]
    t, spare, n_pages = tables(rng, n, extra=30)
    kd, _ = keys(rng, sum(n), h, d)
    vd, _ = bf16(rng, sum(n), h, d)
    qd, _ = bf16(rng, 2, H, d)
    slots = torch.from_numpy(np.concatenate([F.slots_of(t[b], m) for b, m in enumerate(n)])).cuda()
    first = torch.rand((sum(n), h), device="cuda")
    dst = np.zeros((2, 25), np.int32)
    dst[0], dst[1, :5] = spare[:25], spare[25:]
    td, ld, keeps, dd, cu = i32(t), i32(n), i32([400, 80]), i32(dst), i32(cu_of(n))

    def life(stream):
        cache = kv.new_kv4_cache(n_pages, keep_weights=True)
        out = torch.full_like(qd, 7)
        torch.cuda.synchronize()
        kv.kv4_append(cache, kd, vd, slots, first, stream=stream)
        k, v = kv.kv4_read(cache, td, cu, sum(n), stream=stream)
        assert kv.kv4_decode(cache, qd, td, ld, accumulate=True, out=out, stream=stream) is out
        lens, kept = kv.kv4_evict(cache, td, ld, keeps, 9, dd, stream=stream)
        torch.cuda.synchronize()
        return k, v, out, lens, kept, cache.pages, cache.weights

    want = life(None)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        for x, y in zip(life(stream), want):
            assert torch.equal(x, y)
    assert kv.status() == 0
