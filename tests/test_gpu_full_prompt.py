"""GPU tests of full-width prompts: packed causal attention, its weights, and the run from a prompt to evicted decode."""
import numpy as np
import pytest
import torch

from oracle import full_oracle as F

from _full import SHAPES, bf16, context, cu_of, i32, keys, score_error, skv, tables

pytestmark = pytest.mark.gpu


def inputs(rng, shape, n_q, n_k, q_scale=1.0):
    H, h, d = shape
    qd, _ = bf16(rng, sum(n_q), H, d, scale=q_scale)
    kd, _ = keys(rng, sum(n_k), h, d)
    vd, _ = bf16(rng, sum(n_k), h, d)
    return qd, kd, vd


def check_prompt(kv, shape, q, k, v, n_q, n_k, out, lse, weights=None, window=0):
    """out, lse (and the weights of the last `window` queries) of device inputs against the oracle."""
    H, h, d = shape
    q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    cq, ck = cu_of(n_q), cu_of(n_k)
    for b, (n, m) in enumerate(zip(n_q, n_k)):
        Q, K, V = q[cq[b]:cq[b + 1]], k[ck[b]:ck[b + 1]], v[ck[b]:ck[b + 1]]
        seen = [m - n + i + 1 for i in range(n)]
        o, ls, p, mag = F.attend(Q, K, V, seen)
        es = score_error(Q, K)
        got, gl = out[cq[b]:cq[b + 1]], lse[cq[b]:cq[b + 1]]
        # p in bf16 (2^-8 at most), the result in bf16, the score's error in numerator and sum, ex2 and fp32 sums
        tol = 2.0**-8 * (np.abs(o) + mag) + mag * (2 * es[..., None] + 2.0**-18)
        assert (np.abs(got - o) <= tol).all(), (b, n, m, np.abs(got - o).max())
        none = np.isinf(ls)
        assert (np.isneginf(gl) == none).all()
        tl = es + 2.0**-18 + 2.0**-22 * np.abs(np.where(none, 0, ls))
        assert (np.abs(np.where(none, 0, gl) - np.where(none, 0, ls)) <= tl).all()
        if weights is not None:
            w = weights[ck[b]:ck[b + 1]].double().cpu().numpy()
            x = p[max(0, n - window):] if window else p[:0]
            e = es[max(0, n - window):] if window else es[:0]
            want = x.reshape(len(x), h, H // h, m).sum((0, 2)).T
            # each p by the score's error twice (its own, and lse's), lse's rounding, ex2, and a sum of fewer than 2^12 terms
            tw = (x * (2 * e[..., None] + 2.0**-17)).reshape(len(x), h, H // h, m).sum((0, 2)).T + 2.0**-24
            assert (np.abs(w - want) <= tw + 2.0**-14 * want).all(), (b, np.abs(w - want).max())


def run(shape, n_q, n_k, window=0, seed=0, q_scale=1.0):
    rng = np.random.default_rng(seed)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, n_q, n_k, q_scale)
    cq, ck = i32(cu_of(n_q)), i32(cu_of(n_k))
    out, lse = kv.prompt(q, k, v, cq, ck, max(n_q))
    w = kv.prompt_weights(q, k, lse, cq, ck, max(n_k), window)
    assert kv.status() == 0
    check_prompt(kv, shape, q, k, v, n_q, n_k, out, lse, w, window)


@pytest.mark.parametrize("shape", SHAPES + [(40, 1, 64), (150, 1, 64)])
def test_prompt_small(shape):
    run(shape, [1, 2, 0, 40], [1, 2, 0, 40], window=7)


@pytest.mark.parametrize("shape", [(4, 4, 64), (14, 2, 64), (8, 8, 128), (12, 4, 128)])
@pytest.mark.parametrize("n_q,n_k", [([130], [130]), ([257, 64], [257, 64]), ([300], [700]), ([5, 1], [513, 300])])
def test_prompt_tiles(shape, n_q, n_k):
    run(shape, n_q, n_k, window=50, seed=n_q[0])


@pytest.mark.parametrize("shape", [(8, 2, 64), (8, 8, 128)])
def test_prompt_of_more_queries_than_keys(shape):
    run(shape, [150, 3, 20], [40, 0, 300], window=10**6, seed=3)


def test_prompt_without_any_key():
    kv = context(8, 2, 64)
    rng = np.random.default_rng(1)
    q, k, v = inputs(rng, (8, 2, 64), [5], [0])
    out, lse = kv.prompt(q, k, v, i32([0, 5]), i32([0, 0]), 5)
    assert kv.status() == 0 and (out == 0).all() and torch.isneginf(lse).all()


def test_weights_without_any_query():
    kv = context(8, 2, 64)
    rng = np.random.default_rng(1)
    q, k, _ = inputs(rng, (8, 2, 64), [0], [200])
    w = kv.prompt_weights(q, k, torch.empty((0, 8), device="cuda"), i32([0, 0]), i32([0, 200]), 200, 10)
    assert kv.status() == 0 and (w == 0).all()


@pytest.mark.parametrize("window", [0, 1, 64, 129, 1000])
def test_weights_of_a_window(window):
    run((14, 2, 64), [200, 0, 33], [260, 0, 33], window=window, seed=window)


@pytest.mark.parametrize("shape", [(4, 4, 64), (12, 4, 128), (20, 1, 128)])
@pytest.mark.parametrize("n_q,n_k", [([1], [3000]), ([7, 0, 1], [1500, 700, 40]), ([1100], [1100]), ([300, 20, 5], [200, 900, 600])])
def test_prompt_whose_units_are_shared(shape, n_q, n_k):
    """More than 1024 keys in all: key tiles of one unit on several SMs, their parts joined."""
    run(shape, n_q, n_k, window=3, seed=n_k[0])


def test_values_that_are_not_finite_in_a_shared_unit():
    shape = H, h, d = 4, 2, 64
    rng = np.random.default_rng(14)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, [40], [1500])
    cq, ck = i32([0, 40]), i32([0, 1500])
    clean, lse0 = kv.prompt(q, k, v, cq, ck, 40)
    v2 = v.clone()
    v2[1480, 1, 9] = float("inf")  # seen from query 20 on
    out, lse = kv.prompt(q, k, v2, cq, ck, 40)
    assert (out[20:, 2:, 9] == float("inf")).all() and torch.equal(lse, lse0)
    out[20:, 2:, 9], clean[20:, 2:, 9] = 0, 0
    assert torch.equal(out, clean) and kv.status() == 0


def test_prompt_with_scores_far_apart():
    run((8, 2, 128), [200], [200], window=200, q_scale=30.0)   # the running maximum moves often
    run((8, 2, 128), [200], [200], window=200, q_scale=1e-4)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_with_scores_of_large_magnitude(d):
    """Scores of either sign and up to 2^30: a query that sees one key has its value, however low the score."""
    shape = H, h, _ = 8, 2, d
    rng = np.random.default_rng(d)
    kv = context(*shape)
    n = [1] * 20 + [30]
    q, k, v = inputs(rng, shape, n, n, q_scale=2.0**23)
    scores = (q.double() * k.double().repeat_interleave(H // h, 1)).sum(-1) / d**0.5
    one = scores[:20]
    assert one.min() < -2.0**23 and one.max() > 2.0**23
    bound = q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max() / d**0.5  # of all scores, and of their terms' sums
    assert bound < 2.0**30
    cu = i32(cu_of(n))
    out, lse = kv.prompt(q, k, v, cu, cu, 30)
    assert kv.status() == 0
    want = v.double().repeat_interleave(H // h, 1)[:20]
    # p in bf16 and the output in bf16, half a step each
    assert ((out.double()[:20] - want).abs() <= 2.0**-7 * want.abs()).all()
    assert ((lse.double()[:20] - one).abs() <= 2.0**-20 * (one.abs() + bound)).all()
    assert torch.isfinite(out).all() and (out[20:].abs() <= 1.01 * v[20:].abs().max()).all()


def test_prompt_rising_scores_move_the_maximum():
    """Keys that grow along the sequence: each tile's scores pass those before by far more than 2^8."""
    shape = (4, 4, 64)
    rng = np.random.default_rng(5)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, [600], [600])
    q = q.abs()
    k = (k.abs() * torch.linspace(0.1, 6, 600, device="cuda")[:, None, None]).bfloat16()
    cu = i32([0, 600])
    out, lse = kv.prompt(q, k, v, cu, cu, 600)
    w = kv.prompt_weights(q, k, lse, cu, cu, 600, 600)
    assert kv.status() == 0
    check_prompt(kv, shape, q, k, v, [600], [600], out, lse, w, 600)


@pytest.mark.parametrize("shape", [(8, 2, 64), (4, 4, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(shape, bad):
    H, h, d = shape
    rng = np.random.default_rng(6)
    kv = context(*shape)
    n = [300, 90, 40]
    q, k, v = inputs(rng, shape, n, n)
    cu = i32(cu_of(n))
    clean, _ = kv.prompt(q, k, v, cu, cu, 300)
    at, ch = 250, 17
    k2, v2 = k.clone(), v.clone()
    v2[at, 0, ch] = bad          # inside sequence 0
    v2[300:, :, :] = bad         # all of sequences 1 and 2, behind sequence 0's last tile
    k2[300:, :, :] = float("nan")
    out, lse = kv.prompt(q, k2, v2, cu, cu, 300)
    a, b = out[:300].clone(), clean[:300].clone()
    hit = a[at:, :H // h, ch].float()
    assert (torch.isnan(hit) if bad != bad else hit == bad).all()
    a[at:, :H // h, ch] = 0
    b[at:, :H // h, ch] = 0
    assert torch.equal(a, b)
    w = kv.prompt_weights(q, k2, lse, cu, cu, 300, 300)
    assert torch.isfinite(w[:300]).all()


def test_queries_that_are_not_finite_stay_in_their_rows():
    shape = (8, 2, 64)
    rng = np.random.default_rng(7)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, [200, 50], [200, 50])
    cu = i32([0, 200, 250])
    clean, lse0 = kv.prompt(q, k, v, cu, cu, 200)
    q2 = q.clone()
    q2[60, 3] = float("nan")
    q2[200:] = float("inf")
    out, lse = kv.prompt(q2, k, v, cu, cu, 200)
    assert torch.isnan(out[60, 3]).all() and torch.isnan(lse[60, 3])
    keep = torch.ones((200, 8), dtype=torch.bool)
    keep[60, 3] = False
    assert torch.equal(out[:200][keep], clean[:200][keep]) and torch.equal(lse[:200][keep], lse0[:200][keep])
    w0 = kv.prompt_weights(q, k, lse0, cu, cu, 200, 100)
    w = kv.prompt_weights(q2, k, lse, cu, cu, 200, 100)  # query 60 is outside the window
    assert torch.equal(w[:200], w0[:200])


def test_rows_of_one_projection():
    shape = H, h, d = 8, 2, 64
    rng = np.random.default_rng(8)
    kv = context(*shape)
    x, _ = bf16(rng, 150, H + 2 * h, d)
    q, k, v = x[:, :H], x[:, H:H + h], x[:, H + h:]
    cu = i32([0, 150])
    out, lse = kv.prompt(q, k, v, cu, cu, 150)
    w = kv.prompt_weights(q, k, lse, cu, cu, 150, 20)
    again, lse2 = kv.prompt(q.contiguous(), k.contiguous(), v.contiguous(), cu, cu, 150)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    check_prompt(kv, shape, q, k, v, [150], [150], out, lse, w, 20)


def test_bad_spans_leave_their_rows():
    S = skv()
    shape = (8, 2, 64)
    rng = np.random.default_rng(9)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, [60, 40], [60, 40])
    out, lse = torch.full_like(q, 7), torch.full((100, 8), 7.0, device="cuda")
    w = torch.full((100, 2), 7.0, device="cuda")
    cases = [([0, 60, 40], [0, 60, 100], 60, 100), ([0, 60, 100], [0, 120, 100], 60, 100), ([0, 60, 100], [0, 60, 100], 30, 30)]
    for cq, ck, mq, mk in cases:
        S.starkv_prompt_attn(kv.ctx, kv.cfg, q, k, v, i32(cq), i32(ck), mq, out, lse)
        assert kv.status() == S.DEV_BAD_QUERY_SPAN
        S.starkv_prompt_weights(kv.ctx, kv.cfg, q, k, torch.zeros_like(lse), i32(cq), i32(ck), mk, 10, w)
        assert kv.status() == S.DEV_BAD_QUERY_SPAN
    S.starkv_prompt_attn(kv.ctx, kv.cfg, q, k, v, i32([0, 60, 100]), i32([0, 60, 90]), 60, out, lse)
    assert kv.status() == S.DEV_BAD_QUERY_SPAN
    assert (out[60:] == 7).all() and (lse[60:] == 7).all()


def test_prompt_captured_and_on_another_stream():
    shape = (8, 2, 128)
    rng = np.random.default_rng(10)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, [300, 77], [300, 77])
    cu = i32([0, 300, 377])
    out, lse = kv.prompt(q, k, v, cu, cu, 300)
    w = kv.prompt_weights(q, k, lse, cu, cu, 300, 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, l2 = kv.prompt(q, k, v, cu, cu, 300, stream=side)
    o3, l3 = kv.prompt(q, k, v, cu, cu, 300)  # two calls at once
    w2 = kv.prompt_weights(q, k, l2, cu, cu, 300, 64, stream=side)
    torch.cuda.synchronize()
    for a, b in ((o2, out), (o3, out), (l2, lse), (l3, lse), (w2, w)):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o4, l4 = kv.prompt(q, k, v, cu, cu, 300)
        w4 = kv.prompt_weights(q, k, l4, cu, cu, 300, 64)
    keep = [x.clone() for x in (q, k, v)]
    for x in (q, k, v):
        x.copy_(torch.randn_like(x))
    g.replay()
    want = kv.prompt(q, k, v, cu, cu, 300)
    assert torch.equal(o4, want[0]) and torch.equal(l4, want[1])
    for x, y in zip((q, k, v), keep):
        x.copy_(y)
    g.replay()
    assert torch.equal(o4, out) and torch.equal(l4, lse) and torch.equal(w4, w)
    assert kv.status() == 0


@pytest.mark.parametrize("handle", [False, True])
def test_results_on_another_stream_take_no_memory_that_pending_work_still_writes(handle):
    """Tensors given back on the current stream, whose last writes are still to come, while the call's stream is free."""
    shape = H, h, d = 8, 2, 64
    rng = np.random.default_rng(21)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, [300], [1500])
    cq, ck = i32([0, 300]), i32([0, 1500])
    want, want_lse = kv.prompt(q, k, v, cq, ck, 300)
    sizes = [want.shape, want_lse.shape]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        old = [torch.empty(s, dtype=t, device="cuda") for s in sizes for t in (torch.bfloat16, torch.float32)]
        for x in old:
            x.fill_(7.0)
        del old, x
        out, lse = kv.prompt(q, k, v, cq, ck, 300, stream=side.cuda_stream if handle else side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out, lse = kv.prompt(q, k, v, cq, ck, 300, stream=0)  # the default stream by its handle
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and kv.status() == 0


@pytest.mark.parametrize("shape", [(8, 2, 64), (8, 4, 128)])
def test_from_a_prompt_in_two_chunks_to_decode_behind_an_eviction(shape):
    """A full-width layer's life: a first chunk attends and is cached, a second chunk attends to the cache read back and
    itself, its last queries' weights join the cache, the cache is evicted, and decode steps go on in what is kept."""
    H, h, d = shape
    rng = np.random.default_rng(13)
    kv = context(*shape)
    n1, n2, keep, recent, window = [70, 33], [40, 90], [50, 60], 8, 16
    total = [a + b for a, b in zip(n1, n2)]
    steps = 3
    room = [-(-(k + steps) // 16) for k in keep]
    t, spare, n_pages = tables(rng, total, extra=sum(room))
    dst = np.zeros((2, max(room)), np.int32)
    dst[0, :room[0]], dst[1, :room[1]] = spare[:room[0]], spare[room[0]:]
    cache = kv.new_kv4_cache(n_pages, keep_weights=True)
    td = i32(t)

    def slots(table, starts, lens):
        return torch.from_numpy(np.concatenate([F.slots_of(table[b], n, s) for b, (s, n) in enumerate(zip(starts, lens))])).cuda()

    # first chunk
    q1, k1, v1 = inputs(rng, shape, n1, n1)
    c1 = i32(cu_of(n1))
    o1, l1 = kv.prompt(q1, k1, v1, c1, c1, max(n1))
    check_prompt(kv, shape, q1, k1, v1, n1, n1, o1, l1)
    kv.kv4_append(cache, k1, v1, slots(t, [0, 0], n1))
    # second chunk: keys and values of the first come back from the cache
    q2, k2, v2 = inputs(rng, shape, n2, n2)
    kv.kv4_append(cache, k2, v2, slots(t, n1, n2))
    ct = i32(cu_of(total))
    ka, va = kv.kv4_read(cache, td, ct, sum(total))
    o2, l2 = kv.prompt(q2, ka, va, i32(cu_of(n2)), ct, max(n2))
    w = kv.prompt_weights(q2, ka, l2, i32(cu_of(n2)), ct, max(total), window)
    check_prompt(kv, shape, q2, ka, va, n2, total, o2, l2, w, window)
    # the weights enter with the tokens, and eviction goes by them
    kv.kv4_append(cache, ka, va, slots(t, [0, 0], total), w)
    wc = cache.weights.cpu().numpy()
    pages = cache.pages.cpu().numpy()
    lens, kept = kv.kv4_evict(cache, td, i32(total), i32(keep), recent, i32(dst))
    for b in range(2):
        src = F.slots_of(t[b], total[b])
        for head in range(h):
            want = F.kept_tokens(wc[src // 16, head, src % 16], total[b], keep[b], recent)
            np.testing.assert_array_equal(kept[b, head, :keep[b]].cpu().numpy(), want)
    # decode steps behind it
    kk, vv = [], []
    for b in range(2):
        k, v = F.values(pages, F.slots_of(t[b], total[b]), d)
        stay = kept[b, :, :keep[b]].cpu().numpy()
        kk.append(np.stack([k[stay[i], i] for i in range(h)], 1))
        vv.append(np.stack([v[stay[i], i] for i in range(h)], 1))
    lens = lens.cpu().numpy()
    for step in range(steps):
        q, k, v = inputs(rng, shape, [1, 1], [1, 1])
        at = slots(dst, lens, [1, 1])
        kv.kv4_append(cache, k, v, at)
        lens = lens + 1
        out = kv.kv4_decode(cache, q, i32(dst), i32(lens), accumulate=True).double().cpu().numpy()
        now = cache.pages.cpu().numpy()
        for b in range(2):
            k, v = F.values(now, at[b:b + 1].cpu().numpy(), d)
            kk[b], vv[b] = np.concatenate([kk[b], k]), np.concatenate([vv[b], v])
            o, _, _, mag = F.attend(q[b:b + 1].double().cpu().numpy(), kk[b], vv[b], [len(kk[b])])
            assert (np.abs(out[b] - o[0]) <= 2.0**-8 * np.abs(o[0]) + 2.0**-10 * (mag[0] + np.abs(vv[b]).max())).all()
    got = cache.weights.cpu().numpy()
    for b in range(2):
        s = F.slots_of(dst[b], lens[b])
        src = F.slots_of(t[b], total[b])
        stay = kept[b, :, :keep[b]].cpu().numpy()
        before = sum(wc[src[stay[i]] // 16, i, src[stay[i]] % 16].sum() for i in range(h))
        assert abs(got[s // 16, :, s % 16].sum() - before - steps * H) < 1e-3 * steps * H
    assert kv.status() == 0


@pytest.mark.parametrize("shape,n_q,n_k,window", [
    ((8, 2, 64), [3, 70, 0, 200], [900, 70, 300, 1500], 20),      # a window whose queries stay: sequences with fewer of them
    ((8, 2, 128), [64, 1, 130], [1300, 700, 130], 64),
    ((16, 4, 64), [3000], [3000], 3000),                          # many steps an item, few items
    ((4, 4, 64), [700] * 12, [700] * 12, 700),                    # more items than SMs
    ((16, 1, 128), [300, 500], [300, 500], 100),
    ((150, 1, 64), [60], [200], 10),                              # two blocks of heads
    ((8, 2, 64), [900, 40], [100, 40], 900),                      # most queries see nothing
])
def test_weights_of_every_way_to_share_the_work(shape, n_q, n_k, window):
    """The kernel's weights against the formula in 64 bits, from the kernel's own lse."""
    H, h, d = shape
    rng = np.random.default_rng(window)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, n_q, n_k)
    cq, ck = i32(cu_of(n_q)), i32(cu_of(n_k))
    lse = kv.prompt(q, k, v, cq, ck, max(n_q))[1]
    w = torch.full((sum(n_k), h), 7.0, device="cuda")
    for _ in range(2):
        skv().starkv_prompt_weights(kv.ctx, kv.cfg, q, k, lse, cq, ck, max(n_k), window, w)
        assert kv.status() == 0
        for b, (n, m) in enumerate(zip(n_q, n_k)):
            q0, k0 = sum(n_q[:b]), sum(n_k[:b])
            first = max(0, n - window)
            for head in range(h):
                Q = q[q0 + first:q0 + n, head * (H // h):(head + 1) * (H // h)].double()
                K = k[k0:k0 + m, head].double()
                z = torch.einsum("igd,jd->igj", Q, K) / d**0.5
                e = torch.einsum("igd,jd->igj", Q.abs(), K.abs()).amax() * 2.0**-20 / d**0.5 if z.numel() else 0
                seen = torch.arange(m, device="cuda")[None] <= (m - n + first + torch.arange(n - first, device="cuda"))[:, None]
                p = torch.exp(z - lse[q0 + first:q0 + n, head * (H // h):(head + 1) * (H // h), None].double())
                want = torch.where(seen[:, None], p, 0.0).sum((0, 1))
                # the score's error, ex2's and the difference's (lse < 2^5: 2^-18), and fp32 sums of fewer than 2^10 chunks
                tol = want * (e + 2.0**-17 + 2.0**-14) + 2.0**-24
                got = w[k0:k0 + m, head].double()
                assert ((got - want).abs() <= tol).all(), (b, head, (got - want).abs().max())


@pytest.mark.parametrize("shape,n_q,n_k", [
    ((16, 4, 64), [2500], [2500]),
    ((16, 4, 128), [1500, 300], [1500, 300]),
    ((16, 4, 64), [600, 1500], [1500, 1500]),
    ((20, 1, 128), [1, 1490, 0, 33], [700, 1500, 5, 33]),
])
def test_weights_of_items_shared_by_pairs_in_two_rounds(shape, n_q, n_k):
    test_weights_of_every_way_to_share_the_work(shape, n_q, n_k, 4000)


def test_prompt_whose_keys_leave_the_cache():
    """Keys and values of more than 96 MB with units for every SM: whole units a CTA, the longest first."""
    shape = H, h, d = 32, 32, 128
    n, m = 1291, 6400
    kv = context(*shape)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((n, H, d), generator=g, device="cuda").bfloat16()
    k, v = (torch.randn((m, h, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    out, lse = kv.prompt(q, k, v, i32([0, n]), i32([0, m]), n)
    assert kv.status() == 0
    seen = torch.arange(m, device="cuda")[None] <= (m - n + torch.arange(n, device="cuda"))[:, None]
    for head in (0, 13, 31):
        z = (q[:, head].double() @ k[:, head].double().t()) / d**0.5
        e = (q[:, head].double().abs() @ k[:, head].double().abs().t()).amax() * 2.0**-20 / d**0.5
        z = torch.where(seen, z, -torch.inf)
        p = torch.softmax(z, -1)
        o, mag = p @ v[:, head].double(), p @ v[:, head].double().abs()
        assert ((out[:, head].double() - o).abs() <= 2.0**-8 * (o.abs() + mag) + mag * (2 * e + 2.0**-18)).all()
        assert ((lse[:, head].double() - torch.logsumexp(z, -1)).abs() <= e + 2.0**-18 + 2.0**-20).all()


@pytest.mark.parametrize("shape,window", [
    ((14, 2, 64), 50),   # 18 queries a step: three steps an item
    ((14, 2, 64), 75),   # five
    ((5, 1, 64), 60),    # 25 queries a step: three
    ((32, 8, 128), 96),  # 32 queries a step: three
    ((32, 8, 128), 64),  # two
    ((32, 8, 128), 20),  # one
])
def test_weights_of_items_with_an_odd_number_of_steps(shape, window):
    """Several items, of several (sequence, KV head)s, on each SM: a step's columns stay while the items go by."""
    H, h, d = shape
    lens = [100, 77, 130, 96, 101, 60, 20, 99, 100, 140, 100, 75]
    keys_of = [8000, 7000, 8100, 130, 9000, 2000, 8500, 900, 7333, 2500, 4096, 75]
    assert sum(-(-m // 128) for m in keys_of) * h > 2 * 148
    test_weights_of_every_way_to_share_the_work(shape, lens, keys_of, window)
    rng = np.random.default_rng(window)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, lens, keys_of)
    cq, ck = i32(cu_of(lens)), i32(cu_of(keys_of))
    lse = kv.prompt(q, k, v, cq, ck, max(lens))[1]
    first = kv.prompt_weights(q, k, lse, cq, ck, max(keys_of), window)
    for _ in range(50):
        assert torch.equal(kv.prompt_weights(q, k, lse, cq, ck, max(keys_of), window), first)
    assert kv.status() == 0


def test_weights_hold_the_bound_of_each_exponential():
    """One column of a tile at a time: its weight is 2^x alone, x from -130 to 126, half-integers, and what is not finite."""
    kv = context(4, 1, 64)
    rng = np.random.default_rng(22)
    B, n, m = 4096, 32, 160  # a sequence: one step of 32 queries x 4 heads, whose 128 columns all see the first 128 keys
    scale, log2e = np.float32(1.4426950408889634 / 8), np.float32(1.4426950408889634)
    s = ((np.arange(m) - 64) / 16).astype(np.float32)  # scores, bf16 numbers
    base = rng.uniform(-130, 125, B).astype(np.float32)
    base[:300] = np.arange(-130, 20)[np.arange(300) % 150] + np.float32(0.5)
    lse = (base.astype(np.float64) / -np.float64(log2e)).astype(np.float32)
    for step in range(-3, 4):  # lse whose product is the half-integer itself, where there is one
        near = np.where(step < 0, -1, 1).astype(np.float32) * np.inf
        y = lse[:300].copy()
        for _ in range(abs(step)):
            y = np.nextafter(y, near)
        hit = (y * -log2e).astype(np.float32) == base[:300]
        lse[:300][hit] = y[hit]
    base = (lse * -log2e).astype(np.float32)
    assert (base[:300] % 1 == 0.5).sum() > 150
    lse[-2:] = np.nan, np.inf
    col = np.concatenate([np.arange(300) // 150 + 2 + np.arange(300) % 8 * 16, np.arange(B - 300)]) % 128
    q = torch.zeros((B, n, 4, 64), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    k = torch.zeros((B, m, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[..., 0] = torch.from_numpy(s).cuda()[None, :, None]
    ls = torch.full((B, n * 4), float("inf"), device="cuda")
    ls[torch.arange(B), torch.from_numpy(col).cuda()] = torch.from_numpy(lse).cuda()
    cq, ck = i32(np.arange(B + 1) * n), i32(np.arange(B + 1) * m)
    w = kv.prompt_weights(q.view(B * n, 4, 64), k.view(B * m, 1, 64), ls.view(B * n, 4), cq, ck, m, n)
    assert kv.status() == 0
    w = w.view(B, m)[:, :128].cpu().numpy()
    assert np.isnan(w[-2]).all() and (w[-1] == 0).all()
    x = (s[:128].astype(np.longdouble) * np.longdouble(scale) + base[:-2, None].astype(np.longdouble)).astype(np.float32)
    assert x.min() < -130 and x.max() > 125 and (x[:300] % 1 == 0.5).sum() > 150
    want = np.exp2(x.astype(np.longdouble))
    err = np.abs(w[:-2].astype(np.longdouble) - want)
    # 2^-22 relative, of the special function unit's and of the polynomial; below 2^-126 either may be 0
    bad = err > want * np.longdouble(2.0**-22) + np.where(x < -126, 2.0**-126, 0.0)
    assert not bad.any(), (x[bad][:5], np.argwhere(bad)[:5], (err / want)[bad][:5])


@pytest.mark.parametrize("shape,n_q,n_k,window", [
    ((8, 2, 128), [64, 100], [1300, 700], 64),   # a window whose queries stay
    ((14, 2, 64), [300, 90], [300, 400], 300),   # 126 columns of a tile hold heads
    ((4, 4, 64), [700] * 40, [700] * 40, 700),   # items dealt to the SMs
    ((16, 4, 64), [2500], [2500], 4000),         # pairs of CTAs
])
def test_weights_of_exact_scores(shape, n_q, n_k, window):
    """Scores that fp32 holds exactly: what is left is the rounding of the exponent, of the exponential and of the sums."""
    H, h, d = shape
    G = H // h
    kv = context(*shape)
    g = torch.Generator(device="cuda").manual_seed(window)
    q = torch.randint(-2, 3, (sum(n_q), H, d), generator=g, device="cuda").bfloat16()
    k = torch.randint(-2, 3, (sum(n_k), h, d), generator=g, device="cuda").bfloat16()
    cq, ck = cu_of(n_q), cu_of(n_k)
    scale, log2e = float(np.float32(1.4426950408889634 / d**0.5)), 1.4426950408889634
    lse = torch.empty((sum(n_q), H), device="cuda")
    want = torch.zeros((sum(n_k), h), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    for b, (n, m) in enumerate(zip(n_q, n_k)):
        seen = torch.arange(m, device="cuda")[None] <= (m - n + torch.arange(n, device="cuda"))[:, None]
        first = max(0, n - window)
        for i in range(H):
            z = q[cq[b]:cq[b + 1], i].double() @ k[ck[b]:ck[b + 1], i // G].double().t()
            l = torch.logsumexp(torch.where(seen, z, -torch.inf) / d**0.5, -1).float()
            lse[cq[b]:cq[b + 1], i] = l
            x = z * (log2e / d**0.5) - l[:, None].double() * log2e
            p = torch.where(seen, torch.exp2(x), 0.0)[first:]
            # the scale's half step, those of log2(e) and of its product with lse, and of the sum: all times ln 2; and 2^-22
            e = ((z * scale).abs() + 2 * (l[:, None].double() * log2e).abs() + x.abs())[first:] * 2.0**-24 * 0.6932 + 2.0**-22
            want[ck[b]:ck[b + 1], i // G] += p.sum(0)
            tol[ck[b]:ck[b + 1], i // G] += (p * e).sum(0)
    w = kv.prompt_weights(q, k, lse, i32(cq), i32(ck), max(n_k), window).double()
    assert kv.status() == 0
    # fp32 sums: 64 columns in four sums of 16, then those, the steps of an item, four groups of warps, eight CTAs
    steps = max(n_q) // (128 // G) + 1
    assert ((w - want).abs() <= tol + want * ((32 + 3 + steps + 4 + 8) * 2.0**-24) + 2.0**-126).all(), ((w - want).abs() / want).max()


def test_prompt_and_weights_with_loose_bounds():
    """max_q_len and max_k_len far above any length, up to 2^31 - 1."""
    shape = (8, 2, 64)
    rng = np.random.default_rng(31)
    kv = context(*shape)
    for n_q, n_k in (([70, 9, 130], [200, 9, 130]), ([300], [2000]), ([300], [300])):
        q, k, v = inputs(rng, shape, n_q, n_k)
        cq, ck = i32(cu_of(n_q)), i32(cu_of(n_k))
        out, lse = kv.prompt(q, k, v, cq, ck, max(n_q))
        check_prompt(kv, shape, q, k, v, n_q, n_k, out, lse)
        for most in (max(n_q) + 1, 1 << 17, (1 << 31) - 1):
            o2, l2 = kv.prompt(q, k, v, cq, ck, most)
            assert torch.equal(out, o2) and torch.equal(lse, l2)
        for window in (20, 10**6):
            for most in (1 << 17, (1 << 31) - 1):
                w = kv.prompt_weights(q, k, lse, cq, ck, most, window)
                check_prompt(kv, shape, q, k, v, n_q, n_k, out, lse, w, window)
    assert kv.status() == 0


def test_numbers_of_more_than_32_bits_are_refused():
    """They would reach the library cut to their low 32 bits: a window of 2^32 as none."""
    shape = (8, 2, 64)
    kv = context(*shape)
    q, k, v = inputs(np.random.default_rng(1), shape, [20], [20])
    cu = i32([0, 20])
    lse = kv.prompt(q, k, v, cu, cu, 20)[1]
    cache = kv.new_kv4_cache(4, keep_weights=True)
    table, lens = i32([[0, 1]]), i32([20])
    for call in (lambda x: kv.prompt(q, k, v, cu, cu, x), lambda x: kv.prompt_weights(q, k, lse, cu, cu, x, 4),
                 lambda x: kv.prompt_weights(q, k, lse, cu, cu, 20, x), lambda x: kv.kv4_evict(cache, table, lens, lens, x, i32([[2, 3]]))):
        for x in (1 << 32, (1 << 32) + 20, 1 << 31):
            with pytest.raises(ValueError):
                call(x)
    assert kv.status() == 0


def test_workspace_sizes_of_shapes_that_the_calls_refuse_are_refused():
    S = skv()
    kv = context(8, 2, 64)
    most = (1 << 31) - 1
    for call in (lambda: S.starkv_workspace_bytes(kv.ctx, S.OP_KV4_DECODE, 1 << 16, 10, 1),
                 lambda: S.starkv_workspace_bytes(kv.ctx, S.OP_KV4_DECODE, most, most, 1),
                 lambda: S.starkv_workspace_bytes(kv.ctx, S.OP_KV4_DECODE, 1, (1 << 26) + 1, 0),
                 lambda: S.starkv_prompt_workspace_bytes(kv.ctx, 1 << 16, 100, 100),
                 lambda: S.starkv_prompt_workspace_bytes(kv.ctx, 1, 1 << 31, 100),
                 lambda: S.starkv_prompt_workspace_bytes(kv.ctx, 1, 100, 1 << 62)):
        with pytest.raises(S.StarKVError) as e:
            call()
        assert e.value.code == S.ERR_UNSUPPORTED_SHAPE
    with pytest.raises(S.StarKVError) as e:
        S.starkv_workspace_bytes(kv.ctx, 99, 1, 1, 0)
    assert e.value.code == S.ERR_INVALID_ARG
    # the largest that they take: 4 bytes a token and query head, and the parts
    assert 65535 * (1 << 26) * 16 * 8 * 4 <= S.starkv_workspace_bytes(kv.ctx, S.OP_KV4_DECODE, 65535, 1 << 26, 1) < 65535 * (1 << 26) * 16 * 8 * 5
    assert S.starkv_workspace_bytes(kv.ctx, S.OP_KV4_DECODE, 0, 0, 0) >= 0 and S.starkv_prompt_workspace_bytes(kv.ctx, 0, 0, 0) == 0
    assert S.starkv_prompt_workspace_bytes(kv.ctx, 65535, most, most) <= 40 << 20


@pytest.mark.parametrize("shape", [(1, 1, 64), (2, 1, 128), (3, 1, 64), (1024, 8, 64), (200, 200, 64)])
def test_prompt_of_the_fewest_and_the_most_heads(shape):
    run(shape, [5, 0, 140], [9, 3, 140], window=50, seed=shape[0])
    if shape[0] < 100:
        run(shape, [300], [1900], window=290, seed=shape[0])


@pytest.mark.parametrize("shape", [(8, 2, 64), (4, 4, 128)])
def test_prompts_of_more_sequences_than_a_warp_has_lanes(shape):
    """150 sequences, empty ones among them, whose work is cut evenly: where one begins is summed over rounds of 32."""
    rng = np.random.default_rng(44)
    n_q = rng.integers(0, 40, 150)
    n_k = n_q + rng.integers(0, 30, 150) * (rng.random(150) < 0.5)
    n_q[::7] = 0
    n_k[::14] = 0
    n_q[-1], n_k[-1] = 0, 0
    run(shape, n_q.tolist(), n_k.tolist(), window=12, seed=44)     # a window's queries stay
    run(shape, n_q.tolist(), n_k.tolist(), window=10**6, seed=44)


def test_cut_prompts_captured_and_replayed_with_other_lengths():
    """One graph for packed prompts of other lengths in the same rows: work is cut on the device."""
    shape = (12, 4, 128)
    rng = np.random.default_rng(45)
    kv = context(*shape)
    q, k, v = inputs(rng, shape, [700], [2300])
    lens = [([700], [2300]), ([300, 400], [300, 2000]), ([0, 1, 699], [900, 1, 1399]), ([350, 0, 350], [1000, 50, 1250])]
    batch = 3
    cu = [[cu_of(list(x) + [0] * (batch - len(x))) for x in pair] for pair in lens]
    cq, ck = i32(cu[0][0]), i32(cu[0][1])
    plain = []
    for a, b in cu:
        out, lse = kv.prompt(q, k, v, i32(a), i32(b), 700)
        plain.append((out, lse, kv.prompt_weights(q, k, lse, i32(a), i32(b), 2300, 20)))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = kv.prompt(q, k, v, cq, ck, 700)
        w = kv.prompt_weights(q, k, lse, cq, ck, 2300, 20)
    for i in (1, 2, 3, 0, 2):
        cq.copy_(i32(cu[i][0]))
        ck.copy_(i32(cu[i][1]))
        g.replay()
        assert torch.equal(out, plain[i][0]) and torch.equal(lse, plain[i][1]) and torch.equal(w, plain[i][2])
        check_prompt(kv, shape, q, k, v, *lens[i], out, lse, w, 20)
    assert kv.status() == 0


def test_prompt_of_one_chunk_behind_a_million_keys():
    """37 queries of 8 heads over one behind 2^20 keys, on every SM, into a given output; and what they look at."""
    S = skv()
    H, h, d, n, m = 8, 1, 64, 37, (1 << 20) + 37
    kv = context(H, h, d)
    g = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = ((s * torch.randn(x, generator=g, device="cuda")).bfloat16() for s, x in ((2, (n, H, d)), (1, (m, h, d)), (1, (m, h, d))))
    cq, ck = i32([0, n]), i32([0, m])
    given = torch.full_like(q, 7)
    out, lse = kv.prompt(q, k, v, cq, ck, n, out=given)
    assert out is given
    w = kv.prompt_weights(q, k, lse, cq, ck, m, 16)
    assert kv.status() == 0
    bare = torch.empty_like(q)  # without the log-sum-exp
    ws = torch.empty(S.starkv_prompt_workspace_bytes(kv.ctx, 1, n, m), dtype=torch.uint8, device="cuda")
    S.starkv_prompt_attn(kv.ctx, kv.cfg, q, k, v, cq, ck, n, bare, None, ws)
    assert torch.equal(bare, out) and kv.status() == 0
    seen = torch.arange(m, device="cuda")[None] <= (m - n + torch.arange(n, device="cuda"))[:, None]
    kk, vv = k[:, 0].double(), v[:, 0].double()
    want = torch.zeros(m, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    for i in range(H):
        z = torch.where(seen, q[:, i].double() @ kk.t() / 8, -torch.inf)
        es = (q[:, i].double().abs() @ kk.abs().t()).amax() * 2.0**-20 / 8
        p = torch.softmax(z, -1)
        o, mag = p @ vv, p @ vv.abs()
        # p in bf16 and the output in bf16; the score's error twice, ex2 and fp32 sums of parts
        assert ((out[:, i].double() - o).abs() <= 2.0**-8 * (o.abs() + mag) + mag * (2 * es + 2.0**-16)).all()
        ls = torch.logsumexp(z, -1)
        assert ((lse[:, i].double() - ls).abs() <= es + 2.0**-16 + 2.0**-22 * ls.abs()).all()
        x = torch.exp(z - lse[:, i].double()[:, None])[n - 16:]
        want += x.sum(0)
        tol += x.sum(0) * (es + 2.0**-17)
    assert ((w[:, 0].double() - want).abs() <= tol + 2.0**-30).all()
