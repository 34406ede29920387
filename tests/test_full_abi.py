"""Full-width layers without a GPU: exports, the layout, refusals, and the oracle against closed forms."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import full_oracle as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def S():
    from rank_mixed_precision_b200 import starkv
    starkv.lib()
    return starkv


def test_every_declared_symbol_is_exported_and_bound(S):
    text = open(os.path.join(ROOT, "include", "starkv_full.h")).read()
    names = sorted(set(re.findall(r"^STARKV_API[^;(]*?\b(starkv_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(S.EXPORTS_FULL)
    for n in names:
        assert hasattr(ctypes.CDLL(S.LIB_PATH), n) and n in S._SIGS and hasattr(S, n)


def test_the_header_is_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "starkv_full.h"\nint main(void) { starkv_kv4_cache c = {0, 0, 0}; return (int)c.n_pages; }\n')
    assert os.system(f"gcc -std=c99 -Wall -Werror -I{ROOT}/include -fsyntax-only {src}") == 0


@pytest.mark.parametrize("shape", [(4, 4, 64), (32, 8, 128)])
def test_layout(S, shape):
    H, h, d = shape
    got = S.starkv_kv4_layout(S.make_config(H, h, d, 64, 16, 64, 16), 7)
    assert got["head_page_bytes"] == F.page_bytes(d) and got["groups"] == d // 32
    assert got["pages_bytes"] == 7 * h * F.page_bytes(d) and got["weights_bytes"] == 7 * h * 64


def test_layout_refuses(S):
    with pytest.raises(S.StarKVError) as e:
        S.starkv_kv4_layout(S.make_config(4, 4, 96, 64, 16, 64, 16), 1)
    assert e.value.code == S.ERR_UNSUPPORTED_SHAPE
    with pytest.raises(S.StarKVError) as e:
        S.starkv_kv4_layout(S.make_config(4, 4, 64, 64, 16, 64, 16), -1)
    assert e.value.code == S.ERR_INVALID_ARG


def test_a_null_context_is_refused_before_any_device_work(S):
    L = S.lib()
    calls = [lambda: L.starkv_kv4_append(None, None, None, None, 0, 0, None, None, 1, None),
             lambda: L.starkv_kv4_read(None, None, None, None, None, 1, 1, 1, None, None, None),
             lambda: L.starkv_kv4_decode_attn(None, None, None, None, None, 1, 1, 0, None, None, 0, None),
             lambda: L.starkv_kv4_evict(None, None, None, None, None, 0, 1, 1, None, 1, None, None, None),
             lambda: L.starkv_prompt_attn(None, None, None, None, 0, 0, 0, None, None, 1, 1, 1, 1, None, None, None, 0, None),
             lambda: L.starkv_prompt_workspace_bytes(None, 1, 1, 1, None),
             lambda: L.starkv_prompt_weights(None, None, None, 0, 0, None, None, None, 1, 1, 1, 1, 1, None, None),
             lambda: L.starkv_kv4_layout(None, 1, None)]
    for call in calls:
        assert call() == S.ERR_INVALID_ARG and S.starkv_last_error()


def test_the_binding_refuses_wrong_tensors(S):
    cfg = S.make_config(8, 2, 64, 64, 16, 64, 16)
    q = torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a GPU
        S.starkv_prompt_attn(None, cfg, q, q[:, :2], q[:, :2], None, None, 3, q)
    with pytest.raises(TypeError):
        S.starkv_kv4_append(None, cfg, None, q.float(), q, None)
    with pytest.raises(TypeError):
        S.KV4Cache(cfg, pages=torch.zeros((1, 2, 64), dtype=torch.int8))
    with pytest.raises(ValueError):
        S.KV4Cache(cfg)


# ---- the oracle itself
def test_oracle_quantiser_reaches_both_ends():
    x = np.linspace(-2, 1, 32, dtype=np.float32)
    c, s, z, bad = F.quantize(x)
    assert c[0] == 0 and c[-1] == 15 and not bad and z == np.float16(-2) and s == np.float16(np.float32(3) / np.float32(15))
    assert np.abs(c * np.float64(s) + np.float64(z) - x).max() <= 0.5 * s + 15 * 2.0**-12
    assert F.quantize(np.full(32, 0.25, np.float32))[:3] [0].sum() == 0
    assert F.quantize(np.array([np.nan] + [0] * 31, np.float32))[3]
    assert F.quantize(np.array([7e4] + [0] * 31, np.float32))[3]


@pytest.mark.parametrize("d", [64, 128])
def test_oracle_cache_round_trip(d):
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 20, 3, d)).astype(np.float32)
    pages = np.zeros((3, 3, F.page_bytes(d)), np.uint8)
    slots = rng.permutation(48)[:20]
    F.write(pages, k, v, slots)
    for x, y in zip((k, v), F.values(pages, slots, d)):
        c, s, z, _ = F.quantize(x.reshape(20, 3, d // 32, 32))
        want = c * s[..., None].astype(np.float64) + z[..., None].astype(np.float64)
        np.testing.assert_array_equal(y, want.reshape(x.shape))
    # no two tokens share a byte: what the writes left is zero exactly outside them
    alone = np.zeros_like(pages)
    for i, slot in enumerate(slots):
        one = np.zeros_like(pages)
        F.write(one, k[i:i + 1], v[i:i + 1], [slot])
        assert not (alone.astype(bool) & one.astype(bool)).any()
        alone |= one
    np.testing.assert_array_equal(alone, pages)


def test_oracle_attention_is_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((6, 4, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    out, lse, p, _ = F.attend(q, k, v, [4 + i for i in range(6)])
    t = torch.nn.functional.scaled_dot_product_attention(
        *(torch.from_numpy(x).transpose(0, 1)[None] for x in (q, k.repeat(2, 1), v.repeat(2, 1))),
        attn_mask=torch.arange(9)[None] <= 3 + torch.arange(6)[:, None])
    np.testing.assert_allclose(out, t[0].transpose(0, 1).numpy(), atol=1e-12)
    np.testing.assert_allclose(p.sum(-1), 1)
    assert (F.attend(q, k, v, [0, -3, 1, 1, 1, 1])[0][:2] == 0).all()


def test_oracle_eviction_against_a_sort():
    rng = np.random.default_rng(2)
    for n, keep, recent in ((30, 10, 4), (30, 30, 4), (30, 3, 9), (5, 9, 1), (12, 0, 3)):
        w = rng.integers(0, 4, n).astype(np.float32)
        got = F.kept_tokens(w, n, keep, recent)
        keep = min(n, keep)
        w2 = w.copy()
        w2[n - min(keep, recent):] = 100
        want = np.sort(np.argsort(-w2, kind="stable")[:keep])
        np.testing.assert_array_equal(got, want)


def test_whole_numbers_that_a_c_int_cannot_hold_are_refused(S):
    assert S._int32((1 << 31) - 1, "window") == (1 << 31) - 1 and S._int32(np.int64(7), "window") == 7
    for x in (1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 31) - 1, 1 << 63):
        with pytest.raises(ValueError):
            S._int32(x, "window")


def test_layout_of_more_bytes_than_64_bits_count_is_refused(S):
    cfg = S.make_config(8, 4, 64, 64, 16, 64, 16)
    most = ((1 << 63) - 1) // (4 * F.page_bytes(64))
    assert S.starkv_kv4_layout(cfg, most)["pages_bytes"] == most * 4 * F.page_bytes(64)
    for n in (most + 1, 1 << 60, (1 << 63) - 1):
        with pytest.raises(S.StarKVError) as e:
            S.starkv_kv4_layout(cfg, n)
        assert e.value.code == S.ERR_UNSUPPORTED_SHAPE
