"""Pins of the float64 reference of the 8-bit KV cache (tests/kv8_reference.py)."""
import numpy as np
import torch

import kv8_reference as ref


def test_e4m3_rounding_matches_every_code_and_the_cast():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(ref.e4m3(codes), codes, equal_nan=True)
    fin = np.sort(codes[np.isfinite(codes)])
    mid = (fin[1:] + fin[:-1]) / 2  # ties, and values just beside them
    x = np.concatenate([mid, np.nextafter(mid, np.inf), np.nextafter(mid, -np.inf),
                        np.random.default_rng(0).standard_normal(20000) * 40])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.e4m3(x), want)
    assert ref.e4m3(np.inf) == 448 and ref.e4m3(-np.inf) == -448 and np.isnan(ref.e4m3(np.nan))


def test_scale_is_the_least_power_of_two():
    for a in (1e-30, 0.7, 1.75, 1.7500001, 447.9, 448.0, 448.1, 3.0e38):
        s = ref.scale_of(a)
        assert a <= 448 * s and a > 224 * s and np.log2(s) == int(np.log2(s))
    assert ref.scale_of(0.0) == ref.scale_of(1e-40) == 2.0 ** -117


def _cache(B, H, cap, hd, block, seed=0):
    g = np.random.default_rng(seed)
    n = cap // block
    return {"k": ref.e4m3(g.standard_normal((B, H, cap, hd)) * 100), "v": ref.e4m3(g.standard_normal((B, H, cap, hd)) * 100),
            "k_scale": 2.0 ** g.integers(-8, -5, (B, H, n)), "v_scale": 2.0 ** g.integers(-8, -5, (B, H, n)),
            "weight": g.random((B, H, n)), "ids": np.tile(np.arange(n), (B, H, 1))}


def test_attention_of_one_token_and_of_equal_keys():
    c = _cache(1, 2, 32, 16, 8)
    q = np.random.default_rng(1).standard_normal((1, 4, 16))
    out, w, _ = ref.attend(c, 8, [1], q)
    for g in range(4):
        assert np.allclose(out[0, g], c["v"][0, g // 2, 0] * c["v_scale"][0, g // 2, 0], rtol=0, atol=1e-12)
    assert np.allclose(w[0, :, 0], 2.0) and not w[0, :, 1:].any()
    c["k"][:] = 1.0
    c["k_scale"][:] = 0.5
    out, w, _ = ref.attend(c, 8, [20], q)
    v = c["v"][0, 0, :20] * np.repeat(c["v_scale"][0, 0], 8)[:20, None]
    assert np.allclose(out[0, 0], v.mean(0)) and np.allclose(w[0, 0], [0.8, 0.8, 0.4, 0.0])


def test_growing_block_and_token_by_token_append():
    g = np.random.default_rng(2)
    k, v = g.standard_normal((1, 13, 1, 16)), g.standard_normal((1, 13, 1, 16))
    k[0, 9] *= 50  # the second block's scale grows at its second row
    one, many = _cache(1, 1, 16, 16, 8), _cache(1, 1, 16, 16, 8)
    ref.append(many, 8, [0], k, v, [13])
    for t in range(13):
        ref.append(one, 8, [t], k[:, t:t + 1], v[:, t:t + 1], [1])
    assert np.array_equal(one["k_scale"][..., :2], many["k_scale"][..., :2])
    assert one["ids"][0, 0].tolist() == [0, 1] and not one["weight"].any()
    # rows whose rounding was re-done differ by at most one more rounding
    s = np.repeat(many["k_scale"][0, 0], 8)[:13, None]
    assert np.abs((one["k"] - many["k"])[0, 0, :13] * s).max() <= (np.abs(many["k"][0, 0, :13]) * s / 8 + s * 2.0 ** -9).max()
    assert np.array_equal(one["k"][0, 0, 9:13], many["k"][0, 0, 9:13])


def test_eviction_keeps_the_heaviest_and_attention_ignores_order():
    c = _cache(1, 1, 80, 16, 8, seed=3)
    c["weight"][0, 0] = [0.5, 9, 1, 8, 2, 7, 3, 6, 4, 0]
    d = {x: y.copy() for x, y in c.items()}
    after = ref.evict(d, 8, [77], 5, 1, 2)
    assert after == [77 - 5 * 8]
    # kept: 0 (sink), 8 and 9 (recent), 1 and 3 (weight); 0, 1, 3 stay, 8 fills slot 2, 9 the last slot
    assert d["ids"][0, 0, :5].tolist() == [0, 1, 8, 3, 9]
    q = np.random.default_rng(4).standard_normal((1, 2, 16))
    rows = np.concatenate([np.arange(8 * i, 8 * i + 8) for i in (0, 1, 3, 8, 9)])[:37]
    e = {x: (c[x][:, :, rows] if x in "kv" else c[x][:, :, [0, 1, 3, 8, 9]]) for x in c}
    e["k"] = np.concatenate([e["k"], np.zeros((1, 1, 3, 16))], 2)
    e["v"] = np.concatenate([e["v"], np.zeros((1, 1, 3, 16))], 2)
    a, wa, _ = ref.attend(d, 8, after, q)
    b, wb, _ = ref.attend(e, 8, after, q)
    assert np.allclose(a, b, rtol=0, atol=1e-12) and np.allclose(wa[0, 0, [0, 1, 3, 2, 4]], wb[0, 0, :5])
    assert ref.evict(d, 8, after, 5, 1, 2) == after  # nothing more to drop
