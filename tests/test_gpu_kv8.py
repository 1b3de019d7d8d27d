"""The 8-bit KV cache on the GPU against float64 (tests/kv8_reference.py).

Codes, scales, ids and eviction are exact: every rounding they hold is of an exact quotient.  Attention is
f32 arithmetic; with S the largest |logit| of a case, a probability is off by its logit's absolute error (at most
8 half-ulps of a number of size S: the product's accumulation, its scaling and the subtraction) and by 64 half-ulps
for everything else (exp2, the split of the probability into pieces, the sums over tokens and partials, the
division), so an output is within 2^-24 (8 S + 64) of sum_t p_t |v_t|, which no cancellation shrinks.  A row's
probability times its block's value scale enters the product with the codes in fixed point, 28 bits at least (24 for
more than 8 query heads of more than 128 columns) of a number that the largest of the 128-row tile is at least half of:
rounding to half of the last bit, or 1 to the largest number below it, leaves at most 2^-28 (2^-24) and so 2^-27
(2^-23) of the tile's largest, times the rows' codes."""
import numpy as np
import pytest
import torch

import kv8_reference as ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


class Both:
    """One cache on the device, 0xFF behind every written row, and its float64 twin."""

    def __init__(self, xkv, B, H, hd, block, capacity):
        self.xkv, self.block = xkv, block
        self.p = xkv.kv8_params(B, H, hd, block, capacity)
        self.c = xkv.KV8Cache.empty(self.p)
        for t in (self.c.k, self.c.v, self.c.k_scale, self.c.v_scale, self.c.weight, self.c.ids):
            t.view(torch.uint8).fill_(0xFF)
        n = capacity // block
        self.r = {x: np.full((B, H, capacity, hd), np.nan) for x in ("k", "v")}
        self.r |= {x: np.full((B, H, n), np.nan) for x in ("k_scale", "v_scale", "weight")}
        self.r["ids"] = np.full((B, H, n), -1)
        self.lens = [0] * B

    def dev_lens(self):
        return torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def append(self, k, v, counts=None, check=True):
        """k, v [B][n][H][hd] CUDA tensors."""
        B, n = k.shape[:2]
        d = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        self.xkv.xkv_kv8_append(self.p, self.c, self.dev_lens(), k.flatten(2), v.flatten(2), d)
        counts = counts or [n] * B
        ref.append(self.r, self.block, self.lens, k.double().cpu().numpy(), v.double().cpu().numpy(), counts)
        self.lens = [a + b for a, b in zip(self.lens, counts)]
        if check:
            self.check()

    def check(self):
        for x in ("k", "v"):
            got = getattr(self.c, x).float().cpu().numpy().astype(np.float64)
            assert np.array_equal(got, self.r[x], equal_nan=True), x
        for x in ("k_scale", "v_scale", "weight", "ids"):
            got = getattr(self.c, x).cpu().numpy().astype(np.float64)
            assert np.array_equal(got, self.r[x], equal_nan=True), x
        assert self.xkv.get_device_status() == 0


def _rows(g, B, n, H, hd, dt, scale=1.0):
    x = torch.randn((B, n, H, hd), generator=g) * torch.exp(0.5 * torch.randn((H, hd), generator=g)) * scale
    return x.to(_dt(dt)).cuda()


def _fill(xkv, B, H, hd, block, capacity, counts, dt="bf16", seed=0):
    g = torch.Generator().manual_seed(seed)
    b = Both(xkv, B, H, hd, block, capacity)
    n = max(counts)
    if n:
        b.append(_rows(g, B, n, H, hd, dt), _rows(g, B, n, H, hd, dt), counts, check=False)
    b.r["weight"][:] = np.where(np.isnan(b.r["weight"]), np.nan, 0.0)
    return b, g


def _bounds(b, q, top):
    """Output by output: 2^-24 (8 S + 64) sum_t p_t |v_t|, and the fixed point's share."""
    a = dict(b.r)
    a["v"] = np.abs(b.r["v"])
    tol = 2.0 ** -24 * (8 * top + 64) * ref.attend(a, b.block, b.lens, q)[0]
    H = b.r["k"].shape[1]
    gq = q.shape[1] // H
    fixed = 2.0 ** (-23 if gq > 8 and q.shape[2] > 128 else -27)
    for i, n in enumerate(b.lens):
        at = np.arange(n) // b.block
        for h in range(H if n else 0):
            k = b.r["k"][i, h, :n] * b.r["k_scale"][i, h, at][:, None]
            s = q[i, h * gq:(h + 1) * gq] @ k.T / np.sqrt(q.shape[2])
            p = np.exp(s - s.max(1, keepdims=True))
            p *= b.r["v_scale"][i, h, at] / p.sum(1, keepdims=True)
            for t in range(0, n, 128):
                most = p[:, t:t + 128].max(1)
                tol[i, h * gq:(h + 1) * gq] += fixed * most[:, None] * a["v"][i, h, t:min(t + 128, n)].sum(0)
    return tol


def _attend(b, q, accumulate=False, ws=None, stream=None, out=None):
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda") if out is None else out
    b.xkv.xkv_kv8_attention_decode(b.p, b.c, b.dev_lens(), q, out, accumulate=accumulate, ws=ws, stream=stream)
    return out


def _check_attend(b, q, out, weight_before=None):
    want, w, top = ref.attend(b.r, b.block, b.lens, q.double().cpu().numpy())
    got = out.double().cpu().numpy()
    tol = _bounds(b, q.double().cpu().numpy(), top)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol + 1e-300).all(), float((np.abs(got - want) / (tol + 1e-300)).max())
    if weight_before is not None:
        n = [-(-t // b.block) for t in b.lens]
        got_w = b.c.weight.double().cpu().numpy()
        for i, m in enumerate(n):
            err = np.abs(got_w[i, :, :m] - (weight_before[i, :, :m] + w[i, :, :m]))
            bound = 2.0 ** -24 * ((8 * top + 64) * w[i, :, :m] + np.abs(weight_before[i, :, :m]) + w[i, :, :m])
            assert (err <= bound + 1e-300).all(), (i, float((err / (bound + 1e-300)).max()))
            assert np.array_equal(got_w[i, :, m:], weight_before[i, :, m:], equal_nan=True)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dt,B,H,hd,block,capacity,first,then", [
    ("bf16", 1, 1, 16, 8, 8, [1], [7]),
    ("bf16", 2, 3, 128, 64, 256, [64, 1], [1, 64]),
    ("bf16", 3, 2, 80, 16, 160, [0, 37, 5], [33, 0, 100]),
    ("f32", 3, 2, 96, 32, 192, [31, 32, 33], [1, 97, 0]),
    ("f32", 1, 5, 64, 8, 1000, [999], [1]),
    ("bf16", 2, 1, 256, 128, 512, [127, 200], [2, 312]),
    ("f32", 2, 1, 256, 128, 384, [3, 129], [380, 255]),
])
def test_append_is_exact(xkv, dt, B, H, hd, block, capacity, first, then):
    g = torch.Generator().manual_seed(1)
    b = Both(xkv, B, H, hd, block, capacity)
    for counts, scale in ((first, 1.0), (then, 7.0)):  # larger rows join: part-filled blocks are rounded anew
        n = max(counts)
        b.append(_rows(g, B, n, H, hd, dt, scale), _rows(g, B, n, H, hd, dt, 1 / scale), counts)


def test_append_token_by_token(xkv):
    g = torch.Generator().manual_seed(2)
    b = Both(xkv, 2, 2, 32, 16, 64)
    for t in range(40):
        s = 4.0 if t % 7 == 3 else 0.25
        b.append(_rows(g, 2, 1, 2, 32, "bf16", s * (1 + t)), _rows(g, 2, 1, 2, 32, "bf16", s), check=t % 5 == 4 or t > 37)


def test_append_special_values(xkv):
    inf, nan = float("inf"), float("nan")
    b = Both(xkv, 1, 1, 16, 8, 64)
    x = torch.zeros((1, 48, 1, 16))
    x[0, 8:16] = 3e38 * (1 - 0.1 * torch.arange(8))[:, None, None]     # the largest scale
    x[0, 16:24] = 1e-38 * torch.arange(8)[:, None, None]               # clamped to the least scale, and subnormals
    x[0, 24], x[0, 25], x[0, 26, 0, 3] = inf, -inf, 2.0                 # infinities do not count
    x[0, 32, 0, 5], x[0, 33] = nan, 1.0                                 # nor do NaN
    x[0, 40:48] = -0.0
    b.append(x[:, :20].cuda(), -x[:, :20].cuda())
    b.append(x[:, 20:].cuda(), -x[:, 20:].cuda())
    assert b.r["k_scale"][0, 0, 0] == b.r["k_scale"][0, 0, 5] == 2.0 ** -117


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mantissa", [1.0, 1.25, 1.5, 1.75])
def test_append_to_a_block_with_a_scale_of_other_origin(xkv, dt, mantissa):
    # blocks written by another quantiser, their scales no powers of two: what joins them is on the next power, and so
    # are their own codes (times mantissa / 2, which e4m3's four bits times three leave exact in f32)
    B, H, hd, block, held = 2, 2, 64, 16, 21
    b, g = _fill(xkv, B, H, hd, block, 64, [held, held], dt)
    for x in ("k", "v"):
        getattr(b.c, x + "_scale")[:, :, 1].mul_(mantissa)
        b.r[x + "_scale"][:, :, 1] *= mantissa
    before = {x: b.r[x].copy() for x in ("k", "v")}
    new = {x: _rows(g, B, 3, H, hd, dt, 0.25) for x in ("k", "v")}
    want = {}
    for x in ("k", "v"):
        was = b.r[x + "_scale"][:, :, 1].copy()
        rows = new[x].double().cpu().numpy().transpose(0, 2, 1, 3)
        need = np.vectorize(ref.scale_of)(np.abs(rows).max((2, 3)))
        now = np.maximum(np.exp2(np.ceil(np.log2(was))), need)
        b.r[x][:, :, 16:held] = ref.e4m3(b.r[x][:, :, 16:held] * (was / now)[:, :, None, None])
        b.r[x][:, :, held:held + 3] = ref.e4m3(rows / now[:, :, None, None])
        b.r[x + "_scale"][:, :, 1] = now
        want[x] = before[x][:, :, 16:held] * was[:, :, None, None], rows
    xkv.xkv_kv8_append(b.p, b.c, b.dev_lens(), new["k"].flatten(2), new["v"].flatten(2))
    b.lens = [held + 3] * B
    b.check()
    for x in ("k", "v"):  # each within half a step of what it stands for, of a number or of the least one
        now = b.r[x + "_scale"][:, :, 1][:, :, None, None]
        for got, true in zip((b.r[x][:, :, 16:held] * now, b.r[x][:, :, held:held + 3] * now), want[x]):
            assert (np.abs(got - true) <= np.abs(true) * 2.0 ** -4 + now * 2.0 ** -10).all()


def test_append_reads_views_and_writes_only_its_rows(xkv):
    B, H, hd, block, cap, n = 2, 2, 64, 16, 96, 21
    g = torch.Generator().manual_seed(3)
    b = Both(xkv, B, H, hd, block, cap)
    qkv = torch.randn((B, n, 3, H, hd), generator=g).to(torch.bfloat16).cuda()  # q, k, v of one projection
    k, v = qkv[:, :, 1], qkv[:, :, 2]
    xkv.xkv_kv8_append(b.p, b.c, b.dev_lens(), k.flatten(2), v.flatten(2))
    assert k.flatten(2).stride(1) == 3 * H * hd  # a view: nothing was copied
    ref.append(b.r, block, b.lens, k.double().cpu().numpy(), v.double().cpu().numpy(), [n] * B)
    b.check()


def test_append_of_no_rows_and_of_strides_that_nothing_uses(xkv):
    B, H, hd, block = 1, 2, 64, 16
    b, g = _fill(xkv, B, H, hd, block, 64, [21])
    none = torch.empty((B, 0, H * hd), dtype=torch.bfloat16, device="cuda")
    xkv.xkv_kv8_append(b.p, b.c, b.dev_lens(), none, none)
    b.check()
    k = _rows(g, B, 1, H, hd, "bf16")  # one row of one sequence, its value a view into a projection
    qkv = _rows(g, B, 1, 3 * H, hd, "bf16")
    v = qkv.flatten(2)[..., 2 * H * hd:]
    assert v.stride() != k.flatten(2).stride() and v.stride(2) == 1
    xkv.xkv_kv8_append(b.p, b.c, b.dev_lens(), k.flatten(2), v)
    ref.append(b.r, block, b.lens, k.double().cpu().numpy(), v.double().cpu().numpy().reshape(B, 1, H, hd), [1])
    b.lens = [22]
    b.check()
    k, v = _rows(g, B, 5, H, hd, "bf16").flatten(2), _rows(g, 2, 5, H, hd, "bf16").flatten(2)
    wide = torch.empty((1, 9, H * hd), dtype=torch.bfloat16, device="cuda")[:, :5]  # another stride between sequences
    wide.copy_(v[:1])
    xkv.xkv_kv8_append(b.p, b.c, b.dev_lens(), k, wide)
    ref.append(b.r, block, b.lens, k.double().cpu().numpy().reshape(B, 5, H, hd),
               v[:1].double().cpu().numpy().reshape(B, 5, H, hd), [5])
    b.check()
    with pytest.raises(ValueError):  # rows of unlike strides
        xkv.xkv_kv8_append(b.p, b.c, b.dev_lens(), k, torch.empty((1, 5, 2 * H * hd), dtype=torch.bfloat16,
                                                                  device="cuda")[..., :H * hd])


def test_append_past_the_capacity_and_bad_lengths(xkv):
    g = torch.Generator().manual_seed(4)
    b = Both(xkv, 3, 1, 32, 8, 32)
    k, v = _rows(g, 3, 10, 1, 32, "bf16"), _rows(g, 3, 10, 1, 32, "bf16")
    lens = torch.tensor([27, -5, 99], dtype=torch.int32, device="cuda")  # five rows fit; taken as 0; as full
    b.c.k_scale[0, 0, 3], b.c.v_scale[0, 0, 3] = 1.0, 1.0
    b.c.k.view(torch.uint8)[0, 0, 24:27], b.c.v.view(torch.uint8)[0, 0, 24:27] = 0, 0
    xkv.xkv_kv8_append(b.p, b.c, lens, k.flatten(2), v.flatten(2))
    assert xkv.get_device_status() == xkv.XKV_ERR_INVALID_ARG
    for x, new in (("k", k), ("v", v)):
        b.r[x][0, 0, 24:27], b.r[x + "_scale"][0, 0, 3] = 0.0, 1.0
        b.r["ids"][0, 0, 3] = -1
    new_k, new_v = k.double().cpu().numpy(), v.double().cpu().numpy()
    one = {x: y[:1] for x, y in b.r.items()}
    ref.append(one, 8, [27], new_k[:1], new_v[:1], [5])
    two = {x: y[1:2] for x, y in b.r.items()}
    ref.append(two, 8, [0], new_k[1:2], new_v[1:2], [10])
    b.check()


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("dt,H,gq,hd,block,counts", [
    ("bf16", 2, 4, 128, 64, [1, 0, 127, 128, 129, 513]),
    ("bf16", 1, 1, 16, 8, [1]),
    ("bf16", 3, 7, 64, 16, [1000, 3]),
    ("f32", 2, 8, 96, 32, [255, 256, 257, 0]),
    ("f32", 4, 3, 80, 128, [700]),
    ("bf16", 1, 16, 256, 64, [391, 64, 1]),
    ("f32", 1, 16, 256, 8, [140, 129]),
    ("bf16", 8, 2, 192, 8, [33, 1025]),
    ("f32", 5, 1, 48, 16, [2000, 17, 0, 300]),
    ("bf16", 2, 12, 112, 32, [640]),
    ("bf16", 2, 5, 128, 128, [4, 5000]),
    ("bf16", 1, 1, 48, 16, [40000, 129]),   # several tiles to a CTA, odd sizes of the partials
    ("f32", 1, 3, 16, 8, [50001]),
    ("bf16", 3, 16, 128, 64, [20000, 1]),
])
def test_attention_matches_float64(xkv, dt, H, gq, hd, block, counts):
    B = len(counts)
    capacity = -(-max(max(counts), 1) // block) * block + block
    b, g = _fill(xkv, B, H, hd, block, capacity, counts, dt)
    q = (2 * torch.randn((B, H * gq, hd), generator=g)).to(_dt(dt)).cuda()
    _check_attend(b, q, _attend(b, q))
    b.c.weight.copy_(torch.rand(b.c.weight.shape, generator=g))
    before = b.c.weight.double().cpu().numpy()
    out = _attend(b, q, accumulate=True)
    _check_attend(b, q, out, before)
    assert xkv.get_device_status() == 0


@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("gq", [3, 8, 12])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_every_kernel_shape_over_shares_of_several_tiles(xkv, dt, gq, hd):
    # 430 tiles on 148 SMs: each buffer of the pipeline is used again, by both halves of the softmax
    b, g = _fill(xkv, 3, 2, hd, 32, 15040, [12000, 15001, 3], dt)
    q = (2 * torch.randn((3, 2 * gq, hd), generator=g)).to(_dt(dt)).cuda()
    b.c.weight.zero_()
    out = _attend(b, q, accumulate=True)
    assert xkv.get_device_status() == 0
    _check_attend(b, q, out, np.zeros(b.c.weight.shape))
    spoil = torch.empty(64 << 20, dtype=torch.int32, device="cuda")
    for _ in range(8):  # codes from L2 and from memory, whose tiles come at other times
        assert torch.equal(_attend(b, q), out)
        spoil.zero_()
    assert xkv.get_device_status() == 0


def test_attention_over_unlike_scales(xkv):
    # blocks of values from 2^-60 to 2^60, keys from 2^-20 to 2^4, a peaked and a flat head
    b, g = _fill(xkv, 1, 2, 64, 8, 400, [389])
    for x, lo, hi in (("k", -20, 4), ("v", -60, 60)):
        e = torch.randint(lo, hi, b.c.k_scale.shape, generator=g)
        s = torch.exp2(e.float()) / 448
        s = torch.exp2(torch.floor(torch.log2(s)))
        getattr(b.c, x + "_scale").copy_(s)
        b.r[x + "_scale"][:] = s.double().numpy()
    q = torch.randn((1, 8, 64), generator=g)
    q[:, 0] *= 1e-6
    q[:, 1] *= 8
    q = q.cuda()
    _check_attend(b, q, _attend(b, q))


def _tight(b, q, top):
    """_bounds with the probabilities' own precision: what a product of probability and scale loses, beside the f32
    share, is against the largest of its 128-row tile, of which the unit is less than twice: 2^-32 of the unit in 32
    bits (rounding, or 1 to the number below it); in six pieces of four significant bits 2^-38 of it below 2^-14 of it
    (half of the last piece's least code, 2^-10 16^-5 where the unit is 2^8), and above that 2^-24 of the product
    itself, which is one more half-ulp of the f32 share."""
    gq = q.shape[1] // b.r["k"].shape[1]
    six = gq > 8 and q.shape[2] > 128
    a = dict(b.r)
    a["v"] = np.abs(b.r["v"])
    tol = 2.0 ** -24 * (8 * top + 65) * ref.attend(a, b.block, b.lens, q)[0]
    for i, n in enumerate(b.lens):
        at = np.arange(n) // b.block
        for h in range(b.r["k"].shape[1] if n else 0):
            k = b.r["k"][i, h, :n] * b.r["k_scale"][i, h, at][:, None]
            s = q[i, h * gq:(h + 1) * gq] @ k.T / np.sqrt(q.shape[2])
            p = np.exp(s - s.max(1, keepdims=True))
            p *= b.r["v_scale"][i, h, at] / p.sum(1, keepdims=True)
            for t in range(0, n, 128):
                most = p[:, t:t + 128].max(1)
                tol[i, h * gq:(h + 1) * gq] += 2.0 ** (-37 if six else -31) * most[:, None] * a["v"][i, h, t:min(t + 128, n)].sum(0)
    return tol


@pytest.mark.parametrize("kind", ["outlier", "sink", "both"])
@pytest.mark.parametrize("dt,gq,hd,block", [("bf16", 16, 256, 8), ("f32", 16, 256, 8), ("bf16", 9, 144, 16),
                                            ("bf16", 8, 256, 8), ("bf16", 16, 128, 8), ("f32", 3, 64, 8)])
def test_rows_that_weigh_little_beside_their_tile(xkv, kind, dt, gq, hd, block):
    # an outlier value 2^13 times the others makes its block's scale large; a sink has nearly all of the probability
    # and no value.  What the other rows of the tile bring is the whole of most columns, and as exact as ever.
    n = 300
    g = torch.Generator().manual_seed(11)
    b = Both(xkv, 1, 1, hd, block, 320)
    k, v = torch.randn((1, n, 1, hd), generator=g) * 0.1, torch.randn((1, n, 1, hd), generator=g)
    u = torch.sign(torch.randn(hd, generator=g))
    q = u * 0.25 + 0.25 * torch.randn((1, gq, hd), generator=g)
    if kind != "outlier":
        k[0, 5, 0] = u * 48 / hd ** 0.5  # a logit of about 12
        v[0, 5] = 0.0
    if kind != "sink":
        v[0, 43, 0, 7] = 2.0 ** 13
    b.append(k.to(_dt(dt)).cuda(), v.to(_dt(dt)).cuda())
    q = q.to(_dt(dt)).cuda()
    out = _attend(b, q)
    qd = q.double().cpu().numpy()
    want, _, top = ref.attend(b.r, block, b.lens, qd)
    err, tol = np.abs(out.double().cpu().numpy() - want), _tight(b, qd, top)
    assert top < 40 and (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_queries_with_a_column_that_the_keys_do_not_use(xkv, dt):
    # one column 10^5 times the others, zero in the keys: what decides are entries at 2^-17 of the largest
    b, g = _fill(xkv, 1, 1, 64, 16, 320, [300], dt)
    b.c.k.view(torch.uint8)[..., 7] = 0
    b.r["k"][..., 7] = 0.0
    q = (2 * torch.randn((1, 8, 64), generator=g)).to(_dt(dt))
    q[..., 7] = 1e5
    q = q.cuda()
    _check_attend(b, q, _attend(b, q))


def test_attention_of_many_sequences(xkv):
    counts = [(37 * i) % 301 for i in range(700)]  # more sequences than CTAs, some empty
    b, g = _fill(xkv, 700, 1, 32, 16, 320, counts)
    q = torch.randn((700, 2, 32), generator=g).to(torch.bfloat16).cuda()
    b.c.weight.zero_()
    _check_attend(b, q, _attend(b, q, accumulate=True), np.zeros(b.c.weight.shape))


def test_nan_reaches_only_its_own_heads(xkv):
    b, g = _fill(xkv, 2, 2, 64, 16, 256, [200, 130])
    q = torch.randn((2, 8, 64), generator=g).cuda()
    good = _attend(b, q)
    bad = q.clone()
    bad[0, 1, 5], bad[1, 7, 0], bad[1, 6, 3] = float("nan"), float("inf"), -float("inf")
    out = _attend(b, bad)
    for s, h in ((0, 1), (1, 7), (1, 6)):
        assert out[s, h].isnan().all()
        out[s, h] = good[s, h]
    assert torch.equal(out, good)
    b.c.k.view(torch.uint8)[0, 1, 100, 3] = 0x7F  # a NaN key of one KV head
    b.c.v.view(torch.uint8)[1, 0, 129, 9] = 0x7F  # one column of another's values
    out = _attend(b, q)
    assert out[0, 4:].isnan().all() and out[1, :4, 9].isnan().all()
    out[0, 4:], out[1, :4, 9] = good[0, 4:], good[1, :4, 9]
    assert torch.equal(out, good)


@pytest.mark.parametrize("gq,hd,block,counts,unit,rows", [
    (4, 64, 16, [129, 40], (0, 1), (128, 129)),         # a tile's only row
    (2, 128, 64, [512, 512], (1, 0), (128, 256)),       # a whole tile beside finite ones
    (16, 256, 32, [300, 129], (1, 0), (128, 129)),
    (8, 64, 32, [40000, 1], (0, 0), (25600, 25728)),    # one of more slots than a lane holds
    (4, 128, 128, [60000], (0, 1), (59904, 60000)),     # the last tile
    (4, 64, 16, [300], (0, 0), (0, 300)),               # every row
])
def test_nan_keys_with_a_tile_of_their_own(xkv, gq, hd, block, counts, unit, rows):
    # all logits of a partial are NaN, and those of the others are not: the softmax's sum is NaN all the same
    capacity = -(-max(counts) // block) * block + block
    b, g = _fill(xkv, len(counts), 2, hd, block, capacity, counts)
    q = torch.randn((len(counts), 2 * gq, hd), generator=g).to(torch.bfloat16).cuda()
    b.c.weight.zero_()
    good = _attend(b, q, accumulate=True)
    weight = b.c.weight.clone()
    b.c.weight.zero_()
    s, h = unit
    b.c.k.view(torch.uint8)[s, h, rows[0]:rows[1], 3] = 0x7F
    out = _attend(b, q, accumulate=True)
    live = -(-counts[s] // block)
    assert out[s, h * gq:(h + 1) * gq].isnan().all() and b.c.weight[s, h, :live].isnan().all()
    out[s, h * gq:(h + 1) * gq], b.c.weight[s, h, :live] = good[s, h * gq:(h + 1) * gq], weight[s, h, :live]
    assert torch.equal(out, good) and torch.equal(b.c.weight, weight)
    assert xkv.get_device_status() == 0


@pytest.mark.parametrize("gq,hd,block,n,row", [(4, 64, 16, 300, 130), (16, 256, 32, 200, 128), (2, 128, 64, 60000, 30000),
                                              (8, 64, 8, 129, 128)])
def test_nan_values_of_rows_without_weight(xkv, gq, hd, block, n, row):
    # logits of 800 for the first rows and 0 for the others, whose probabilities are 0 in f32: 0 * NaN stays NaN,
    # whichever partial has the row
    b, g = _fill(xkv, 1, 2, hd, block, -(-n // block) * block, [n])
    b.c.k.view(torch.uint8).zero_()
    b.c.k[:, :, :8] = torch.full((1, 2, 8, hd), 8.0).to(F8).cuda()
    b.c.k_scale.fill_(1.0)
    q = torch.full((1, 2 * gq, hd), 100.0 / hd ** 0.5, dtype=torch.float32, device="cuda")
    good = _attend(b, q)
    b.c.v.view(torch.uint8)[0, 1, row, 9] = 0x7F
    out = _attend(b, q)
    assert out[0, gq:, 9].isnan().all()
    out[0, gq:, 9] = good[0, gq:, 9]
    assert torch.equal(out, good)


def test_largest_values_of_rows_without_weight(xkv):
    # a tile whose values sum past f32's largest, and whose probabilities are all 0 in f32: nothing of it is left
    n, hd, gq = 200, 64, 4
    b, g = _fill(xkv, 1, 1, hd, 8, n, [n])
    b.c.k.view(torch.uint8).zero_()
    b.c.k[:, :, :8] = torch.full((1, 1, 8, hd), 8.0).to(F8).cuda()
    b.c.k_scale.fill_(1.0)
    q = torch.full((1, gq, hd), 100.0 / hd ** 0.5, dtype=torch.float32, device="cuda")
    good = _attend(b, q)
    b.c.v[:, :, 128:] = torch.full((1, 1, n - 128, hd), 448.0).to(F8).cuda()
    b.c.v_scale[:, :, 16:] = 2.0 ** 119
    out = _attend(b, q)
    assert out.isfinite().all() and torch.equal(out, good)


def test_attention_writes_only_its_outputs(xkv):
    counts = [77, 0, 300]
    b, g = _fill(xkv, 3, 2, 80, 16, 304, counts)
    q = torch.randn((3, 6, 80), generator=g).to(torch.bfloat16).cuda()
    n = b.xkv.xkv_kv8_workspace_size(b.p, 6)
    ws = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    buf = torch.full((q.numel() + 2048,), float("nan"), device="cuda")
    out = buf[1024:1024 + q.numel()].view(q.shape)
    b.c.weight.zero_()
    before = [t.clone() for t in (b.c.k.view(torch.uint8), b.c.v.view(torch.uint8), b.c.k_scale, b.c.v_scale, b.c.ids)]
    _attend(b, q, True, ws[:n], out=out)
    assert out.isfinite().all() and buf[:1024].isnan().all() and buf[-1024:].isnan().all()
    assert bool((ws[n:] == 0xFF).all())
    after = (b.c.k.view(torch.uint8), b.c.v.view(torch.uint8), b.c.k_scale, b.c.v_scale, b.c.ids)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, after))
    for i, t in enumerate(counts):
        assert not b.c.weight[i, :, -(-t // 16):].any()


def test_bad_lengths_are_clamped_and_recorded(xkv):
    b, g = _fill(xkv, 2, 1, 32, 8, 64, [64, 64])
    q = torch.randn((2, 2, 32), generator=g).cuda()
    want = _attend(b, q)
    assert xkv.get_device_status() == 0
    out = torch.empty_like(want)
    xkv.xkv_kv8_attention_decode(b.p, b.c, torch.tensor([65, -1], dtype=torch.int32, device="cuda"), q, out)
    assert xkv.get_device_status() == xkv.XKV_ERR_INVALID_ARG
    assert torch.equal(out[0], want[0]) and not out[1].any()


def test_offsets_past_32_bits(xkv):
    # 34 sequences of 2^20 x 128 codes: the last one starts past 2^32
    B, cap, hd, block, n = 34, 1 << 20, 128, 64, 700
    b = Both.__new__(Both)
    b.xkv, b.block, b.p = xkv, block, xkv.kv8_params(B, 1, hd, block, cap)
    b.c = xkv.KV8Cache.empty(b.p)
    b.c.weight.zero_()
    g = torch.Generator().manual_seed(5)
    k, v = _rows(g, 1, n, 1, hd, "bf16"), _rows(g, 1, n, 1, hd, "bf16")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    counts = lens.clone()
    counts[-1] = n
    xkv.xkv_kv8_append(b.p, b.c, lens, k.expand(B, n, 1, hd).flatten(2), v.expand(B, n, 1, hd).flatten(2), counts)
    q = torch.randn((B, 4, hd), generator=g).cuda()
    out = torch.empty_like(q)
    xkv.xkv_kv8_attention_decode(b.p, b.c, counts, q, out, accumulate=True)
    nb = -(-n // block)
    b.r = {x: getattr(b.c, x)[-1:, :, :nb * block].float().double().cpu().numpy() for x in ("k", "v")}
    b.r |= {x: getattr(b.c, x)[-1:, :, :nb].double().cpu().numpy() for x in ("k_scale", "v_scale")}
    b.lens = [n]
    want, w, top = ref.attend(b.r, block, [n], q[-1:].double().cpu().numpy())
    tol = _bounds(b, q[-1:].double().cpu().numpy(), top)
    assert (np.abs(out[-1:].double().cpu().numpy() - want) <= tol).all() and not out[:-1].any()
    kept = torch.empty_like(counts)
    xkv.xkv_kv8_evict(b.p, b.c, counts, 4, 1, 1, kept)
    assert kept[-1] == n - (nb - 4) * block and not kept[:-1].any()
    assert b.c.ids[-1, 0, 0] == 0 and b.c.ids[-1, 0, 3] == nb - 1
    assert xkv.get_device_status() == 0


# ---------------------------------------------------------------- eviction
def _evict(b, budget, sink, recent):
    out = torch.full((len(b.lens),), -7, dtype=torch.int32, device="cuda")
    b.xkv.xkv_kv8_evict(b.p, b.c, b.dev_lens(), budget, sink, recent, out)
    b.lens = ref.evict(b.r, b.block, b.lens, budget, sink, recent)
    assert out.tolist() == b.lens
    b.check()


def _set_weight(b, w):
    live = ~np.isnan(b.r["k_scale"])
    w = np.where(live, w, b.r["weight"])
    b.c.weight.copy_(torch.from_numpy(w.astype(np.float32)))
    b.r["weight"] = w.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("B,H,hd,block,counts,budget,sink,recent", [
    (1, 1, 16, 8, [80], 1, 0, 1),           # one block is left
    (2, 2, 64, 16, [333, 100], 7, 1, 2),    # one sequence is below the budget
    (3, 1, 128, 64, [1000, 0, 641], 10, 2, 3),
    (1, 3, 80, 32, [32 * 40], 39, 0, 39),   # everything kept is recent
    (1, 2, 48, 8, [8 * 70 + 3], 33, 3, 1),  # the budget's edge on a mask word's first bit
    (1, 1, 32, 8, [8 * 97], 32, 31, 1),     # and on its last
    (2, 2, 256, 128, [1280, 1281], 6, 1, 1),
    (1, 1, 16, 8, [8 * 5000 + 1], 1234, 5, 100),
    (2, 1, 16, 8, [8 * 16384, 8 * 2049 - 7], 2000, 0, 1),  # the most keys that are kept, and the least that need room
    (2, 1, 16, 8, [8 * 16384 + 1, 8 * 2048], 2047, 3, 5),  # past them
])
def test_eviction_is_exact(xkv, B, H, hd, block, counts, budget, sink, recent):
    capacity = -(-max(counts) // block) * block + block
    b, g = _fill(xkv, B, H, hd, block, capacity, counts)
    n = np.random.default_rng(6)
    _set_weight(b, np.exp(2 * n.standard_normal(b.r["weight"].shape)))
    _evict(b, budget, sink, recent)


@pytest.mark.parametrize("kind", ["equal", "few", "special", "tiny"])
def test_eviction_ties_and_special_weights(xkv, kind):
    b, g = _fill(xkv, 1, 2, 16, 8, 8 * 130, [8 * 129 + 2])
    r, shape = np.random.default_rng(7), b.r["weight"].shape
    w = {"equal": np.ones(shape), "few": r.integers(0, 3, shape).astype(float),
         "special": r.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -2.0], shape),
         "tiny": r.choice([1e-45, 2e-45, 1e-38, 0.0], shape)}[kind]
    live = ~np.isnan(b.r["k_scale"])
    b.c.weight.copy_(torch.from_numpy(np.where(live, w, np.nan).astype(np.float32)))
    b.r["weight"] = np.where(live, w, np.nan).astype(np.float32).astype(np.float64)
    for x in ("weight",):  # 0xFF behind the last block is a NaN of its own
        assert np.isnan(b.r[x][~live]).all()
    _evict(b, 50, 2, 3)


def test_repeated_eviction_between_appends(xkv):
    # blocks change slots and keep their numbers, the newest block stays last and goes on growing
    g, r = torch.Generator().manual_seed(8), np.random.default_rng(8)
    b = Both(xkv, 2, 2, 32, 8, 160)
    b.append(_rows(g, 2, 150, 2, 32, "bf16"), _rows(g, 2, 150, 2, 32, "bf16"), [150, 91])
    for step in range(5):
        _set_weight(b, np.exp(r.standard_normal(b.r["weight"].shape)))
        _evict(b, 9, 1, 2)
        b.append(_rows(g, 2, 29, 2, 32, "bf16", 2.0), _rows(g, 2, 29, 2, 32, "bf16", 2.0), [29, 13 + step])
    q = torch.randn((2, 6, 32), generator=g).cuda()
    _check_attend(b, q, _attend(b, q))


# ---------------------------------------------------------- used together
def test_serving_run(xkv):
    """A padded batch of prompts, then decode steps (append, attend with weights, evict when a sequence is past the
    budget), in f32 on the device against float64 with the device's own codes."""
    B, H, gq, hd, block, budget = 3, 2, 4, 64, 16, 12
    g = torch.Generator().manual_seed(9)
    b = Both(xkv, B, H, hd, block, 320)
    b.append(_rows(g, B, 180, H, hd, "bf16"), _rows(g, B, 180, H, hd, "bf16"), [180, 64, 0])
    ws = xkv.workspace(xkv.xkv_kv8_workspace_size(b.p, H * gq))
    for step in range(40):
        b.append(_rows(g, B, 1, H, hd, "bf16"), _rows(g, B, 1, H, hd, "bf16"), check=step % 10 == 0)
        q = (2 * torch.randn((B, H * gq, hd), generator=g)).to(torch.bfloat16).cuda()
        before = b.r["weight"].copy()
        out = _attend(b, q, accumulate=True, ws=ws)
        _check_attend(b, q, out, before)
        b.r["weight"] = b.c.weight.double().cpu().numpy()  # the eviction below is by the device's sums
        if step % 8 == 7:
            _evict(b, budget, 1, 2)
    assert max(b.lens) <= (budget + 1) * block


def test_repeats_give_the_same_bits(xkv):
    b, g = _fill(xkv, 4, 2, 128, 32, 2048, [2047, 5, 1000, 300])
    q = torch.randn((4, 8, 128), generator=g).to(torch.bfloat16).cuda()
    first, w = None, None
    for _ in range(4):
        b.c.weight.zero_()
        out = _attend(b, q, accumulate=True)
        if first is not None:
            assert torch.equal(out, first) and torch.equal(b.c.weight, w)
        first, w = out, b.c.weight.clone()


def test_graphs_streams_and_a_shared_workspace(xkv):
    """A decode step captured once replays at other lengths and inputs; two graphs use one workspace in turn; a call
    on a stream of its own gives the same bits."""
    B, H, gq, hd, block = 2, 2, 4, 128, 64
    b, g = _fill(xkv, B, H, hd, block, 1024, [700, 333])
    ws = xkv.workspace(xkv.xkv_kv8_workspace_size(b.p, H * gq))
    q = torch.randn((B, H * gq, hd), generator=g).to(torch.bfloat16).cuda()
    k = torch.randn((B, 1, H * hd), generator=g).to(torch.bfloat16).cuda()
    lens, after = b.dev_lens(), torch.empty(B, dtype=torch.int32, device="cuda")
    out = torch.empty((B, H * gq, hd), device="cuda")
    b.c.weight.zero_()
    plain = torch.empty_like(out)

    def step(o):
        xkv.xkv_kv8_append(b.p, b.c, lens, k, k)
        torch.add(lens, 1, out=after)
        xkv.xkv_kv8_attention_decode(b.p, b.c, after, q, o, accumulate=True, ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(plain)
    torch.cuda.current_stream().wait_stream(s)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        step(out)
    other, q2 = torch.empty_like(out), torch.randn((B, H * gq, hd), generator=g).cuda()
    with torch.cuda.graph(g2):
        xkv.xkv_kv8_attention_decode(b.p, b.c, after, q2, other, ws=ws)
    for trial in range(3):
        lens.copy_(torch.tensor([700 + trial, 333 + 40 * trial], dtype=torch.int32))
        if trial:  # rows that the earlier lengths did not reach
            xkv.xkv_kv8_append(b.p, b.c, lens - trial * 40 + 1, k.expand(B, 1, H * hd).repeat(1, 40 * trial - 1, 1),
                               k.repeat(1, 40 * trial - 1, 1), torch.tensor([trial - 1, 40 * trial - 1], dtype=torch.int32,
                                                                            device="cuda"))
        q.normal_(generator=None)
        want, want2 = torch.empty_like(out), torch.empty_like(out)
        step(want)
        xkv.xkv_kv8_attention_decode(b.p, b.c, after, q2, want2)
        out.fill_(float("nan"))
        other.fill_(float("nan"))
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want2)
    assert xkv.get_device_status() == 0


@pytest.mark.parametrize("raw", [False, True])
def test_a_call_on_another_stream_takes_its_workspace_there(xkv, raw):
    # the call's own workspace goes back when the call returns, long before it has run: what the current stream
    # allocates meanwhile is other memory
    b, g = _fill(xkv, 2, 2, 128, 64, 4096, [4000, 333])
    q = torch.randn((2, 8, 128), generator=g).to(torch.bfloat16).cuda()
    want, lens = _attend(b, q), b.dev_lens()
    out = torch.full_like(want, float("nan"))
    n = xkv.xkv_kv8_workspace_size(b.p, 8)
    s, x = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    torch.empty(n, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(s):
        torch.empty(n, dtype=torch.uint8, device="cuda")
        x = torch.clamp(x @ x, -1, 1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(40):
            x = torch.clamp(x @ x, -1, 1)
    xkv.xkv_kv8_attention_decode(b.p, b.c, lens, q, out, stream=s.cuda_stream if raw else s)
    for _ in range(200):
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    assert not s.query()  # the call was still to run
    torch.cuda.synchronize()
    assert torch.equal(out, want) and xkv.get_device_status() == 0


def _chain(xkv, seed, steps, wait):
    """Steps of append, attention with weights and eviction, one behind the other; every output and the last cache."""
    B, H, gq, hd, block, budget = 5, 2, 8, 64, 16, 9
    g = torch.Generator().manual_seed(seed)
    b, _ = _fill(xkv, B, H, hd, block, 192, [100, 1, 40, 144, 0], seed=seed)
    k = torch.randn((steps, B, 3, H * hd), generator=g).to(torch.bfloat16).cuda()
    q = torch.randn((steps, B, H * gq, hd), generator=g).to(torch.bfloat16).cuda()
    outs = torch.full((steps, B, H * gq, hd), float("nan"), device="cuda")
    ws = xkv.workspace(xkv.xkv_kv8_workspace_size(b.p, H * gq))
    lens, after = b.dev_lens(), torch.empty(B, dtype=torch.int32, device="cuda")
    b.c.weight.nan_to_num_()
    torch.cuda.synchronize()
    for i in range(steps):
        for call in (lambda: xkv.xkv_kv8_append(b.p, b.c, lens, k[i], k[i].flip(0)), lambda: lens.add_(3),
                     lambda: xkv.xkv_kv8_attention_decode(b.p, b.c, lens, q[i], outs[i], accumulate=True, ws=ws),
                     lambda: xkv.xkv_kv8_evict(b.p, b.c, lens, budget, 1, 2, after), lambda: lens.copy_(after)):
            call()
            if wait:
                torch.cuda.synchronize()
    return [outs, lens, b.c.k.view(torch.uint8), b.c.v.view(torch.uint8), b.c.k_scale, b.c.weight, b.c.ids]


def test_calls_behind_one_another_and_side_by_side(xkv):
    # nothing waits between the calls, which prepare themselves while the one before still runs; then two such runs
    # on streams of their own
    want = [[t.clone() for t in _chain(xkv, seed, 60, True)] for seed in (1, 2)]
    for got, ref_ in ((_chain(xkv, 1, 60, False), want[0]), (_chain(xkv, 2, 60, False), want[1])):
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, ref_))
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s, seed in zip(streams, (1, 2)):
        with torch.cuda.stream(s):
            got.append(_chain(xkv, seed, 60, False))
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(x, y))
    assert xkv.get_device_status() == 0


def test_a_replaced_tensor_is_read_and_written(xkv):
    # sequences in another order, and weights started anew
    b, g = _fill(xkv, 3, 2, 64, 16, 256, [200, 0, 77])
    q = torch.randn((3, 8, 64), generator=g).to(torch.bfloat16).cuda()
    b.c.weight.zero_()
    want, weight = _attend(b, q, accumulate=True), b.c.weight.clone()
    order = torch.tensor([2, 0, 1], device="cuda")
    old = b.c.weight
    for x in ("k", "v"):
        setattr(b.c, x, getattr(b.c, x).view(torch.uint8)[order].view(F8))
    for x in ("k_scale", "v_scale", "ids"):
        setattr(b.c, x, getattr(b.c, x)[order])
    b.c.weight = torch.zeros_like(old)
    b.lens = [b.lens[i] for i in order.tolist()]
    assert torch.equal(_attend(b, q[order], accumulate=True), want[order])
    assert torch.equal(b.c.weight, weight[order]) and torch.equal(old, weight)


def test_binding_refuses_what_the_library_cannot_see(xkv):
    b, g = _fill(xkv, 2, 2, 64, 16, 64, [10, 20])
    q, out = torch.zeros((2, 4, 64), device="cuda"), torch.empty((2, 4, 64), device="cuda")
    lens, rows = b.dev_lens(), torch.zeros((2, 3, 128), device="cuda")
    att, app, ev = xkv.xkv_kv8_attention_decode, xkv.xkv_kv8_append, xkv.xkv_kv8_evict
    for call in (lambda: att(b.p, b.c, lens.long(), q, out), lambda: att(b.p, b.c, lens[:1], q, out),
                 lambda: att(b.p, b.c, lens.cpu(), q, out), lambda: att(b.p, b.c, lens, q[:1], out[:1]),
                 lambda: att(b.p, b.c, lens, q[..., :32], out[..., :32]), lambda: att(b.p, b.c, lens, q, out.half()),
                 lambda: att(b.p, b.c, lens, q.half(), out), lambda: att(b.p, b.c, lens, q.cpu(), out),
                 lambda: att(xkv.kv8_params(2, 2, 64, 16, 128), b.c, lens, q, out),
                 lambda: att(xkv.kv8_params(2, 2, 64, 32, 64), b.c, lens, q, out),
                 lambda: att(b.p, b.c, lens, q.transpose(0, 1).contiguous().transpose(0, 1), out),
                 lambda: app(b.p, b.c, lens, rows, rows.bfloat16()), lambda: app(b.p, b.c, lens, rows, rows[:, :2]),
                 lambda: app(b.p, b.c, lens, rows[:1], rows[:1]), lambda: app(b.p, b.c, lens, rows.cpu(), rows.cpu()),
                 lambda: app(b.p, b.c, lens, rows, rows, counts=lens.float()),
                 lambda: app(b.p, b.c, lens, rows.transpose(1, 2).contiguous().transpose(1, 2), rows),
                 lambda: ev(b.p, b.c, lens, 2, 0, 1, lens.long())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(xkv.XKVError):
        ev(b.p, b.c, lens, 2, 0, 1, lens)
    with pytest.raises(xkv.XKVError):
        att(b.p, b.c, lens, q, out, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
