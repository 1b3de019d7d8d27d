"""The cases that the 8-bit KV cache's operators are measured on: writing K and V rows into the cache (append), single-token
attention over it (attend), and eviction of whole blocks by accumulated attention weight (evict).

A cache holds, for every (sequence, KV head), `capacity` token rows of K and of V as e4m3 codes, and one power-of-two f32 scale
for each block of tokens.  Lengths are on the device, one for each sequence.  With `own` false, run() computes each operator in
its plain form, elementary torch operations in 32 bits; with `own` true it makes the calls a user makes of the framework."""
import math

import torch

own = False

E_MIN = -117  # the least exponent of a scale: 2^-117 times e4m3's least code 2^-9 is the least normal f32


def listed():
    a, t, e = {"op": "append"}, {"op": "attend"}, {"op": "evict"}
    return [
        # one generated token for each of 32 sequences: the smallest call of a decode step
        dict(a, name="append_token_b32", dtype="bf16", B=32, Hkv=8, hd=128, block=64, n=1, held=2000, ragged=True),
        # a padded batch of f32 rows joining part-filled blocks: ragged counts, small heads and blocks
        dict(a, name="append_f32_ragged", dtype="f32", B=6, Hkv=3, hd=64, block=16, n=777, held=333, ragged=True),
        # the prompts of the 64K-token, batch-4 decode workload
        dict(a, name="append_prompt_64k_b4", dtype="bf16", B=4, Hkv=8, hd=128, block=64, n=65536, held=0, ragged=False),
        # the smallest attention call: one short sequence, where latency counts
        dict(t, name="attend_short", dtype="bf16", B=1, Hkv=8, gq=4, hd=128, block=64, T=513, ragged=False, weight=False),
        # a serving batch of ragged sequences, from single tokens to 8K, accumulating weights
        dict(t, name="attend_ragged_b48", dtype="bf16", B=48, Hkv=4, gq=8, hd=64, block=32, T=8192, ragged=True, weight=True),
        # f32 queries of a model without grouped heads, odd length and head size
        dict(t, name="attend_f32_mha", dtype="f32", B=2, Hkv=12, gq=1, hd=96, block=8, T=10007, ragged=True, weight=False),
        # the 128K-token, batch-2 workload with seven query heads to a KV head, accumulating weights
        dict(t, name="attend_128k_b2", dtype="bf16", B=2, Hkv=4, gq=7, hd=128, block=128, T=131071, ragged=False, weight=True),
        # the 64K-token, batch-4 workload: the largest call
        dict(t, name="attend_64k_b4", dtype="bf16", B=4, Hkv=8, gq=4, hd=128, block=64, T=65536, ragged=False, weight=False),
        # wide heads shared by sixteen query heads
        dict(t, name="attend_wide_hd256", dtype="bf16", B=8, Hkv=1, gq=16, hd=256, block=64, T=20000, ragged=True, weight=True),
        # eviction of a few small blocks from one short sequence
        dict(e, name="evict_small", B=1, Hkv=2, hd=64, block=8, T=1021, budget=96, sink=1, recent=4, ragged=False),
        # a batch cut from 16K to 8K tokens
        dict(e, name="evict_16k_b4", B=4, Hkv=8, hd=128, block=64, T=16384, budget=128, sink=1, recent=8, ragged=False),
        # ragged long sequences cut to 24K tokens; those below it stay
        dict(e, name="evict_ragged_b16", B=16, Hkv=4, hd=128, block=32, T=40000, budget=768, sink=2, recent=16, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict"])
    c = {"op": op, "B": _log(rng, 1, 48), "Hkv": rng.choice([1, 2, 3, 4, 6, 8, 10]), "hd": rng.choice([16, 48, 64, 80, 96, 128, 128, 192, 256]),
         "block": rng.choice([8, 16, 32, 64, 128]), "ragged": rng.random() < 0.6}
    row = c["B"] * c["Hkv"] * c["hd"]  # elements of K of one token of all sequences
    if op == "append":
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        c["held"] = rng.choice([0, rng.randint(1, 200), _log(rng, 1, 4000)])
        c["n"] = 1 if rng.random() < 0.3 else _log(rng, 1, max(2, min(65536, (1 << 26) // row)))
    elif op == "attend":
        c["dtype"], c["gq"] = rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        c["T"] = _log(rng, 1, max(2, min(131072, (1 << 27) // row)))
        c["weight"] = rng.random() < 0.5
    else:
        c["T"] = _log(rng, 4 * c["block"], max(8 * c["block"], min(65536, (1 << 27) // row)))
        n = -(-c["T"] // c["block"])
        c["recent"], c["sink"] = rng.randint(1, max(1, n // 8)), rng.randint(0, max(1, n // 8))
        c["budget"] = rng.randint(max(c["recent"] + c["sink"], n // 4), max(c["recent"] + c["sink"], n - 1))
    return c


# ------------------------------------------------------------------ inputs
def _lens(case, most, least, seed):
    """One length for each sequence: `most`, or spread evenly over the logarithm from `least` to `most` in an order of the seed's."""
    B = case["B"]
    if not case["ragged"]:
        return [most] * B
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(B, generator=g).tolist()
    v = [int(round(math.exp(math.log(max(1, least)) + x * (math.log(max(1, most)) - math.log(max(1, least)))))) for x in u]
    at = int(torch.randint(B, (1,), generator=g))
    v[at] = most
    if B > 2 and least == 0:
        v[at - 1] = 0  # a sequence with nothing in it
    return [min(most, x) for x in v]


def _exponent(a):
    """The least e >= E_MIN with a <= 448 2^e, for finite a >= 0 (frexp: a = m 2^x, m in [0.5, 1); 448 = 0.875 2^9)."""
    m, x = torch.frexp(a)
    e = x - 9 + (m > 0.875).to(torch.int32)
    return torch.where(a > 0, e, torch.full_like(e, E_MIN)).clamp(min=E_MIN)


def _pow2(e):
    return ((e + 127) << 23).view(torch.float32)


def _rows(g, shape, dt, chan):
    """Rows of keys or values: normal, with channels of unlike size as trained models have them, and a slow drift over the tokens."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    t = torch.arange(shape[1], device="cuda", dtype=torch.float32)
    x *= chan
    x *= (1.0 + 0.5 * torch.sin(t * 0.013))[None, :, None, None]
    return x.to(dt)


def _filled(case, tokens, capacity, g):
    """A cache that holds `tokens` rows of every sequence, and bytes of no meaning behind them."""
    B, H, hd, block = case["B"], case["Hkv"], case["hd"], case["block"]
    c = {}
    nb = -(-tokens // block)
    for x in ("k", "v"):
        codes = torch.randint(0, 256, (B, H, capacity, hd), generator=g, device="cuda", dtype=torch.uint8)
        scale = torch.ones((B, H, capacity // block), device="cuda")
        chan = torch.exp(0.5 * torch.randn((H, hd), generator=g, device="cuda"))
        for b in range(B):
            if nb:
                r = _rows(g, (1, nb * block, H, hd), torch.float32, chan)[0].permute(1, 0, 2).reshape(H, nb, block, hd)
                s = _pow2(_exponent(r.abs().amax((2, 3))))
                scale[b, :, :nb] = s
                codes[b, :, :nb * block] = (r / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(H, nb * block, hd)
        c[x], c[x + "_scale"] = codes.view(torch.float8_e4m3fn), scale
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, hd, block = case["B"], case["Hkv"], case["hd"], case["block"]
    s = {"case": case}
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}.get(case.get("dtype"))
    if case["op"] == "append":
        n, held = case["n"], case["held"]
        lens = _lens(case, held, 1, seed) if held else [0] * B
        counts = _lens(case, n, 0, seed + 1)
        capacity = -(-(held + n) // block) * block + block
        s |= _filled(case, held, capacity, g)
        chan = torch.exp(0.5 * torch.randn((H, hd), generator=g, device="cuda"))
        for x in ("k", "v"):  # what stands behind a sequence's last row is finite there, so that outputs can be compared
            live = torch.arange(capacity, device="cuda")[None, :] < torch.tensor(lens, device="cuda")[:, None]
            s[x].view(torch.uint8).mul_(live[:, None, :, None])
            s[x + "_new"] = _rows(g, (B, n, H, hd), dt, chan).reshape(B, n, H * hd)
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda") if case["ragged"] else None
    elif case["op"] == "attend":
        lens = _lens(case, case["T"], 0, seed)
        capacity = -(-case["T"] // block) * block
        s |= _filled(case, case["T"], capacity, g)
        for x in ("k", "v"):  # NaN codes behind the last row, as a reused buffer may hold
            live = torch.arange(capacity, device="cuda")[None, :] < torch.tensor(lens, device="cuda")[:, None]
            s[x].view(torch.uint8).masked_fill_(~live[:, None, :, None], 0x7F)
        s["q"] = (2.0 * torch.randn((B, H * case["gq"], hd), generator=g, device="cuda")).to(dt)
        s["out"] = torch.empty((B, H * case["gq"], hd), dtype=torch.float32, device="cuda")
    else:
        lens = _lens(case, case["T"], case["T"] // 4, seed)
        capacity = -(-case["T"] // block) * block
        s |= _filled(case, case["T"], capacity, g)
        for x in ("k", "v"):
            live = torch.arange(capacity, device="cuda")[None, :] < torch.tensor(lens, device="cuda")[:, None]
            s[x].view(torch.uint8).mul_(live[:, None, :, None])
        s["lens_out"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # weights and block numbers in one buffer, so that one copy puts both back
    nblk = s["k_scale"].shape[2]
    s["meta"] = torch.empty((2, B, H, nblk), dtype=torch.int32, device="cuda")
    s["weight"], s["ids"] = s["meta"][0].view(torch.float32), s["meta"][1]
    # the attention that blocks have had is heavy-tailed; a step's own is measured on an accumulator that starts at zero
    s["weight"].copy_(torch.exp(1.5 * torch.randn((B, H, nblk), generator=g, device="cuda")))
    if case["op"] == "attend":
        s["weight"].zero_()
    s["ids"].copy_(torch.arange(nblk, device="cuda", dtype=torch.int32).expand(B, H, nblk))
    s["meta0"] = s["meta"].clone()
    if own:
        import cross_layer_rank_b200 as xkv
        s["p"] = xkv.kv8_params(B, H, hd, block, s["k"].shape[2])
        s["cache"] = xkv.KV8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["weight"], s["ids"])
        if case["op"] == "attend":
            s["ws"] = xkv.workspace(xkv.xkv_kv8_workspace_size(s["p"], H * case["gq"]))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if op == "append":
        return _append_own(s) if own else _append_plain(s)
    if op == "attend":
        return _attend_own(s) if own else _attend_plain(s)
    # a pass changes weights and block numbers: put those of the step back, so that every pass has the same blocks to move
    s["meta"].copy_(s["meta0"])
    return _evict_own(s) if own else _evict_plain(s)


def _append_out(s):
    return {x: s[x] for x in ("k", "v", "k_scale", "v_scale", "weight", "ids")}


def _append_own(s):
    import cross_layer_rank_b200 as xkv
    xkv.xkv_kv8_append(s["p"], s["cache"], s["lens"], s["k_new"], s["v_new"], s["counts"])
    return _append_out(s)


def _append_plain(s):
    c = s["case"]
    B, H, hd, block, n = c["B"], c["Hkv"], c["hd"], c["block"], c["n"]
    lens = s["lens"].long()
    counts = s["counts"].long() if s["counts"] is not None else torch.full_like(lens, n)
    nb = (n + block - 2) // block + 1  # blocks that n rows can touch
    blk = lens[:, None] // block + torch.arange(nb, device="cuda")
    i = blk[:, :, None] * block + torch.arange(block, device="cuda") - lens[:, None, None]  # row of the call, [B, nb, block]
    new = (i >= 0) & (i < counts[:, None, None])
    touched = new.any(2)
    blk = torch.minimum(blk, torch.full_like(blk, s["k_scale"].shape[2] - 1))  # past the last block nothing is touched
    bi = torch.arange(B, device="cuda")[:, None]
    started = touched & (blk * block < lens[:, None])  # held rows before
    for x in ("k", "v"):
        rows = s[x + "_new"].view(B, n, H, hd)[bi[:, :, None], i.clamp(0, n - 1)].float()  # [B, nb, block, H, hd]
        a = torch.where(new[..., None, None] & torch.isfinite(rows), rows.abs(), 0.0).amax((2, 4))  # [B, nb, H]
        scale = s[x + "_scale"].permute(0, 2, 1)[bi, blk]  # [B, nb, H]
        need = _pow2(_exponent(a))
        now = torch.where(started[..., None], torch.maximum(need, scale), need)
        now = torch.where(touched[..., None], now, scale)
        codes = s[x].view(B, H, -1, block, hd).permute(0, 2, 3, 1, 4)
        old = codes.view(torch.uint8)[bi, blk].view(torch.float8_e4m3fn)
        kept = (old.float() * (scale / now)[:, :, None, :, None]).to(torch.float8_e4m3fn)
        made = (rows / now[:, :, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        grown = started[:, :, None] & (i < 0)
        both = torch.where(new[..., None, None], made.view(torch.uint8),
                           torch.where(grown[..., None, None], kept.view(torch.uint8), old.view(torch.uint8)))
        both = torch.where(touched[:, :, None, None, None], both, old.view(torch.uint8))
        codes.view(torch.uint8)[bi, blk] = both
        s[x + "_scale"].permute(0, 2, 1)[bi, blk] = now
    opened = (touched & ~started)[..., None]
    before = torch.where(lens > 0, (lens + block - 1) // block, torch.zeros_like(lens))  # blocks in use
    last = s["ids"].permute(0, 2, 1)[bi[:, 0], (before - 1).clamp(min=0)]  # [B, H]
    first = torch.where(before[:, None] > 0, last + 1, torch.zeros_like(last))
    ids = first[:, None, :] + (blk - before[:, None])[..., None].to(torch.int32)
    s["ids"].permute(0, 2, 1)[bi, blk] = torch.where(opened, ids, s["ids"].permute(0, 2, 1)[bi, blk])
    s["weight"].permute(0, 2, 1)[bi, blk] = torch.where(opened, 0.0, s["weight"].permute(0, 2, 1)[bi, blk])
    return _append_out(s)


def _attend_own(s):
    import cross_layer_rank_b200 as xkv
    xkv.xkv_kv8_attention_decode(s["p"], s["cache"], s["lens"], s["q"], s["out"], accumulate=s["case"]["weight"], ws=s["ws"])
    return {"out": s["out"], "weight": s["weight"]} if s["case"]["weight"] else s["out"]


def _attend_plain(s):
    c = s["case"]
    B, H, hd, block, gq = c["B"], c["Hkv"], c["hd"], c["block"], c["gq"]
    nb = -(-c["T"] // block)
    live = torch.arange(nb * block, device="cuda")[None, :] < s["lens"][:, None]  # [B, T]

    def values(x):
        w = s[x][:, :, :nb * block].float().view(B, H, nb, block, hd) * s[x + "_scale"][:, :, :nb, None, None]
        return torch.where(live[:, None, :, None], w.view(B, H, nb * block, hd), 0.0)

    q = s["q"].float().view(B, H, gq, hd)
    logit = torch.matmul(q, values("k").transpose(2, 3)) / math.sqrt(hd)  # [B, H, gq, T]
    logit = torch.where(live[:, None, None, :], logit, -math.inf)
    top = logit.amax(3, keepdim=True)
    p = torch.exp(logit - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(3, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    s["out"].copy_(torch.matmul(p, values("v")).view(B, H * gq, hd))
    if not c["weight"]:
        return s["out"]
    s["weight"][:, :, :nb] += p.sum(2).view(B, H, nb, block).sum(3)
    return {"out": s["out"], "weight": s["weight"]}


def _evict_out(s):
    return {x: s[x] for x in ("k", "v", "k_scale", "v_scale", "weight", "ids", "lens_out")}


def _evict_own(s):
    import cross_layer_rank_b200 as xkv
    c = s["case"]
    xkv.xkv_kv8_evict(s["p"], s["cache"], s["lens"], c["budget"], c["sink"], c["recent"], s["lens_out"])
    return _evict_out(s)


def _evict_plain(s):
    c = s["case"]
    B, H, hd, block, budget = c["B"], c["Hkv"], c["hd"], c["block"], c["budget"]
    nblk = s["ids"].shape[2]
    lens = s["lens"].long()
    n = (lens + block - 1) // block
    slot = torch.arange(nblk, device="cuda")
    held = (slot < n[:, None])[:, None]  # [B, 1, nblk]
    last = s["ids"].gather(2, (n - 1).clamp(min=0)[:, None, None].expand(B, H, 1))
    safe = ((s["ids"] < c["sink"]) | (s["ids"] > last - c["recent"]) | (slot == (n - 1)[:, None])[:, None]) & held
    key = torch.where(safe, math.inf, torch.where(held, s["weight"].double(), -math.inf))
    rank = torch.argsort(torch.argsort(key, dim=2, descending=True, stable=True), dim=2)
    keep = (rank < budget) & held
    low = slot < budget - 1
    moves = keep & ~low
    free = (low & ~keep) | (slot == budget - 1)
    source = torch.argsort((~moves).to(torch.int8), dim=2, stable=True)  # the moving blocks, ascending, come first
    source = source.gather(2, (free.long().cumsum(2) - 1).clamp(min=0))
    source = torch.where(free & (n > budget)[:, None, None], source, slot)[:, :, :budget]  # [B, H, budget]
    for x in ("k", "v"):
        codes = s[x].view(torch.uint8).view(B, H, nblk, block * hd)
        codes[:, :, :budget] = codes.gather(2, source[..., None].expand(B, H, source.shape[2], block * hd))
    for x in ("k_scale", "v_scale", "weight", "ids"):
        s[x][:, :, :budget] = s[x].gather(2, source)
    s["lens_out"].copy_(torch.where(n > budget, lens - (n - budget) * block, lens))
    return _evict_out(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    B, H, hd, block = case["B"], case["Hkv"], case["hd"], case["block"]
    # the mean length of lengths spread evenly over the logarithm from lo to hi
    mean = lambda lo, hi: (hi - lo) / math.log(hi / lo) if case["ragged"] and hi > lo else hi  # noqa: E731
    if case["op"] == "append":
        rows = B * mean(1, case["n"]) * H * hd
        el = 2 if case["dtype"] == "bf16" else 4
        blocks = B * H * max(1.0, mean(1, case["n"]) / block)
        return {"bytes": 2 * rows * (el + 1) + blocks * 16, "flops": 4 * rows}
    if case["op"] == "attend":
        tokens = B * mean(1, case["T"]) * H
        el = 2 if case["dtype"] == "bf16" else 4
        q = B * H * case["gq"] * hd
        return {"bytes": 2 * tokens * hd + 8 * tokens / block + q * (el + 4) + (8 * tokens / block if case["weight"] else 0),
                "flops": 4 * tokens * case["gq"] * hd}
    # every unit's block weights are read; of the blocks above the budget, those kept are read and written
    moved = read = 0.0
    for i in range(64):
        t = case["T"] * 4.0 ** (-(i + 0.5) / 64) if case["ragged"] else case["T"]
        n = -(-int(t) // block)
        cut = max(0, n - case["budget"])
        fresh = min(cut, case["recent"])
        moved += B * H * (fresh + (cut - fresh) * case["budget"] / n) / 64
        read += B * H * n / 64
    return {"bytes": moved * (2 * 2 * block * hd + 32) + read * 8, "flops": read}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _append_exact, "attend": _attend_exact, "evict": _evict_exact}[case["op"]](s, case)


def _e4m3(x):
    """float64 values to the nearest e4m3 number, ties to even: steps of 2^(floor(log2|x|) - 3), and of 2^-9 below 2^-6."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    step = torch.where(a / step < 8, step / 2, torch.where(a / step >= 16, step * 2, step)).clamp(min=2.0 ** -9)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _append_exact(s, c):
    H, hd, block = c["Hkv"], c["hd"], c["block"]
    got = {x: s[x].double() for x in ("k", "v", "k_scale", "v_scale", "weight")} | {"ids": s["ids"].clone()}
    lens = s["lens"].tolist()
    counts = s["counts"].tolist() if s["counts"] is not None else [c["n"]] * c["B"]
    for b in range(c["B"]):
        lo, hi = lens[b], lens[b] + counts[b]
        first, past = lo // block, -(-hi // block)
        for x in ("k", "v"):
            new = s[x + "_new"][b, :counts[b]].double().view(counts[b], H, hd).permute(1, 0, 2)
            buf = torch.zeros((H, (past - first) * block, hd), dtype=torch.float64, device="cuda")
            buf[:, lo - first * block:hi - first * block] = new
            most = buf.view(H, past - first, block * hd).abs().amax(2)
            # the least power of two that is not below most / 448
            e = torch.ceil(torch.log2(most.clamp(min=1e-300) / 448.0))
            e = torch.where(torch.exp2(e) * 448.0 < most, e + 1, e)
            e = torch.where(torch.exp2(e - 1) * 448.0 >= most, e - 1, e).clamp(min=float(E_MIN))
            scale = torch.exp2(e)
            head = lo - first * block
            if head:  # the part-filled block keeps the larger of its scale and the new one
                was = got[x + "_scale"][b, :, first]
                scale[:, 0] = torch.maximum(scale[:, 0], was)
                ratio = (was / scale[:, 0])[:, None, None]
                got[x][b, :, first * block:lo] = _e4m3(got[x][b, :, first * block:lo] * ratio)
            codes = _e4m3(buf.view(H, past - first, block, hd) / scale[:, :, None, None]).view(H, -1, hd)
            got[x][b, :, lo:hi] = codes[:, head:head + counts[b]]
            got[x + "_scale"][b, :, first:past] = scale
        begin = -(-lo // block)
        if past > begin:
            at = got["ids"][b, :, begin - 1] + 1 if begin else torch.zeros(H, dtype=torch.int32, device="cuda")
            got["ids"][b, :, begin:past] = at[:, None] + torch.arange(past - begin, dtype=torch.int32, device="cuda")
            got["weight"][b, :, begin:past] = 0.0
    return got


def _attend_exact(s, c):
    H, hd, block, gq = c["Hkv"], c["hd"], c["block"], c["gq"]
    out = torch.zeros((c["B"], H * gq, hd), dtype=torch.float64, device="cuda")
    weight = s["weight"].double()
    for b, t in enumerate(s["lens"].tolist()):
        nb = -(-t // block)
        for h in range(H):
            kv = [s[x][b, h, :t].double() * s[x + "_scale"][b, h, :nb].double().repeat_interleave(block)[:t, None] for x in ("k", "v")]
            p = torch.softmax(kv[0] @ s["q"][b, h * gq:(h + 1) * gq].double().T / hd ** 0.5, 0)  # [t, gq]
            out[b, h * gq:(h + 1) * gq] = p.T @ kv[1]
            weight[b, h].index_add_(0, torch.arange(t, device="cuda") // block, p.sum(1))
    return {"out": out, "weight": weight} if c["weight"] else out


def _evict_exact(s, c):
    block, budget = c["block"], c["budget"]
    got = {x: s[x].double() for x in ("k", "v", "k_scale", "v_scale", "weight")} | {"ids": s["ids"].clone()}
    lens, lens_out = s["lens"].tolist(), []
    weights, numbers = s["weight"].double().cpu().tolist(), s["ids"].cpu().tolist()
    for b, t in enumerate(lens):
        n = -(-t // block)
        lens_out.append(t if n <= budget else t - (n - budget) * block)
        for h in range(c["Hkv"] if n > budget else 0):
            w, num = weights[b][h], numbers[b][h]
            safe = lambda i: num[i] < c["sink"] or num[i] > num[n - 1] - c["recent"] or i == n - 1  # noqa: E731
            keep = sorted(sorted(range(n), key=lambda i: (not safe(i), -w[i], i))[:budget])
            stay = {i for i in keep if i < budget - 1}
            src = [i for i in keep if i >= budget - 1]
            dst = [i for i in range(budget) if i not in stay]
            i, j = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
            for x in ("k", "v"):
                v = got[x][b, h].view(-1, block * c["hd"])
                v[j] = v[i].clone()
            for x in ("k_scale", "v_scale", "weight", "ids"):
                got[x][b, h, j] = got[x][b, h, i].clone()
    return got | {"lens_out": torch.tensor(lens_out, dtype=torch.int32, device="cuda")}
