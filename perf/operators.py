"""Cases of the serving operators for 8-bit and windowed caches, with their plain forms.

Four operators of the verify step, by `case["op"]`:

  kv8      verify attention over a paged cache held in e4m3 with one float32 scale for each block of 64 tokens and KV
           head, after quantising the verify tokens' own K/V into it (mtp_verify_attention_kv8)
  window   verify attention over the bf16 (or float32) cache in which a row sees the last `window` positions and the
           first `sinks` tokens (mtp_verify_attention_window)
  append   quantising a ragged batch of new K/V (prefill chunks, accepted tokens) into the 8-bit cache (mtp_kv8_append)
  release  returning the blocks that have left the window to the free list (kv_window_release)

The quantisation, which has to agree to the bit: with a the largest finite |x| that a call writes into a block's head,
a block whose first slot the call writes gets the scale s = 2^e with the smallest e >= -100 for which a <= 448 s; any
other block's scale s is doubled until a <= 448 s, and the bytes before the written ones are rounded again to
(value * old s / new s). A byte is e4m3(x / s), to nearest even; what is not finite becomes NaN.
"""
import math

import torch

own = False

BLOCK = 64
MIN_EXP = -100


# ------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's greedy decode with one draft: latency
        dict(name="kv8 one request", op="kv8", B=1, D=1, Hq=32, Hkv=8, d=128, lo=997, hi=997, window=0, sinks=0, t="bf16"),
        # the tiny fp32 workload (SIMT path)
        dict(name="kv8 tiny fp32", op="kv8", B=4, D=3, Hq=8, Hkv=8, d=64, lo=128, hi=128, window=0, sinks=0, t="f32"),
        # Llama-70B-shaped heads, 5 drafts, 64 requests of 4096 tokens: many query rows a KV head
        dict(name="kv8 70B-shaped", op="kv8", B=64, D=5, Hq=64, Hkv=8, d=128, lo=4096, hi=4096, window=0, sinks=0, t="bf16"),
        # a large mixed batch with contexts of 1k to 32k tokens
        dict(name="kv8 mixed 1k-32k", op="kv8", B=64, D=3, Hq=32, Hkv=8, d=128, lo=1024, hi=32768, window=0, sinks=0, t="bf16"),
        # an 8-bit cache with a window, odd sizes, head dim 64 and the most drafts
        dict(name="kv8 windowed odd", op="kv8", B=5, D=15, Hq=12, Hkv=4, d=64, lo=100, hi=5000, window=333, sinks=7, t="bf16"),
        # one long conversation behind a window: latency
        dict(name="window one request", op="window", B=1, D=3, Hq=32, Hkv=8, d=128, lo=32768, hi=32768, window=4096, sinks=4, t="bf16"),
        # an ordinary batch, 48 query rows a KV head, no sinks
        dict(name="window 70B-shaped", op="window", B=16, D=5, Hq=64, Hkv=8, d=128, lo=500, hi=8192, window=1000, sinks=0, t="bf16"),
        # the large mixed batch behind a window
        dict(name="window mixed 1k-32k", op="window", B=256, D=3, Hq=32, Hkv=8, d=128, lo=1024, hi=32768, window=4096, sinks=4, t="bf16"),
        # a step's accepted tokens of a decode batch
        dict(name="append decode", op="append", B=33, Hkv=8, d=128, lo=0, hi=2000, nlo=0, nhi=16, t="bf16"),
        # prefill chunks of a batch
        dict(name="append prefill", op="append", B=64, Hkv=8, d=128, lo=0, hi=3000, nlo=500, nhi=1500, t="bf16"),
        # the blocks that a small and a large batch give back after prefill
        dict(name="release 16", op="release", B=16, lo=100, hi=8192, window=1024, sinks=4),
        dict(name="release 512", op="release", B=512, lo=1024, hi=131072, window=4096, sinks=100),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kv8", "kv8", "window", "window", "append", "release"])
    if op == "release":
        hi = _between(rng, 200, 131072)
        return dict(op=op, B=_between(rng, 1, 512), lo=rng.randint(1, hi), hi=hi, window=_between(rng, 1, 8192),
                    sinks=rng.choice([0, 1, 4, 64, 100]))
    d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 8, 16])
    t = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append":
        B = _between(rng, 1, 128)
        nhi = _between(rng, 1, 65536 // B)
        return dict(op=op, B=B, Hkv=Hkv if Hkv < 16 else 8, d=d, lo=0, hi=_between(rng, 1, 4096), nlo=rng.randint(min(1, nhi // 2), nhi), nhi=max(2, nhi), t=t)
    group, D = rng.choice([1, 2, 3, 4, 7, 8]), rng.randint(0, 15)
    budget = 30e6 if t == "f32" else 1.0e9   # keys of all requests x KV heads x head dim
    B = _between(rng, 1, 128)
    hi = _between(rng, 1, max(1, min(32768, int(budget / (B * Hkv * d)))))
    lo = rng.choice([hi, rng.randint(0, hi)])
    sinks = rng.choice([0, 1, 4, 64, 100])
    window = _between(rng, 1, 8192) if op == "window" or rng.random() < 0.3 else 0
    return dict(op=op, B=B, D=D, Hq=group * Hkv, Hkv=Hkv, d=d, lo=lo, hi=hi, window=window, sinks=sinks if window else 0, t=t)


# ------------------------------------------------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _spread(lo, hi, n):
    """n lengths spread evenly from lo to hi."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * n) for i in range(n)]


def _lens(lo, hi, n, gen):
    """The same in an order of the seed's: what a case reads and computes is the same for every seed."""
    return torch.tensor(_spread(lo, hi, n))[torch.randperm(n, generator=gen)]


def _tables(first_free, need, max_blocks, num_blocks, gen, device):
    """Block tables in which request b has the entries 0 .. need[b]-1 except first_free[b][0] .. first_free[b][1]-1, in
    random physical order."""
    i = torch.arange(max_blocks)
    a, z = first_free
    has = (i < need[:, None]) & ~((i >= a[:, None]) & (i < z[:, None]))
    used = int(has.sum())
    perm = torch.randperm(num_blocks, generator=gen)
    table = torch.full((len(need), max_blocks), -1, dtype=torch.int64)
    table[has] = perm[:used]
    return table.to(torch.int32).to(device)


def _normal(shape, gen, device, dtype, times=1.0):
    out = torch.empty(shape, dtype=dtype, device=device)
    flat = out.reshape(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = torch.randn(min(1 << 28, flat.numel() - i), generator=gen, device=device)
        flat[i:i + part.numel()] = (part * times).to(dtype)
    return out


def _scales(num_blocks, Hkv, gen, device):
    """What caches quantised from unit normal values have: 2^-6, some blocks and heads larger or smaller."""
    return torch.exp2(torch.randint(-7, -4, (num_blocks, Hkv), generator=gen, device=device).float())


def _cache8(num_blocks, Hkv, d, gen, device):
    k = _normal((num_blocks, BLOCK, Hkv, d), gen, device, torch.float8_e4m3fn, 64.0)
    v = _normal((num_blocks, BLOCK, Hkv, d), gen, device, torch.float8_e4m3fn, 64.0)
    return dict(k_cache=k, v_cache=v, k_scale=_scales(num_blocks, Hkv, gen, device), v_scale=_scales(num_blocks, Hkv, gen, device))


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    op, B = case["op"], case["B"]
    s = dict(case=case, op=op)
    zero = torch.zeros(B, dtype=torch.int64)
    if op == "release":
        lens = _lens(case["lo"], case["hi"], B, host)
        s["window"], s["sinks"] = case["window"], case["sinks"]
        max_blocks = -(-(case["hi"] + 16) // BLOCK)
        need = (lens + 16 + BLOCK - 1) // BLOCK
        num_blocks = int(need.sum()) + 4
        s["table0"] = _tables((zero, zero), need, max_blocks, num_blocks, host, device)
        s["table"] = s["table0"].clone()
        s["seq_lens"] = lens.to(torch.int32).to(device)
        s["free_list0"] = torch.full((num_blocks,), -1, dtype=torch.int32, device=device)
        s["free_list0"][:4] = torch.arange(4, dtype=torch.int32, device=device)
        s["free_list"] = s["free_list0"].clone()
        s["free_count"] = torch.full((1,), 4, dtype=torch.int32, device=device)
        return s
    Hkv, d, dtype = case["Hkv"], case["d"], _TYPES[case["t"]]
    ctx = _lens(case["lo"], case["hi"], B, host)
    if op == "append":
        n = _lens(case["nlo"], case["nhi"], B, host)
        max_blocks = -(-(case["hi"] + case["nhi"]) // BLOCK)
        need = (ctx + n + BLOCK - 1) // BLOCK
        # the whole cache of such a program, of which a call touches the written blocks
        num_blocks = B * max_blocks
        s["table"] = _tables((zero, zero), need, max_blocks, num_blocks, host, device)
        starts = torch.cat([zero[:1], n.cumsum(0)])
        T = int(starts[-1])
        s.update(_cache8(num_blocks, Hkv, d, gen, device))
        s["starts"] = starts.to(torch.int32).to(device)
        s["k_new"] = _normal((T, Hkv, d), gen, device, dtype)
        s["v_new"] = _normal((T, Hkv, d), gen, device, dtype)
        s["ctx"] = ctx.to(torch.int32).to(device)
        return s
    R, Hq, window, sinks = case["D"] + 1, case["Hq"], case["window"], case["sinks"]
    max_blocks = -(-(case["hi"] + R) // BLOCK)
    need = (ctx + R + BLOCK - 1) // BLOCK
    gone = (zero, zero)   # with a window, the blocks that have left it were given back
    if window:
        gone = (zero + -(-sinks // BLOCK), ((ctx - window + 1).clamp(min=0) // BLOCK).clamp(min=-(-sinks // BLOCK)))
    num_blocks = int((need - (gone[1] - gone[0])).sum()) + 4
    s["table"] = _tables(gone, need, max_blocks, num_blocks, host, device)
    if op == "kv8":
        s.update(_cache8(num_blocks, Hkv, d, gen, device))
    else:
        s["k_cache"] = _normal((num_blocks, BLOCK, Hkv, d), gen, device, dtype)
        s["v_cache"] = _normal((num_blocks, BLOCK, Hkv, d), gen, device, dtype)
    s["q"] = _normal((B, R, Hq, d), gen, device, dtype)
    s["k_new"] = _normal((B, R, Hkv, d), gen, device, dtype)
    s["v_new"] = _normal((B, R, Hkv, d), gen, device, dtype)
    s["ctx"] = ctx.to(torch.int32).to(device)
    s["out"] = torch.empty((B, R, Hq, d), dtype=dtype, device=device)
    s["window"], s["sinks"], s["scale"] = window, sinks, d ** -0.5
    return s


# --------------------------------------------------------------------------------------------------------------- run
def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "release":
        s["table"].copy_(s["table0"])
        return _plain_release(s)
    if s["op"] == "append":
        _plain_append(s, s["k_new"], s["v_new"], s["starts"])
        return _cache_of(s)
    R = s["q"].shape[1]
    if s["op"] == "kv8":
        starts = torch.arange(s["q"].shape[0] + 1, device=s["q"].device) * R
        _plain_append(s, s["k_new"].flatten(0, 1), s["v_new"].flatten(0, 1), starts)
    else:
        slot = s["ctx"].long()[:, None] + torch.arange(R, device=s["q"].device)
        at = torch.gather(s["table"].long(), 1, slot // BLOCK) * BLOCK + slot % BLOCK
        s["k_cache"].view(-1, *s["k_cache"].shape[2:])[at] = s["k_new"]
        s["v_cache"].view(-1, *s["v_cache"].shape[2:])[at] = s["v_new"]
    s["out"].copy_(_plain_attention(s))
    return dict(out=s["out"], **_cache_of(s))


def _cache_of(s):
    names = ("k_cache", "v_cache") + (("k_scale", "v_scale") if "k_scale" in s else ())
    return {n: s[n] for n in names}


def _run_own(s):
    import mtp_speculative_decoding_verify_gb300 as mv
    if s["op"] == "release":
        s["table"].copy_(s["table0"])   # the call works in place: each pass begins from the same tables
        s["free_list"].copy_(s["free_list0"])
        s["free_count"].fill_(4)
        mv.kv_window_release(s["table"], s["seq_lens"], s["free_list"], s["free_count"], window=s["window"], sinks=s["sinks"])
        return dict(table=s["table"], free_list=s["free_list"], free_count=s["free_count"])
    if s["op"] == "append":
        mv.mtp_kv8_append(s["k_new"], s["v_new"], s["starts"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["ctx"])
        return _cache_of(s)
    if s["op"] == "kv8":
        mv.mtp_verify_attention_kv8(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                    s["table"], s["ctx"], s["out"], window=s["window"], sinks=s["sinks"], sm_scale=s["scale"])
    else:
        mv.mtp_verify_attention_window(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["out"],
                                       window=s["window"], sinks=s["sinks"], sm_scale=s["scale"])
    return dict(out=s["out"], **_cache_of(s))


# ------------------------------------------------------------------------------------------------------- plain forms
def _plain_append(s, k_new, v_new, starts):
    table, ctx, starts = s["table"].long(), s["ctx"].long(), starts.long()
    b = torch.bucketize(torch.arange(k_new.shape[0], device=ctx.device), starts[1:], right=True)
    slot = ctx[b] + torch.arange(k_new.shape[0], device=ctx.device) - starts[b]
    block, off = table[b, slot // BLOCK], slot % BLOCK
    some = starts[1:] > starts[:-1]
    first = table.gather(1, (ctx // BLOCK).clamp(max=table.shape[1] - 1)[:, None])[some, 0]   # each request's first written block
    before = ctx[some] % BLOCK                                    # and the slots of it that are kept
    for x, cache, scale in ((k_new, s["k_cache"], s["k_scale"]), (v_new, s["v_cache"], s["v_scale"])):
        x = x.float()
        a = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)                     # [T, Hkv]
        most = torch.zeros_like(scale).scatter_reduce_(0, block[:, None].expand_as(a), a, "amax")   # by block and head
        fresh = torch.zeros_like(scale[:, 0]).index_fill_(0, block[off == 0], 1.0).bool()[:, None]
        start = torch.where(fresh, 2.0 ** MIN_EXP, scale)
        k = (torch.frexp(most)[1] - torch.frexp(start)[1] - 10).clamp(min=0)
        for _ in range(3):   # the exponents' difference leaves at most three doublings
            k = torch.where(448.0 * torch.ldexp(start, k) < most, k + 1, k)
        new = torch.ldexp(start, k)
        kept = cache[first]
        again = (kept.float() * torch.exp2(-k[first].float())[:, None, :, None]).to(cache.dtype)
        keep = torch.arange(BLOCK, device=ctx.device) < before[:, None]
        cache[first] = torch.where(keep[:, :, None, None], again.view(torch.uint8), kept.view(torch.uint8)).view(cache.dtype)
        scale[block] = new[block]
        cache[block, off] = (x / new[block][:, :, None]).to(cache.dtype)


def _plain_attention(s):
    """Softmax over the visible positions, in float32."""
    q, ctx, table = s["q"], s["ctx"].long(), s["table"].long()
    B, R, Hq, d = q.shape
    Hkv = s["k_cache"].shape[2]
    j = torch.arange(R, device=q.device)
    if s["window"]:
        low = (ctx - s["window"] + 1).clamp(min=0)                 # the first position in a row's window
        span = torch.arange(min(s["window"] + R - 1, table.shape[1] * BLOCK), device=q.device)
        first = torch.arange(s["sinks"], device=q.device).expand(B, -1)
        t = torch.cat([first, low[:, None] + span], 1)
        once = torch.cat([first < low[:, None], torch.ones_like(low[:, None] + span, dtype=torch.bool)], 1)
        at = (ctx[:, None] + j)[:, :, None]
        seen = once[:, None] & (t[:, None] <= at) & ((t[:, None] > at - s["window"]) | (t[:, None] < s["sinks"]))
    else:
        t = torch.arange(table.shape[1] * BLOCK, device=q.device).expand(B, -1)
        seen = t[:, None] <= (ctx[:, None] + j)[:, :, None]
    block = torch.gather(table, 1, (t // BLOCK).clamp(max=table.shape[1] - 1)).clamp(min=0)

    def rows(cache, scale):                                        # [B, Hkv, keys, d]
        x = cache.view(-1, Hkv, d)[block * BLOCK + t % BLOCK].permute(0, 2, 1, 3).float()
        return x if scale is None else x.mul_(scale[block].permute(0, 2, 1)[..., None])

    rows_q = q.float().view(B, R, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    x = torch.matmul(rows_q, rows(s["k_cache"], s.get("k_scale")).transpose(2, 3)).mul_(s["scale"])
    x = x.view(B, Hkv, R, Hq // Hkv, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp_()
    x = x.div_(x.sum(-1, keepdim=True)).view(B, Hkv, R * (Hq // Hkv), -1)
    y = torch.matmul(x, rows(s["v_cache"], s.get("v_scale")))
    return y.view(B, Hkv, R, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, d)


def _plain_release(s):
    table, lens = s["table"], s["seq_lens"].long()
    i = torch.arange(table.shape[1], device=table.device)
    out = (lens - s["window"] + 1).clamp(min=0) // BLOCK           # blocks before this one hold no position in a window
    gone = (i >= -(-s["sinks"] // BLOCK)) & (i < out[:, None]) & (table >= 0)
    s["free_list"].copy_(s["free_list0"])
    place = 4 + gone.reshape(-1).cumsum(0) - 1
    s["free_list"][place[gone.reshape(-1)]] = table[gone]
    s["free_count"].copy_(4 + gone.sum())
    table.masked_fill_(gone, -1)
    return dict(table=table, free_list=s["free_list"], free_count=s["free_count"])


# ------------------------------------------------------------------------------------------------------ work, exact
def _mean_keys(case):
    """The mean over the requests of the positions that a request's rows see between them."""
    R = case["D"] + 1
    most = case["window"] + R - 1 + case["sinks"] if case["window"] else math.inf
    return sum(min(c + R, most) for c in _spread(case["lo"], case["hi"], case["B"])) / case["B"]


def work(case):
    op, B = case["op"], case["B"]
    if op == "release":
        kept = -(-case["sinks"] // BLOCK)
        mean = sum(max(0, (c - case["window"] + 1) // BLOCK - kept) for c in _spread(case["lo"], case["hi"], B)) / B
        return {"bytes": B * (4 + 12 * mean) + 8, "flops": B * mean}
    Hkv, d, size = case["Hkv"], case["d"], 2 if case["t"] == "bf16" else 4
    if op == "append":
        n = sum(_spread(case["nlo"], case["nhi"], B))
        return {"bytes": n * 2 * Hkv * d * (size + 1) + n / BLOCK * 2 * Hkv * 4 + B * 12, "flops": n * 2 * Hkv * d * 2}
    R, Hq, held = case["D"] + 1, case["Hq"], 1 if op == "kv8" else size
    keys = _mean_keys(case)
    moved = B * keys * 2 * Hkv * (d * held + (4 / BLOCK if op == "kv8" else 0))           # the cache
    moved += B * R * (2 * Hq * d * size + 2 * Hkv * d * (size + held))                     # q, out, new K/V in and out
    return {"bytes": moved + B * keys / BLOCK * 4, "flops": 4.0 * B * R * Hq * d * keys}


def _exact_quantised(case, s):
    """The cache after a call's tokens went in: e4m3 values and scales, request by request in 64 bits."""
    grid = torch.arange(127, dtype=torch.uint8, device=s["ctx"].device).view(torch.float8_e4m3fn).double()   # 0 .. 448

    def nearest(x):   # of the e4m3 values, ties to the even byte
        m = x.abs().clamp(max=448.0)
        up = torch.searchsorted(grid, m.contiguous()).clamp(max=126)
        dn = (up - 1).clamp(min=0)
        a, b = m - grid[dn], grid[up] - m
        return torch.sign(x) * grid[torch.where((a < b) | ((a == b) & (dn % 2 == 0)), dn, up)]

    if case["op"] == "append":
        edges = s["starts"].tolist()
    else:
        edges = [i * (case["D"] + 1) for i in range(case["B"] + 1)]
    ctx, table, got = s["ctx"].tolist(), s["table"].tolist(), {}
    for x, n in ((s["k_new"], "k"), (s["v_new"], "v")):
        x = x.reshape(-1, case["Hkv"], case["d"]).double()
        cache, scale = s[n + "_cache"].to(torch.float32), s[n + "_scale"].double()
        for b in range(case["B"]):
            at, end = ctx[b], ctx[b] + edges[b + 1] - edges[b]
            while at < end:
                stop, blk, off = min(end, (at // BLOCK + 1) * BLOCK), table[b][at // BLOCK], at % BLOCK
                part = x[edges[b] + at - ctx[b]:edges[b] + stop - ctx[b]]
                a = part.abs().amax((0, 2))
                old = scale[blk].clone() if off else torch.full_like(scale[blk], 2.0 ** MIN_EXP)
                ratio = torch.exp2(torch.ceil(torch.log2((a / (448.0 * old)).clamp(min=1.0))))
                if off:
                    cache[blk, :off] = nearest(cache[blk, :off].double() / ratio[:, None]).float()
                scale[blk] = old * ratio
                cache[blk, off:off + stop - at] = nearest(part / (old * ratio)[:, None]).float()
                at = stop
        got[n + "_cache"], got[n + "_scale"] = cache, scale
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "release":
        return None
    if case["op"] == "append":
        return _exact_quantised(case, s)
    B, R, Hq, Hkv, d = case["B"], case["D"] + 1, case["Hq"], case["Hkv"], case["d"]
    ctx, table = s["ctx"].tolist(), s["table"].long()
    if case["op"] == "kv8":
        got = _exact_quantised(case, s)
    else:
        got = dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
        for n in "kv":
            for b in range(B):
                for j in range(R):
                    p = ctx[b] + j
                    got[n + "_cache"][table[b, p // BLOCK], p % BLOCK] = s[n + "_new"][b, j]
    out = torch.empty((B, R, Hq, d), dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        t = torch.arange(ctx[b] + R, device=out.device)
        if case["window"]:
            t = t[(t < case["sinks"]) | (t > ctx[b] - case["window"])]
        blk = table[b, t // BLOCK]
        k, v = (got[n + "_cache"][blk, t % BLOCK].double() * (got[n + "_scale"][blk][..., None] if case["op"] == "kv8" else 1.0) for n in "kv")
        for j in range(R):
            see = t <= ctx[b] + j
            if case["window"]:
                see &= (t > ctx[b] + j - case["window"]) | (t < case["sinks"])
            qh = s["q"][b, j].double().view(Hkv, Hq // Hkv, d)
            x = torch.einsum("hgd,thd->hgt", qh, k[see]) * s["scale"]
            out[b, j] = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v[see]).reshape(Hq, d)
    return dict(out=out, **got)
