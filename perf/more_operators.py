"""Cases of the serving operators for requests that share a prompt, with their plain forms.

Three operators of a server around the verify step, by `case["op"]`:

  assign   blocks for the tokens that each request is about to append, taken from the free list into the block tables,
           and the cache slot of every such token (kv_block_assign)
  append   K/V of new tokens into the paged cache by those slots: prefill chunks, a step's tokens, latent rows
           (mtp_kv_append)
  prefix   verify attention of groups of requests whose tables begin with the same blocks: the shared blocks are read
           once for the whole group (mtp_verify_attention_prefix)

The assignment, which has to agree to the last entry: request b holds seq_lens[b] = L tokens and appends n = starts[b+1]
- starts[b]; the table entries of blocks ceil(L/64) .. (L+n-1)/64 that are below 0 take blocks from the end of the free
list, requests in order and blocks ascending. A request is served whole or not at all, and none overtakes: it is refused
(taken -1, slots -1, its table row as it was) when its blocks and those of all earlier requests are more than the list
holds. The slot of a token at position p is table[b][p/64] * 64 + p%64.
"""
import math

import torch

own = False

BLOCK = 64


# ------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the blocks of one verify step of a large mixed batch: latency, every step
        dict(name="assign step", op="assign", B=256, lo=1024, hi=32768, nlo=4, nhi=4, short=False),
        # a prefill batch of chunks, some requests with tokens in the cache already
        dict(name="assign prefill", op="assign", B=64, lo=0, hi=3000, nlo=500, nhi=1500, short=False),
        # long prompts of many requests, more than the pool holds: the last ones are refused
        dict(name="assign long prompts short pool", op="assign", B=32, lo=0, hi=100, nlo=5000, nhi=65000, short=True),
        # a step's tokens of a batch, K and V as views of the fused projection's output
        dict(name="append step fused", op="append", T=1024, Hq=32, Hkv=8, d=128, latent=False, t="bf16", pad=0),
        # prefill chunks of a batch, padded to a fixed number of tokens
        dict(name="append prefill padded", op="append", T=65536, Hq=0, Hkv=8, d=128, latent=False, t="bf16", pad=977),
        # latent rows (576 values a token) of a DeepSeek-V3-shaped prefill chunk
        dict(name="append latent", op="append", T=8192, Hq=0, Hkv=1, d=576, latent=True, t="bf16", pad=0),
        # four samples drawn from one prompt: latency
        dict(name="prefix four samples", op="prefix", B=4, D=1, Hq=32, Hkv=8, d=128, G=1, plo=32, phi=32, lo=0, hi=100, tree=False, t="bf16"),
        # the tiny fp32 workload's heads, a shared prompt (SIMT path)
        dict(name="prefix tiny fp32", op="prefix", B=4, D=3, Hq=8, Hkv=8, d=64, G=1, plo=16, phi=16, lo=1, hi=128, tree=False, t="f32"),
        # Llama-70B-shaped heads, 5 drafts, a system prompt of 4096 tokens
        dict(name="prefix 70B-shaped", op="prefix", B=32, D=5, Hq=64, Hkv=8, d=128, G=1, plo=64, phi=64, lo=50, hi=500, tree=False, t="bf16"),
        # a large batch behind one long prompt
        dict(name="prefix large batch", op="prefix", B=256, D=3, Hq=32, Hkv=8, d=128, G=1, plo=128, phi=128, lo=64, hi=1000, tree=False, t="bf16"),
        # several system prompts of different lengths, groups of different sizes, one of a few requests
        dict(name="prefix five prompts", op="prefix", B=61, D=3, Hq=32, Hkv=8, d=128, G=5, plo=9, phi=301, lo=1, hi=1500, tree=False, t="bf16"),
        # trees of 15 drafts, odd sizes, head dim 64
        dict(name="prefix trees odd", op="prefix", B=13, D=15, Hq=12, Hkv=4, d=64, G=2, plo=11, phi=37, lo=0, hi=333, tree=True, t="bf16"),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "append", "prefix", "prefix", "prefix"])
    if op == "assign":
        B = _between(rng, 1, 512)
        nhi = rng.choice([1, rng.randint(2, 16), _between(rng, 16, max(17, min(65536, (1 << 20) // B)))])
        return dict(op=op, B=B, lo=0, hi=_between(rng, 1, 32768), nlo=rng.randint(min(1, nhi // 2), nhi), nhi=nhi,
                    short=rng.random() < 0.25)
    if op == "append":
        latent, t = rng.random() < 0.3, rng.choice(["bf16", "bf16", "f32"])
        Hkv, d = (1, 576) if latent else (rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128]))
        T = _between(rng, 1, 65536 if t == "bf16" else 32768)
        return dict(op=op, T=T, Hq=rng.choice([0, 4 * Hkv]), Hkv=Hkv, d=d, latent=latent, t=t, pad=rng.choice([0, 0, T // 7]))
    t = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d, Hkv, group, D = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([1, 2, 3, 4, 7, 8]), rng.randint(0, 15)
    B = _between(rng, 1, 256)
    G = rng.randint(1, min(B, 8))
    flops = 6e9 if t == "f32" else 1.3e11
    rows, token = B * (D + 1) * group * Hkv, Hkv * d * (8 if t == "f32" else 4)      # bytes of a token's K and V
    phi = _between(rng, 1, int(max(1, min(512, 0.25e9 / (G * token * BLOCK), flops / (4 * rows * d * BLOCK)))))
    hi = _between(rng, 1, int(max(2, min(2048, 0.25e9 / (B * token), 0.1 * flops / (4 * rows * d)))))
    return dict(op=op, B=B, D=D, Hq=group * Hkv, Hkv=Hkv, d=d, G=G, plo=rng.randint(0, phi), phi=phi, lo=rng.randint(0, hi), hi=hi,
                tree=rng.random() < 0.3, t=t)


# ------------------------------------------------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _spread(lo, hi, n):
    """n lengths spread evenly from lo to hi."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * n) for i in range(n)]


def _lens(lo, hi, n, gen):
    """The same in an order of the seed's: what a case reads and computes is the same for every seed."""
    return torch.tensor(_spread(lo, hi, n))[torch.randperm(n, generator=gen)]


def _normal(shape, gen, device, dtype):
    out = torch.empty(shape, dtype=dtype, device=device)
    flat = out.reshape(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = torch.randn(min(1 << 28, flat.numel() - i), generator=gen, device=device)
        flat[i:i + part.numel()] = part.to(dtype)
    return out


def _group_sizes(B, G):
    """Sizes of G groups of B requests, the last ones larger; at least one request each."""
    cuts = [max(i, B * i * (i + 1) // (G * (G + 1))) for i in range(G)] + [B]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    return dict(assign=_prepare_assign, append=_prepare_append, prefix=_prepare_prefix)[case["op"]](case, host, gen, device)


def _prepare_assign(case, host, gen, device):
    B = case["B"]
    lens, n = _lens(case["lo"], case["hi"], B, host), _lens(case["nlo"], case["nhi"], B, host)
    held, need = (lens + BLOCK - 1) // BLOCK, (lens + n + BLOCK - 1) // BLOCK
    max_blocks = -(-(case["hi"] + case["nhi"]) // BLOCK) + 1
    want = int((need - held).sum())
    free = max(1, want * 3 // 5) if case["short"] else want + 100
    perm = torch.randperm(int(held.sum()) + free, generator=host).to(torch.int32)
    table = torch.full((B, max_blocks), -1, dtype=torch.int32)
    table[torch.arange(max_blocks) < held[:, None]] = perm[free:]
    free_list = torch.full((perm.numel(),), -1, dtype=torch.int32)
    free_list[:free] = perm[:free]
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    T = int(starts[-1])
    s = dict(op="assign", T=T, free=free, table0=table.to(device), seq_lens=lens.to(torch.int32).to(device),
             starts=starts.to(torch.int32).to(device), free_list=free_list.to(device))
    s["table"] = s["table0"].clone()
    s["free_count"] = torch.full((1,), free, dtype=torch.int32, device=device)
    s["slot_map"] = torch.empty(T, dtype=torch.int64, device=device)
    s["taken"] = torch.empty(B, dtype=torch.int32, device=device)
    return s


def _prepare_append(case, host, gen, device):
    T, Hkv, d, dtype = case["T"], case["Hkv"], case["d"], _TYPES[case["t"]]
    # chunks of a few hundred tokens in random blocks, as an assignment leaves them; the padded tokens have no slot
    num_blocks = T // BLOCK + T // 300 + 40
    order, live, slots = torch.randperm(num_blocks, generator=host), T - case["pad"], []
    at, off, left = 0, 0, live
    while left > 0:
        off = int(torch.randint(0, BLOCK, (1,), generator=host)) if at % 8 == 0 else 0
        k = min(BLOCK - off, left)
        slots.append(int(order[at]) * BLOCK + off + torch.arange(k))
        at, left = at + 1, left - k
        if at == num_blocks - 1 and left > BLOCK:
            raise ValueError("blocks")
    slots = torch.cat(slots + [torch.full((case["pad"],), -1, dtype=torch.int64)])
    s = dict(op="append", slot_map=slots.to(device))
    if case["Hq"]:
        rows = _normal((T, case["Hq"] + 2 * Hkv, d), gen, device, dtype)
        s["k_new"], s["v_new"] = rows[:, case["Hq"]:case["Hq"] + Hkv], None if case["latent"] else rows[:, case["Hq"] + Hkv:]
    else:
        s["k_new"] = _normal((T, Hkv, d), gen, device, dtype)
        s["v_new"] = None if case["latent"] else _normal((T, Hkv, d), gen, device, dtype)
    s["k_cache"] = torch.zeros((num_blocks, BLOCK, Hkv, d), dtype=dtype, device=device)
    s["v_cache"] = None if case["latent"] else torch.zeros_like(s["k_cache"])
    return s


def _prefixes(case):
    """(blocks of the group's prefix, requests) for every group."""
    return list(zip(_spread(case["plo"], case["phi"], case["G"]), _group_sizes(case["B"], case["G"])))


def _prepare_prefix(case, host, gen, device):
    B, R, Hq, Hkv, d, dtype = case["B"], case["D"] + 1, case["Hq"], case["Hkv"], case["d"], _TYPES[case["t"]]
    tail = _lens(case["lo"], case["hi"], B, host)          # tokens of a request's own
    groups = _prefixes(case)
    blocks = torch.tensor([p for p, n in groups for _ in range(n)])
    need = blocks + (tail + R + BLOCK - 1) // BLOCK
    max_blocks = int(need.max())
    num_blocks = int((need - blocks).sum()) + sum(p for p, _ in groups) + 4
    order = torch.randperm(num_blocks, generator=host).to(torch.int32)
    table = torch.full((B, max_blocks), -1, dtype=torch.int32)
    i = torch.arange(max_blocks)
    mine = (i >= blocks[:, None]) & (i < need[:, None])
    used = int(mine.sum())
    table[mine] = order[:used]
    b = 0
    for p, n in groups:
        table[b:b + n, :p] = order[used:used + p]
        used, b = used + p, b + n
    starts = torch.tensor([0] + [n for _, n in groups]).cumsum(0)
    s = dict(op="prefix", case=case, table=table.to(device), ctx=(blocks * BLOCK + tail).to(torch.int32).to(device),
             group_starts=starts.to(torch.int32).to(device),
             prefix_blocks=torch.tensor([p for p, _ in groups], dtype=torch.int32, device=device), scale=d ** -0.5)
    for name in ("k_cache", "v_cache"):
        s[name] = _normal((num_blocks, BLOCK, Hkv, d), gen, device, dtype)
    s["q"] = _normal((B, R, Hq, d), gen, device, dtype)
    for name in ("k_new", "v_new"):
        s[name] = _normal((B, R, Hkv, d), gen, device, dtype)
    s["parents"] = None
    if case["tree"]:
        k = torch.arange(R)
        par = (torch.rand((B, R), generator=host) * k).long().minimum((k - 1).clamp(min=0))
        par[:, 0] = -1
        s["parents"] = par.to(torch.int32).to(device)
    s["out"] = torch.empty_like(s["q"])
    return s


# --------------------------------------------------------------------------------------------------------------- run
def run(state):
    s = state
    if s["op"] == "assign":      # the call works in place: each pass begins from the same tables
        s["table"].copy_(s["table0"])
        s["free_count"].fill_(s["free"])
    if own:
        import mtp_speculative_decoding_verify_gb300 as mv
        if s["op"] == "assign":
            mv.kv_block_assign(s["table"], s["seq_lens"], s["starts"], s["free_list"], s["free_count"], s["slot_map"], s["taken"])
        elif s["op"] == "append":
            mv.mtp_kv_append(s["k_new"], s["v_new"], s["slot_map"], s["k_cache"], s["v_cache"])
        else:
            mv.mtp_verify_attention_prefix(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["ctx"],
                                           s["group_starts"], s["prefix_blocks"], s["out"], sm_scale=s["scale"],
                                           parents=s["parents"])
    else:
        dict(assign=_plain_assign, append=_plain_append, prefix=_plain_prefix)[s["op"]](s)
    names = dict(assign=("table", "free_count", "slot_map", "taken"), append=("k_cache", "v_cache"),
                 prefix=("out", "k_cache", "v_cache"))[s["op"]]
    return {n: s[n] for n in names if s[n] is not None}


# ------------------------------------------------------------------------------------------------------- plain forms
def _plain_assign(s):
    table, lens, starts = s["table"], s["seq_lens"].long(), s["starts"].long()
    n, i = starts[1:] - starts[:-1], torch.arange(table.shape[1], device=table.device)
    held, need = (lens + BLOCK - 1) // BLOCK, (lens + n + BLOCK - 1) // BLOCK
    miss = (i >= held[:, None]) & (i < need[:, None]) & (table < 0)
    count = miss.sum(1)
    served = (count == 0) | (count.cumsum(0) <= s["free_count"])
    miss &= served[:, None]
    rank = miss.reshape(-1).cumsum(0).view_as(miss)               # counted from 1
    table.copy_(torch.where(miss, s["free_list"][(s["free_count"] - rank).clamp(min=0)], table))
    s["free_count"] -= miss.sum()
    s["taken"].copy_(torch.where(served, count, -1))
    t = torch.arange(s["T"], device=table.device)
    b = torch.bucketize(t, starts[1:], right=True)
    p = lens[b] + t - starts[b]
    s["slot_map"].copy_(torch.where(served[b], table[b, p // BLOCK].long() * BLOCK + p % BLOCK, -1))


def _plain_append(s):
    live = s["slot_map"] >= 0
    at = s["slot_map"][live]
    for new, cache in ((s["k_new"], s["k_cache"]), (s["v_new"], s["v_cache"])):
        if new is not None:
            cache.view(-1, *cache.shape[2:])[at] = new[live]


def _plain_prefix(s):
    """Softmax over a group's shared positions and each request's own, in float32."""
    q, ctx, table = s["q"], s["ctx"].long(), s["table"].long()
    B, R, Hq, d = q.shape
    Hkv = s["k_cache"].shape[2]
    group = Hq // Hkv
    j = torch.arange(R, device=q.device)
    slot = ctx[:, None] + j
    at = torch.gather(table, 1, slot // BLOCK) * BLOCK + slot % BLOCK
    caches = [s[n].view(-1, Hkv, d) for n in ("k_cache", "v_cache")]
    for cache, new in zip(caches, (s["k_new"], s["v_new"])):
        cache[at] = new
    path = torch.tril(torch.ones(R, R, dtype=torch.bool, device=q.device)).expand(B, R, R)   # row sees verify key
    if s["parents"] is not None:
        up = torch.nn.functional.one_hot(s["parents"].long().clamp(min=0), R).bool()   # (the root is its own parent here)
        path = torch.eye(R, dtype=torch.bool, device=q.device).expand(B, R, R)
        for _ in range(R - 1):
            path = path | (path.float() @ up.float() > 0)
    rows = q.float().view(B, R, Hkv, group, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * group, d)
    b = 0
    for p, n in _prefixes(s["case"]):
        # the group's prefix: one set of keys for all of its rows
        first = (table[b, :p, None] * BLOCK + torch.arange(BLOCK, device=q.device)).reshape(-1)
        kp, vp = (c[first].permute(1, 0, 2).float() for c in caches)                       # [Hkv, P, d]
        qg = rows[b:b + n].transpose(0, 1).reshape(Hkv, -1, d)
        xp = torch.matmul(qg, kp.transpose(1, 2)).mul_(s["scale"])
        # each request's own positions
        most = int(s["table"].shape[1]) - p
        t = p * BLOCK + torch.arange(most * BLOCK, device=q.device)
        blk = table[b:b + n, p:].clamp(min=0)
        ko, vo = (c.view(-1, BLOCK, Hkv, d)[blk].flatten(1, 2).transpose(1, 2).float() for c in caches)   # [n, Hkv, K, d]
        rel = t[None, :] - ctx[b:b + n, None]                                              # [n, K]
        seen = torch.gather(path[b:b + n], 2, rel.clamp(0, R - 1)[:, None, :].expand(-1, R, -1)) & (rel < R)[:, None]
        seen = seen | (rel < 0)[:, None]                                                   # [n, R, K]
        xo = torch.matmul(rows[b:b + n], ko.transpose(2, 3)).mul_(s["scale"])
        xo = xo.view(n, Hkv, R, group, -1).masked_fill_(~seen[:, None, :, None], -math.inf).view(n, Hkv, R * group, -1)
        m = xo.amax(-1, keepdim=True)
        if p:
            xp = xp.view(Hkv, n, R * group, -1)
            m = torch.maximum(m, xp.amax(-1, keepdim=True).transpose(0, 1))
        xo = (xo - m).exp_()
        total, y = xo.sum(-1, keepdim=True), torch.matmul(xo, torch.where(seen.any(1)[:, None, :, None], vo, 0.0))
        if p:
            xp = xp.sub_(m.transpose(0, 1)).exp_()
            total = total + xp.sum(-1, keepdim=True).transpose(0, 1)
            y = y + torch.matmul(xp.view(Hkv, n * R * group, -1), vp).view(Hkv, n, R * group, d).transpose(0, 1)
        y = (y / total).view(n, Hkv, R, group, d).permute(0, 2, 1, 3, 4).reshape(n, R, Hq, d)
        s["out"][b:b + n] = y.to(q.dtype)
        b += n


# ------------------------------------------------------------------------------------------------------ work, exact
def work(case):
    B = case["B"] if "B" in case else 0
    if case["op"] == "assign":
        n = sum(_spread(case["nlo"], case["nhi"], B))
        blocks = n / BLOCK * (0.6 if case["short"] else 1.0)
        return {"bytes": n * 8 + blocks * 12 + B * 12, "flops": float(n)}
    size = 2 if case["t"] == "bf16" else 4
    if case["op"] == "append":
        live = case["T"] - case["pad"]
        row = case["Hkv"] * case["d"] * size * (1 if case["latent"] else 2)
        return {"bytes": live * row * 2 + case["T"] * 8, "flops": float(live)}
    R, Hq, Hkv, d = case["D"] + 1, case["Hq"], case["Hkv"], case["d"]
    tails = sum(_spread(case["lo"], case["hi"], B))
    once = sum(p for p, _ in _prefixes(case)) * BLOCK
    seen = sum(p * n for p, n in _prefixes(case)) * BLOCK + tails + B * R
    moved = (once + tails + B * R) * 2 * Hkv * d * size                            # the cache
    moved += B * R * (2 * Hq * d * size + 2 * Hkv * d * size)                      # q, out, new K/V
    return {"bytes": moved, "flops": 4.0 * R * Hq * d * seen}


def exact(case, seed):
    if case["op"] != "prefix":
        return None                                                                # integers and copies
    s = prepare(case, seed)
    B, R, Hq, Hkv, d = case["B"], case["D"] + 1, case["Hq"], case["Hkv"], case["d"]
    ctx, table = s["ctx"].tolist(), s["table"].long()
    parents = None if s["parents"] is None else s["parents"].tolist()
    out = torch.empty((B, R, Hq, d), dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        for j in range(R):
            p = ctx[b] + j
            for n in "kv":
                s[n + "_cache"][table[b, p // BLOCK], p % BLOCK] = s[n + "_new"][b, j]
        t = torch.arange(ctx[b] + R, device=out.device)
        k, v = (s[n + "_cache"][table[b, t // BLOCK], t % BLOCK].double().transpose(0, 1) for n in "kv")   # [Hkv, K, d]
        see = torch.ones((R, ctx[b] + R), dtype=torch.bool, device=out.device)
        for j in range(R):
            nodes, at = set(), j
            while at >= 0:
                nodes.add(at)
                at = at - 1 if parents is None else parents[b][at]
            for i in range(R):
                see[j, ctx[b] + i] = i in nodes
        qh = s["q"][b].double().view(R, Hkv, Hq // Hkv, d).permute(1, 0, 2, 3)
        x = torch.einsum("hrgd,htd->hrgt", qh, k) * s["scale"]
        x = x.masked_fill(~see[None, :, None], -math.inf)
        y = torch.einsum("hrgt,htd->hrgd", torch.softmax(x, -1), v)
        out[b] = y.permute(1, 0, 2, 3).reshape(R, Hq, d)
    return dict(out=out, k_cache=s["k_cache"], v_cache=s["v_cache"])
