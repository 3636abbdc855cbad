"""Measured calls of the 8-bit paged cache: its write and read, decode and prefill attention, page selection with
attention over the chosen pages, and eviction of pages by accumulated attention weight.

``run`` computes a case either with the framework's operators (``own``) or in plain torch.  The cache is the paged
one of ``include/tq.h`` with ``int8 = 1``: pages of 16 tokens; for a (page, KV head) int8 codes of keys and of values
with one float scale each, and the smallest and largest key code of every channel; the newest tokens in a float16 ring.
"""
import math

import torch

own = False

PAGE = 16
LOG_DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a prompt's keys and values written into the cache, and the cache handed on as plain tensors
        dict(name="write_prompt", op="write", batch=4, ctx=8192, hkv=8, g=4, d=128, window=128, dtype="bf16"),
        # a short odd prompt, wide heads, half precision
        dict(name="write_short_odd", op="write", batch=3, ctx=1037, hkv=2, g=4, d=256, window=33, dtype="f16"),
        # one user, short context: the latency of a decode step's attention
        dict(name="decode_short", op="decode", batch=1, ctx=517, hkv=8, g=4, d=128, window=128, dtype="bf16"),
        # a serving batch of sequences of mixed lengths
        dict(name="decode_batch", op="decode", batch=32, ctx=8192, hkv=8, g=4, d=128, window=128, dtype="bf16"),
        # wide heads, eight query heads a KV head, float queries, no multiple of anything
        dict(name="decode_wide", op="decode", batch=5, ctx=16411, hkv=4, g=8, d=256, window=100, dtype="f32"),
        # one user, a very long document
        dict(name="decode_long", op="decode", batch=1, ctx=262144, hkv=8, g=5, d=128, window=64, dtype="f16"),
        # a small chunk of a prompt (or a draft to verify) over a few thousand cached tokens
        dict(name="prefill_small", op="prefill", batch=3, ctx=4100, nq=17, hkv=4, g=6, d=128, window=64, dtype="f16"),
        # a large chunk of a long prompt
        dict(name="prefill_chunk", op="prefill", batch=1, ctx=16384, nq=2048, hkv=8, g=4, d=128, window=128, dtype="bf16"),
        # long contexts read through a fixed budget of pages
        dict(name="sparse_batch", op="sparse", batch=8, ctx=65536, k=128, sink=1, recent=2, hkv=8, g=4, d=128, window=128,
             dtype="bf16"),
        # the same for one user with wide heads
        dict(name="sparse_one", op="sparse", batch=1, ctx=9001, k=37, sink=2, recent=0, hkv=2, g=8, d=256, window=40, dtype="f16"),
        # attention weights of one decode step added to the pages' totals
        dict(name="track_step", op="track", batch=16, ctx=8192, hkv=8, g=4, d=128, window=128, dtype="bf16"),
        # half of the pages dropped from every sequence of a batch
        dict(name="evict_half", op="evict", batch=32, ctx=16384, budget=512, sink=4, recent=16, hkv=8, g=4, d=128, window=128,
             dtype="bf16"),
    ]


#: tokens x KV heads x d of the largest drawn case of each operator: no more than its largest listed one
MOST = {"write": 4 * 8192 * 8 * 128, "decode": 32 * 8192 * 8 * 128, "prefill": 16384 * 8 * 128, "sparse": 8 * 65536 * 8 * 128,
        "track": 16 * 8192 * 8 * 128, "evict": 32 * 16384 * 8 * 128}


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "decode", "decode", "prefill", "sparse", "track", "evict"])
    d = rng.choice([128, 128, 256])
    hkv, g = between(1, 8), rng.randint(1, 8)
    room = MOST[op] // (hkv * d)
    batch = between(1, 32)
    if op == "prefill":
        batch = min(batch, 4)
    ctx = between(1 if op in ("write", "decode") else 300, max(301, min(room // batch, 131072)))
    case = dict(op=op, batch=batch, ctx=ctx, hkv=hkv, g=g, d=d, window=between(1, 300), dtype=rng.choice(list(LOG_DTYPE)))
    if op == "prefill":
        most = max(1, (2048 * 16384 * 32 * 128) // (ctx * hkv * g * d * batch))
        case["nq"] = between(1, min(ctx, most, 2048))
    elif op == "sparse":
        case["sink"], case["recent"] = rng.randint(0, 4), rng.randint(0, 4)
        case["k"] = case["sink"] + case["recent"] + between(1, 200)
    elif op == "evict":
        case["sink"], case["recent"] = rng.randint(0, 4), rng.randint(0, 20)
        case["budget"] = case["sink"] + case["recent"] + between(1, max(2, ctx // PAGE))
    return case


def lengths(case):
    """Tokens of every sequence: the first has them all, the others down to about half."""
    n, b = case["ctx"], case["batch"]
    least = case.get("nq", 1)
    return [max(least, n - (i * 7919) % (n // 2 + 1)) for i in range(b)] if case["op"] != "write" else [n] * b


def compressed(case):
    return [PAGE * (max(0, t - case["window"]) // PAGE) for t in lengths(case)]


def work(case):
    b, hkv, g, d, w = case["batch"], case["hkv"], case["g"], case["d"], case["window"]
    hq, T, nc = hkv * g, lengths(case), compressed(case)
    e = 4 if case["dtype"] == "f32" else 2
    page = hkv * (2 * PAGE * d + 8)                       # codes and scales of one page
    bounds = hkv * 2 * d                                  # and its channel bounds
    pages, left = [n // PAGE for n in nc], sum(t - n for t, n in zip(T, nc))
    ring = left * hkv * d * 2 * 2
    qo = b * hq * (d * e + d * 4 + 4)
    op = case["op"]
    if op == "write":
        dense = 2 * sum(T) * hkv * d * e
        return {"bytes": 2 * dense + sum(pages) * (2 * page + bounds) + 2 * ring, "flops": 0}
    if op == "decode":
        return {"bytes": sum(pages) * page + ring + qo, "flops": 4 * hq * d * sum(T)}
    if op == "prefill":
        nq = case["nq"]
        seen = sum(nq * t - nq * (nq - 1) // 2 for t in T)
        return {"bytes": sum(pages) * page + ring + nq * qo, "flops": 4 * hq * d * seen}
    if op == "sparse":
        taken = sum(min(p, case["k"]) for p in pages)
        return {"bytes": sum(pages) * (bounds + 4 * hkv) + taken * page + ring + qo + b * hkv * (4 * case["k"] + 4),
                "flops": 4 * hq * d * (sum(pages) + taken * PAGE + left)}
    table = b * max_pages(case)
    if op == "track":
        return {"bytes": 4 * hq * sum(nc) + 2 * 4 * sum(pages) + 4 * b * hq, "flops": 2 * hq * sum(nc)}
    moved = b * hkv * (w + PAGE) * d * 2 * 2
    return {"bytes": 4 * sum(pages) + 3 * 4 * table + 4 * b * case["budget"] + 2 * moved, "flops": 0}


def max_pages(case):
    return max(1, -(-case["ctx"] // PAGE))


# ---------------------------------------------------------------------------------------------- page format

def page_codes(x):
    """Codes (int8 values) and float scale of pages [..., 16, d]: scale = max |x| / 127, code = nearest to x / scale
    with ties to even.  The quotient is taken in 64 bits: next to a half step 32 bits would round twice."""
    a = x.double().abs().amax((-1, -2))
    s = a.float() / 127
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    c = torch.where(s[..., None, None] > 0, x.double() / s.double()[..., None, None], torch.zeros((), dtype=torch.float64, device=x.device))
    return c.round().clamp(-127, 127).to(torch.int8), s


def pack_pages(k, v):
    """The bytes of pages from keys and values [n, Hkv, 16, d]: [n, Hkv, 34 d + 32]."""
    n, h, _, d = k.shape
    (kc, ks), (vc, vs) = page_codes(k), page_codes(v)
    head = torch.zeros(n, h, 8, dtype=torch.float32, device=k.device)
    head[..., 0], head[..., 1] = ks, vs
    ku = (kc.short() + 128).to(torch.uint8).reshape(n, h, 4, 2, 2, d // 64, 4, 16).permute(0, 1, 3, 5, 2, 4, 6, 7)
    vu = (vc.short() + 128).to(torch.uint8).reshape(n, h, 4, 4, d // 64, 8, 2, 4).permute(0, 1, 4, 6, 5, 2, 7, 3)
    return torch.cat([kc.amin(2).view(torch.uint8), kc.amax(2).view(torch.uint8), head.view(torch.uint8),
                      ku.reshape(n, h, 16 * d), vu.reshape(n, h, 16 * d)], -1)


def unpack_pages(raw, d):
    """Key codes, value codes [n, Hkv, 16, d] (float), their scales and the keys' smallest and largest codes."""
    n, h, _ = raw.shape
    o = 2 * d + 32
    lo, hi = raw[..., :d].contiguous().view(torch.int8).float(), raw[..., d:2 * d].contiguous().view(torch.int8).float()
    head = raw[..., 2 * d:o].contiguous().view(torch.float32)
    kc = raw[..., o:o + 16 * d].reshape(n, h, 2, d // 64, 4, 2, 4, 16).permute(0, 1, 4, 2, 5, 3, 6, 7).reshape(n, h, 16, d)
    vc = raw[..., o + 16 * d:].reshape(n, h, d // 64, 2, 8, 4, 4, 4).permute(0, 1, 5, 7, 2, 4, 3, 6).reshape(n, h, 16, d)
    return kc.float() - 128, vc.float() - 128, head[..., 0], head[..., 1], lo, hi


# ---------------------------------------------------------------------------------------------- inputs

def dense(shape, gen, dtype):
    """Keys, values or queries as attention layers have them: unit scale, some channels several times larger."""
    chan = 1 + 5 * torch.rand(shape[-1], device="cuda", generator=gen).pow(8)
    return (torch.randn(shape, device="cuda", generator=gen) * chan).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b, hkv, g, d, w = case["batch"], case["hkv"], case["g"], case["d"], case["window"]
    dt, op, mp, ring = LOG_DTYPE[case["dtype"]], case["op"], max_pages(case), w + PAGE
    T, nc = lengths(case), compressed(case)
    s = dict(case=case, scale=d ** -0.5)
    if op == "write":
        s["k"], s["v"] = (dense((b, case["ctx"], hkv, d), gen, dt) for _ in range(2))
    s["seq_len"] = torch.tensor(T, dtype=torch.int32, device="cuda")
    s["n_compressed"] = torch.tensor(nc, dtype=torch.int32, device="cuda")
    # pages in the order a shared pool hands them out
    s["table"] = torch.randperm(b * mp, device="cuda", generator=gen).to(torch.int32).reshape(b, mp)
    if op in ("decode", "prefill", "sparse"):
        s["raw"] = torch.zeros(b * mp, hkv, 34 * d + 32, dtype=torch.uint8, device="cuda")
        for p in range(0, b * mp, 8192):
            n = min(8192, b * mp - p)
            s["raw"][p:p + n] = pack_pages(dense((n, hkv, PAGE, d), gen, torch.float32), dense((n, hkv, PAGE, d), gen, torch.float32))
        shape = (b, case["nq"], hkv * g, d) if op == "prefill" else (b, hkv * g, d)
        s["q"] = dense(shape, gen, dt)
    if op in ("decode", "prefill", "sparse", "evict"):
        s["win_k"], s["win_v"] = (dense((b, hkv, ring, d), gen, torch.float16) for _ in range(2))
    if op == "track":
        sc = 2 * torch.randn((b, hkv * g, case["ctx"]), device="cuda", generator=gen)
        live = torch.arange(case["ctx"], device="cuda")[None] < s["seq_len"][:, None]
        s["scores"], s["lse"] = sc, torch.where(live[:, None], sc.double(), -math.inf).logsumexp(-1).float()
    if op in ("track", "evict"):
        full = torch.arange(mp, device="cuda")[None] < (s["n_compressed"] // PAGE)[:, None]
        s["mass"] = torch.where(full, torch.randn((b, mp), device="cuda", generator=gen).mul(1.5).exp(), 0.0)
    if own:
        handles(s)
    return s


def handles(s):
    """What a program of the framework keeps next to the tensors: the layer, the cache, workspaces and outputs."""
    import kv_cache_vector_head_gb300 as tq

    case = s["case"]
    b, hkv, g, d, w, op = case["batch"], case["hkv"], case["g"], case["d"], case["window"], case["op"]
    s["tq"] = tq
    layer = s["layer"] = tq.TQLayer(d, hkv, hkv * g, 8, 8, tq.TQ_FWHT, window=w, key_qjl=tq.KEY_MSE, int8=True)
    pages = None if op in ("write", "decode", "prefill", "sparse") else 1  # track and evict never look into a page
    pc = s["pc"] = tq.PagedCache(layer, b, case["ctx"], pool_pages=pages)
    if op == "write":
        pc.block_table.copy_(s["table"])
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        return
    pc.block_table.copy_(s["table"])
    pc.seq_len.copy_(s["seq_len"])
    pc.n_compressed.copy_(s["n_compressed"])
    if "raw" in s:
        pc.pool.copy_(s.pop("raw").reshape(-1))
    if "win_k" in s:
        pc.win_k.copy_(s["win_k"])
        pc.win_v.copy_(s["win_v"])
    if "q" in s:
        s["out"] = torch.empty(s["q"].shape, dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty(s["q"].shape[:-1], dtype=torch.float32, device="cuda")
    if op == "decode":
        n = tq.decode_workspace_size(layer.params, b, case["ctx"])
    elif op == "prefill":
        n = tq.prefill_workspace_size(layer.params, b, case["nq"], case["ctx"])
    elif op == "sparse":
        n = max(tq.select_workspace_size(layer.params, b, case["ctx"]), tq.decode_pages_workspace_size(layer.params, b, case["k"]))
        s["pages"] = torch.empty(b, hkv, case["k"], dtype=torch.int32, device="cuda")
        s["counts"] = torch.empty(b, hkv, dtype=torch.int32, device="cuda")
    elif op == "evict":
        n = tq.evict_workspace_size(layer.params, b, pc.max_pages)
        s["after"] = tq.PagedCache(layer, b, case["ctx"], pool_pages=1)
        s["after"].share_pages(pc)
        s["mass_out"] = torch.empty_like(s["mass"])
        s["kept"] = torch.empty(b, case["budget"], dtype=torch.int32, device="cuda")
    else:
        n = 1
    s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------------------------- the passes

def run(s):
    return run_own(s) if own else PLAIN[s["case"]["op"]](s)


def run_own(s):
    tq, case, pc, p = s["tq"], s["case"], s["pc"], s["layer"].params
    op = case["op"]
    if op == "write":
        pc.prefill(s["k"], s["v"])
        tq.read_cache(p, pc.cache, s["k_out"], s["v_out"], 0, case["ctx"])
        return s["k_out"], s["v_out"], pc.seq_len, pc.n_compressed
    if op == "decode":
        tq.decode_attention(p, pc.cache, s["q"], s["scale"], s["out"], s["lse"], None, s["ws"], case["ctx"])
        return s["out"], s["lse"]
    if op == "prefill":
        tq.prefill_attention(p, pc.cache, case["nq"], s["q"], s["scale"], s["out"], s["lse"], s["ws"], case["ctx"])
        return s["out"], s["lse"]
    if op == "sparse":
        tq.select_pages(p, pc.cache, s["q"], case["k"], case["sink"], case["recent"], s["pages"], s["counts"], s["ws"], case["ctx"])
        tq.decode_attention_pages(p, pc.cache, s["q"], s["scale"], s["pages"], s["counts"], case["k"], s["out"], s["lse"], s["ws"],
                                  case["ctx"])
        return s["pages"], s["counts"], s["out"], s["lse"]
    if op == "track":
        tq.track_pages(p, pc.cache, s["scores"], s["lse"], s["mass"], case["ctx"])
        return s["mass"]
    after = s["after"]
    tq.evict_pages(p, pc.cache, after.cache, s["mass"], s["mass_out"], case["budget"], case["sink"], case["recent"], s["kept"], s["ws"])
    return after.block_table, after.seq_len, after.n_compressed, after.win_k, after.win_v, s["mass_out"], s["kept"]


def window_positions(s, dev="cuda"):
    """Ring slots of the window's tokens [b, W + 15] and which of them are there."""
    w = s["case"]["window"]
    pos = s["n_compressed"].long()[:, None] + torch.arange(w + PAGE - 1, device=dev)
    return pos % (w + PAGE), pos < s["seq_len"].long()[:, None], pos


def gathered(s, table=None):
    """Keys and values of the cache as floats, pages first, then the window: [b, Hkv, n, d], their positions [b, 1, n]
    and which are there.  `table`: [b, Hkv, k] page ordinals to take instead of all (-1: none)."""
    case = s["case"]
    b, hkv, d = case["batch"], case["hkv"], case["d"]
    slot, there, wpos = window_positions(s)
    np_ = (s["n_compressed"].long() // PAGE)[:, None]
    if table is None:
        n = max(1, max(compressed(case)) // PAGE)
        ordinal = torch.arange(n, device="cuda").expand(b, n)
        have = ordinal < np_
        raw = s["raw"][s["table"][:, :n].long()].transpose(1, 2)                      # [b, Hkv, n, bytes]
        ordinal, have = ordinal[:, None], have[:, None]
    else:
        have = table >= 0
        ordinal = table.clamp(min=0).long()
        page = s["table"].long()[:, None].expand(b, hkv, -1).gather(2, ordinal)
        raw = s["raw"][page, torch.arange(hkv, device="cuda")[None, :, None]]
    n = raw.shape[2]
    kc, vc, ks, vs, _, _ = unpack_pages(raw.reshape(b * hkv, n, -1), d)
    k = (kc * ks[..., None, None]).reshape(b, hkv, n * PAGE, d)
    v = (vc * vs[..., None, None]).reshape(b, hkv, n * PAGE, d)
    row = slot[:, None, :, None].expand(b, hkv, -1, d)
    k = torch.cat([k, s["win_k"].gather(2, row).float()], 2)
    v = torch.cat([v, s["win_v"].gather(2, row).float()], 2)
    pos = (ordinal[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(-2)
    pos = torch.cat([pos, wpos[:, None].expand(b, pos.shape[1], -1)], -1)
    live = torch.cat([have[..., None].expand(*have.shape, PAGE).flatten(-2), there[:, None].expand(b, have.shape[1], -1)], -1)
    return k, v, pos, live


def attend(q, k, v, live, scale):
    """q [b, Hkv, rows, d] over k, v [b, Hkv, n, d] where live [b, Hkv or 1, rows or 1, n]: outputs and log-sum-exp."""
    l = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    l = l.masked_fill_(~live, -math.inf)
    m = l.amax(-1, keepdim=True)
    p = l.sub_(m.masked_fill(m == -math.inf, 0)).exp_()
    z = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / z.clamp(min=1e-38), (m + z.log()).squeeze(-1)


def plain_write(s):
    case = s["case"]
    b, T, hkv, d, w = case["batch"], case["ctx"], case["hkv"], case["d"], case["window"]
    nc = compressed(case)[0]

    def held(x):
        pages = x[:, :nc].reshape(b, nc // PAGE, PAGE, hkv, d).transpose(2, 3)
        c, sc = page_codes(pages)
        y = (c.float() * sc[..., None, None]).transpose(2, 3).reshape(b, nc, hkv, d)
        return torch.cat([y, x[:, nc:].half().float()], 1).to(x.dtype)

    return held(s["k"]), held(s["v"]), s["seq_len"], s["n_compressed"]


def plain_decode(s):
    case = s["case"]
    b, hkv, g, d = case["batch"], case["hkv"], case["g"], case["d"]
    k, v, _, live = gathered(s)
    o, lse = attend(s["q"].float().reshape(b, hkv, g, d), k, v, live[:, :, None], s["scale"])
    return o.reshape(b, hkv * g, d), lse.reshape(b, hkv * g)


def plain_prefill(s):
    case = s["case"]
    b, hkv, g, d, nq = case["batch"], case["hkv"], case["g"], case["d"], case["nq"]
    k, v, pos, live = gathered(s)
    at = s["seq_len"].long()[:, None] - nq + torch.arange(nq, device="cuda")          # the queries' positions [b, nq]
    seen = live[:, :, None] & (pos[:, :, None] <= at[:, None, :, None])               # [b, 1, nq, n]
    q = s["q"].float().reshape(b, nq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * nq, d)
    o, lse = attend(q, k, v, seen.repeat(1, 1, g, 1), s["scale"])
    o = o.reshape(b, hkv, g, nq, d).permute(0, 3, 1, 2, 4).reshape(b, nq, hkv * g, d)
    return o, lse.reshape(b, hkv, g, nq).permute(0, 3, 1, 2).reshape(b, nq, hkv * g)


def plain_select(s):
    case = s["case"]
    b, hkv, g, d, kk = case["batch"], case["hkv"], case["g"], case["d"], case["k"]
    n = max(1, max(compressed(case)) // PAGE)
    raw = s["raw"][s["table"][:, :n].long()].transpose(1, 2)[..., :2 * d + 32]
    lo = raw[..., :d].contiguous().view(torch.int8).float()
    hi = raw[..., d:2 * d].contiguous().view(torch.int8).float()
    ks = raw[..., 2 * d:].contiguous().view(torch.float32)[..., 0]
    qi, _ = page_codes(s["q"].reshape(b, hkv, g, d))
    qi = qi.float()
    # products of codes: every sum is a whole number below 2^24, exact in 32 bits in any order
    top = torch.matmul(qi.clamp(min=0), hi.transpose(-1, -2)) + torch.matmul(qi.clamp(max=0), lo.transpose(-1, -2))
    score = top.amax(2) * ks                                                           # [b, Hkv, n]
    np_ = (s["n_compressed"].long() // PAGE)[:, None, None]
    i = torch.arange(n, device="cuda")
    score = torch.where((i < case["sink"]) | (i >= np_ - case["recent"]), math.inf, score)
    score = torch.where(i < np_, score, -math.inf)
    first = score.sort(dim=-1, descending=True, stable=True).indices[..., :kk]
    taken = np_.clamp(max=kk)                                                          # [b, 1, 1]
    rank = torch.arange(first.shape[-1], device="cuda")
    first = torch.where(rank < taken, first, 1 << 30).sort(dim=-1).values
    pages = torch.full((b, hkv, kk), -1, dtype=torch.int32, device="cuda")
    pages[..., :first.shape[-1]] = torch.where(rank < taken, first, -1).int()
    return pages, taken[..., 0].expand(b, hkv).int().contiguous()


def plain_sparse(s):
    case = s["case"]
    b, hkv, g, d = case["batch"], case["hkv"], case["g"], case["d"]
    pages, counts = plain_select(s)
    k, v, _, live = gathered(s, pages)
    live = live.expand(b, hkv, -1)
    o, lse = attend(s["q"].float().reshape(b, hkv, g, d), k, v, live[:, :, None], s["scale"])
    return pages, counts, o.reshape(b, hkv * g, d), lse.reshape(b, hkv * g)


def plain_track(s):
    case = s["case"]
    n = max(compressed(case))
    live = torch.arange(n, device="cuda")[None, None] < s["n_compressed"][:, None, None]
    p = torch.where(live, (s["scores"][..., :n] - s["lse"][..., None]).exp(), 0.0)
    add = p.reshape(case["batch"], case["hkv"] * case["g"], n // PAGE, PAGE).sum((1, 3))
    s["mass"][:, :n // PAGE] += add
    return s["mass"]


def plain_evict(s):
    case = s["case"]
    b, mp, budget, ring = case["batch"], max_pages(case), case["budget"], case["window"] + PAGE
    np_ = (s["n_compressed"].long() // PAGE)[:, None]
    i = torch.arange(mp, device="cuda")[None]
    key = torch.where((i < case["sink"]) | (i >= np_ - case["recent"]), math.inf, s["mass"])
    key = torch.where(i < np_, key, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices
    stay = torch.zeros(b, mp, dtype=torch.bool, device="cuda").scatter_(1, order, i.expand(b, mp) < budget) & (i < np_)
    kind = torch.where(stay, 0, torch.where(i < np_, 1, 2))
    perm = kind.sort(dim=-1, stable=True).indices
    n_keep = np_.clamp(max=budget)
    table = s["table"].gather(1, perm)
    mass = torch.where(i < n_keep, s["mass"].gather(1, perm), 0.0)
    kept = torch.full((b, budget), -1, dtype=torch.int32, device="cuda")
    m = min(budget, mp)
    kept[:, :m] = torch.where(i < n_keep, perm, -1)[:, :m].int()
    gone = PAGE * (np_ - n_keep)                                                       # tokens
    slot = (torch.arange(ring, device="cuda")[None] + gone) % ring
    row = slot[:, None, :, None].expand_as(s["win_k"])
    return (table, (s["seq_len"] - gone[:, 0]).int(), (s["n_compressed"] - gone[:, 0]).int(), s["win_k"].gather(2, row),
            s["win_v"].gather(2, row), mass, kept)


PLAIN = {"write": plain_write, "decode": plain_decode, "prefill": plain_prefill, "sparse": plain_sparse, "track": plain_track,
         "evict": plain_evict}


# ---------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits, one sequence after the other."""
    if own:
        return None
    s = prepare(case, seed)
    op, b, hkv, g, d, w = case["op"], case["batch"], case["hkv"], case["g"], case["d"], case["window"]
    T, nc, ring = lengths(case), compressed(case), w + PAGE
    if op == "write":
        outs = []
        for x in (s["k"], s["v"]):
            y = x.double()
            for i in range(0, nc[0], PAGE):
                t = y[:, i:i + PAGE]
                a = (t.abs().amax((1, 3), keepdim=True).float() / 127).double()
                y[:, i:i + PAGE] = torch.round(t / a) * a if float(a.min()) > 0 else torch.where(a > 0, torch.round(t / a) * a, 0.0)
            y[:, nc[0]:] = x[:, nc[0]:].half().double()
            outs.append(y)
        return outs[0], outs[1], None, None
    if op == "track":
        m = s["mass"].double()
        for i in range(b):
            p = torch.exp(s["scores"][i, :, :nc[i]].double() - s["lse"][i].double()[:, None]).sum(0)
            m[i, :nc[i] // PAGE] += p.reshape(-1, PAGE).sum(1)
        return m
    if op == "evict":
        out = [None] * 7
        m = torch.zeros_like(s["mass"]).double()
        wk, wv = s["win_k"].double().clone(), s["win_v"].double().clone()
        for i in range(b):
            n = nc[i] // PAGE
            if n <= case["budget"]:
                m[i, :n] = s["mass"][i, :n].double()
                continue
            forced = set(range(min(n, case["sink"]))) | set(range(max(0, n - case["recent"]), n))
            mass = s["mass"][i, :n].double().tolist()
            rest = sorted((j for j in range(n) if j not in forced), key=lambda j: (-mass[j], j))
            keep = sorted(list(forced) + rest[:case["budget"] - len(forced)])
            m[i, :len(keep)] = torch.tensor([mass[j] for j in keep], dtype=torch.float64, device="cuda")
            by = (PAGE * (n - len(keep))) % ring
            wk[i], wv[i] = wk[i].roll(-by, 1), wv[i].roll(-by, 1)
        out[3], out[4], out[5] = wk, wv, m
        return tuple(out)
    nq = case.get("nq", 1)
    q = s["q"].double().reshape(b, nq, hkv, g, d)
    outs, lses = [], []
    chosen = plain_choice(s) if op == "sparse" else None
    for i in range(b):
        at = torch.tensor([(j % ring) for j in range(nc[i], T[i])], dtype=torch.long, device="cuda")
        for h in range(hkv):
            ords = torch.arange(nc[i] // PAGE, device="cuda") if chosen is None else chosen[i][h]
            rows = s["raw"][s["table"][i].long()[ords], h]
            where = (ords[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)
            where = torch.cat([where, torch.arange(nc[i], T[i], device="cuda")])
            z = [x.double() for x in unpack_pages(rows[:, None], d)]
            k = torch.cat([(z[0][:, 0] * z[2][:, :, None]).reshape(-1, d), s["win_k"][i, h, at].double()])
            v = torch.cat([(z[1][:, 0] * z[3][:, :, None]).reshape(-1, d), s["win_v"][i, h, at].double()])
            for r in range(0, nq, 512):
                qs = q[i, r:r + 512, h]                                                # [rows, g, d]
                l = torch.einsum("rgd,nd->rgn", qs, k) * s["scale"]
                pos = T[i] - nq + r + torch.arange(qs.shape[0], device="cuda")
                l = l.masked_fill((where[None] > pos[:, None])[:, None], -math.inf)
                outs.append((i, h, r, torch.einsum("rgn,nd->rgd", torch.softmax(l, -1), v)))
                lses.append((i, h, r, torch.logsumexp(l, -1)))
    o = torch.zeros(b, nq, hkv, g, d, dtype=torch.float64, device="cuda")
    z = torch.zeros(b, nq, hkv, g, dtype=torch.float64, device="cuda")
    for i, h, r, x in outs:
        o[i, r:r + x.shape[0], h] = x
    for i, h, r, x in lses:
        z[i, r:r + x.shape[0], h] = x
    o, z = o.reshape(s["q"].shape), z.reshape(s["q"].shape[:-1])
    return (None, None, o, z) if op == "sparse" else (o, z)


def plain_choice(s):
    """The pages that the definition takes, from whole-number scores, one (sequence, KV head) after the other."""
    case = s["case"]
    b, hkv, g, d = case["batch"], case["hkv"], case["g"], case["d"]
    nc, found = compressed(case), []
    for i in range(b):
        n, of = nc[i] // PAGE, []
        for h in range(hkv):
            rows = s["raw"][s["table"][i, :n].long(), h]
            lo, hi = rows[:, :d].contiguous().view(torch.int8).long(), rows[:, d:2 * d].contiguous().view(torch.int8).long()
            ks = rows[:, 2 * d:2 * d + 4].contiguous().view(torch.float32)[:, 0]
            q = s["q"][i, h * g:(h + 1) * g].double()
            step = (q.abs().max().float() / 127).double()
            qi = (torch.round(q / step) if float(step) > 0 else q * 0).long()
            best = torch.maximum(qi[:, None] * lo, qi[:, None] * hi).sum(-1).amax(0) if n else ks.long()
            value = (best.float() * ks).tolist()
            forced = set(range(min(n, case["sink"]))) | set(range(max(0, n - case["recent"]), n))
            rest = sorted((j for j in range(n) if j not in forced), key=lambda j: (-value[j], j))
            take = sorted(list(forced) + rest[:case["k"] - len(forced)]) if n > case["k"] else list(range(n))
            of.append(torch.tensor(take, dtype=torch.long, device="cuda"))
        found.append(of)
    return found
