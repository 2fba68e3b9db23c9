"""Cases for timing the operators on a paged key-value cache: attention of new tokens, attention of prompts, appending, and page
keeping (forks, releases, compaction).

Each case has a plain form in elementary torch operations and, where `own` is set, the framework's call. Sizes stand for one layer
of the decoders this repository serves (hidden 5120 as 40 heads of 128; hidden 2048 as 32 heads of 64; up to 32 rows in a
speculative verify step) and generic grouped-query layouts.
"""
import math

import torch

own = False

WORKSPACE_BYTES = 64 << 20


def listed():
    A = dict(op="attend", window=0, sinks=0, kv="bf16")
    P = dict(op="prompt", window=0, sinks=0, kv="bf16")
    return [
        # one user, a chat of two thousand tokens: latency
        dict(A, name="token_b1_2k", batch=1, new=1, lo=1999, hi=1999, heads=8, group=4, dim=128, page=64),
        # speculative verify: 8 sequences x 4 positions (32 rows), 40 heads on 8, 8-bit cache of small pages
        dict(A, name="verify_b8_e4m3", batch=8, new=4, lo=517, hi=24001, heads=8, group=5, dim=128, page=16, kv="e4m3"),
        # a full serving batch over long contexts
        dict(A, name="token_b64_16k", batch=64, new=1, lo=9001, hi=22003, heads=8, group=4, dim=128, page=64),
        # a serving batch of long streams: a window and a few first tokens; the pages in between were given up
        dict(A, name="token_b96_window", batch=96, new=1, lo=40, hi=131072, heads=4, group=8, dim=64, page=32, window=4096, sinks=7),
        # a few short prompts at once, 64-wide heads, nothing cached before, 8-bit cache
        dict(P, name="prompt_ragged_small", batch=3, lo_new=1, hi_new=197, past=0, heads=8, group=4, dim=64, page=16, kv="e4m3"),
        # a long prompt under a sliding window
        dict(P, name="prompt_8k_window", batch=1, lo_new=8192, hi_new=8192, past=0, heads=8, group=5, dim=128, page=64, window=1024, sinks=16),
        # chunks of a prompt that continue long contexts
        dict(P, name="prompt_chunk_2k_on_14k", batch=2, lo_new=1500, hi_new=2048, past=14336, heads=8, group=4, dim=128, page=64),
        # the new token of each sequence into an 8-bit cache
        dict(op="append", name="append_b64_e4m3", batch=64, lo_new=1, hi_new=1, past=3000, heads=8, dim=128, page=16, kv="e4m3"),
        # ragged prompts of 16 thousand tokens in all
        dict(op="append", name="append_16k", batch=6, lo_new=1001, hi_new=4460, past=0, heads=8, dim=128, page=64, kv="bf16"),
        # 48 prompts sampled four ways each, then the prompts let go
        dict(op="fork", name="fork_48x4", sources=48, ways=4, lo=700, hi=6001, heads=8, dim=128, page=64, kv="bf16"),
        # a small pool tidied up
        dict(op="compact", name="compact_1k", pages=1024, used=0.3, seqs=16, heads=8, dim=128, page=16, kv="e4m3"),
        # a large pool, half full, tidied up
        dict(op="compact", name="compact_24k", pages=24576, used=0.5, seqs=128, heads=8, dim=128, page=32, kv="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("attend", "attend", "prompt", "prompt", "append", "fork", "compact"))
    heads, dim, page = rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 128)), rng.choice((16, 32, 64, 128))
    kv = rng.choice(("bf16", "e4m3"))
    if op == "attend":
        batch = log(1, 96)
        hi = log(16, min(131072, 900000 // batch))
        w = rng.choice((0, 0, 1)) * log(16, 8192)
        # few rows of a key-value head at once: single tokens, and verify steps of up to 32 rows
        group = rng.randint(1, 8)
        return dict(op=op, batch=batch, new=rng.choice((1, 1, min(4, 32 // group))), lo=log(8, hi), hi=hi, heads=heads, group=group, dim=dim, page=page,
                    kv=kv, window=w, sinks=rng.choice((0, 1, 4, 130)) if w else 0)
    if op == "prompt":
        batch = rng.choice((1, 1, 2, 3, 5))
        hi_new = log(64, 8192 // batch)
        past = rng.choice((0, log(32, 8192)))
        w = rng.choice((0, 1)) * log(64, 4096)
        case = dict(op=op, batch=batch, lo_new=log(1, hi_new), hi_new=hi_new, past=past, heads=heads, group=rng.randint(1, 5), dim=dim, page=page,
                    kv=kv, window=w, sinks=rng.choice((0, 1, 4, 130)) if w else 0)
        while work(case)["flops"] > 8e11:
            case["hi_new"] //= 2
            case["lo_new"] = min(case["lo_new"], case["hi_new"])
        return case
    if op == "append":
        batch = log(1, 64)
        hi_new = log(1, 16384 // batch)
        return dict(op=op, batch=batch, lo_new=log(1, hi_new), hi_new=hi_new, past=rng.choice((0, log(8, 2048))), heads=heads, dim=dim, page=page, kv=kv)
    if op == "fork":
        hi = log(32, 6000)
        return dict(op=op, sources=log(1, 48), ways=rng.randint(1, 4), lo=log(8, hi), hi=hi, heads=heads, dim=dim, page=page, kv=kv)
    return dict(op=op, pages=log(100, 24576), used=round(rng.uniform(0.05, 0.95), 3), seqs=log(1, 64), heads=heads, dim=dim, page=min(page, 32), kv=kv)


# ------------------------------------------------------------------------------------------------ sizes that follow from a case


def spread(lo, hi, n):
    """n lengths between lo and hi, both reached, in an order that is not sorted."""
    if n == 1:
        return [hi]
    step = next(s for s in (7, 11, 13, 17, 1) if math.gcd(s, n) == 1)
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def lengths(case):
    """(new tokens, tokens with the new ones) of each sequence."""
    b = case["batch"]
    if case["op"] == "attend":
        new = [case["new"]] * b
        return new, [max(x, case["new"]) for x in spread(case["lo"], case["hi"], b)]
    new = spread(case["lo_new"], case["hi_new"], b)
    return new, [n + (case["past"] * (3 + i % 2) // 4 if i else case["past"]) for i, n in enumerate(new)]


def seen(case, new, length):
    """The positions that some new token of a sequence sees, as two ranges: [0, a) and [b, length)."""
    w = case["window"]
    if not w:
        return 0, 0
    b = max(0, length - new - w + 1)
    a = min(case["sinks"], length)
    return (0, 0) if b <= a else (a, b)


def pairs(case, new, length):
    """Sum over the new tokens of the number of positions that they see."""
    w, s, total = case["window"], case["sinks"], 0
    for p in range(length - new, length):
        total += p + 1 if not w else min(w, p + 1) + min(s, max(0, p + 1 - w))
    return total


def work(case):
    op = case["op"]
    size = 2 if case["kv"] == "bf16" else 1
    row = case["heads"] * case["dim"]
    if op in ("attend", "prompt"):
        news, lens = lengths(case)
        kept = sum(a + n - b for n, (a, b) in zip(lens, (seen(case, m, n) for m, n in zip(news, lens))))
        q = sum(news) * row * case["group"]
        return {"bytes": 2.0 * kept * row * size + 4.0 * q,
                "flops": 4.0 * row * case["group"] * sum(pairs(case, m, n) for m, n in zip(news, lens))}
    if op == "append":
        t = sum(lengths(case)[0])
        return {"bytes": 2.0 * t * row * (2 + size), "flops": 2.0 * t * row}
    if op == "fork":
        lens = spread(case["lo"], case["hi"], case["sources"])
        tails = sum(n % case["page"] for n in lens) * case["ways"]
        entries = sum(-(-n // case["page"]) for n in lens) * (2 + 3 * case["ways"])
        return {"bytes": 4.0 * tails * row * size + 4.0 * entries, "flops": 1.0 * entries}
    live, moved = layout(case)[2:]
    return {"bytes": 4.0 * moved * row * case["page"] * size + 12.0 * case["pages"], "flops": 1.0 * case["pages"]}


def layout(case):
    """A pool in use: (pages of each sequence, pages shared by two sequences, live pages, live pages that have to move)."""
    n = max(1, int(case["pages"] * case["used"]))
    each = [n * (i + 1) // case["seqs"] - n * i // case["seqs"] for i in range(case["seqs"])]
    mul = next(m for m in (7919, 7907, 7901, 1) if math.gcd(m, case["pages"]) == 1)
    ids = [(i * mul + 3) % case["pages"] for i in range(n)]
    return each, ids, n, sum(i >= n for i in ids)


# ------------------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    op, heads, dim, page = case["op"], case["heads"], case["dim"], case["page"]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def pool(pages):
        x = normal(pages, heads, page, dim)
        if case["kv"] == "bf16":
            return x
        x.mul_(64)
        return x.to(torch.float8_e4m3fn)

    if case["kv"] == "e4m3":
        s["k_scale"] = (torch.rand(heads, generator=g, device="cuda") + 0.5) / 64
        s["v_scale"] = (torch.rand(heads, generator=g, device="cuda") + 0.5) / 64
    else:
        s["k_scale"] = s["v_scale"] = None
    if op in ("attend", "prompt", "append"):
        news, lens = lengths(case)
        widest = -(-max(lens) // page)
        ends = [0]
        for m in news:
            ends.append(ends[-1] + m)
        s["max_new"] = max(news)
        s["lens"], s["start"] = ints(lens), ints(ends) if min(news) < max(news) else None
        s["seq"] = ints([b for b, m in enumerate(news) for _ in range(m)]).long()
        s["nth"] = ints([i for m in news for i in range(m)]).long()
        s["news"] = ints(news)
        s["longest"] = max(lens)
        # pages that no position in use lies in are not there: the cache gave them up
        have = torch.zeros(len(lens), widest, dtype=torch.bool, device="cuda")
        for b, (m, n) in enumerate(zip(news, lens)):
            lo, hi = seen(case, m, n) if op != "append" else (0, max(0, n - m))
            have[b, : -(-lo // page)] = True
            have[b, hi // page: -(-n // page)] = True
        count = int(have.sum())
        s["table"] = torch.full((len(lens), widest), -1, dtype=torch.int32, device="cuda")
        s["table"][have] = torch.randperm(count, generator=g, device="cuda").int()
        s["k"], s["v"] = pool(count), pool(count)
        if op == "append":
            # the keys and values of a fused projection's output
            qkv = normal(ends[-1], 2, heads, dim)
            s["new_k"], s["new_v"] = qkv[:, 0], qkv[:, 1]
        else:
            s["q"] = normal(ends[-1], heads * case["group"], dim) * 1.5
            s["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        return s
    if op == "fork":
        lens = spread(case["lo"], case["hi"], case["sources"])
        n_seq, widest = case["sources"] * (1 + case["ways"]), -(-max(lens) // page)
        held = [-(-n // page) for n in lens]
        pages = sum(held) + case["sources"] * case["ways"] + 5
        ids = torch.randperm(pages, generator=g, device="cuda").int()
        have = torch.arange(widest, device="cuda")[None] < ints(held)[:, None]
        table = torch.full((n_seq, widest), -1, dtype=torch.int32, device="cuda")
        table[: case["sources"]][have] = ids[: sum(held)]
        refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        refs[ids[: sum(held)].long()] = 1
        all_lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
        all_lens[: case["sources"]] = ints(lens)
        s["src"] = torch.arange(case["sources"], device="cuda", dtype=torch.int32).repeat_interleave(case["ways"])
        s["dst"] = torch.arange(case["sources"], n_seq, device="cuda", dtype=torch.int32)
        s["gone"] = torch.arange(case["sources"], device="cuda", dtype=torch.int32)
    else:
        each, ids, n, _ = layout(case)
        pages, widest = case["pages"], max(each)
        have = torch.arange(widest, device="cuda")[None] < ints(each)[:, None]
        table = torch.full((case["seqs"] + 1, widest), -1, dtype=torch.int32, device="cuda")
        table[:-1][have] = ints(ids)[torch.randperm(n, generator=g, device="cuda")]
        # a fork of the first sequence shares its pages
        table[-1] = table[0]
        refs = torch.bincount(table[table >= 0].long(), minlength=pages).int()
        all_lens = ints(each + [each[0]]) * page
    s["k"], s["v"] = pool(pages), pool(pages)
    # the bookkeeping in one buffer, and as it stands before the pass
    s["before"] = torch.cat([table.reshape(-1), all_lens, refs])
    s["now"] = s["before"].clone()
    a, b = table.numel(), table.numel() + all_lens.numel()
    s["table"], s["lens"], s["refs"] = s["now"][:a].view(table.shape), s["now"][a:b], s["now"][b:]
    return s


# ------------------------------------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if op in ("fork", "compact"):
        s["now"].copy_(s["before"])
    return (run_own if own else run_plain)(s, op)


def run_own(s, op):
    import nvfp4_block_scaled_04_gb300 as nv

    cache = nv.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if op in ("attend", "prompt"):
        c = s["case"]
        return nv.paged_attention(s["q"], cache, s["table"], s["lens"], start=s["start"], max_new=s["max_new"], window=c["window"], sinks=c["sinks"],
                                  workspace=s["workspace"])
    if op == "append":
        nv.kv_append(cache, s["new_k"], s["new_v"], s["table"], s["lens"], start=s["start"], max_new=s["max_new"])
        return s["k"], s["v"]
    if op == "fork":
        nv.kv_fork(cache, s["table"], s["lens"], s["refs"], s["src"], s["dst"])
        nv.kv_release(s["table"], s["lens"], s["refs"], s["gone"])
        return s["k"], s["v"], s["table"], s["lens"], s["refs"]
    live = nv.kv_compact(cache, s["table"], s["refs"])
    return s["k"], s["v"], s["table"], s["refs"], live


def raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def rows(pool, page, nth, scale):
    """pool[page, :, nth] as 32-bit values: [..., heads, dim]."""
    x = raw(pool)[page, :, nth]
    if scale is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * scale[:, None]


def run_plain(s, op):
    if op in ("attend", "prompt"):
        return plain_attention(s)
    if op == "append":
        at = (s["lens"] - s["news"]).long()[s["seq"]] + s["nth"]
        size = s["k"].shape[2]
        page = s["table"][s["seq"], at // size].long()
        for pool, x, scale in ((s["k"], s["new_k"], s["k_scale"]), (s["v"], s["new_v"], s["v_scale"])):
            if scale is not None:
                x = (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            raw(pool)[page, :, at % size] = raw(x)
        return s["k"], s["v"]
    if op == "fork":
        return plain_fork(s)
    return plain_compact(s)


def plain_attention(s):
    c, q, table, lens = s["case"], s["q"], s["table"], s["lens"].long()
    heads, group, dim, size = c["heads"], c["group"], c["dim"], c["page"]
    window, sinks, most = c["window"], c["sinks"], s["max_new"]
    first = lens - s["news"]
    at = torch.arange(s["longest"], device=q.device)[None].expand(len(lens), -1)
    if window:
        # the sinks, then what the first new token's window reaches
        skip = (first - window + 1 - sinks).clamp(min=0)
        width = min(s["longest"], sinks + window + most)
        at = at[:, :width]
        at = torch.where(at < sinks, at, at + skip[:, None])
    there = at < lens[:, None]
    page = table.gather(1, at.clamp(max=s["longest"] - 1) // size).long()
    there = there & (page >= 0)
    page = page.clamp(min=0)
    k = rows(s["k"], page, at % size, s["k_scale"]).permute(0, 2, 3, 1)
    padded = torch.zeros(len(lens), most, heads, group, dim, device=q.device)
    padded[s["seq"], s["nth"]] = q.float().view(-1, heads, group, dim)
    p = padded.permute(0, 2, 3, 1, 4).reshape(len(lens), heads, group * most, dim) @ k
    del k
    pos = first[:, None] + torch.arange(most, device=q.device)
    ok = there[:, None] & (at[:, None] <= pos[:, :, None])
    if window:
        ok = ok & ((pos[:, :, None] - at[:, None] < window) | (at[:, None] < sinks))
    p = p.view(len(lens), heads, group, most, -1).mul_(dim ** -0.5).masked_fill_(~ok[:, None, None], -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e38)).exp_()
    total = p.sum(-1)
    v = rows(s["v"], page, at % size, s["v_scale"]).permute(0, 2, 1, 3)
    out = (p.view(len(lens), heads, group * most, -1) @ v).view(len(lens), heads, group, most, dim)
    out = torch.where(total[..., None] > 0, out / total[..., None], torch.zeros((), device=q.device))
    return out.permute(0, 3, 1, 2, 4)[s["seq"], s["nth"]].reshape(q.shape).bfloat16()


def plain_fork(s):
    table, lens, refs, size = s["table"], s["lens"], s["refs"], s["case"]["page"]
    src, dst = s["src"].long(), s["dst"].long()
    n = lens[src].long()
    full, tail = n // size, n % size
    rest = tail > 0
    shared = torch.arange(table.shape[1], device=table.device)[None] < full[:, None]
    mine = torch.where(shared, table[src], -1)
    refs.index_add_(0, mine.clamp(min=0).view(-1).long(), (mine >= 0).view(-1).int())
    # the lowest free pages, in the order of the forks that need one
    free = torch.argsort((refs > 0).int(), stable=True)
    fresh = free[(rest.long().cumsum(0) - 1).clamp(min=0)]
    mine = torch.where(rest[:, None] & (torch.arange(table.shape[1], device=table.device)[None] == full[:, None]), fresh[:, None].int(), mine)
    refs.index_put_((fresh,), rest.int(), accumulate=True)
    old = table[src, full.clamp(max=table.shape[1] - 1)].long().clamp(min=0)
    keep = rest[:, None, None, None] & (torch.arange(size, device=table.device)[None, None, :, None] < tail[:, None, None, None])
    fresh = torch.where(rest, fresh, old)
    for pool in (raw(s["k"]), raw(s["v"])):
        pool[fresh] = torch.where(keep, pool[old], pool[fresh])
    table[dst], lens[dst] = mine, n.int()
    gone = s["gone"].long()
    held = table[gone]
    refs.index_add_(0, held.clamp(min=0).view(-1).long(), -(held >= 0).view(-1).int())
    table[gone] = -1
    lens[gone] = 0
    return s["k"], s["v"], table, lens, refs


def plain_compact(s):
    table, refs = s["table"], s["refs"]
    used = refs > 0
    live = used.sum(dtype=torch.int32)
    page = torch.arange(len(refs), device=refs.device)
    moves, holes = used & (page >= live), ~used & (page < live)
    src, dst = page[moves], page[holes]
    to = page.clone()
    to[src] = dst
    for pool in (raw(s["k"]), raw(s["v"])):
        pool[dst] = pool[src]
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    return s["k"], s["v"], table, refs, live


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """The definition, sequence by sequence and head by head."""
    s = prepare(case, seed)
    op, size = case["op"], case["page"]

    def value(x):
        return raw(x).view(torch.float8_e4m3fn).double() if x.dtype == torch.float8_e4m3fn else x.double()

    if op == "append":
        news, lens = lengths(case)
        k, v = value(s["k"]), value(s["v"])
        t = 0
        for b, (m, n) in enumerate(zip(news, lens)):
            at = torch.arange(n - m, n, device="cuda")
            page = s["table"][b].long()[at // size]
            k[page, :, at % size] = value(s["new_k"][t:t + m]) / (1 if s["k_scale"] is None else s["k_scale"].double()[:, None])
            v[page, :, at % size] = value(s["new_v"][t:t + m]) / (1 if s["v_scale"] is None else s["v_scale"].double()[:, None])
            t += m
        return k, v
    if op in ("fork", "compact"):
        return None  # whole pages and whole numbers: nothing is computed
    news, lens = lengths(case)
    out, t = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (m, n) in enumerate(zip(news, lens)):
        a, lo = seen(case, m, n)
        at = torch.cat([torch.arange(a, device="cuda"), torch.arange(lo, n, device="cuda")])
        page = s["table"][b].long()[at // size]
        pos = torch.arange(n - m, n, device="cuda")
        ok = at[None] <= pos[:, None]
        if case["window"]:
            ok &= (pos[:, None] - at[None] < case["window"]) | (at[None] < case["sinks"])
        for h in range(case["heads"]):
            k = value(raw(s["k"])[page, h, at % size].view(s["k"].dtype))
            v = value(raw(s["v"])[page, h, at % size].view(s["v"].dtype))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for i in range(h * case["group"], (h + 1) * case["group"]):
                x = (s["q"][t:t + m, i].double() @ k.T) / math.sqrt(case["dim"])
                x.masked_fill_(~ok, -math.inf)
                out[t:t + m, i] = torch.softmax(x, -1) @ v
        t += m
    return out
