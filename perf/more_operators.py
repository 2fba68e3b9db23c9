"""Cases for timing what stands between the 4-bit linears of a decoder and behind its head: the root-mean-square norm with the
residual's addition (outputs in bf16, in E4M3 with a scale for each row, and in NVFP4 in front of a W4A4 linear), and the draw of
the next token (temperature, top-k, top-p, min-p, from given random numbers), alone and as a speculative verification.

Each case has a plain form in elementary torch operations and, where `own` is set, the framework's calls. Sizes are the hidden
size and the vocabulary that this repository serves (5120; 248,320 rows of the head), its mixture-of-experts hidden size (2048),
heads of 128, and generic odd ones.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


def listed():
    N = dict(op="norm", heads=1, others=0, residual="bf16", out="bf16", offset=0.0)
    S = dict(op="sample", dtype="bf16", masked=False)
    return [
        # one token in front of a W4A16 linear: latency
        dict(N, name="norm_1x5120", tokens=1, dim=5120),
        # the query heads of a fused projection's output, each normalised by itself, for a prompt
        dict(N, name="norm_heads_4096x40x128", tokens=4096, dim=128, heads=40, others=16, residual="none"),
        # a prefill batch, bf16 stream
        dict(N, name="norm_8192x5120", tokens=8192, dim=5120),
        # a ragged batch of decode and prompt rows into an 8-bit linear, gains stored as what is added to one
        dict(N, name="norm_e4m3_333x2048", tokens=333, dim=2048, out="e4m3", offset=1.0),
        # a prefill batch into an 8-bit linear, the stream kept in 32 bits
        dict(N, name="norm_e4m3_8192x5120_f32", tokens=8192, dim=5120, out="e4m3", residual="f32"),
        # in front of a W4A4 linear: a prompt's key and value projection, tensor scale from the data
        dict(N, name="norm_w4a4_4096x5120", tokens=4096, dim=5120, out="w4a4", columns=2048, given=False),
        # the same for a few rows, with a calibrated tensor scale
        dict(N, name="norm_w4a4_17x2048", tokens=17, dim=2048, out="w4a4", columns=1536, given=True),
        # one user: the usual settings of a chat
        dict(S, name="sample_1_chat", rows=1, vocab=248320, mode="chat"),
        # a serving batch, every row with settings of its own, some under a grammar's mask, some greedy
        dict(S, name="sample_64_mixed", rows=64, vocab=248320, mode="mixed", masked=True),
        # many samples of a model's own distribution
        dict(S, name="sample_256_plain", rows=256, vocab=248320, mode="plain"),
        # logits that a program has worked on in 32 bits, odd vocabulary
        dict(S, name="sample_f32_24_nucleus", rows=24, vocab=151937, mode="nucleus", dtype="f32"),
        # verification of 8 sequences x (3 drafts + 1)
        dict(S, name="verify_8x4", op="verify", batch=8, drafts=3, vocab=248320, mode="chat"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("norm", "norm", "norm", "sample", "sample", "verify"))
    if op == "norm":
        out = rng.choice(("bf16", "bf16", "e4m3", "e4m3", "w4a4"))
        heads = rng.choice((1, 1, 1, rng.randint(2, 40))) if out != "w4a4" else 1
        unit = 64 if out == "w4a4" else 8
        dim = unit * log(max(1, 64 // unit), (512 if heads > 1 else 16384 if out != "w4a4" else 8192) // unit)
        case = dict(op=op, heads=heads, others=rng.randint(0, 16) if heads > 1 else 0, residual=rng.choice(("none", "bf16", "bf16", "f32")) if heads == 1 else "none",
                    out=out, offset=rng.choice((0.0, 1.0)), dim=dim, tokens=log(1, min(16384, 8192 * 5120 // (heads * dim))))
        if out == "w4a4":
            case["columns"], case["given"] = 8 * log(8, 256), rng.choice((False, True))
        return case
    mode = rng.choice(("chat", "plain", "nucleus", "floor", "mixed", "mixed"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    vocab = log(1000, 262144)
    if op == "sample":
        most = 256 * 248320 // (1 if dtype == "bf16" else 2) // vocab
        return dict(op=op, rows=log(1, min(512, most)), vocab=vocab, mode=mode, dtype=dtype, masked=rng.choice((False, True)))
    drafts = rng.randint(0, 7)
    return dict(op=op, batch=log(1, 64 // (drafts + 1)), drafts=drafts, vocab=vocab, mode=mode, dtype=dtype, masked=False)


def row_count(case):
    return case["rows"] if case["op"] == "sample" else case["batch"] * (case["drafts"] + 1)


def work(case):
    if case["op"] == "norm":
        n = case["tokens"] * case["heads"] * case["dim"]
        size = 2.0 + {"none": 0, "bf16": 4, "f32": 8}[case["residual"]]
        rows = case["tokens"] * case["heads"]
        if case["out"] == "w4a4":
            m, c, k = case["tokens"], case["columns"], case["dim"]
            return {"bytes": n * size + 2.0 * k + c * k * 9 / 16 + 2.0 * m * c, "flops": 2.0 * m * c * k + 12.0 * n}
        return {"bytes": n * (size + (2 if case["out"] == "bf16" else 1)) + 2.0 * case["dim"] + (0 if case["out"] == "bf16" else 4.0 * rows),
                "flops": 8.0 * n}
    rows = row_count(case)
    return {"bytes": rows * case["vocab"] * (2.0 if case["dtype"] == "bf16" else 4.0) + 28.0 * rows, "flops": 2.0 * rows * case["vocab"]}


# ------------------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    if case["op"] == "norm":
        tokens, heads, dim = case["tokens"], case["heads"], case["dim"]
        shape = (tokens, heads, dim) if heads > 1 else (tokens, dim)
        if heads > 1:  # a slice of a fused projection's output
            s["x"] = normal(tokens, heads + case["others"], dim).bfloat16()[:, :heads]
        else:
            s["x"] = normal(*shape).bfloat16()
        s["weight"] = (normal(dim) * 0.1 + (1 - case["offset"])).bfloat16()
        s["residual"] = s["residual_out"] = None
        if case["residual"] != "none":
            # a stream with a few channels far above the others
            r = normal(*shape) * 2
            r[..., torch.randint(0, dim, (max(1, dim // 512),), generator=g, device="cuda")] *= 30
            s["residual"] = r.bfloat16() if case["residual"] == "bf16" else r
            s["residual_out"] = torch.empty_like(s["residual"])
        if case["out"] == "w4a4":
            n = case["columns"]
            s["codes"] = torch.randint(0, 256, (n, dim // 2), generator=g, device="cuda", dtype=torch.uint8)
            scales = (rand(n, dim // 16) * 200 + 20).to(torch.float8_e4m3fn).view(torch.uint8)
            # the layout of the tensor cores: 128 x 4 tiles, row r and column c of a tile at (r % 32) * 16 + (r / 32) * 4 + c
            high, wide = -(-n // 128), -(-(dim // 16) // 4)
            padded = torch.zeros(high * 128, wide * 4, dtype=torch.uint8, device="cuda")
            padded[:n, : dim // 16] = scales
            s["scales"] = padded.view(high, 4, 32, wide, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
            s["scale"] = (rand(1) + 0.5) * 1e-4
            s["s_t"] = (rand(1) + 4) / 2688 if case["given"] else None
        return s
    rows, vocab = row_count(case), case["vocab"]
    # logits that fall with the logarithm of a rank, as steep as a row is sure of what comes next
    steep = rand(rows, 1) * 1.5 + 1.0
    x = rand(rows, vocab).mul_(vocab).add_(1).log_().mul_(-steep).add_(normal(rows, vocab), alpha=0.5).add_(18.0)
    if case["masked"]:
        # every fourth row under a grammar: a hundredth of the vocabulary is left
        x[::4].masked_fill_(rand(x[::4].shape[0], vocab) > 0.01, -math.inf)
    s["logits"] = x.bfloat16() if case["dtype"] == "bf16" else x
    s["uniform"] = rand(rows)
    n = case["batch"] if case["op"] == "verify" else rows  # a sequence's settings serve all its rows
    one = torch.ones(n, device="cuda")
    chat, free = (0.7, 20, 0.8, 0.0), (1.0, 0, 1.0, 0.0)
    t, k, p, m = {"chat": chat, "plain": free, "nucleus": (1.0, 0, 0.95, 0.0), "floor": (1.2, 0, 1.0, 0.05), "mixed": free}[case["mode"]]
    s["temperature"], s["top_p"], s["min_p"] = one * t, one * p, one * m
    s["top_k"] = torch.full((n,), k, dtype=torch.int32, device="cuda")
    if case["mode"] == "mixed":
        kind = torch.arange(n, device="cuda") % 5  # a greedy row, top-k, top-p, min-p, all three
        s["temperature"] = torch.where(kind == 0, 0.0, 0.6 + 0.8 * rand(n))
        s["top_k"] = torch.where((kind == 1) | (kind == 4), torch.randint(1, 200, (n,), generator=g, device="cuda"), 0).int()
        s["top_p"] = torch.where((kind == 2) | (kind == 4), 0.5 + 0.49 * rand(n), 1.0)
        s["min_p"] = torch.where((kind == 3) | (kind == 4), 0.2 * rand(n), 0.0)
    if case["op"] == "verify":
        # drafts that are often the likeliest token
        best = s["logits"].float().argmax(-1).view(n, -1)[:, : case["drafts"]]
        other = torch.randint(0, vocab, best.shape, generator=g, device="cuda")
        s["draft_ids"] = torch.where(rand(*best.shape) < 0.8, best, other).int()
    return s


# ------------------------------------------------------------------------------------------------ one pass


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import nvfp4_block_scaled_04_gb300 as nv

    c = s["case"]
    if c["op"] == "norm":
        given = dict(eps=EPS, residual=s["residual"], residual_out=s["residual_out"], weight_offset=c["offset"])
        if c["out"] == "bf16":
            return nv.rms_norm(s["x"], s["weight"], **given)
        if c["out"] == "e4m3":
            return nv.rms_norm_e4m3(s["x"], s["weight"], **given)
        got = nv.rms_norm_quantize(s["x"], s["weight"], s_t=s["s_t"], scale_layout=nv.SCALES_MMA, **given)
        q, *stream = got if isinstance(got, tuple) else (got,)
        w = nv.QTensor(s["codes"], s["scales"], s["scale"], c["columns"], c["dim"], 1, nv.SCALES_MMA)
        return (nv.gemm_w4a4(q, w), q.s_t, *stream)
    settings = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    if c["op"] == "sample":
        return nv.sample(s["logits"], s["uniform"], **settings)
    return nv.verify_sample(s["logits"], s["uniform"], s["draft_ids"], **settings)


def run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return plain_norm(s)
    each = 1 if c["op"] == "sample" else c["drafts"] + 1
    t, k, p, m = (s[n].repeat_interleave(each)[:, None] for n in ("temperature", "top_k", "top_p", "min_p"))
    ids, probs = plain_sample(s["logits"], s["uniform"], t.double(), k.long(), p.double(), m.double())
    if c["op"] == "sample":
        return ids, probs
    tokens = ids.view(c["batch"], each)
    same = (tokens[:, :-1] == s["draft_ids"]).int()
    return tokens, same.cumprod(1).sum(1).int(), probs.view(tokens.shape)


def plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    stream = ()
    if s["residual"] is not None:
        s["residual_out"].copy_(x + s["residual"].float())
        stream = (s["residual_out"],)
        x = s["residual_out"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (s["weight"].float() + c["offset"])
    if c["out"] == "bf16":
        y = y.bfloat16()
        return (y, *stream) if stream else y
    if c["out"] == "e4m3":
        most = y.abs().amax(-1)
        scale = torch.where(most > 0, most / 448, 1.0)
        return ((y / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale.view(-1), *stream)
    rows, dim, n = c["tokens"], c["dim"], c["columns"]
    s_t = s["s_t"] if c["given"] else (y.abs().amax() / 2688).view(1)
    blocks = y.view(rows, dim // 16, 16)
    sb = (blocks.abs().amax(-1, keepdim=True) / (s_t * 6)).clamp(max=448).to(torch.float8_e4m3fn).float()
    a = torch.where(sb > 0, blocks / (sb * s_t), 0.0)
    m = a.abs()
    # 0, 0.5, 1, 1.5, 2, 3, 4, 6: halves go to the even code
    m = 0.5 * ((m > 0.25).float() + (m >= 0.75).float() + (m > 1.25).float() + (m >= 1.75).float()) + ((m > 2.5).float() + (m >= 3.5).float()) + 2 * (m > 5).float()
    q = (torch.copysign(m, a) * sb).view(rows, dim)
    return ((q @ weight_of(s, torch.float32).T * (s_t * s["scale"])).bfloat16(), s_t, *stream)


def weight_of(s, dtype):
    """The weight's values without its tensor scale."""
    n, dim = s["case"]["columns"], s["case"]["dim"]
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda", dtype=dtype)
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(n, dim)
    high, wide = -(-n // 128), -(-(dim // 16) // 4)
    scales = s["scales"].view(high, wide, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(high * 128, wide * 4)[:n, : dim // 16]
    scales = scales.contiguous().view(torch.float8_e4m3fn).to(dtype)
    return (values[codes.int()].view(n, dim // 16, 16) * scales[..., None]).view(n, dim)


def plain_sample(logits, u, t, k, p, m):
    """Rows in falling order, ties by index, and the kept tokens a first part of it. (64 bits: the draw falls next to a border.)"""
    x = logits.double()
    x = torch.where(x.isnan(), -math.inf, x)
    x, at = torch.sort(x, dim=-1, descending=True, stable=True)
    best = x[:, :1]
    greedy = ~(t > 0)
    w = ((x - best) / torch.where(greedy, 1.0, t)).exp_()
    w = torch.where(x == best, 1.0, w).masked_fill_(x == -math.inf, 0.0)
    w.masked_fill_((torch.arange(x.shape[1], device=x.device) >= k) & (k > 0), 0.0)
    before = w.cumsum(-1)
    total = before[:, -1:].clone()
    before -= w
    keep = (before < p * total) | (p >= 1)
    keep &= w >= m.clamp(max=1.0)
    keep[:, 0] = True
    w.masked_fill_(~keep, 0.0)
    c = w.cumsum(-1)
    total = c[:, -1:]
    j = (c <= u.double()[:, None] * total).sum(-1, keepdim=True).clamp(max=x.shape[1] - 1)
    j = torch.where(greedy, 0, j)
    none = best == -math.inf
    ids = torch.where(none, -1, at.gather(1, j)).int().view(-1)
    probs = torch.where(none, 0.0, torch.where(greedy, 1.0, w.gather(1, j) / total)).float().view(-1)
    return ids, probs


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """The definitions: the norm by rows in 64 bits, the draw by counting equal logits."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        return exact_norm(case, s)
    rows = row_count(case)
    each = rows // len(s["temperature"])
    u = s["uniform"].cpu().numpy().astype(np.float64)
    t, k, p, m = (s[n].cpu().numpy().astype(np.float64).repeat(each) for n in ("temperature", "top_k", "top_p", "min_p"))
    x = s["logits"].double().cpu().numpy()
    ids, probs = np.empty(rows, dtype=np.int32), np.empty(rows, dtype=np.float64)
    for r in range(rows):
        ids[r], probs[r] = exact_draw(x[r], u[r], t[r], int(k[r]), p[r], m[r])
    if case["op"] == "sample":
        return ids, probs
    tokens = ids.reshape(case["batch"], each)
    drafts = s["draft_ids"].cpu().numpy()
    accepted = [next((i for i in range(each - 1) if a[i] != d[i]), each - 1) for a, d in zip(tokens, drafts)]
    return tokens, np.array(accepted, dtype=np.int32), probs.reshape(tokens.shape)


def exact_draw(x, u, t, k, p, m):
    there = np.flatnonzero(x > -math.inf)
    if not len(there):
        return -1, 0.0
    values, counts = np.unique(x[there], return_counts=True)
    values, counts = values[::-1], counts[::-1]
    if not t > 0:
        return int(np.flatnonzero(x == values[0])[0]), 1.0
    w = np.exp((values - values[0]) / t)
    ends = np.cumsum(counts)
    if 0 < k < ends[-1]:  # the first k
        i = int(np.searchsorted(ends, k))
        counts = counts[: i + 1].copy()
        counts[i] -= ends[i] - k
        w = w[: i + 1]
    if p < 1:  # the shortest first part that reaches its share
        mass = np.cumsum(counts * w)
        i = int(np.searchsorted(mass, p * mass[-1]))
        over = (p * mass[-1] - (mass[i - 1] if i else 0.0)) / w[i]
        counts = counts[: i + 1].copy()
        counts[i] = min(counts[i], max(1, math.ceil(over)))
        w = w[: i + 1]
    if m > 0:
        i = max(1, int((w >= m).sum()))
        counts, w = counts[:i], w[:i]
    mass = np.cumsum(counts * w)
    i = min(int(np.searchsorted(mass, u * mass[-1], side="right")), len(mass) - 1)
    nth = min(int((u * mass[-1] - (mass[i - 1] if i else 0.0)) / w[i]), int(counts[i]) - 1)
    return int(np.flatnonzero(x == values[i])[max(nth, 0)]), float(w[i] / mass[-1])


def exact_norm(case, s):
    x, stream = s["x"].double(), ()
    if s["residual"] is not None:
        x = x + s["residual"].double()
        stream = (x,)
        x = x.to(s["residual"].dtype).double()  # the stream as it goes on
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS) * (s["weight"].double() + case["offset"])
    if case["out"] == "bf16":
        return (y, *stream) if stream else y
    if case["out"] == "e4m3":
        scale = y.abs().amax(-1, keepdim=True) / 448
        scale[scale == 0] = 1
        return (y / scale, scale.view(-1), *stream)
    s_t = s["s_t"].double() if case["given"] else y.abs().max().view(1) / 2688
    b = y.view(case["tokens"], -1, 16)
    sb = (b.abs().amax(-1, keepdim=True) / 6 / s_t).clamp(max=448).float().to(torch.float8_e4m3fn).double()
    steps = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
    a = torch.where(sb > 0, b / (sb * s_t), 0)
    q = steps[torch.bucketize(a.abs(), (steps[1:] + steps[:-1]) / 2)] * a.sign() * sb
    return (q.view(case["tokens"], -1) @ weight_of(s, torch.float64).T * (s_t * s["scale"].double()), s_t, *stream)
