"""The paged-cache operators and the cases they are timed at.

    fm_attend_window   causal attention over paged keys and values, sliding window and sinks
    fm_attend_tree     the same for a tree of drafted tokens
    fm_qk_norm_rope    per-head norms of queries and keys, rotation, and the write into the pages
    fm_cache_*         forking, growing, compacting and freeing the pages of requests

A case is a dict of plain values.  `run` computes it in elementary torch operations (32 bits, 64
for the angles), or, where `own` is true, through the library.  Pages hold 64 entries, a key or
value pool is [pages, kv heads, 64, row], a row is head_dim values or 128 e4m3 codes and a
float32 scale.
"""
import math
import random

import torch

own = False

PAGE = 64
DEV = "cuda" if torch.cuda.is_available() else "cpu"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}
ROPE = dict(rope_base=160000.0, rope_factor=16.0, rope_orig_len=65536, beta_fast=32.0, beta_slow=1.0)
EPS = 1e-6


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one chat, next token, a window of 128 entries: latency alone
        dict(name="window_decode_1", op="window", B=1, rows=1, ragged=False, ctx=1000, window=128, sink=4,
             heads=16, kv=2, dim=128, kind="bf16"),
        # a full decode batch at 64K context whose cache keeps a 4K window
        dict(name="window_decode_32", op="window", B=32, rows=1, ragged=True, ctx=65536, window=4096, sink=64,
             heads=64, kv=8, dim=128, kind="bf16"),
        # long-context decode over an fp8 cache
        dict(name="window_decode_fp8_30", op="window", B=30, rows=1, ragged=True, ctx=40000, window=32768, sink=16,
             heads=64, kv=8, dim=128, kind="fp8"),
        # one chunk of a long prompt
        dict(name="window_prefill_4096", op="window", B=1, rows=4096, ragged=False, ctx=16384, window=4096, sink=4,
             heads=32, kv=8, dim=128, kind="bf16"),
        # a mixed batch: prompt chunks of any length beside single tokens, no window
        dict(name="window_mixed_8", op="window", B=8, rows=1024, ragged=True, ctx=8192, window=1 << 20, sink=0,
             heads=32, kv=8, dim=128, kind="bf16"),
        # small fp32 model, 64-wide heads, three query heads to a kv head
        dict(name="window_f32_3", op="window", B=3, rows=333, ragged=True, ctx=2500, window=500, sink=1,
             heads=12, kv=4, dim=64, kind="f32"),
        # speculative decoding of one chat, sixteen drafts
        dict(name="tree_1", op="tree", B=1, rows=16, ragged=False, ctx=2000, window=1 << 20, sink=0,
             heads=32, kv=8, dim=128, kind="bf16"),
        # speculative decoding of a batch: 64 drafts each over 384 pages of fp8 cache
        dict(name="tree_fp8_30", op="tree", B=30, rows=64, ragged=True, ctx=24576, window=1 << 20, sink=0,
             heads=32, kv=8, dim=128, kind="fp8"),
        # one token of every request of a batch
        dict(name="qk_decode_32", op="qk", T=32, heads=64, kv=8, dim=128, rope=64, halves=False, kind="bf16"),
        # a prompt chunk into an fp8 cache
        dict(name="qk_prefill_fp8_4096", op="qk", T=4096, heads=32, kv=8, dim=128, rope=128, halves=True, kind="fp8"),
        # beam search: the losing beams are dropped and the winners forked, eight pools
        dict(name="fork_12_of_16", op="fork", B=16, n=12, ctx=8000, pools=8, kv=8, row=256, deep=False),
        # after verification: the accepted path of every tree moved to the front, eight pools
        dict(name="compact_32", op="compact", B=32, drafts=64, ctx=4000, pools=8, kv=8, row=256),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "tree", "tree", "qk", "qk", "fork", "compact"])
    if op in ("window", "tree"):
        kind = rng.choice(["bf16", "bf16", "fp8", "f32"])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 7, 8, 16])
        dim = 128 if kind == "fp8" else rng.choice([64, 128, 128])
        B = _between(rng, 1, 32)
        if op == "tree":
            rows = _between(rng, 2, 100)
        else:
            rows = 1 if rng.random() < 0.4 else _between(rng, 2, 4096)
        ctx = _between(rng, max(rows, 16), 40000)
        window = _between(rng, 16, 32768) if rng.random() < 0.7 else 1 << 20
        sink = rng.choice([0, 0, 1, 4, 64, 100])
        # no dearer than the largest listed ones: scores a pass, and entries gathered a pass
        while B > 1 and (B * heads * rows * min(ctx, window + rows + sink) > 1 << 30
                         or B * kv * min(ctx, window + rows + sink) > 1 << 22):
            B = max(1, B // 2)
        while heads > kv and heads * rows * min(ctx, window + rows + sink) > 1 << 30:
            heads = kv
        if heads * rows * min(ctx, window + rows + sink) > 1 << 30:
            ctx = max(rows, 4096)
        return dict(op=op, B=B, rows=rows, ragged=rng.random() < 0.7, ctx=ctx, window=window, sink=sink,
                    heads=heads, kv=kv, dim=dim, kind=kind)
    if op == "qk":
        kind = rng.choice(["bf16", "fp8", "f32"])
        kv = rng.choice([1, 2, 4, 8])
        dim = 128 if kind == "fp8" else rng.choice([64, 128])
        return dict(op="qk", T=_between(rng, 1, 4096), heads=kv * rng.choice([1, 3, 4, 8]), kv=kv, dim=dim,
                    rope=rng.choice([dim, dim // 2]), halves=rng.random() < 0.5, kind=kind)
    kv, row = rng.choice([(8, 256), (1, 132), (2, 512), (4, 128), (8, 132)])
    if op == "fork":
        B = rng.randint(4, 48)
        return dict(op="fork", B=B, n=rng.randint(1, B - 2), ctx=_between(rng, 50, 16000), pools=rng.randint(1, 12),
                    kv=kv, row=row, deep=rng.random() < 0.3)
    return dict(op="compact", B=_between(rng, 1, 64), drafts=_between(rng, 2, 100), ctx=_between(rng, 70, 8000),
                pools=rng.randint(1, 12), kv=kv, row=row)


def _lens(c):
    """(rows, length) of every request: set by the case alone."""
    r = random.Random("%(B)d %(rows)d %(ctx)d" % c)
    out = []
    for _ in range(c["B"]):
        n = c["rows"] if not c["ragged"] or c["op"] == "tree" else r.randint(max(1, c["rows"] // 8), c["rows"])
        out.append((n, c["ctx"] if not c["ragged"] else r.randint(max(n, c["ctx"] * 3 // 4), c["ctx"])))
    if c["ragged"] and c["B"] > 2 and c["rows"] > 1 and c["op"] == "window":
        out[1] = (1, out[1][1])          # a single token among the chunks
    return out


# ---------------------------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _quant(x):
    """132-byte rows of x [..., 128]: e4m3 codes, then the float32 scale."""
    a = x.abs().amax(-1, keepdim=True)
    scale = torch.where(a > 0, a / 448.0, torch.ones_like(a))
    codes = (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([codes, scale.float().contiguous().view(torch.uint8)], -1)


def _dequant(rows):
    """(codes, scales) of 132-byte rows, in 32 bits."""
    codes = rows[..., :128].view(torch.float8_e4m3fn).float()
    return codes, rows[..., 128:].contiguous().view(torch.float32)


def _pool(g, c, pages):
    x = _normal(g, pages, c["kv"], PAGE, c["dim"])
    return _quant(x) if c["kind"] == "fp8" else x.to(DT[c["kind"]])


def _prepare_attn(c, seed):
    g = _gen(seed)
    lens = _lens(c)
    B, D = c["B"], c["dim"]
    n = torch.tensor([x[0] for x in lens], device=DEV)
    length = torch.tensor([x[1] for x in lens], device=DEV)
    ml = max(x[1] for x in lens)
    P = -(-ml // PAGE)
    at = torch.arange(P, device=DEV)[None] * PAGE
    lo = (length - n - c["window"] + 1).clamp(min=0)[:, None]
    need = (at < length[:, None]) & ((at + PAGE > lo) | (at < c["sink"]))   # pages before the window are freed
    count = int(need.sum())
    bt = torch.full((B, P), -1, dtype=torch.int32, device=DEV)
    bt[need] = torch.randperm(count, generator=g, device=DEV).to(torch.int32)
    T = sum(x[0] for x in lens)
    start = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    start[1:] = n.cumsum(0).to(torch.int32)
    dt = DT[c["kind"]]
    s = dict(case=c, q=_normal(g, T, c["heads"], D, std=1.5).to(dt), k=_pool(g, c, count), v=_pool(g, c, count),
             bt=bt, length=length.to(torch.int32), start=start, max_rows=max(x[0] for x in lens), max_len=ml,
             out=torch.empty(T, c["heads"], D, dtype=dt, device=DEV),
             lse=torch.empty(T, c["heads"], dtype=torch.float32, device=DEV))
    if c["op"] == "tree":
        # every draft hangs below an earlier one (two in three below one of the last four)
        r = random.Random(seed)
        words = -(-c["rows"] // 64)
        masks = []
        for rows, _ in lens:
            seen = []
            for i in range(rows):
                up = r.randrange(max(0, i - 4), i) if i and r.random() < 0.67 else r.randrange(i) if i else -1
                seen.append((seen[up] if up >= 0 else 0) | 1 << i)
            masks += [[(m >> 64 * w) & (1 << 64) - 1 for w in range(words)] for m in seen]
        s["mask"] = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in m] for m in masks],
                                 dtype=torch.int64, device=DEV)
    return s


def _prepare_qk(c, seed):
    g = _gen(seed)
    T, H, K, D = c["T"], c["heads"], c["kv"], c["dim"]
    dt = DT[c["kind"]]
    qkv = _normal(g, T, (H + 2 * K) * D, std=2.0).to(dt)       # one projection's output
    B = 1 if T > 256 else T                                    # a prompt chunk, or one token a request
    first = torch.randint(0, 200000, (B,), generator=g, device=DEV)
    base = first % PAGE + (PAGE * 3 if T <= 256 else 0)        # the cache holds what is left of the window
    slot = base + (torch.arange(T, device=DEV) if B == 1 else 0)
    req = torch.zeros(T, dtype=torch.int32, device=DEV) if B == 1 else torch.arange(T, dtype=torch.int32, device=DEV)
    length = (slot.max() + 1).repeat(1) if B == 1 else slot + 1
    P = -(-int(length.max()) // PAGE)
    bt = torch.randperm(B * P, generator=g, device=DEV).to(torch.int32).view(B, P)
    return dict(case=c, qkv=qkv, qn=(1 + 0.2 * _normal(g, D)).to(dt), kn=(1 + 0.2 * _normal(g, D)).to(dt),
                pos=(first[req.long()] + (torch.arange(T, device=DEV) if B == 1 else 0)).to(torch.int32),
                slot=slot.to(torch.int32), req=req, bt=bt, length=length.to(torch.int32),
                max_len=int(length.max()), k=_pool(g, c, B * P), v=_pool(g, c, B * P),
                qo=torch.empty(T, H, D, dtype=dt, device=DEV))


def _bytes(g, *shape):
    return torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)


def _prepare_fork(c, seed):
    """B requests; the last n of them are beams forked from the others a step ago."""
    g = _gen(seed)
    B, n = c["B"], c["n"]
    r = random.Random("%(B)d %(n)d %(ctx)d" % c)
    keep = B - n
    lens = [r.randint(max(1, c["ctx"] * 3 // 4), c["ctx"]) for _ in range(keep)]
    P = -(-c["ctx"] // PAGE) + 1
    used = sum(-(-x // PAGE) for x in lens)
    spare = n * P if c["deep"] else n
    N = used + spare + 8
    ids = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
    bt = torch.full((B, P), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, x in enumerate(lens):
        p = -(-x // PAGE)
        bt[b, :p] = ids[at:at + p]
        at += p
    free = torch.zeros(N, dtype=torch.int32, device=DEV)
    free[:N - used] = ids[used:].sort().values
    ref = torch.zeros(N, dtype=torch.int32, device=DEV)
    ref[ids[:used].long()] = 1
    src = torch.randint(0, keep, (n,), generator=g, device=DEV).to(torch.int32)
    return dict(case=c, pools=[_bytes(g, N, c["kv"], PAGE, c["row"]) for _ in range(c["pools"])], bt=bt,
                length=torch.tensor(lens + [0] * n, dtype=torch.int32, device=DEV), ref=ref, free=free,
                n_free=torch.tensor([N - used], dtype=torch.int32, device=DEV), src=src,
                dst=torch.arange(keep, B, dtype=torch.int32, device=DEV),
                ok=torch.zeros(n, dtype=torch.int32, device=DEV))


def _prepare_compact(c, seed):
    """B requests of committed length; a step appends the drafts and keeps one path of them."""
    g = _gen(seed)
    B, n = c["B"], c["drafts"]
    r = random.Random("%(B)d %(drafts)d %(ctx)d" % c)
    lens = [r.randint(max(1, c["ctx"] * 3 // 4), c["ctx"]) for _ in range(B)]
    P = -(-(c["ctx"] + n) // PAGE)
    used = sum(-(-x // PAGE) for x in lens)
    N = used + B * (n // PAGE + 2)
    ids = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
    bt = torch.full((B, P), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, x in enumerate(lens):
        p = -(-x // PAGE)
        bt[b, :p] = ids[at:at + p]
        at += p
    free = torch.zeros(N, dtype=torch.int32, device=DEV)
    free[:N - used] = ids[used:].sort().values
    ref = torch.zeros(N, dtype=torch.int32, device=DEV)
    ref[ids[:used].long()] = 1
    q = random.Random(seed)
    D = min(8, n)
    keep = torch.full((B, D), -1, dtype=torch.int32)
    count = []
    for b, x in enumerate(lens):
        k = min(D, q.randint(1, 8))
        keep[b, :k] = torch.tensor(sorted(q.sample(range(n), k)), dtype=torch.int32) + x
        count.append(k)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(case=c, pools=[_bytes(g, N, c["kv"], PAGE, c["row"]) for _ in range(c["pools"])], bt=bt,
                length=i32(lens), ref=ref, free=free, n_free=i32([N - used]), req=torch.arange(B, dtype=torch.int32, device=DEV),
                start=i32(lens), drafted=i32([x + n for x in lens]), keep=keep.to(DEV), count=i32(count),
                ok=torch.zeros(2, B, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    return {"window": _prepare_attn, "tree": _prepare_attn, "qk": _prepare_qk, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](dict(case), seed)


# ---------------------------------------------------------------------------------- plain forms
def _plain_attn(s):
    c = s["case"]
    B, H, K, D, W, S = c["B"], c["heads"], c["kv"], c["dim"], c["window"], c["sink"]
    G, R = H // K, s["max_rows"]
    start, length = s["start"].long(), s["length"].long()
    n = start[1:] - start[:-1]
    lo = (length - n - W + 1).clamp(min=0)
    lo = torch.maximum(lo, torch.full_like(lo, S))
    C = min(S, s["max_len"]) + min(max(s["max_len"] - S, 0), W + R - 1)     # columns: the sinks, then from lo on
    sinks = min(S, s["max_len"])
    col = torch.arange(C, device=DEV)
    at = torch.where(col < sinks, col, lo[:, None] + (col - sinks))          # [B, C]: entry of a column
    page = s["bt"].gather(1, (at // PAGE).clamp(max=s["bt"].shape[1] - 1)).long()
    live = (at < length[:, None]) & (page >= 0)

    def rows(pool):
        x = pool[page.clamp(min=0), :, at % PAGE]                             # [B, C, K, row]
        if c["kind"] == "fp8":
            codes, scale = _dequant(x)
            x = codes * scale
        x = torch.where(live[:, :, None, None], x.float(), torch.zeros((), device=DEV))
        return x.permute(0, 2, 1, 3).contiguous()                             # [B, K, C, D]

    i = torch.arange(R, device=DEV)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)               # [B, R]
    q = s["q"][row].float().view(B, R, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * R, D)
    pos = length[:, None] - n[:, None] + i                                    # [B, R]
    if c["op"] == "tree":
        m = s["mask"][row]                                                    # [B, R, words]
        bit = torch.arange(64, device=DEV)
        bits = ((m[..., None] >> bit) & 1).flatten(2)                         # [B, R, 64 words]
        base = length - n
        pos = base[:, None] + bits.sum(-1) - 1
        j = (at - base[:, None])                                              # [B, C]
        drafted = bits.gather(2, j.clamp(0, bits.shape[2] - 1)[:, None].expand(B, R, C)) > 0
        a = at[:, None]
        see = torch.where(j[:, None] >= 0, drafted & (j[:, None] < n[:, None, None]),
                          (a <= pos[..., None]) & ((a < S) | (a > pos[..., None] - W)))
    else:
        a = at[:, None]
        see = (a <= pos[..., None]) & ((a < S) | (a > pos[..., None] - W))
    see = see & live[:, None] & (i < n[:, None])[..., None]                   # [B, R, C]
    x = torch.matmul(q, rows(s["k"]).transpose(2, 3).contiguous()).view(B, K, G, R, C)
    x.mul_(1.0 / math.sqrt(D)).masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top.isinf(), torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, K, G * R, C), rows(s["v"])).view(B, K, G, R, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(B, R, H, D)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, R, H)
    mine = i < n[:, None]
    return o[mine].to(s["q"].dtype), lse[mine]


def _freqs(d, base, factor, orig, fast, slow):
    i = torch.arange(d // 2, dtype=torch.float64, device=DEV)
    th = base ** (-2.0 * i / d)
    if factor == 1.0:
        return th
    corr = lambda beta: d * math.log(orig / (beta * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(corr(fast)), 0), min(math.ceil(corr(slow)), d // 2 - 1)
    ramp = ((i - lo) / (hi - lo if hi != lo else 0.001)).clamp(0, 1)
    return th / factor * ramp + th * (1 - ramp)


def _plain_qk(s):
    c = s["case"]
    T, H, K, D, R = c["T"], c["heads"], c["kv"], c["dim"], c["rope"]
    x = s["qkv"].float().view(T, H + 2 * K, D)
    q, k, v = x[:, :H], x[:, H:H + K], x[:, H + K:]
    ang = s["pos"].double()[:, None] * _freqs(R, *ROPE.values())              # 64 bits: far positions
    co, si = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def turn(x, w):
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        keep, y = x[..., :D - R], x[..., D - R:]                              # the last dims turn
        if c["halves"]:
            a, b = y[..., :R // 2], y[..., R // 2:]
            y = torch.cat([a * co - b * si, a * si + b * co], -1)
        else:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack([a * co - b * si, a * si + b * co], -1).flatten(-2)
        return torch.cat([keep, y], -1)

    slot, req = s["slot"].long(), s["req"].long()
    page = s["bt"][req, slot // PAGE].long()
    store = _quant if c["kind"] == "fp8" else lambda y: y.to(DT[c["kind"]])
    s["k"][page, :, slot % PAGE] = store(turn(k, s["kn"]))
    s["v"][page, :, slot % PAGE] = store(v)
    return [turn(q, s["qn"]).to(s["qkv"].dtype)] + _shown(s)


def _shown(s):
    """The pools as the values they hold."""
    if s["case"]["kind"] != "fp8":
        return [s["k"], s["v"]]
    return [f(p) for p in (s["k"], s["v"]) for f in (lambda p: p[..., :128].view(torch.float8_e4m3fn),
                                                     lambda p: p[..., 128:].view(torch.float32))]


def _pages(x):
    return (x + PAGE - 1) // PAGE


def _plain_free(s, req, new):
    """Requests req cut to new entries; a page nobody holds any more goes back, in page order."""
    N = s["ref"].shape[0]
    old = s["length"][req].long()
    cell = torch.arange(s["bt"].shape[1], device=DEV)[None]
    gone = (cell >= _pages(new)[:, None]) & (cell < _pages(old)[:, None])
    rows = s["bt"][req]
    page = torch.where(gone & (rows >= 0), rows, torch.full_like(rows, N)).long()
    drop = torch.zeros(N + 1, dtype=torch.int32, device=DEV).index_add_(
        0, page.flatten(), torch.ones_like(page.flatten(), dtype=torch.int32))[:N]
    free = (drop > 0) & (s["ref"] == drop)
    s["ref"].sub_(drop)
    s["bt"][req] = torch.where(gone, torch.full_like(rows, -1), rows)
    s["length"][req] = new.to(torch.int32)
    # the r-th freed page goes to place n_free + r of the list; the others to a place past its end
    place = torch.where(free, s["n_free"].long() + free.long().cumsum(0) - 1, torch.full((N,), N, device=DEV))
    grown = torch.cat([s["free"], s["free"].new_zeros(1)])
    grown[place] = torch.arange(N, dtype=torch.int32, device=DEV)
    s["free"].copy_(grown[:N])
    s["n_free"].add_(free.sum().to(torch.int32))


def _plain_fork(s):
    deep = s["case"]["deep"]
    _plain_free(s, s["dst"].long(), torch.zeros_like(s["dst"]).long())
    src, dst = s["src"].long(), s["dst"].long()
    N = s["ref"].shape[0]
    length = s["length"][src].long()
    need = _pages(length) if deep else (length % PAGE != 0).long()
    ok = need.cumsum(0) <= s["n_free"]
    base = need.cumsum(0) - need
    cell = torch.arange(s["bt"].shape[1], device=DEV)[None]
    rows = s["bt"][src]
    full = (length // PAGE)[:, None]
    new = ok[:, None] & (cell < _pages(length)[:, None]) & (torch.ones_like(full, dtype=torch.bool) if deep else cell >= full)
    rank = base[:, None] + (cell if deep else torch.zeros_like(cell))
    fresh = s["free"][(s["n_free"].long() - 1 - rank).clamp(0, N - 1)]
    held = ok[:, None] & (cell < _pages(length)[:, None])
    s["bt"][dst] = torch.where(new, fresh, torch.where(held, rows, s["bt"][dst]))
    shared = held & ~new
    spare = torch.full_like(rows, N)
    ref = torch.cat([s["ref"], s["ref"].new_zeros(1)])
    ref.index_add_(0, torch.where(shared, rows, spare).flatten().long(), torch.ones_like(rows).flatten())
    ref[torch.where(new, fresh, spare).flatten().long()] = 1
    s["ref"].copy_(ref[:N])
    s["length"][dst] = torch.where(ok, length, torch.zeros_like(length)).to(torch.int32)
    s["n_free"].sub_((need * ok).sum().to(torch.int32))
    a, b = rows[new].long(), fresh[new].long()
    for p in s["pools"]:
        p[b] = p[a]
    return dict(ok=ok.to(torch.int32), **_tables(s))


def _plain_compact(s):
    req = s["req"].long()
    # the drafts' pages
    old, new = s["length"][req].long(), s["drafted"].long()
    need = _pages(new) - _pages(old)
    grown = need.cumsum(0) <= s["n_free"]
    base = need.cumsum(0) - need
    N = s["ref"].shape[0]
    cell = torch.arange(s["bt"].shape[1], device=DEV)[None]
    more = grown[:, None] & (cell >= _pages(old)[:, None]) & (cell < _pages(new)[:, None])
    rank = base[:, None] + cell - _pages(old)[:, None]
    fresh = s["free"][(s["n_free"].long() - 1 - rank).clamp(0, N - 1)]
    s["bt"][req] = torch.where(more, fresh, s["bt"][req])
    ref = torch.cat([s["ref"], s["ref"].new_zeros(1)])
    ref[torch.where(more, fresh, torch.full_like(fresh, N)).flatten().long()] = 1
    s["ref"].copy_(ref[:N])
    s["n_free"].sub_((need * grown).sum().to(torch.int32))
    s["length"][req] = torch.where(grown, new, old).to(torch.int32)
    # the kept ones to the front
    i = torch.arange(s["keep"].shape[1], device=DEV)[None]
    kept = i < s["count"][:, None]
    a = s["keep"].long()[kept]
    b = (s["start"].long()[:, None] + i)[kept]
    r = req[:, None].expand(kept.shape)[kept]
    pa, pb = s["bt"][r, a // PAGE].long(), s["bt"][r, b // PAGE].long()
    for p in s["pools"]:
        p[pb, :, b % PAGE] = p[pa, :, a % PAGE]
    _plain_free(s, req, s["start"].long() + s["count"].long())
    return dict(ok=torch.stack([grown.to(torch.int32), torch.ones_like(s["count"])]), **_tables(s))


def _tables(s):
    return dict(bt=s["bt"], length=s["length"], ref=s["ref"], free=s["free"], n_free=s["n_free"],
                **{"pool%02d" % i: p for i, p in enumerate(s["pools"])})


# ---------------------------------------------------------------------------------- the library
def _own_attn(s):
    from top_selection_fm_amd import api
    c = s["case"]
    if "desc" not in s:                      # a serving loop keeps its descriptors and workspace
        kind = "fp8x132" if c["kind"] == "fp8" else c["kind"]
        s["cache"] = api.kv_desc([s["k"], s["v"]], kind, s["bt"], s["length"], s["max_len"], head_dim=c["dim"])
        s["desc"] = api.attn_desc(s["q"], "f32" if c["kind"] == "f32" else "bf16", s["out"], s["start"], s["max_rows"],
                                  n_kv_heads=c["kv"], scale=1.0 / math.sqrt(c["dim"]), lse=s["lse"])
        s["nb"] = api.fm_attend_workspace_bytes(s["desc"], s["cache"], c["window"], c["sink"])
        s["ws"] = torch.empty(max(s["nb"], 256), dtype=torch.uint8, device=DEV)
    if c["op"] == "tree":
        api.fm_attend_tree(s["desc"], s["cache"], s["mask"], s["mask"].shape[1], c["window"], c["sink"], s["ws"], s["nb"])
    else:
        api.fm_attend_window(s["desc"], s["cache"], c["window"], c["sink"], s["ws"], s["nb"])
    return s["out"], s["lse"]


def _own_qk(s):
    from top_selection_fm_amd import api
    c = s["case"]
    if "desc" not in s:
        H, K, D = c["heads"], c["kv"], c["dim"]
        x = s["qkv"].view(c["T"], H + 2 * K, D)
        kind = "fp8x132" if c["kind"] == "fp8" else c["kind"]
        s["cache"] = api.kv_desc([s["k"], s["v"]], kind, s["bt"], s["length"], s["max_len"], head_dim=D)
        s["desc"] = api.qk_desc(x[:, :H], x[:, H:H + K], x[:, H + K:], "f32" if c["kind"] == "f32" else "bf16", s["qo"],
                                s["qn"], s["kn"], s["pos"], rms_eps=EPS, rope_dim=c["rope"], rope_first=D - c["rope"],
                                rope_halves=c["halves"], row_req=s["req"], slot=s["slot"], **ROPE)
    api.fm_qk_norm_rope(s["desc"], s["cache"])
    return [s["qo"]] + _shown(s)


def _own_cache(s):
    from top_selection_fm_amd import api
    c = s["case"]
    if "desc" not in s:
        s["desc"] = api.cache_desc(s["pools"], s["bt"], s["length"], s["ref"], s["free"], s["n_free"])
        s["nb"] = api.fm_cache_workspace_bytes(s["desc"], c["B"])
        s["ws"] = torch.empty(max(s["nb"], 256), dtype=torch.uint8, device=DEV)
    d, ok, ws, nb = s["desc"], s["ok"], s["ws"], s["nb"]
    if c["op"] == "fork":
        api.fm_cache_free(d, s["dst"], None, c["n"], None)
        api.fm_cache_fork(d, s["src"], s["dst"], c["n"], c["deep"], ok, ws, nb)
    else:
        api.fm_cache_grow(d, s["req"], s["drafted"], c["B"], ok[0], ws, nb)
        api.fm_cache_compact(d, s["req"], s["start"], s["keep"], s["keep"].shape[1], s["count"], c["B"], ok[1])
    return dict(ok=ok, **_tables(s))


def run(state):
    op = state["case"]["op"]
    if own:
        return (_own_attn if op in ("window", "tree") else _own_qk if op == "qk" else _own_cache)(state)
    return {"window": _plain_attn, "tree": _plain_attn, "qk": _plain_qk, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


# ---------------------------------------------------------------------------------- floors
def _seen(c):
    """(entries read at least once, visible (row, entry) pairs) of an attention case."""
    S, W, entries, pairs = c["sink"], c["window"], 0, 0
    for n, L in _lens(c):
        first = max(0, L - n - W + 1)
        entries += L - first + min(S, first)
        if c["op"] == "tree":
            pairs += n * (min(L - n, W) + min(S, max(0, L - n - W))) + n * 6
        else:
            for pos in range(L - n, L):
                lo = max(0, pos - W + 1)
                pairs += pos + 1 - lo + min(S, lo)
    return entries, pairs


def work(case):
    c = case
    if c["op"] in ("window", "tree"):
        entries, pairs = _seen(c)
        T = sum(n for n, _ in _lens(c))
        size = 4 if c["kind"] == "f32" else 2
        row = 132 if c["kind"] == "fp8" else size * c["dim"]
        return {"bytes": 2 * entries * c["kv"] * row + T * c["heads"] * (2 * size * c["dim"] + 4),
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "qk":
        size = 4 if c["kind"] == "f32" else 2
        row = 132 if c["kind"] == "fp8" else size * c["dim"]
        return {"bytes": c["T"] * (2 * c["heads"] * size * c["dim"] + 2 * c["kv"] * (size * c["dim"] + row)),
                "flops": c["T"] * (c["heads"] + c["kv"]) * c["dim"] * 7}
    page = c["kv"] * PAGE * c["row"]
    cells = c["B"] * (c["ctx"] // PAGE)
    if c["op"] == "fork":
        pages = c["n"] * (c["ctx"] * 7 // 8 // PAGE if c["deep"] else 1)
        return {"bytes": 2 * pages * page * c["pools"] + 16 * cells, "flops": 0}
    return {"bytes": 2 * 4 * c["B"] * c["kv"] * c["row"] * c["pools"] + 16 * c["B"], "flops": 0}


# ---------------------------------------------------------------------------------- in 64 bits
def _exact_values(pool, kind):
    if kind != "fp8":
        return pool.double()
    return pool[..., :128].view(torch.float8_e4m3fn).double() * pool[..., 128:].contiguous().view(torch.float32).double()


def _exact_attn(c, seed):
    s = _prepare_attn(c, seed)
    H, K, D = c["heads"], c["kv"], c["dim"]
    G = H // K
    outs, lses, t = [], [], 0
    for b, (n, L) in enumerate(_lens(c)):
        pos = torch.arange(L - n, L, device=DEV)
        see = torch.zeros(n, L, dtype=torch.bool, device=DEV)
        if c["op"] == "tree":
            m = s["mask"][t:t + n]
            bits = torch.stack([(m[:, j // 64] >> (j % 64)) & 1 for j in range(n)], 1).bool()
            see[:, L - n:] = bits
            pos = L - n + bits.sum(1) - 1
        s_at = torch.arange(L - n if c["op"] == "tree" else L, device=DEV)[None]
        see[:, :s_at.shape[1]] = (s_at <= pos[:, None]) & ((s_at > pos[:, None] - c["window"]) | (s_at < c["sink"]))
        table = s["bt"][b].long().repeat_interleave(PAGE)[:L]
        used = torch.nonzero(see.any(0) & (table >= 0))[:, 0]
        see = see[:, used]
        out = torch.zeros(n, H, D, dtype=torch.float64, device=DEV)
        lse = torch.zeros(n, H, dtype=torch.float64, device=DEV)
        for h in range(K):
            k = _exact_values(s["k"][table[used], h, used % PAGE], c["kind"])
            v = _exact_values(s["v"][table[used], h, used % PAGE], c["kind"])
            for g in range(h * G, h * G + G):
                x = s["q"][t:t + n, g].double() @ k.T / math.sqrt(D)
                x = torch.where(see, x, -math.inf)
                lse[:, g] = torch.logsumexp(x, 1)
                out[:, g] = torch.where(see.any(1)[:, None], torch.softmax(x, 1), 0.0) @ v
        outs.append(out)
        lses.append(lse)
        t += n
    return torch.cat(outs), torch.cat(lses)


def _exact_qk(c, seed):
    s = _prepare_qk(c, seed)
    T, H, K, D, R = c["T"], c["heads"], c["kv"], c["dim"], c["rope"]
    x = s["qkv"].double().view(T, H + 2 * K, D)
    i = torch.arange(R // 2, device=DEV)
    u, w = (2 * i, 2 * i + 1) if not c["halves"] else (i, i + R // 2)
    u, w = u + D - R, w + D - R
    turn = torch.exp(1j * s["pos"].double()[:, None] * _freqs(R, *ROPE.values()))[:, None]

    def norm(y, weight):
        y = y / (y.square().sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
        z = torch.complex(y[..., u], y[..., w]) * turn
        y = y.clone()
        y[..., u], y[..., w] = z.real, z.imag
        return y

    q, k, v = norm(x[:, :H], s["qn"]), norm(x[:, H:H + K], s["kn"]), x[:, H + K:]
    found = [q]
    for pool, y in ((s["k"], k), (s["v"], v)):
        if c["kind"] == "fp8":
            codes, scale = pool[..., :128].view(torch.float8_e4m3fn).double(), pool[..., 128:].contiguous().view(torch.float32).double()
            top = y.abs().amax(-1, keepdim=True) / 448.0
            full = [(codes, y / top), (scale, top)]
        else:
            full = [(pool.double(), y)]
        for whole, rows in full:
            for t in range(T) if T <= 256 else [slice(None)]:
                slot = s["slot"].long()[t]
                whole[s["bt"][s["req"].long()[t], slot // PAGE].long(), :, slot % PAGE] = rows[t]
            found.append(whole)
    return found


def exact(case, seed):
    c = dict(case)
    if c["op"] in ("window", "tree"):
        return _exact_attn(c, seed)
    if c["op"] == "qk":
        return _exact_qk(c, seed)
    return None                              # whole numbers and moved bytes
