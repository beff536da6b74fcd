"""Rotary positions, and eviction from the paged cache by accumulated attention weight, as a serving program calls
them: cases, inputs, plain forms and calls.

  rope    turn the queries and keys of a packed stream by their tokens' positions: pairs (j, j + rot/2) or (2j, 2j+1)
          of a head's first `rot` numbers, frequencies scaled for long contexts or not; transposed for gradients
  mass    after a decode step, add to every cached row of one layer the weight that the step's queries gave it:
          mass <- decay * mass + sum over the key head's query heads of exp(q . K_i * dk^-0.5 - lse)
  evict   choose the rows of every request and key head that stay: `budget` of them, the first `sinks` and the last
          `recent` tokens before the others, those by mass; rows that stay beyond the new length move into the holes
  move    the rows' keys, values, scales and records to their new places

The cache is pages of B tokens, [pages, Hkv, B, dk], in bf16 or in e4m3 with one power-of-two scale (a biased
exponent, uint8) per token and head; mass (fp32) and born (int32, the token's number in its layer's stream) lie
beside it as [pages, Hkv, B].

`own` false: elementary torch operations in 32 bits (angles in 64).  `own` true: the calls of
long_context_prefill_varlen_gb300.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
LLAMA, QWEN, GEMMA = (32, 8, 128), (16, 2, 256), (16, 8, 256)      # the layer geometries of bench.py's workloads


# ------------------------------------------------------------------------------------------ cases

def _rope(name, heads, tokens, requests=1, first=0, rot=0, layout="halves", theta=500000.0, scaling="none", factor=1.0,
          original=8192, transpose=False, fused=True, gaps=0.0):
    """tokens of each request; first position; rot = 0: the whole head; gaps: share of positions that a drop left out"""
    hq, hkv, dk = heads
    c = dict(op="rope", Hq=hq, Hkv=hkv, dk=dk, tokens=tokens, requests=requests, first=first, rot=rot or dk, layout=layout,
             theta=theta, scaling=scaling, factor=factor, original=original, transpose=transpose, fused=fused, gaps=gaps)
    return dict(c, name=name) if name else c


def _cache(name, op, fmt, heads, page, lengths, **more):
    """heads = (Hq, Hkv, dk); lengths = (requests, shortest, longest, how they are spread)"""
    hq, hkv, dk = heads
    r, lo, hi, spread = lengths
    c = dict(op=op, fmt=fmt, Hq=hq, Hkv=hkv, dk=dk, page=page, requests=r, shortest=lo, longest=hi, spread=spread, **more)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request's new token: the smallest call, latency counts
        _rope("rope 1 new token", LLAMA, 1, first=32768, scaling="bands", factor=8.0),
        # the tokens that a drop kept of a 32K prefill, from the fused projection's output
        _rope("rope 32K kept", LLAMA, 32513, scaling="bands", factor=8.0, gaps=0.01),
        # the gradient through a quarter of wide heads, four long documents, stretched past their trained length
        _rope("rope 4 x 128K part", QWEN, 131072, requests=4, rot=64, layout="pairs", theta=10000000.0, scaling="ramp",
              factor=4.0, original=32768, transpose=True, fused=False),
        # a single 4K request's decode step: the smallest call
        _cache("mass 1 x 4K bf16", "mass", "bf16", LLAMA, 16, (1, 4096, 4096, "even"), decay=1.0, fresh=False),
        # a batch in continuous batching, an empty and a one-token request among them
        _cache("mass 64 x 0-8K e4m3", "mass", "e4m3", LLAMA, 16, (64, 0, 8192, "even"), decay=1.0, fresh=False),
        # the packed batch of 16 requests of 4K to 128K tokens, older steps counting for less
        _cache("mass 16 x 4K-128K bf16", "mass", "bf16", LLAMA, 64, (16, 4096, 131072, "log"), decay=0.98, fresh=False),
        # a full cache that makes room for one token
        _cache("evict 1 x 4K one row", "evict", "none", LLAMA, 16, (1, 4097, 4097, "even"), keep=4096, share=0.0, sinks=4,
               recent=128),
        # a ragged batch cut to half of every request
        _cache("evict 64 x 0-8K half", "evict", "none", LLAMA, 16, (64, 0, 8192, "even"), keep=0, share=0.5, sinks=128,
               recent=128),
        # four long documents cut to 16K, few and long lists
        _cache("evict 4 x 128K to 16K", "evict", "none", QWEN, 32, (4, 131072, 131072, "even"), keep=16384, share=0.0,
               sinks=128, recent=1024),
        # a batch's step: a row of every head makes place for the newest
        _cache("move 64 x one row e4m3", "move", "e4m3", LLAMA, 16, (64, 1025, 1025, "even"), keep=1024, share=0.0),
        # the long documents' rows to their 16K places
        _cache("move 4 x 128K to 16K e4m3", "move", "e4m3", QWEN, 32, (4, 131072, 131072, "even"), keep=16384, share=0.0),
        # the packed batch cut to half, unquantised
        _cache("move 16 x 4K-128K half", "move", "bf16", LLAMA, 64, (16, 4096, 131072, "log"), keep=0, share=0.5),
    ]


GEOMETRIES = [LLAMA, LLAMA, QWEN, GEMMA, (8, 8, 64), (28, 4, 128), (16, 1, 64), (40, 8, 128), (32, 1, 128)]


def draw(rng):
    op = rng.choice(["rope", "mass", "evict", "move"])
    heads = rng.choice(GEOMETRIES)
    hq, hkv, dk = heads
    if op == "rope":
        budget = math.exp(rng.uniform(math.log(3e4), math.log(3e9)))       # bytes of the stream
        total = max(1, int(budget / (2 * (hq + hkv) * dk)))
        requests = min(64, total, int(math.exp(rng.uniform(0, math.log(64)))))
        rot = rng.choice([dk, dk, dk // 2, dk // 4])
        scaling, factor = rng.choice([("none", 1.0), ("linear", 4.0), ("bands", 8.0), ("ramp", 4.0), ("ramp", 40.0)])
        return _rope(None, heads, total // requests, requests, rng.choice([0, 0, 1, 100_003, 7_654_321]), rot,
                     rng.choice(["halves", "pairs"]), rng.choice([10000.0, 500000.0, 1000000.0]), scaling, factor,
                     rng.choice([4096, 8192, 32768]), rng.random() < 0.3, rng.random() < 0.5, rng.choice([0.0, 0.0, 0.3]))
    fmt = rng.choice(["bf16", "e4m3"])
    page = rng.choice([8, 16, 16, 24, 32, 48, 64, 128, 256])
    budget = math.exp(rng.uniform(math.log(1e7 if op == "evict" else 1e6), math.log(1.4e9)))       # bytes of a bf16 cache
    tokens = min(1_000_000, max(2, int(budget / (4 * hkv * dk))))
    if op == "evict":
        tokens = min(tokens, 2_000_000 // hkv)
    requests = min(128, tokens // 2, int(math.exp(rng.uniform(0, math.log(100)))))
    longest = max(2, tokens // requests) + rng.choice([0, 0, 1, 3])
    spread = rng.choice(["even", "log", "same"])
    shortest = longest if spread == "same" else rng.choice([0, 1, longest // 30, longest // 3])
    lengths = (requests, shortest, longest, spread)
    if op == "mass":
        return _cache(None, op, fmt, heads, page, lengths, decay=rng.choice([1.0, 1.0, 0.95]), fresh=rng.random() < 0.2)
    cut = rng.choice(["one", "share", "share", "to"])
    keep = longest - 1 if cut == "one" else max(1, longest // rng.choice([2, 5, 30])) if cut == "to" else 0
    share = rng.choice([0.1, 0.5, 0.8]) if cut == "share" else 0.0
    if op == "move":
        return _cache(None, op, fmt, heads, page, lengths, keep=keep, share=share)
    return _cache(None, op, "none", heads, page, lengths, keep=keep, share=share, sinks=rng.choice([0, 4, 128]),
                  recent=rng.choice([0, 1, 128, 1000]))


def _lengths(c):
    """the case's lengths, the same for every seed; a ragged batch has its shortest and its longest"""
    r, lo, hi = c["requests"], c["shortest"], c["longest"]
    rng = random.Random("%d %d %d %s" % (r, lo, hi, c["spread"]))
    if c["spread"] == "log":
        n = [int(round(math.exp(rng.uniform(math.log(max(1, lo)), math.log(max(1, hi)))))) for _ in range(r)]
    else:
        n = [rng.randint(lo, hi) for _ in range(r)]
    n[0] = lo
    if r > 2:
        n[1] = min(hi, max(lo, 1))
    n[-1] = hi
    return n


def _budgets(c):
    """rows that stay of every request"""
    return [min(n, int(n * c["share"]) if c["share"] else c["keep"]) for n in _lengths(c)]


def _moved(c):
    """rows of a request and head that move, where the rows that stay are spread evenly"""
    return [-(-k * (n - k) // n) if n else 0 for n, k in zip(_lengths(c), _budgets(c))]


def _row_bytes(c):
    """one token and head of the cache, keys or values"""
    return 2 * c["dk"] if c["fmt"] == "bf16" else c["dk"] + 1


def work(c):
    if c["op"] == "rope":
        t, h = c["tokens"] * c["requests"], c["Hq"] + c["Hkv"]
        return {"bytes": 4 * t * h * c["dk"] + 8 * t, "flops": 3 * t * h * c["rot"]}
    n, hkv = sum(_lengths(c)), c["Hkv"]
    pages = sum(-(-x // c["page"]) for x in _lengths(c))
    if c["op"] == "mass":
        old = 0 if c["fresh"] else 4
        return {"bytes": n * hkv * (_row_bytes(c) + 4 + old) + 4 * pages + c["requests"] * (2 * c["Hq"] * c["dk"] + 4 * c["Hq"] + 12),
                "flops": 2 * n * c["Hq"] * c["dk"] + 3 * n * c["Hq"]}
    moves = sum(_moved(c)) * hkv
    if c["op"] == "evict":
        return {"bytes": 8 * n * hkv + 8 * moves + 4 * pages + 4 * c["requests"] * (4 + hkv), "flops": n * hkv}
    return {"bytes": moves * (2 * (2 * _row_bytes(c) + 8) + 8) + 4 * pages + 4 * c["requests"] * hkv, "flops": 0}


# ------------------------------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _frequencies(c):
    """radians per position of every pair, and what the rotated numbers are multiplied by"""
    rot, s, length = c["rot"], c["factor"], float(c["original"])
    f = c["theta"] ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    if c["scaling"] == "linear":
        return f / s, 1.0
    if c["scaling"] == "bands":                            # long waves stretched, short ones kept, a blend between
        turns = length * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (1 - keep) * f / s + keep * f, 1.0
    if c["scaling"] == "ramp":                             # by the pair's index, between 32 turns and 1 of the length
        low, high = (rot * math.log(length / (b * 2 * math.pi)) / (2 * math.log(c["theta"])) for b in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0
    return f, 1.0


def _prepare_rope(c, seed):
    g = _generator(seed)
    t, hq, hkv, dk = c["tokens"] * c["requests"], c["Hq"], c["Hkv"], c["dk"]
    step = 1 + (torch.rand(c["requests"], c["tokens"], generator=g, device="cuda") < c["gaps"]).long()
    positions = (c["first"] + step.cumsum(1) - 1).flatten()
    if c["first"] and c["tokens"] == 1:                    # single tokens: every request at its own
        positions = positions + torch.randint(0, c["first"], (t,), generator=g, device="cuda")
    wide = _randn(g, (t, hq + hkv * (2 if c["fused"] else 1), dk), torch.bfloat16)
    q, k = wide[:, :hq], wide[:, hq:hq + hkv]
    if not c["fused"]:
        q, k = q.contiguous(), k.contiguous()
    freq, gain = _frequencies(c)
    return {"case": c, "q": q, "k": k, "positions": positions, "freq": freq.cuda(), "gain": gain,
            "q_out": torch.zeros(t, hq, dk, dtype=torch.bfloat16, device="cuda"),
            "k_out": torch.zeros(t, hkv, dk, dtype=torch.bfloat16, device="cuda"),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _exponents(x):
    """the biased exponent of the power-of-two scale of every row of x: the least with max|x| / scale <= 448"""
    m, e = torch.frexp(x.float().abs().amax(-1))
    b = e - 9 + (m > E4M3_MAX / 512) + 127
    return torch.where(m == 0, 127, b.clamp(1, 254)).to(torch.uint8)


def _fill(s, g, names, shape, f8):
    """pages of keys with a few strong channels and values whose size differs from token to token"""
    pages, hkv, b, dk = shape
    step = max(1, (1 << 28) // (hkv * b * dk))
    for name in names:
        cache = torch.zeros(shape, dtype=torch.uint8 if f8 else torch.bfloat16, device="cuda")
        if f8:
            s[name + "_scale"] = torch.zeros(pages, hkv, -(-b // 16) * 16, dtype=torch.uint8, device="cuda")
        for p in range(0, pages, step):
            x = _randn(g, (min(step, pages - p), hkv, b, dk), torch.bfloat16)
            if name == "k":
                x[..., :: dk // 4] *= 6.0
            else:
                x *= torch.exp2(_randn(g, x.shape[:3] + (1,))).to(torch.bfloat16)
            if f8:
                e = _exponents(x)
                s[name + "_scale"][p:p + step, :, :b] = e
                x = torch.ldexp(x.float(), 127 - e.int()[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            cache[p:p + step] = x
        s[name + "_cache"] = cache.view(torch.float8_e4m3fn) if f8 else cache


def _prepare_cache(c, seed):
    g, rng = _generator(seed), random.Random(seed)
    hkv, dk, b, lens, r = c["Hkv"], c["dk"], c["page"], _lengths(c), c["requests"]
    need = [-(-n // b) for n in lens]
    pages = sum(need) + 1 + max(1, sum(need)) // 16
    # pages are handed out in no order; entries past a request's last page are -1
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int64)
    wide = max(1, max(need)) + rng.randint(0, 3)
    start = torch.tensor([0] + need, device="cuda").cumsum(0)
    col = torch.arange(wide, device="cuda")
    at = (start[:-1, None] + col[None, :]).clamp(max=pages - 1)
    table = torch.where(col[None, :] < torch.tensor(need, device="cuda")[:, None], perm[at], -1).to(torch.int32)
    # what older steps gave a row: most have little, some nothing
    mass = torch.exp(2.0 * _randn(g, (pages, hkv, b)) - 4.0)
    mass[torch.rand(mass.shape, generator=g, device="cuda") < 0.2] = 0.0
    s = {"case": c, "table": table, "seqused": _int32(lens), "mass": mass,
         "born": torch.zeros(pages, hkv, b, dtype=torch.int32, device="cuda"),
         "total": _int32([n + n // 3 for n in lens]), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    # tokens that went left the stream's order: the first are where they were, the others about so
    live, page, tok, pos = _places(s)
    order = torch.where(live[:, None], pos[None, None] + 0.1 * _rows_of(s) * _randn(g, (r, hkv, pos.numel())), math.inf)
    order[:, :, :4] = -math.inf
    rank = order.argsort(dim=-1, stable=True).argsort(dim=-1, stable=True)
    gap = torch.where(rank < 4, 0, (s["total"] - s["seqused"])[:, None, None])
    s["born"][_rows(s, live, page, tok, hkv)] = (rank + gap).to(torch.int32)[live[:, None].expand(r, hkv, -1)]
    if c["op"] == "mass":
        _fill(s, g, "k", (pages, hkv, b, dk), c["fmt"] == "e4m3")
        if c["fmt"] == "e4m3":                             # the values' side of the cache is not looked at
            s["v_cache"], s["v_scale"] = s["k_cache"], s["k_scale"]
        else:
            s["v_cache"] = s["k_cache"]
        s["q"] = _randn(g, (r, c["Hq"], dk), torch.bfloat16)
        s["mass_out"] = torch.zeros_like(mass)
        s["counted"] = _int32([0 if c["fresh"] else max(0, n - 1) for n in lens])
        s["lse"] = torch.full((r, c["Hq"]), -math.inf, device="cuda")
        for i, n in enumerate(lens):
            if n:
                at = torch.arange(n, device="cuda")
                k = _value(s, "k", table[i].long()[at // b], slice(None), at % b).transpose(0, 1)
                x = (s["q"][i].view(hkv, -1, dk).float() @ k.transpose(1, 2)) * dk ** -0.5
                s["lse"][i] = torch.logsumexp(x.flatten(0, 1), -1)
        return s
    if c["op"] == "evict":
        s["budget"] = _int32(_budgets(c))
        most = max(1, max(min(k, n - k) for n, k in zip(lens, _budgets(c))))
        s["new_len"] = torch.zeros(r, dtype=torch.int32, device="cuda")
    else:
        _fill(s, g, "kv", (pages, hkv, b, dk), c["fmt"] == "e4m3")
        most = max(1, max(_moved(c)))
    s["moves"] = torch.full((r, hkv, most, 2), -1, dtype=torch.int32, device="cuda")
    s["num_moves"] = torch.zeros(r, hkv, dtype=torch.int32, device="cuda")
    if c["op"] == "move":
        for i, (n, k, m) in enumerate(zip(lens, _budgets(c), _moved(c))):
            for j, (lo, hi) in enumerate(((k, n), (0, k))):
                x = torch.rand(hkv, hi - lo, generator=g, device="cuda").argsort(-1)[:, :m].sort(-1).values + lo
                s["moves"][i, :, :m, j] = x.to(torch.int32)
            s["num_moves"][i] = m
    return s


def prepare(c, seed):
    return _prepare_rope(c, seed) if c["op"] == "rope" else _prepare_cache(c, seed)


# ------------------------------------------------------------------------------------------ plain forms

def _plain_turn(s, x, out, cos, sin):
    c, h = s["case"], s["case"]["rot"] // 2
    turned, rest = x[..., :2 * h].float(), x[..., 2 * h:]
    if c["layout"] == "halves":
        a, b = turned[..., :h], turned[..., h:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    out[..., :2 * h] = turned
    out[..., 2 * h:] = rest


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["gain"]).float()[:, None] for f in (torch.cos, torch.sin))
    if s["case"]["transpose"]:
        sin = -sin
    _plain_turn(s, s["q"], s["q_out"], cos, sin)
    _plain_turn(s, s["k"], s["k_out"], cos, sin)
    return {"q": s["q_out"], "k": s["k_out"]}


def _value(s, name, *at):
    """what `at` picks out of the cache [pages, Hkv, B, dk], in 32 bits"""
    if name + "_scale" not in s:
        return s[name + "_cache"][at].float()
    x = s[name + "_cache"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    return x * torch.exp2(s[name + "_scale"][..., :s["case"]["page"]][at].float() - 127)[..., None]


def _rows_of(s):
    return s["seqused"].long()[:, None, None]


def _places(s):
    """every position of the tables: whether it holds a row [R, P], its page [R, P] and its place there [P]"""
    b = s["case"]["page"]
    pos = torch.arange(s["table"].shape[1] * b, device=s["table"].device)
    return pos[None] < _rows_of(s)[..., 0], s["table"].long()[:, pos // b], pos % b, pos


def _rows(s, live, page, tok, hkv):
    """(page, head, token) of every live row, in the order of [R, Hkv, P]"""
    at = live[:, None].expand(-1, hkv, -1).nonzero(as_tuple=True)
    return page[at[0], at[2]], at[1], tok[at[2]]


def _plain_mass(s):
    c, q = s["case"], s["q"]
    r, hkv, dk = q.shape[0], c["Hkv"], c["dk"]
    live, page, tok, pos = _places(s)
    k = _value(s, "k", s["table"].long().clamp(min=0)).transpose(1, 2).flatten(2, 3)      # [R, Hkv, P, dk]
    a = (q.view(r, hkv, -1, dk).float() * dk ** -0.5) @ k.transpose(-1, -2)
    w = torch.exp(a - s["lse"].view(r, hkv, -1, 1)).sum(2)
    at, mine = _rows(s, live, page, tok, hkv), live[:, None].expand(r, hkv, -1)
    new = (pos[None, None] >= s["counted"].long()[:, None, None]).expand(r, hkv, -1)
    s["mass_out"][at] = torch.where(new[mine], 0.0, c["decay"] * s["mass"][at]) + w[mine]
    born = (s["total"] - s["seqused"])[:, None, None] + pos[None, None]
    s["born"][at] = torch.where(new[mine], born.expand(r, hkv, -1)[mine].to(torch.int32), s["born"][at])
    return {"mass": s["mass_out"], "born": s["born"]}


def _plain_evict(s):
    c, r, hkv = s["case"], s["case"]["requests"], s["case"]["Hkv"]
    live, page, tok, pos = _places(s)
    page, head = page.clamp(min=0)[:, None], torch.arange(hkv, device=page.device)[None, :, None]
    mass, born = s["mass"][page, head, tok], s["born"][page, head, tok]
    safe = (born < c["sinks"]) | (born >= s["total"][:, None, None] - c["recent"])
    order = torch.where(live[:, None], mass, -math.inf).argsort(dim=-1, descending=True, stable=True)
    kind = torch.where(live[:, None], torch.where(safe, 0, 1), 2)
    order = order.gather(-1, kind.gather(-1, order).argsort(dim=-1, stable=True))
    keep = torch.minimum(s["budget"], s["seqused"])
    kept = torch.zeros_like(safe).scatter_(-1, order, (pos < keep[:, None]).unsqueeze(1).expand(r, hkv, -1))
    low = pos < keep[:, None, None]
    hole, tail = low & ~kept, ~low & kept
    for j, x in enumerate((tail, hole)):
        at = x.nonzero(as_tuple=True)
        s["moves"][at[0], at[1], (x.cumsum(-1) - 1)[at], j] = at[2].to(torch.int32)
    s["num_moves"].copy_(hole.sum(-1))
    s["new_len"].copy_(keep)
    return {"moves": s["moves"], "num_moves": s["num_moves"], "new_len": s["new_len"]}


def _plain_move(s):
    b, moves = s["case"]["page"], s["moves"].long()
    at = (torch.arange(moves.shape[2], device=moves.device) < s["num_moves"][..., None]).nonzero(as_tuple=True)
    page, tok = s["table"].long()[at[0][:, None], moves[at] // b], moves[at] % b
    out = {}
    for name in ("k_cache", "v_cache", "k_scale", "v_scale", "mass", "born"):
        if name in s:
            x = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
            x[page[:, 1], at[1], tok[:, 1]] = x[page[:, 0], at[1], tok[:, 0]]
            out[name] = s[name]
    return out


# ------------------------------------------------------------------------------------------ the calls

def _own_rope(s):
    import long_context_prefill_varlen_gb300 as up
    c = s["case"]
    if "plan" not in s:                                    # the plan is the program's, kept from step to step
        s["plan"] = up.up_rope_plan(c["rot"], theta=c["theta"], layout=c["layout"], scaling=c["scaling"], factor=c["factor"],
                                    original_len=c["original"])
    up.up_rope(s["plan"], s["positions"], s["status"], q=s["q"], q_out=s["q_out"], k=s["k"], k_out=s["k_out"],
               transpose=c["transpose"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_mass(s):
    import long_context_prefill_varlen_gb300 as up
    up.up_kv_mass(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seqused"], s["lse"], s["mass"], s["born"], s["status"],
                  k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), mass_out=s["mass_out"], counted=s["counted"],
                  total=s["total"], decay=s["case"]["decay"])
    return {"mass": s["mass_out"], "born": s["born"]}


def _own_evict(s):
    import long_context_prefill_varlen_gb300 as up
    up.up_kv_evict(s["mass"], s["born"], s["table"], s["seqused"], s["budget"], s["moves"], s["num_moves"], s["new_len"],
                   s["status"], total=s["total"], sinks=s["case"]["sinks"], recent=s["case"]["recent"])
    return {"moves": s["moves"], "num_moves": s["num_moves"], "new_len": s["new_len"]}


def _own_move(s):
    import long_context_prefill_varlen_gb300 as up
    up.up_kv_move(s["k_cache"], s["v_cache"], s["table"], s["moves"], s["num_moves"], s["status"], k_scale=s.get("k_scale"),
                  v_scale=s.get("v_scale"), mass=s["mass"], born=s["born"])
    return {name: s[name] for name in ("k_cache", "v_cache", "k_scale", "v_scale", "mass", "born") if name in s}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "mass": _own_mass, "evict": _own_evict, "move": _own_move}[op](s)
    return {"rope": _plain_rope, "mass": _plain_mass, "evict": _plain_evict, "move": _plain_move}[op](s)


# ------------------------------------------------------------------------------------------ 64 bits

def _exact_frequency(c, j):
    rot = c["rot"]
    f = math.exp(-math.log(c["theta"]) * 2 * j / rot)
    wave = 2 * math.pi / f
    if c["scaling"] == "linear":
        return f / c["factor"]
    if c["scaling"] == "bands":
        if wave < c["original"] / 4.0:
            return f
        if wave > c["original"] / 1.0:
            return f / c["factor"]
        smooth = (c["original"] / wave - 1.0) / 3.0
        return (1 - smooth) * f / c["factor"] + smooth * f
    if c["scaling"] == "ramp":
        def index(turns):                                  # the pair that turns so often over the trained length
            return rot / 2 * math.log(c["original"] / (2 * math.pi * turns)) / math.log(c["theta"])
        low, high = max(0, math.floor(index(32))), min(rot - 1, math.ceil(index(1)))
        x = (j - low) / (high - low) if high > low else (j - low) * 1000.0
        x = min(1.0, max(0.0, x))
        return f * (x / c["factor"] + 1 - x)
    return f


def _exact_rope(c, s):
    pairs = c["rot"] // 2
    gain = 1 + math.log(c["factor"]) / 10 if c["scaling"] == "ramp" else 1.0
    freq = torch.tensor([_exact_frequency(c, j) for j in range(pairs)], dtype=torch.float64, device="cuda")
    first = torch.arange(pairs, device="cuda") * (1 if c["layout"] == "halves" else 2)
    second = first + (pairs if c["layout"] == "halves" else 1)
    out = {}
    for name in "qk":
        y = s[name].double()
        for t in range(0, y.shape[0], 1 << 16):
            z = torch.polar(torch.full((), gain, dtype=torch.float64, device="cuda"),
                            s["positions"][t:t + (1 << 16), None].double() * freq * (-1 if c["transpose"] else 1))[:, None]
            x = s[name][t:t + (1 << 16)].double()
            z = torch.complex(x[..., first], x[..., second]) * z
            y[t:t + (1 << 16), :, first] = z.real
            y[t:t + (1 << 16), :, second] = z.imag
        out[name] = y
    return out


def _exact_keys(s, page, head, off):
    """rows of the keys as 64-bit numbers, from the formats' definitions"""
    if "k_scale" not in s:
        return s["k_cache"][page, head, off].double()
    code = s["k_cache"].view(torch.uint8)[page, head, off].int()
    sign, e, m = 1.0 - 2.0 * (code >> 7).double(), (code >> 3) & 15, (code & 7).double()
    size = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).double()))
    return sign * size * torch.exp2(s["k_scale"][page, head, off].double() - 127)[..., None]


def _exact_mass(c, s):
    group, b = c["Hq"] // c["Hkv"], c["page"]
    mass, born = torch.zeros(s["mass"].shape, dtype=torch.float64, device="cuda"), s["born"].clone()
    for r, n in enumerate(_lengths(c)):
        pos = torch.arange(n, device="cuda")
        page, off = s["table"][r].long()[pos // b], pos % b
        old = int(s["counted"][r])
        born[page[old:], :, off[old:]] = (pos[old:] + int(s["total"][r]) - n).to(torch.int32)[:, None]
        for h in range(c["Hkv"] if n else 0):
            q, k = s["q"][r, h * group:(h + 1) * group].double(), _exact_keys(s, page, h, off)
            w = torch.exp(q @ k.T / math.sqrt(c["dk"]) - s["lse"][r, h * group:(h + 1) * group, None].double()).sum(0)
            w[:old] += c["decay"] * s["mass"][page[:old], h, off[:old]].double()
            mass[page, h, off] = w
    return {"mass": mass, "born": born}


def _exact_evict(c, s):
    moves, number = s["moves"].clone(), s["num_moves"].clone()
    keep, b = _budgets(c), c["page"]
    for r, n in enumerate(_lengths(c)):
        pos, total = torch.arange(n, device="cuda"), int(s["total"][r])
        page, off = s["table"][r].long()[pos // b], pos % b
        for h in range(c["Hkv"]):
            born, x = s["born"][page, h, off], s["mass"][page, h, off].double()
            x = torch.where((born < c["sinks"]) | (born >= total - c["recent"]), x + 1e30, x)
            safe = x >= 1e30                               # protected rows that do not all fit: by mass as well
            if int(safe.sum()) > keep[r]:
                x = torch.where(safe, s["mass"][page, h, off].double(), -1.0)
            least = x.sort(descending=True).values[keep[r] - 1] if keep[r] else torch.tensor(math.inf, device="cuda")
            stay, ties = x > least, (x == least).nonzero()[:, 0]
            stay[ties[:keep[r] - int(stay.sum())]] = True
            tail = stay[keep[r]:].nonzero()[:, 0] + keep[r]
            moves[r, h, :tail.numel(), 0] = tail.to(torch.int32)
            moves[r, h, :tail.numel(), 1] = (~stay[:keep[r]]).nonzero()[:, 0].to(torch.int32)
            number[r, h] = tail.numel()
    return {"moves": moves, "num_moves": number, "new_len": _int32(keep)}


def _exact_move(c, s):
    """the rows, moved in 64 bits: the codes' values, as the outputs are"""
    out = {}
    for name in ("k_cache", "v_cache", "k_scale", "v_scale", "mass", "born"):
        if name in s:
            x = s[name]
            y = x.double() if x.is_floating_point() else x.clone()
            for r, m in enumerate(_moved(c)):
                for h in range(c["Hkv"]):
                    src, dst = (s["moves"][r, h, :m, j].long() for j in (0, 1))
                    table = s["table"][r].long()
                    y[table[dst // c["page"]], h, dst % c["page"]] = y[table[src // c["page"]], h, src % c["page"]]
            out[name] = y
    return out


def exact(c, seed):
    s = prepare(c, seed)
    return {"rope": _exact_rope, "mass": _exact_mass, "evict": _exact_evict, "move": _exact_move}[c["op"]](c, s)
