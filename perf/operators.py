"""The paged key-value cache's operators as a serving program calls them: cases, inputs, plain forms and calls.

Three operators work on one layer's cache, pages of B tokens laid out [pages, Hkv, B, dk], held in bf16 or in
e4m3 with one power-of-two scale (a biased exponent, uint8) per token and head:
  write   quantise (or copy) the new keys and values [T, Hkv, dk] into the rows that `slots` names
  read    bring the rows that `slots` names back to a packed bf16 stream [T, Hkv, dk]
  decode  attention of one new token per request over its pages, with the layer's own lengths (`seqused`)

`own` false: elementary torch operations in 32 bits.  `own` true: the calls of long_context_prefill_varlen_gb300.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------ cases

def _case(name, op, fmt, heads, page, lengths, window=0, fused=False, padded=0):
    """heads = (Hq, Hkv, dk); lengths = (requests, shortest, longest, how they are spread)"""
    hq, hkv, dk = heads
    r, lo, hi, spread = lengths
    c = dict(op=op, fmt=fmt, Hq=hq, Hkv=hkv, dk=dk, page=page, requests=r, shortest=lo, longest=hi, spread=spread,
             window=window, fused=fused, padded=padded)
    if name:
        c["name"] = name
    return c


LLAMA, QWEN, GEMMA = (32, 8, 128), (16, 2, 256), (16, 8, 256)      # the layer geometries of bench.py's workloads


def listed():
    return [
        # the first generated token of a single 4K request: the smallest call, latency counts
        _case("decode 1 x 4K bf16", "decode", "bf16", LLAMA, 16, (1, 4096, 4096, "even")),
        # a batch in continuous batching, an empty and a one-token request among them
        _case("decode 64 x 0-8K e4m3", "decode", "e4m3", LLAMA, 16, (64, 0, 8192, "even")),
        # the packed batch of 16 requests of 4K to 128K tokens, generating
        _case("decode 16 x 4K-128K bf16", "decode", "bf16", LLAMA, 64, (16, 4096, 131072, "log")),
        # four long documents on wide heads, eight query heads to a key head
        _case("decode 4 x 128K e4m3", "decode", "e4m3", QWEN, 32, (4, 131072, 131072, "even")),
        # the largest batch that bench.py scores, generating from a bf16 cache
        _case("decode 64 x 32K bf16", "decode", "bf16", GEMMA, 16, (64, 32768, 32768, "even")),
        # a sliding-window layer beside it: 1,024 of up to 32K tokens, pages of an odd size
        _case("decode window e4m3", "decode", "e4m3", GEMMA, 24, (64, 300, 32768, "log"), window=1024),
        # one step's new tokens, a batch padded to 64 rows
        _case("write 64 new e4m3", "write", "e4m3", LLAMA, 16, (64, 1, 1, "even"), padded=5),
        # the tokens that a drop kept of a 32K prefill, straight from the fused projection's output
        _case("write 32K kept e4m3", "write", "e4m3", LLAMA, 16, (1, 32513, 32513, "even"), fused=True),
        # the packed batch of 16 requests into an unquantised cache
        _case("write 16 x 4K-128K bf16", "write", "bf16", LLAMA, 64, (16, 4096, 131072, "log")),
        # a short cached prefix brought back for the next chunk's scores
        _case("read 1000 bf16", "read", "bf16", LLAMA, 16, (1, 1000, 1000, "even")),
        # a 32K cached prefix
        _case("read 32K e4m3", "read", "e4m3", LLAMA, 16, (1, 32768, 32768, "even")),
        # the prefixes of a packed batch on wide heads
        _case("read 4 x 100K-128K e4m3", "read", "e4m3", QWEN, 32, (4, 100000, 131072, "even")),
    ]


GEOMETRIES = [LLAMA, LLAMA, QWEN, GEMMA, (8, 8, 64), (28, 4, 128), (16, 1, 64), (40, 8, 128), (32, 1, 128)]


def draw(rng):
    op = rng.choice(["decode", "decode", "write", "read"])
    fmt = rng.choice(["bf16", "e4m3"])
    hq, hkv, dk = rng.choice(GEOMETRIES)
    page = rng.choice([8, 16, 16, 24, 32, 48, 64, 128, 256])
    budget = math.exp(rng.uniform(math.log(2e6), math.log(6e9)))           # bytes of a bf16 cache
    tokens = min(2_000_000, max(1, int(budget / (4 * hkv * dk))))
    requests = min(256, tokens, int(math.exp(rng.uniform(0, math.log(100)))))
    longest = min(1_000_000, max(1, tokens // requests)) + rng.choice([0, 0, 1, 3])
    spread = rng.choice(["even", "log", "same"])
    shortest = longest if spread == "same" else rng.choice([0, 1, longest // 30, longest // 3])
    window = rng.choice([0, 0, 0, 128, 1000, 4096]) if op == "decode" else 0
    padded = rng.choice([0, 0, 7]) if op == "write" and requests > 16 and longest < 64 else 0
    return _case(None, op, fmt, (hq, hkv, dk), page, (requests, shortest, longest, spread), window,
                 op == "write" and rng.random() < 0.3, padded)


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


def _attended(c):
    return [min(n, c["window"]) if c["window"] else n for n in _lengths(c)]


def _row_bytes(c):
    """one token and head of the cache, keys or values"""
    return 2 * c["dk"] if c["fmt"] == "bf16" else c["dk"] + 1


def work(c):
    tokens, hkv, dk = sum(_lengths(c)), c["Hkv"], c["dk"]
    if c["op"] == "decode":
        seen, r = sum(_attended(c)), c["requests"]
        pages = sum(-(-n // c["page"]) for n in _attended(c))
        return {"bytes": 2 * seen * hkv * _row_bytes(c) + 4 * pages + r * (4 * c["Hq"] * dk + 4 * c["Hq"] + 4),
                "flops": 4 * seen * c["Hq"] * dk}
    return {"bytes": 2 * tokens * hkv * (2 * dk + _row_bytes(c)) + 8 * (tokens + c["padded"]),
            "flops": 4 * tokens * hkv * dk if c["fmt"] == "e4m3" else 0}


# ------------------------------------------------------------------------------------------ inputs

def _exponents(x):
    """the biased exponent of the power-of-two scale of every row of x: the least with max|x| / scale <= 448"""
    m, e = torch.frexp(x.float().abs().amax(-1))
    b = e - 9 + (m > E4M3_MAX / 512) + 127
    return torch.where(m == 0, 127, b.clamp(1, 254)).to(torch.uint8)


def _codes(x, b):
    """x over its rows' scales, in e4m3"""
    return torch.ldexp(x.float(), 127 - b.int()[..., None]).to(torch.float8_e4m3fn)


def _rows(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _kv(g, t, hkv, dk, spread):
    """keys with a few strong channels and values whose size differs from token to token, as projections give"""
    k, v = _rows(g, (t, hkv, dk)), _rows(g, (t, hkv, dk))
    k[..., :: dk // 4] *= 6.0
    v *= torch.exp2(spread * torch.randn((t, hkv, 1), generator=g, device="cuda")).to(torch.bfloat16)
    return k, v


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)
    hkv, dk, b = c["Hkv"], c["dk"], c["page"]
    lens = _lengths(c)
    need = [-(-n // b) for n in lens]
    spare = 1 + max(1, sum(need)) // 16
    pages = sum(need) + spare
    # pages are handed out in no order; entries past a request's last page are -1
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int64)
    wide = max(1, max(need)) + rng.randint(0, 3)
    start = torch.tensor([0] + need, device="cuda").cumsum(0)
    col = torch.arange(wide, device="cuda")
    at = (start[:-1, None] + col[None, :]).clamp(max=pages - 1)
    table = torch.where(col[None, :] < torch.tensor(need, device="cuda")[:, None], perm[at], -1).to(torch.int32)
    f8 = c["fmt"] == "e4m3"
    s = {"case": c, "table": table, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    shape = (pages, hkv, b, dk)
    if f8:
        s["k_cache"], s["v_cache"] = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                                      for _ in "kv")
        s["k_scale"], s["v_scale"] = (torch.zeros(pages, hkv, -(-b // 16) * 16, dtype=torch.uint8, device="cuda")
                                      for _ in "kv")
    else:
        s["k_cache"], s["v_cache"] = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    if c["op"] == "write":
        # prefill writes from position 0; a step's single tokens go to the last position of their pages so far
        tokens = sum(lens)
        req = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"),
                                      output_size=tokens)
        cu = torch.tensor([0] + lens, device="cuda").cumsum(0)
        pos = torch.arange(tokens, device="cuda") - cu[req]
        if max(lens) == 1:
            pos = torch.randint(0, b, (tokens,), generator=g, device="cuda")
        slots = table[req, pos // b].long() * b + pos % b
        t = tokens + c["padded"]
        s["slots"] = torch.cat([slots, slots.new_full((c["padded"],), -1)])
        k, v = _kv(g, t, hkv, dk, 1.0)
        if c["fused"]:                                     # the rows of the fused projection: q heads, k heads, v heads
            qkv = torch.zeros(t, c["Hq"] + 2 * hkv, dk, dtype=torch.bfloat16, device="cuda")
            qkv[:, c["Hq"]:c["Hq"] + hkv], qkv[:, c["Hq"] + hkv:] = k, v
            k, v = qkv[:, c["Hq"]:c["Hq"] + hkv], qkv[:, c["Hq"] + hkv:]
        s["k"], s["v"] = k, v
        return s
    step = max(1, (1 << 28) // (hkv * b * dk))
    for p in range(0, pages, step):                        # every page holds something: masked places too
        n = min(step, pages - p)
        k, v = _kv(g, n * b, hkv, dk, 1.0)
        for name, x in (("k", k), ("v", v)):
            x = x.view(n, b, hkv, dk).transpose(1, 2)
            if f8:
                e = _exponents(x)
                s[name + "_scale"][p:p + n, :, :b] = e
                s[name + "_cache"].view(torch.uint8)[p:p + n] = _codes(x, e).view(torch.uint8)
            else:
                s[name + "_cache"][p:p + n] = x
    if c["op"] == "read":
        tokens = sum(lens)
        req = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"),
                                      output_size=tokens)
        cu = torch.tensor([0] + lens, device="cuda").cumsum(0)
        pos = torch.arange(tokens, device="cuda") - cu[req]
        s["slots"] = table[req, pos // b].long() * b + pos % b
        s["k"], s["v"] = (torch.zeros(tokens, hkv, dk, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        return s
    s["seqused"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q"] = _rows(g, (len(lens), c["Hq"], dk))
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(len(lens), c["Hq"], device="cuda")
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _plain_write(s):
    b = s["case"]["page"]
    live = s["slots"] >= 0
    page, off = s["slots"][live] // b, s["slots"][live] % b
    out = {}
    for name in ("k", "v"):
        x = s[name][live]
        if "k_scale" in s:
            e = _exponents(x)
            s[name + "_scale"][page, :, off] = e
            s[name + "_cache"].view(torch.uint8)[page, :, off] = _codes(x, e).view(torch.uint8)
            out[name + "_scale"] = s[name + "_scale"]
        else:
            s[name + "_cache"][page, :, off] = x
        out[name] = s[name + "_cache"]
    return out


def _plain_value(s, name, *at):
    """what `at` picks out of the cache [pages, Hkv, B, dk], in 32 bits"""
    if "k_scale" not in s:
        return s[name + "_cache"][at].float()
    x = s[name + "_cache"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    return x * torch.exp2(s[name + "_scale"][..., :s["case"]["page"]][at].float() - 127)[..., None]


def _plain_read(s):
    b = s["case"]["page"]
    at = (s["slots"] // b, slice(None), s["slots"] % b)
    s["k"].copy_(_plain_value(s, "k", *at))
    s["v"].copy_(_plain_value(s, "v", *at))
    return {"k": s["k"], "v": s["v"]}


def _plain_pages(s, name, pages):
    """the requests' pages side by side: [R, Hkv, positions, dk]"""
    return _plain_value(s, name, pages).transpose(1, 2).flatten(2, 3)


def _plain_decode(s):
    c, q, pages = s["case"], s["q"], s["table"].long().clamp(min=0)
    b, r, n = c["page"], q.shape[0], s["seqused"].long()[:, None]
    pos = torch.arange(pages.shape[1] * b, device=q.device).expand(r, -1)
    if c["window"]:                                        # the pages that hold the window alone
        col = (n - c["window"]).clamp(min=0) // b + torch.arange(-(-c["window"] // b) + 1, device=q.device)
        pos = (col[:, :, None] * b + torch.arange(b, device=q.device)).flatten(1)
        pages = pages.gather(1, col.clamp(max=pages.shape[1] - 1))
    seen = pos < n
    if c["window"]:
        seen &= pos >= n - c["window"]
    qg = q.view(r, c["Hkv"], -1, c["dk"]).float() * c["dk"] ** -0.5
    logits = qg @ _plain_pages(s, "k", pages).transpose(-1, -2)
    logits = torch.where(seen[:, None, None, :], logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    o = p @ _plain_pages(s, "v", pages) / torch.where(total == 0, 1.0, total)
    s["out"].copy_(o.view_as(q))
    s["lse"].copy_((top + torch.log(total)).view_as(s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------ the calls

def _own_write(s):
    import long_context_prefill_varlen_gb300 as up
    up.up_kv_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["status"], k_scale=s.get("k_scale"),
                   v_scale=s.get("v_scale"))
    out = {"k": s["k_cache"], "v": s["v_cache"]}
    if "k_scale" in s:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _own_read(s):
    import long_context_prefill_varlen_gb300 as up
    up.up_kv_read(s["k_cache"], s["v_cache"], s["slots"], s["k"], s["v"], s["status"], k_scale=s.get("k_scale"),
                  v_scale=s.get("v_scale"))
    return {"k": s["k"], "v": s["v"]}


def _own_decode(s):
    import long_context_prefill_varlen_gb300 as up
    c, q, table = s["case"], s["q"], s["table"]
    if "ws" not in s:                                      # the workspace is the program's, kept from step to step
        nbytes = up.up_paged_decode_workspace_bytes(q.shape[0], c["Hq"], c["Hkv"], c["dk"], c["page"],
                                                    table.shape[1], c["window"])
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    up.up_paged_decode(q, s["k_cache"], s["v_cache"], table, s["seqused"], s["out"], s["ws"], s["status"],
                       k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), lse=s["lse"], window=c["window"])
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "decode": _own_decode}[op](s)
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode}[op](s)


# ------------------------------------------------------------------------------------------ 64 bits

def _e4m3_value(y):
    """the e4m3 number nearest to every y (|y| <= 448), ties to the even one, from the format's definition: four
    significant bits down to 2^-6, steps of 2^-9 below"""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(y / step) * step


def _value(s, name, page, off, head=slice(None)):
    """rows of the cache as 64-bit numbers, of every head or of one"""
    if "k_scale" not in s:
        return s[name + "_cache"][page, head, off].double()
    code = s[name + "_cache"].view(torch.uint8)[page, head, off].int()
    sign, e, m = 1.0 - 2.0 * (code >> 7).double(), (code >> 3) & 15, (code & 7).double()
    size = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).double()))
    return sign * size * torch.exp2(s[name + "_scale"][page, head, off].double() - 127)[..., None]


def exact(c, seed):
    s = prepare(c, seed)
    b, out = c["page"], {}
    if c["op"] == "write":
        for name in ("k", "v"):
            cache = torch.zeros(s[name + "_cache"].shape, dtype=torch.float64, device="cuda")
            if "k_scale" in s:
                out[name + "_scale"] = torch.zeros_like(s[name + "_scale"])
            for i in range(0, s["slots"].numel(), 1 << 16):
                slots = s["slots"][i:i + (1 << 16)]
                keep = (slots >= 0).nonzero()[:, 0]
                slots, x = slots[keep], s[name][i:i + (1 << 16)][keep].double()
                if "k_scale" in s:
                    top = x.abs().amax(-1)
                    e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(-126, 127)
                    e = torch.where(top == 0, 0.0, torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e))
                    e = torch.where((top <= E4M3_MAX * torch.exp2(e - 1)) & (e > -126) & (top > 0), e - 1, e)
                    out[name + "_scale"][slots // b, :, slots % b] = (e + 127).to(torch.uint8)
                    x = _e4m3_value(x * torch.exp2(-e)[..., None])
                cache[slots // b, :, slots % b] = x
            out[name] = cache
        return out
    if c["op"] == "read":
        for name in ("k", "v"):
            out[name] = torch.cat([_value(s, name, i // b, i % b) for i in s["slots"].split(1 << 16)])
        return out
    group, scale = c["Hq"] // c["Hkv"], 1.0 / math.sqrt(c["dk"])
    o = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for r, n in enumerate(_lengths(c)):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == first:
            continue
        pos = torch.arange(first, n, device="cuda")
        page, off = s["table"][r].long()[pos // b], pos % b
        q = s["q"][r].double()
        for h in range(0, c["Hq"], group):
            k, v = (_value(s, name, page, off, h // group) for name in ("k", "v"))
            a = scale * (q[h:h + group] @ k.T)
            lse[r, h:h + group] = torch.logsumexp(a, -1)
            o[r, h:h + group] = torch.exp(a - lse[r, h:h + group, None]) @ v
    return {"out": o, "lse": lse}
