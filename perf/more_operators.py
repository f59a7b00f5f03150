"""What the paged key/value cache's operators are measured on, and their plain forms.

Every rank holds H key/value heads of size d and two pools of pages, [pages, H, page, d]: bf16, or e4m3 with one power of
two for each position and head.  Sequence b has len[b] positions; position j lies in row j % page of page table[b, j // page].
The rows start[b] .. start[b + 1] - 1 of a call's token arrays are the sequence's newest positions.

  append     writes the rows' keys and values into the pages.  e4m3: 2^k is the least power of two (k >= -64) with
             max|x| <= 448 * 2^k over a row's d values, and the pages hold x / 2^k, rounded to e4m3
  gather     reads the rows' keys and values back, in bf16
  attention  softmax(scale q k) v of the rows' queries over the positions up to their own (with a window: over the last
             `window` of those), Hq = G * H query heads, and each row's log of the sum of exponentials

The cache's e4m3 pools are returned as e4m3 values beside the exponents' bytes (k + 127).
"""
import math

import torch

own = False


def _case(name, op, R, B, n, ctx, H, d, page, dtype, G=1, window=0, ragged=False):
    c = dict(op=op, R=R, B=B, n=n, ctx=ctx, H=H, d=d, page=page, dtype=dtype, G=G, window=window, ragged=ragged)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one running request writes its newest token: only the launch counts
        _case("append 1 token bf16", "append", 1, 1, 1, 777, 8, 128, 16, "bf16"),
        # the prompts of a prefill step, quantised, heads split over two ranks
        _case("append 4 x 4096 e4m3 tp2", "append", 2, 4, 4096, 9000, 8, 128, 64, "e4m3"),
        # a few short prefixes copied out to be handed on, odd lengths
        _case("gather 3 short bf16 d64", "gather", 1, 3, 333, 333, 5, 64, 16, "bf16", ragged=True),
        # whole contexts read back to be moved to another server
        _case("gather 16 x 8192 e4m3", "gather", 1, 16, 8192, 8192, 8, 128, 64, "e4m3"),
        # the smallest decode step: one request with a short context
        _case("decode 1 x 1023 bf16", "attention", 1, 1, 1, 1023, 8, 128, 16, "bf16", G=4),
        # a decode batch of requests at all stages
        _case("decode 64 x 8192 bf16", "attention", 1, 64, 1, 8192, 8, 128, 16, "bf16", G=8, ragged=True),
        # the same with a quantised cache, heads split over eight ranks, and more requests
        _case("decode 201 x 8000 e4m3 tp8", "attention", 8, 201, 1, 8000, 1, 128, 64, "e4m3", G=8, ragged=True),
        # one request with a very long context: its positions are all the parallelism there is
        _case("decode 1 x 1000003 e4m3", "attention", 1, 1, 1, 1000003, 8, 128, 64, "e4m3", G=8),
        # speculative decoding: five proposed tokens of each request are verified
        _case("verify 40 x 5 e4m3", "attention", 1, 40, 5, 6000, 8, 128, 32, "e4m3", G=8, ragged=True),
        # a chunk of a long prompt over what the chunks before it left
        _case("chunk 2048 over 32768 bf16", "attention", 1, 1, 2048, 32768, 8, 128, 64, "bf16", G=4),
        # prefill and decode in one step, odd head counts and lengths, a sliding window, quantised
        _case("mixed 9 x 1-700 e4m3 window", "attention", 1, 9, 700, 5003, 4, 64, 16, "e4m3", G=7, window=1000, ragged=True),
        # a whole prompt, heads split over two ranks
        _case("prompt 8192 bf16 tp2", "attention", 2, 1, 8192, 8192, 4, 128, 64, "bf16", G=8),
    ]


def _lens(c):
    """Each sequence's newest positions and all its positions: by the case alone, so that its work is known."""
    n, l = [], []
    for b in range(c["B"]):
        u = (0.5 + b * 0.6180339887498949) % 1.0
        n.append(max(1, int(c["n"] * (u * u if c["ragged"] else 1.0))))
        full = c["ctx"] == c["n"]
        l.append(n[-1] if full else max(n[-1], int(c["ctx"] * ((0.25 + 0.75 * u) if c["ragged"] else 1.0))))
    n[0], l[0] = c["n"], c["ctx"]
    return n, l


def _seen(c):
    """(row, position) pairs that a rank's one query head sees, and positions that are read, over all sequences."""
    pairs = read = 0
    w = c["window"] or 1 << 60
    for n, l in zip(*_lens(c)):
        first = l - n  # position of the first row
        ramp = max(0, min(l, w) - first)  # rows whose visible positions still grow
        pairs += sum((first + 1, first + ramp)) * ramp // 2 + (n - ramp) * min(w, l)
        read += l - max(0, first - w + 1)
    return pairs, read


def _cost(c):
    w = work(c)
    return w["bytes"] / 7e12 + w["flops"] / 1.5e15


def _plain_values(c):
    """Values of the largest intermediates that the plain form holds."""
    rows = c["B"] * c["H"] * c["G"] * c["n"]
    L = c["ctx"]
    return rows * L + 2 * c["B"] * L * c["H"] * c["d"] if c["op"] == "attention" else c["R"] * c["B"] * c["n"] * c["H"] * c["d"]


def draw(rng):
    every = listed()
    most = {op: max(_cost(c) for c in every if c["op"] == op) for op in ("append", "gather", "attention")}
    held = max(_plain_values(c) for c in every if c["op"] == "attention")

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["append", "gather", "attention", "attention"])
        n = log(1, 9000) if op != "attention" or rng.random() < 0.5 else rng.choice([1, 1, 1, log(1, 16)])
        ctx = max(n, log(1, 300000))
        c = _case(None, op, rng.choice([1, 1, 2, 4, 8]), log(1, 300), n, ctx, rng.choice([1, 2, 3, 4, 5, 8]),
                  rng.choice([64, 128]), rng.choice([16, 16, 32, 64, 128, 1]), rng.choice(["bf16", "e4m3"]),
                  ragged=rng.random() < 0.7)
        if op == "attention":
            c.update(G=rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16]), window=rng.choice([0, 0, 0, log(1, ctx)]))
        if _cost(c) <= most[op] and _plain_values(c) <= held and c["B"] * ctx * c["H"] * c["d"] * c["R"] < 1 << 32:
            return c


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    R, B, H, d, P = c["R"], c["B"], c["H"], c["d"], c["page"]
    n, l = _lens(c)
    T, wide = sum(n), max(-(-x // P) for x in l)
    used = sum(-(-x // P) for x in l)
    pages = used + 1 + used // 16  # some are free
    dev = torch.device("cuda")

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    # pages were handed out as sequences grew: no order, and a table's entries past a sequence's end are stale
    s = dict(c, T=T, pages=pages, max_pages=wide, Hq=H * c["G"], scale=1.0 / math.sqrt(d), start=ints([0] + n).cumsum(0).to(torch.int32), len=ints(l))
    own_pages = (s["len"][:, None].long() + P - 1) // P
    perm = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
    at = torch.arange(wide, device=dev)[None]
    first = torch.cumsum(own_pages, 0) - own_pages
    s["table"] = torch.where(at < own_pages, perm[(first + at).clamp(max=pages - 1)], perm[0]).contiguous()

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g, dtype=torch.bfloat16)

    def pool():
        if c["dtype"] == "bf16":
            return normal(pages, H, P, d)
        x = torch.empty(pages, H, P, d, device=dev, dtype=torch.float8_e4m3fn)
        # rows of maximum 4 or so, as the scale 2^-6 leaves them
        for a in range(0, pages, 8192):
            x[a:a + 8192] = (torch.randn(x[a:a + 8192].shape, device=dev, generator=g) * 64).clamp_(-448, 448).to(x.dtype)
        return x

    s["K"], s["V"] = [pool() for _ in range(R)], [pool() for _ in range(R)]
    if c["dtype"] == "e4m3":
        for name in ("K_exp", "V_exp"):
            s[name] = [torch.randint(120, 123, (pages, H, P), device=dev, generator=g, dtype=torch.uint8) for _ in range(R)]
    if c["op"] == "append":
        # keys have channels that stand out; now and then a head's row is nearly nothing
        loud = 1 + 7 * (torch.rand(H, d, device=dev, generator=g) < 0.03)
        quiet = torch.where(torch.rand(T, H, 1, device=dev, generator=g) < 0.01, 2.0 ** -20, 1.0)
        s["k_new"] = [(normal(T, H, d) * loud).to(torch.bfloat16) for _ in range(R)]
        s["v_new"] = [(normal(T, H, d) * quiet).to(torch.bfloat16) for _ in range(R)]
    elif c["op"] == "gather":
        s["k_out"], s["v_out"] = ([torch.empty(T, H, d, device=dev, dtype=torch.bfloat16) for _ in range(R)] for _ in range(2))
    else:
        # most rows' scores are spread out, some look for one position (a key near their own query)
        seq, pos = _rows(s)
        low = torch.clamp(pos - c["window"] + 1, min=0) if c["window"] else torch.zeros_like(pos)
        s["Q"] = []
        for r in range(R):
            aim = low + (torch.rand(T, device=dev, generator=g) * (pos + 1 - low)).long()
            k = _at(s, "K", r, seq, torch.minimum(aim, pos))
            near = torch.rand(T, H, c["G"], 1, device=dev, generator=g) * 1.2
            s["Q"].append((normal(T, H, c["G"], d) + near * k[:, :, None]).to(torch.bfloat16).view(T, s["Hq"], d))
        s["O"] = [torch.empty(T, s["Hq"], d, device=dev, dtype=torch.bfloat16) for _ in range(R)]
        s["lse"] = [torch.empty(T, s["Hq"], device=dev) for _ in range(R)]
    return s


def _rows(s):
    """Each row's sequence and position."""
    n = s["start"].diff().long()
    seq = torch.repeat_interleave(torch.arange(s["B"], device="cuda"), n, output_size=s["T"])
    return seq, torch.arange(s["T"], device="cuda") - s["start"][seq].long() + s["len"][seq].long() - n[seq]


def _where(s, seq, pos):
    """Page and row of positions."""
    return s["table"][seq, pos // s["page"]].long(), pos % s["page"]


def _two_to(k):
    """2^k of whole numbers in 32 bits, exactly."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _at(s, name, r, seq, pos):
    """The cache's values at positions: [..., H, d] in 32 bits."""
    page, row = _where(s, seq, pos)
    h = torch.arange(s["H"], device="cuda")
    if s["dtype"] == "bf16":
        return s[name][r][page[..., None], h, row[..., None]].float()
    # (indexed as bytes, read as e4m3)
    x = s[name][r].view(torch.uint8)[page[..., None], h, row[..., None]].view(torch.float8_e4m3fn).float()
    return x * _two_to(s[name + "_exp"][r][page[..., None], h, row[..., None]].int() - 127)[..., None]


def _quantise(x):
    """Rows of d values as e4m3 and the byte of their power of two."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(dim=-1))  # max = m 2^e, 1/2 <= m < 1: 448 = 7/8 2^9
    k = torch.where(m == 0, -64, torch.clamp(torch.where(m > 0.875, e - 8, e - 9), min=-64))
    return (x * _two_to(-k)[..., None]).to(torch.float8_e4m3fn), (k + 127).to(torch.uint8)


def _plain_append(s):
    seq, pos = _rows(s)
    page, row = _where(s, seq, pos)
    at = page[:, None], torch.arange(s["H"], device="cuda"), row[:, None]

    def put(pool, x):
        pool[at] = x

    if s["dtype"] == "bf16":
        _ = [put(pool, x) for name in ("K", "V") for pool, x in zip(s[name], s[name.lower() + "_new"])]
        return {"K": s["K"], "V": s["V"]}
    made = {name: [_quantise(x) for x in s[name.lower() + "_new"]] for name in ("K", "V")}
    _ = [put(pool.view(torch.uint8), q.view(torch.uint8)) for name in made for pool, (q, _) in zip(s[name], made[name])]
    _ = [put(pool, e) for name in made for pool, (_, e) in zip(s[name + "_exp"], made[name])]
    return {name: s[name] for name in ("K", "V", "K_exp", "V_exp")}


def _plain_gather(s):
    seq, pos = _rows(s)
    return {name: [_at(s, name, r, seq, pos).to(torch.bfloat16) for r in range(s["R"])] for name in ("K", "V")}


def _plain_attention(s, r):
    """All sequences at once, padded to the longest."""
    B, H, G, d = s["B"], s["H"], s["G"], s["d"]
    seq, pos = _rows(s)
    n = s["start"].diff().long()
    rows, L = s["n"], s["ctx"]
    j = torch.arange(L, device="cuda")[None]
    there = j < s["len"][:, None]
    at = torch.arange(B, device="cuda")[:, None].expand(B, L), torch.where(there, j, 0)
    k = _at(s, "K", r, *at).permute(0, 2, 3, 1)                                       # [B, H, d, L]
    v = torch.where(there[..., None, None], _at(s, "V", r, *at), 0.0).transpose(1, 2)  # [B, H, L, d]
    i = torch.arange(s["T"], device="cuda") - s["start"][seq].long()
    q = torch.zeros(B, rows, H * G, d, device="cuda")
    q[seq, i] = s["Q"][r].float()
    q = q.view(B, rows, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * rows, d)
    x = torch.matmul(q, k).mul_(s["scale"]).view(B, H, G, rows, L)
    p = s["len"][:, None].long() - n[:, None] + torch.arange(rows, device="cuda")  # [B, rows]
    out = (j[:, None] > p[..., None]) | ~there[:, None]
    if s["window"]:
        out |= j[:, None] <= p[..., None] - s["window"]
    x = x.masked_fill_(out[:, None, None], -torch.inf)
    m = x.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(m).exp_()
    z = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x.view(B, H, G * rows, L), v).view(B, H, G, rows, d) / z
    lse = (m + torch.log(z))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, rows, H * G, d)
    return o[seq, i].to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(B, rows, H * G)[seq, i]


def _handles(s):
    """The descriptions of the cache and of the step's sequences that a serving loop keeps beside its buffers."""
    import gemm_collective_gb300 as fcc

    if "handles" not in s:
        e4m3 = s["dtype"] == "e4m3"
        cache = fcc.make_cache(s["K"], s["V"], s["pages"], s["page"], s["H"], s["d"], fcc.FCC_E4M3 if e4m3 else fcc.FCC_BF16,
                               s["K_exp"] if e4m3 else None, s["V_exp"] if e4m3 else None)
        s["handles"] = fcc, cache, fcc.make_batch(s["start"], s["len"], s["table"], s["T"], s["B"], s["max_pages"])
    return s["handles"]


def _own(s):
    fcc, cache, batch = _handles(s)
    st = torch.cuda.current_stream()
    if s["op"] == "append":
        fcc.fcc_cache_append(s["R"], s["k_new"], s["v_new"], cache, batch, stream=st)
        return {name: s[name] for name in ("K", "V", "K_exp", "V_exp") if name in s}
    if s["op"] == "gather":
        fcc.fcc_cache_gather(s["R"], cache, batch, s["k_out"], s["v_out"], stream=st)
        return {"K": s["k_out"], "V": s["v_out"]}
    fcc.fcc_paged_attention(s["R"], s["Q"], cache, batch, s["Hq"], s["O"], s["lse"], scale=s["scale"], window=s["window"], stream=st)
    return {"O": s["O"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "append":
        return _plain_append(state)
    if state["op"] == "gather":
        return _plain_gather(state)
    made = [_plain_attention(state, r) for r in range(state["R"])]
    return {"O": [o for o, _ in made], "lse": [x for _, x in made]}


def work(case):
    c = case
    T = sum(_lens(c)[0])
    held = 2 * c["H"] * (c["d"] + 1 if c["dtype"] == "e4m3" else 2 * c["d"])  # of one position
    if c["op"] != "attention":
        return {"bytes": c["R"] * T * (held + 4 * c["H"] * c["d"]), "flops": 0}
    pairs, read = _seen(c)
    Hq = c["H"] * c["G"]
    return {"bytes": c["R"] * (read * held + T * Hq * (4 * c["d"] + 4)), "flops": 4 * c["R"] * c["d"] * Hq * pairs}


def _power(k):
    """2^k of whole numbers in 64 bits, exactly."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _value(codes, byte):
    """e4m3 codes (as whole numbers) and their row's byte as 64-bit numbers, by the format's own definition."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _power(e - 10))
    return torch.where(c >= 128, -x, x) * _power(byte.to(torch.int64) - 127)[..., None]


def _exact_rows(s, name, r, b, upto):
    """Positions 0 .. upto - 1 of sequence b: [H, upto, d]."""
    P = s["page"]
    page = s["table"][b, :-(-upto // P)].long()
    x = s[name][r][page] if s["dtype"] == "bf16" else s[name][r].view(torch.uint8)[page]
    x = x.double() if s["dtype"] == "bf16" else _value(x, s[name + "_exp"][r][page])
    return x.transpose(0, 1).reshape(s["H"], -1, s["d"])[:, :upto]


def _exact_e4m3(x):
    """The nearest e4m3 value (ties to the even one) of each x / 2^k, and k's byte."""
    x = x.double()
    top = x.abs().amax(-1)
    k = torch.full_like(top, -64)
    for step in (64, 32, 16, 8, 4, 2, 1):  # the largest k that is still too small, by halving, and one more
        k = torch.where(448 * _power(k + step - 1) < top, k + step, k)
    x = x * _power(-k)[..., None]
    lo = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    unit = _power(lo - 3)
    return torch.round(x / unit) * unit, (k + 127).to(torch.uint8)


def exact(case, seed):
    """From the definitions, in 64 bits, a sequence and a head at a time."""
    c = case
    if c["op"] == "attention" and (work(c)["flops"] > 6e12 or c["R"] * sum(_lens(c)[1]) * c["H"] * c["d"] > 3e9):
        return None
    s = prepare(case, seed)
    R, B, H, G, d, P = (s[k] for k in ("R", "B", "H", "G", "d", "page"))
    n, l = _lens(c)
    if c["op"] == "append":
        out = {}
        for name in ("K", "V"):
            out[name] = [x.double() for x in s[name]]
            if s["dtype"] == "e4m3":
                out[name + "_exp"] = s[name + "_exp"]
            t = 0
            for b in range(B):
                pos = torch.arange(l[b] - n[b], l[b], device="cuda")
                page, row = s["table"][b, pos // P].long(), pos % P
                for r in range(R):
                    x = s[name.lower() + "_new"][r][t:t + n[b]]
                    if s["dtype"] == "e4m3":
                        x, e = _exact_e4m3(x)
                        out[name + "_exp"][r][page, :, row] = e
                    out[name][r][page, :, row] = x.double()
                t += n[b]
        return out
    if c["op"] == "gather":
        made = {name: [torch.cat([_exact_rows(s, name, r, b, l[b])[:, l[b] - n[b]:].transpose(0, 1) for b in range(B)]) for r in range(R)]
                for name in ("K", "V")}
        return made
    O, lse = [], []
    for r in range(R):
        o_r = torch.zeros(s["T"], H, G, d, dtype=torch.float64, device="cuda")
        z_r = torch.zeros(s["T"], H, G, dtype=torch.float64, device="cuda")
        t = 0
        for b in range(B):
            K, V = _exact_rows(s, "K", r, b, l[b]), _exact_rows(s, "V", r, b, l[b])
            q = s["Q"][r][t:t + n[b]].double().view(n[b], H, G, d)
            p = torch.arange(l[b] - n[b], l[b], device="cuda")[:, None]
            j = torch.arange(l[b], device="cuda")[None]
            hide = (j > p) | (j <= p - (s["window"] or 1 << 40))
            for h in range(H):
                x = torch.einsum("igd,jd->igj", q[:, h], K[h]) * s["scale"]
                x.masked_fill_(hide[:, None], float("-inf"))
                z = torch.logsumexp(x, -1)
                o_r[t:t + n[b], h] = torch.einsum("igj,jd->igd", torch.exp_(x.sub_(z[..., None])), V[h])
                z_r[t:t + n[b], h] = z
            t += n[b]
        O.append(o_r.view(s["T"], H * G, d))
        lse.append(z_r.view(s["T"], H * G))
    return {"O": O, "lse": lse}
