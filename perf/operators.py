"""What the vocabulary-parallel losses are measured on, and their plain forms.

The head's weights W [V, D] are split by rows over R ranks; every rank holds a copy of the tokens' last hidden states
X [T, D].  Two losses on the logits l = X W^T (optionally capped, l = c tanh(x / c)), each forward and backward:

  xent     lse - (1 - eps) l_y - eps / V sum_v l_v + z lse^2,  lse = log sum_v exp(l_v)
  distill  tau^2 KL(q || p), q the softmax over a teacher's top logits / tau, p the softmax over all l / tau

"forward" gives every rank's loss and lse; "backward" takes lse and the losses' upstream gradients and gives every rank's
dX (the sum over the ranks) and dW (its own rows).
"""
import math

import torch

own = False

IGNORE = -100


def _case(name, op, dir, T, V, D, R=1, K=0, smoothing=0.0, z=0.0, softcap=0.0, tau=1.0):
    c = dict(op=op, dir=dir, T=T, V=V, D=D, R=R, K=K, smoothing=smoothing, z=z, softcap=softcap, tau=tau)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a unit test's size: only launches and latency count
        _case("xent fwd 5 tokens", "xent", "forward", 5, 1009, 256, smoothing=0.1),
        # scoring one token of a running request
        _case("xent fwd 1 token", "xent", "forward", 1, 32000, 4096),
        # scoring a decode batch with the head split over eight ranks: the weights' bytes bound it
        _case("xent fwd 64 tokens tp8", "xent", "forward", 64, 131072, 8192, R=8),
        # a training micro-batch on one rank
        _case("xent fwd 4096 tokens", "xent", "forward", 4096, 32000, 4096),
        # the largest forward: a long sequence, the head split over eight ranks
        _case("xent fwd 8192 tokens tp8", "xent", "forward", 8192, 131072, 4096, R=8, z=1e-4),
        # an adapter's or a short prompt's step: the gradient of the weights is most of the bytes
        _case("xent bwd 96 tokens", "xent", "backward", 96, 32000, 4096),
        # odd sizes everywhere, with smoothing and capped logits
        _case("xent bwd odd capped", "xent", "backward", 1999, 50257, 2048, smoothing=0.1, softcap=30.0),
        # the largest backward
        _case("xent bwd 4096 tokens tp8", "xent", "backward", 4096, 131072, 4096, R=8, z=1e-4),
        # a small distillation batch
        _case("distill fwd 33 tokens", "distill", "forward", 33, 4099, 512, K=8),
        # a distillation micro-batch, softened
        _case("distill fwd 4096 tokens", "distill", "forward", 4096, 32000, 4096, K=64, tau=2.0),
        # its backward at odd sizes with capped logits
        _case("distill bwd odd capped", "distill", "backward", 777, 50257, 1024, K=20, tau=1.5, softcap=30.0),
        # its backward on two ranks with a long list of teacher entries
        _case("distill bwd 4096 tokens tp2", "distill", "backward", 4096, 65536, 4096, R=2, K=128),
    ]


def _cost(c):
    return c["T"] * c["V"] * c["D"] * (1 if c["dir"] == "forward" else 3)


def draw(rng):
    most = max(_cost(c) for c in listed())

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op, dir = rng.choice(["xent", "distill"]), rng.choice(["forward", "backward"])
        R = rng.choice([1, 1, 2, 4, 8])
        c = _case(None, op, dir, log(1, 8192), log(500, 131072) // R * R, 8 * log(16, 1024), R,
                  softcap=rng.choice([0.0, 0.0, 30.0]))
        if op == "xent":
            c.update(smoothing=rng.choice([0.0, 0.1]), z=rng.choice([0.0, 1e-4]))
        else:
            c.update(K=log(1, 128), tau=rng.choice([1.0, 2.0, 0.75]))
        if _cost(c) <= most:
            return c


def _lse(X, W, softcap, tau):
    """log sum exp of the capped logits / tau, in 32 bits, rank after rank."""
    m = s = None
    for x, w in zip(X, W):
        l = _cap(x.float() @ w.float().T, softcap) / tau
        top = l.max(dim=1, keepdim=True).values if m is None else torch.maximum(m, l.max(dim=1, keepdim=True).values)
        part = torch.exp(l - top).sum(dim=1, keepdim=True)
        s = part if m is None else s * torch.exp(m - top) + part
        m = top
    return (m + torch.log(s))[:, 0]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, V, D, R = c["T"], c["V"], c["D"], c["R"]

    def rand(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    # logits of standard deviation 1.28, whatever D; the token's own word stands out by about 10, as in a trained model
    W = torch.randn(V, D, device="cuda", generator=g, dtype=torch.bfloat16) * (1.28 / math.sqrt(D))
    word = torch.randint(0, V, (T,), device="cuda", generator=g)
    X = torch.randn(T, D, device="cuda", generator=g)
    X += 6.0 * W[word].float() * rand(T, 1)
    X = X.to(torch.bfloat16)
    s = dict(c, X=[X.clone() for _ in range(R)], W=[w.clone() for w in W.split(V // R)])
    masked = rand(T) < 0.1  # a prompt's or a padding's tokens
    masked[0] = False
    if c["op"] == "xent":
        s["labels"] = torch.where(masked, IGNORE, word).to(torch.int32)
    else:
        # distinct entries of every row, the word first; lists end early here and there, and masked rows have none
        K = c["K"]
        step = 1 + (rand(T, 1) * (V // K - 1)).long()
        idx = (word[:, None] + step * torch.arange(K, device="cuda")) % V
        val = torch.sort(torch.randn(T, K, device="cuda", generator=g) * 2.0, dim=1, descending=True).values
        val[:, 0] += 4.0
        count = torch.where(rand(T) < 0.2, (1 + rand(T) * K).long(), K)
        count = torch.where(masked, 0, count)
        over = torch.arange(K, device="cuda")[None] >= count[:, None]
        s["teacher_idx"] = torch.where(over, -1, idx).to(torch.int32)
        s["teacher"] = val.float()
    if c["dir"] == "forward":
        s["loss"] = [torch.empty(T, device="cuda") for _ in range(R)]
        s["lse"] = [torch.empty(T, device="cuda") for _ in range(R)]
    else:
        # the mean over the tokens that count, of a loss scaled per sequence
        s["dloss"] = (0.5 + rand(T)) / max(1.0, 0.9 * T)
        s["lse"] = [_lse(s["X"], s["W"], c["softcap"], c["tau"]).clone() for _ in range(R)]
        s["dX"] = [torch.empty(T, D, device="cuda", dtype=torch.bfloat16) for _ in range(R)]
        s["dW"] = [torch.empty(V // R, D, device="cuda", dtype=torch.bfloat16) for _ in range(R)]
    return s


def _cap(x, softcap):
    return softcap * torch.tanh(x / softcap) if softcap else x


def _teacher(s):
    """The teacher's probabilities over each row's entries (0 where it has none), and which rows have any."""
    there = s["teacher_idx"] >= 0
    t = torch.where(there, s["teacher"] / s["tau"], -torch.inf)
    live = there.any(dim=1)
    e = torch.where(there, torch.exp(t - torch.where(live, t.max(dim=1).values, 0.0)[:, None]), 0.0)
    return e / torch.where(live, e.sum(dim=1), 1.0)[:, None], live


def _plain_forward(s):
    l = _cap(torch.cat([x.float() @ w.float().T for x, w in zip(s["X"], s["W"])], dim=1), s["softcap"]) / s["tau"]
    m = l.max(dim=1).values
    lse = m + torch.log(torch.exp(l - m[:, None]).sum(dim=1))
    if s["op"] == "xent":
        live = s["labels"] != IGNORE
        at = torch.where(live, s["labels"], 0).long()
        ly = l.gather(1, at[:, None])[:, 0]
        eps = s["smoothing"]
        loss = lse - (1 - eps) * ly + s["z"] * lse * lse
        if eps:
            loss = loss - eps / s["V"] * l.sum(dim=1)
    else:
        q, live = _teacher(s)
        lk = l.gather(1, s["teacher_idx"].clamp(min=0).long())
        logq = torch.log(torch.where(q > 0, q, 1.0))
        loss = s["tau"] ** 2 * ((q * (logq - lk)).sum(dim=1) + lse)
    loss = torch.where(live, loss, 0.0)
    return {"loss": [loss] * s["R"], "lse": [lse] * s["R"]}


def _plain_backward(s):
    l = _cap(torch.cat([x.float() @ w.float().T for x, w in zip(s["X"], s["W"])], dim=1), s["softcap"])
    p = torch.exp(l / s["tau"] - s["lse"][0][:, None])
    if s["op"] == "xent":
        live = s["labels"] != IGNORE
        at = torch.where(live, s["labels"], 0).long()
        eps = s["smoothing"]
        d = p * (1 + 2 * s["z"] * s["lse"][0])[:, None] - eps / s["V"]
        d.scatter_add_(1, at[:, None], torch.full_like(at, -(1 - eps), dtype=torch.float32)[:, None])
        d = d * s["dloss"][:, None]
    else:
        q, live = _teacher(s)
        d = p.scatter_add_(1, s["teacher_idx"].clamp(min=0).long(), -q)
        d = d * (s["tau"] * s["dloss"])[:, None]
    if s["softcap"]:
        d = d * (1 - (l / s["softcap"]) ** 2)
    d = torch.where(live[:, None], d, 0.0).split(s["V"] // s["R"], dim=1)
    dX = sum(x @ w.float() for x, w in zip(d, s["W"])).to(torch.bfloat16)
    return {"dX": [dX] * s["R"], "dW": [(x.T @ h.float()).to(torch.bfloat16) for x, h in zip(d, s["X"])]}


def _own(s):
    import gemm_collective_gb300 as fcc

    st = torch.cuda.current_stream()
    sizes = s["T"], s["V"], s["D"]
    if s["op"] == "xent":
        kw = dict(ignore_index=IGNORE, smoothing=s["smoothing"], z_weight=s["z"], softcap=s["softcap"], stream=st)
        if s["dir"] == "forward":
            fcc.fcc_linear_xent(s["R"], s["X"], s["W"], s["labels"], *sizes, s["loss"], s["lse"], **kw)
        else:
            fcc.fcc_linear_xent_grad(s["R"], s["X"], s["W"], s["labels"], s["lse"], s["dloss"], *sizes, s["dX"], s["dW"], **kw)
    else:
        kw = dict(temperature=s["tau"], softcap=s["softcap"], stream=st)
        if s["dir"] == "forward":
            fcc.fcc_linear_distill(s["R"], s["X"], s["W"], s["teacher_idx"], s["teacher"], *sizes, s["K"], s["loss"], s["lse"], **kw)
        else:
            fcc.fcc_linear_distill_grad(s["R"], s["X"], s["W"], s["teacher_idx"], s["teacher"], s["lse"], s["dloss"], *sizes,
                                        s["K"], s["dX"], s["dW"], **kw)
    if s["dir"] == "forward":
        return {"loss": s["loss"], "lse": s["lse"]}
    return {"dX": s["dX"], "dW": s["dW"]}


def run(state):
    if own:
        return _own(state)
    return _plain_forward(state) if state["dir"] == "forward" else _plain_backward(state)


def work(case):
    T, V, D, R, K = (case[k] for k in ("T", "V", "D", "R", "K"))
    rows = R * T * D * 2 + V * D * 2
    aims = T * 8 * K if case["op"] == "distill" else T * 4
    if case["dir"] == "forward":
        return {"bytes": rows + aims + R * T * 8, "flops": 2 * T * V * D}
    # the logits are not kept: the backward pass computes them again
    return {"bytes": 2 * rows + aims + T * 4 + R * T * 4, "flops": 6 * T * V * D}


def exact(case, seed):
    """From the definitions, in 64 bits, a slice of the vocabulary at a time."""
    if _cost(case) * 2 > 1.4e13:
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    T, V, D, R, cap, tau = s["T"], s["V"], s["D"], s["R"], s["softcap"], s["tau"]
    X, W = s["X"][0].to(f64), torch.cat(s["W"])
    slices = [slice(a, min(V, a + 16384)) for a in range(0, V, 16384)]

    def scores(at):
        raw = torch.mm(X, W[at].to(f64).t())
        return (torch.tanh(raw / cap) * cap if cap else raw).div_(tau)

    parts = [scores(at) for at in slices]
    lse = torch.logsumexp(torch.stack([torch.logsumexp(p, 1) for p in parts]), 0)
    aim = torch.zeros(T, V, dtype=f64, device="cuda")  # the probabilities that the scores are drawn to
    rows = torch.arange(T, device="cuda")
    if s["op"] == "xent":
        live = s["labels"] >= 0
        aim += s["smoothing"] / V
        aim[rows[live], s["labels"][live].long()] += 1 - s["smoothing"]
        entropy = torch.zeros(T, dtype=f64, device="cuda")
        scale, pull = 1.0, 1 + 2 * s["z"] * lse
        extra = s["z"] * lse.square()
    else:
        has = s["teacher_idx"] >= 0
        live = has.sum(1) > 0
        t = (s["teacher"].to(f64) / tau).masked_fill(~has, float("-inf"))
        q = torch.softmax(t[live], 1)
        r, k = torch.nonzero(has[live], as_tuple=True)
        aim.index_put_((rows[live][r], s["teacher_idx"][live][r, k].long()), q[r, k], accumulate=True)
        entropy = torch.zeros(T, dtype=f64, device="cuda")
        entropy[live] = torch.special.xlogy(q, q).sum(1)
        scale, pull = tau, torch.ones_like(lse)
        extra = torch.zeros_like(lse)
    if s["dir"] == "forward":
        hit = sum((aim[:, at] * p).sum(1) for at, p in zip(slices, parts))
        loss = (scale * scale * (entropy - hit + lse) + extra).masked_fill(~live, 0.0)
        return {"loss": [loss] * R, "lse": [lse] * R}
    dX = torch.zeros(T, D, dtype=f64, device="cuda")
    dW = torch.empty(V, D, dtype=f64, device="cuda")
    up = (s["dloss"].to(f64) * scale).masked_fill(~live, 0.0)[:, None]
    for at, p in zip(slices, parts):
        d = (torch.exp(p - lse[:, None]) * pull[:, None] - aim[:, at]) * up
        if cap:
            d *= 1 - (p * (tau / cap)).square()
        dX += torch.mm(d, W[at].to(f64))
        dW[at] = torch.mm(d.t(), X)
    return {"dX": [dX] * R, "dW": list(dW.split(V // R))}
