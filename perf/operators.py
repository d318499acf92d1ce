"""Cases of the operators that stand around the MoE layer in a serving step.

`run(state)` makes one pass through one operator: in its plain form (`own` false:
elementary torch operations in 32 bits, 64 where 32 would lose what matters) or
through this package (`own` true).  The operators:

  linear   y = x W^T with e4m3 weights that carry one fp32 scale per 128 x 128
           block; the bf16 tokens are quantised per token and 128 inputs
  step     the gated delta rule for the next 1..8 tokens of each sequence,
           states in a slot pool, updated in place
  prefill  the gated delta rule over packed prompts of any lengths
  select   beam search: the best W continuations of W beams over the vocabulary
  reorder  beam search: states of the surviving beams moved to their new places,
           in place
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
BLOCK = 128   # inputs (and outputs of the weights) that share a scale
CHUNK = 16    # tokens per chunk of the plain prefill


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token through a square projection of the hidden size
        dict(name="linear decode", op="linear", T=1, N=2560, K=2560, out="bf16"),
        # a verify window of 8 tokens through a wide projection
        dict(name="linear verify", op="linear", T=8, N=8192, K=2560, out="bf16"),
        # a chunk of a prompt whose sizes fill no tile and no scale block
        dict(name="linear ragged", op="linear", T=517, N=1544, K=1000, out="fp32"),
        # a long prompt through a large projection: bound by the tensor cores
        dict(name="linear prefill", op="linear", T=8192, N=8192, K=4096, out="bf16"),
        # one sequence, one token: the latency of a decode step
        dict(name="step decode", op="step", B=1, n=1, Hk=32, Hv=32, dk=128, dv=128, decay="channel"),
        # 64 sequences in a 4-token verify window: the states' traffic
        dict(name="step verify", op="step", B=64, n=4, Hk=32, Hv=32, dk=128, dv=128, decay="channel"),
        # one prompt chunk of 2048 tokens, a decay per channel
        dict(name="prefill one", op="prefill", T=2048, S=1, Hk=32, Hv=32, dk=128, dv=128, decay="channel"),
        # seven prompts of ragged lengths packed together, grouped heads, a decay per head
        dict(name="prefill ragged", op="prefill", T=8192, S=7, Hk=16, Hv=32, dk=128, dv=128, decay="head"),
        # the first step of one request: only one beam lives, logits from the LM head
        dict(name="select first", op="select", G=1, W=4, V=157184, dtype="fp32", finished=0, first=True),
        # a batch in the middle of its search, some beams finished
        dict(name="select batch", op="select", G=32, W=8, V=157184, dtype="bf16", finished=1, first=False),
        # two requests whose beams mostly stay where they are
        dict(name="reorder few", op="reorder", G=2, W=4, moved=2, cycle=False, row=2097152, small=0),
        # eight requests whose beams change places, a second, small state beside
        dict(name="reorder cycle", op="reorder", G=8, W=8, moved=6, cycle=True, row=2097152, small=24576),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "step", "prefill", "select", "reorder"])
    if op == "linear":
        while True:
            c = dict(op=op, T=_log(rng, 1, 8192), N=8 * _log(rng, 16, 1024), K=8 * _log(rng, 16, 1024),
                     out=rng.choice(["bf16", "fp32"]))
            if c["T"] * c["N"] * c["K"] <= 8192 * 8192 * 4096:
                return c
    if op in ("step", "prefill"):
        Hk = rng.choice([2, 4, 8, 16, 32])
        c = dict(op=op, Hk=Hk, Hv=Hk * rng.choice([1, 1, 2]), dk=rng.choice([64, 128, 128]),
                 dv=rng.choice([64, 128, 128]), decay=rng.choice(["channel", "channel", "head"]))
        if op == "step":
            c.update(n=rng.randint(1, 8), B=_log(rng, 1, max(1, 64 * 32 * 16384 // (c["Hv"] * c["dk"] * c["dv"]))))
        else:
            c.update(T=_log(rng, 1, 8192), S=rng.randint(1, 12))
            c["S"] = min(c["S"], c["T"])
        return c
    if op == "select":
        W = rng.randint(1, 16)
        return dict(op=op, W=W, G=_log(rng, 1, 256 // W), V=_log(rng, 1000, 157184), dtype=rng.choice(["fp32", "bf16"]),
                    finished=rng.randint(0, W - 1), first=rng.random() < 0.2)
    W = rng.randint(2, 16)
    return dict(op=op, W=W, G=_log(rng, 1, max(1, 64 // W)), moved=rng.randint(1, W - 1), cycle=rng.random() < 0.5,
                row=16 * _log(rng, 1024, 131072), small=rng.choice([0, 4096, 24576]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _lengths(T, S):
    """S ragged lengths that sum to T: each about 0.6 of the one before it, none empty."""
    w = [0.6 ** i for i in range(S)]
    n = [max(1, int(T * x / sum(w))) for x in w]
    n[0] += T - sum(n)
    return n if n[0] > 0 else [T - S + 1] + [1] * (S - 1)


def _blocks(t, rows):
    """[R, K] -> [R / rows, K / 128] scales max|.| / 448 and e4m3 codes of a matrix, zero-padded to whole blocks."""
    R, K = t.shape
    p = torch.nn.functional.pad(t.float(), (0, -K % BLOCK, 0, -R % rows))
    b = p.view(p.shape[0] // rows, rows, p.shape[1] // BLOCK, BLOCK)
    s = b.abs().amax(dim=(1, 3)) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    c = (b / s[:, None, :, None]).clamp(-448.0, 448.0).to(F8)
    return c.view(p.shape)[:R, :K].contiguous(), s


def _delta_inputs(c, tokens, g):
    """q, k, v as slices of one projection's output; log-decays and write strengths as their gates give them."""
    Hk, Hv, dk, dv = c["Hk"], c["Hv"], c["dk"], c["dv"]
    qkv = torch.randn(tokens, 2 * Hk * dk + Hv * dv, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = qkv.split([Hk * dk, Hk * dk, Hv * dv], dim=1)
    ch = dk if c["decay"] == "channel" else 1
    rate = 1.0 + 15.0 * torch.rand(Hv, 1, generator=g, device=DEV)
    dt = torch.exp(math.log(1e-3) + (math.log(1e-1) - math.log(1e-3)) * torch.rand(Hv, ch, generator=g, device=DEV))
    raw = torch.randn(tokens, Hv, ch, generator=g, device=DEV) + torch.log(torch.expm1(dt))
    decay = -rate * torch.nn.functional.softplus(raw)
    beta = torch.sigmoid(torch.randn(tokens, Hv, generator=g, device=DEV))
    return dict(q=q.view(tokens, Hk, dk), k=k.view(tokens, Hk, dk), v=v.view(tokens, Hv, dv),
                g=decay if c["decay"] == "channel" else decay.squeeze(-1), beta=beta)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=case)
    if c["op"] == "linear":
        w = torch.randn(c["N"], c["K"], generator=g, device=DEV) * 0.02
        s["codes"], s["scales"] = _blocks(w, BLOCK)
        s["x"] = torch.randn(c["T"], c["K"], generator=g, device=DEV).to(torch.bfloat16)
        if own:
            import weight_only_int4_fp32_b200 as lm
            s["op"] = lm.BlockFP8Linear(s["codes"], s["scales"], max_tokens=c["T"])
    elif c["op"] in ("step", "prefill"):
        n = c["B"] if c["op"] == "step" else c["S"]
        tokens = c["B"] * c["n"] if c["op"] == "step" else c["T"]
        s.update(_delta_inputs(c, tokens, g))
        slots = n + 1  # a pool with a slot that no sequence holds
        s["state"] = 0.3 * torch.randn(slots, c["Hv"], c["dk"], c["dv"], generator=g, device=DEV)
        s["slots"] = torch.randperm(slots, generator=g, device=DEV)[:n].to(torch.int32)
        if c["op"] == "prefill":
            s["lengths"] = _lengths(c["T"], c["S"])
            s["cu"] = torch.tensor([sum(s["lengths"][:i]) for i in range(c["S"] + 1)], dtype=torch.int32, device=DEV)
        if own:
            import weight_only_int4_fp32_b200 as lm
            s["op"] = lm.GatedDeltaRule(c["Hk"], c["Hv"], c["dk"], c["dv"], max_tokens=tokens, max_seqs=n)
    elif c["op"] == "select":
        G, W, V = c["G"], c["W"], c["V"]
        dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
        s["logits"] = (2.5 * torch.randn(G, W, V, generator=g, device=DEV)).to(dt)
        hot = torch.randint(0, V, (G, W, 20), generator=g, device=DEV)  # the head of the distribution
        s["logits"].scatter_add_(2, hot, (6.0 * torch.rand(G, W, 20, generator=g, device=DEV)).to(dt))
        s["scores"] = -torch.sort(30.0 * torch.rand(G, W, generator=g, device=DEV))[0]
        s["finished"] = torch.rand(G, W, generator=g, device=DEV).argsort(-1) < c["finished"]
        if c["first"]:
            s["scores"][:, 0], s["scores"][:, 1:], s["finished"][:] = 0.0, -math.inf, False
        s["eos"] = V - 1
        if own:
            import weight_only_int4_fp32_b200 as lm
            s["op"] = lm.BeamSearch(max_groups=G, beams=W, vocab=V)
    else:
        G, W = c["G"], c["W"]
        s["states"] = [torch.randn(G * W, c["row"] // 4, generator=g, device=DEV)]
        if c["small"]:
            s["states"].append(torch.randn(G * W, c["small"] // 2, generator=g, device=DEV).to(torch.bfloat16))
        order = torch.rand(G, W, generator=g, device=DEV).argsort(-1)
        moved = order[:, :c["moved"]]
        # the moved beams change places among themselves, or take the states of beams that stay
        src = moved.roll(1, -1) if c["cycle"] else order[:, c["moved"] + torch.arange(c["moved"], device=DEV) % (W - c["moved"])]
        place = torch.arange(W, device=DEV).expand(G, W).clone()
        s["parents"] = place.scatter(1, moved, src).to(torch.int32)
        if own:
            import weight_only_int4_fp32_b200 as lm
            s["op"] = lm.BeamSearch(max_groups=G, beams=W, vocab=1)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if c["op"] == "linear":
        dt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        return s["op"].forward(s["x"], out_dtype=dt) if own else _plain_linear(s["x"], s["codes"], s["scales"], dt)
    if c["op"] == "step":
        shape = lambda t: t.view(c["B"], c["n"], *t.shape[1:])  # noqa: E731
        a = [shape(s[k]) for k in ("q", "k", "v", "g", "beta")]
        if own:
            out = s["op"].step(*a, s["state"], slots=s["slots"])
        else:
            out = _plain_step(*a, s["state"], s["slots"])
        return dict(out=out, state=s["state"])
    if c["op"] == "prefill":
        a = [s[k] for k in ("q", "k", "v", "g", "beta")]
        if own:
            out = s["op"].prefill(*a, s["state"], s["cu"], slots=s["slots"])
        else:
            out = _plain_prefill(*a, s["state"], s["cu"], s["slots"], max(s["lengths"]))
        return dict(out=out, state=s["state"])
    if c["op"] == "select":
        f = s["op"].select if own else _plain_select
        tokens, parents, scores, finished = f(s["logits"], s["scores"], s["finished"], s["eos"])
        return dict(tokens=tokens, parents=parents, scores=scores, finished=finished)
    if own:
        s["op"].reorder(s["states"], s["parents"])
    else:
        _plain_reorder(s["states"], s["parents"])
    return dict(enumerate(s["states"]))


# ------------------------------------------------------------------ plain forms
def _plain_linear(x, codes, scales, dt):
    T, K = x.shape
    xb = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).view(T, -1, BLOCK)
    sx = xb.abs().amax(-1, keepdim=True) / 448.0
    sx = torch.where(sx > 0, sx, torch.ones_like(sx))
    xq = (xb / sx).clamp(-448.0, 448.0).to(F8).float() * sx
    ws = scales.repeat_interleave(BLOCK, 0)[:codes.shape[0]].repeat_interleave(BLOCK, 1)[:, :K]
    return (xq.view(T, -1)[:, :K] @ (codes.float() * ws).t()).to(dt)


def _unit(t):
    return t * torch.rsqrt(t.square().sum(-1, keepdim=True) + 1e-6)


def _heads(q, k, v, g, beta):
    """fp32, unit keys and queries of every value head, queries scaled, decays per channel."""
    r = v.shape[-2] // k.shape[-2]
    q = _unit(q.float()).repeat_interleave(r, -2) * q.shape[-1] ** -0.5
    k = _unit(k.float()).repeat_interleave(r, -2)
    return q, k, v.float(), g if g.dim() == k.dim() else g.unsqueeze(-1).expand(k.shape), beta


def _plain_step(q, k, v, g, beta, state, slots):
    q, k, v, g, beta = _heads(q, k, v, g, beta)
    S = state[slots.long()]
    outs = []
    for i in range(q.shape[1]):
        S = S * torch.exp(g[:, i]).unsqueeze(-1)
        u = beta[:, i].unsqueeze(-1) * (v[:, i] - (S * k[:, i].unsqueeze(-1)).sum(-2))
        S = S + k[:, i].unsqueeze(-1) * u.unsqueeze(-2)
        outs.append((S * q[:, i].unsqueeze(-1)).sum(-2))
    state[slots.long()] = S
    return torch.stack(outs, 1).to(torch.bfloat16)


def _plain_prefill(q, k, v, g, beta, state, cu, slots, longest):
    """Chunks of 16 tokens: inside a chunk every pair's decay is formed on its own and the writes are solved by
    (I + A)^-1 = (I - A)(I + A^2)(I + A^4)(I + A^8), A strictly lower triangular; chunks follow one another."""
    dt, T = torch.bfloat16, q.shape[0]
    t = _heads(q, k, v, g, beta)
    L = -(-longest // CHUNK) * CHUNK
    at = cu[:-1, None].long() + torch.arange(L, device=cu.device)
    live = at < cu[1:, None]
    at = at.clamp(max=T - 1)
    # [sequence, chunk, head, token, channel], zeros behind each sequence's end
    pack = lambda x: (x[at] * live.view(*live.shape, *[1] * (x.dim() - 1))).view(  # noqa: E731
        at.shape[0], L // CHUNK, CHUNK, *x.shape[1:]).transpose(2, 3)
    q, k, v, g = (pack(x) for x in t[:4])
    beta = pack(t[4].unsqueeze(-1))
    G = torch.cumsum(g, -2)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    pair = (G.unsqueeze(-2) - G.unsqueeze(-3)).masked_fill(~low[..., None], -math.inf).exp() * k.unsqueeze(-3)
    Aqk = (q.unsqueeze(-2) * pair).sum(-1)
    A = (beta * (k.unsqueeze(-2) * pair).sum(-1)).tril(-1)
    I = torch.eye(CHUNK, device=q.device)
    A2 = A @ A
    A4 = A2 @ A2
    P = (I - A) @ (I + A2) @ (I + A4) @ (I + A4 @ A4)
    E = torch.exp(G)
    w, u = P @ (beta * k * E), P @ (beta * v)
    qe, last = q * E, G[..., -1:, :]
    ke, ge = (k * torch.exp(last - G)).transpose(-1, -2), torch.exp(last).transpose(-1, -2)
    S = state[slots.long()]
    outs = []
    for i in range(L // CHUNK):
        d = u[:, i] - w[:, i] @ S
        outs.append(qe[:, i] @ S + Aqk[:, i] @ d)
        S = ge[:, i] * S + ke[:, i] @ d
    state[slots.long()] = S
    o = torch.stack(outs, 1).transpose(2, 3).reshape(at.shape[0], L, *v.shape[2:3], v.shape[-1])
    return o[live].to(dt)


def _plain_select(logits, scores, finished, eos):
    G, W, V = logits.shape
    x = logits.float()
    x = torch.where(x.isnan(), -math.inf, x)
    m = x.amax(-1, keepdim=True).double()
    lse = m + torch.exp(x.double() - m).sum(-1, keepdim=True).log()
    # the best of each row by (logit, then the lower token): one whole number for both
    b = x.view(torch.int32).long()
    key = torch.where(b < 0, -(b & 0x7FFFFFFF), b) * 2**31 + (2**31 - 1 - torch.arange(V, device=x.device))
    key, tok = key.topk(min(W, V), dim=-1)
    val = x.gather(-1, tok).double() - lse + scores.double().unsqueeze(-1)
    only = torch.full_like(val, -math.inf)
    only[..., 0] = scores.double()
    val = torch.where(finished.unsqueeze(-1), only, val)
    tok = torch.where(finished.unsqueeze(-1), eos, tok)
    val = torch.where(val.isnan(), -math.inf, val).flatten(1)
    val, at = torch.sort(val, dim=-1, descending=True, stable=True)
    val, at = val[:, :W], at[:, :W]
    none = val == -math.inf
    tokens = torch.where(none, -1, tok.flatten(1).gather(1, at))
    parents = torch.where(none, torch.arange(W, device=x.device), at // tok.shape[-1])
    done = none | finished.gather(1, parents) | (tokens == eos)
    return tokens.to(torch.int32), parents.to(torch.int32), val.float(), done


def _plain_reorder(states, parents):
    G, W = parents.shape
    src = (parents.long() + W * torch.arange(G, device=parents.device).unsqueeze(-1)).flatten()
    for t in states:
        t.copy_(t[src])


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        if T * N * K > 1 << 39:
            return None
        y = torch.zeros(T, N, dtype=torch.float64, device=DEV)
        for j in range(-(-K // BLOCK)):  # block by block: codes are exact, each pair of scales stands apart
            a, b = j * BLOCK, min(K, (j + 1) * BLOCK)
            xj = s["x"][:, a:b].float()
            sx = xj.abs().amax(1) / 448.0
            sx[sx == 0] = 1.0
            xq = (xj / sx[:, None]).clamp(-448.0, 448.0).to(F8).double()
            sw = s["scales"][:, j].double().repeat_interleave(BLOCK)[:N]
            y += (xq @ s["codes"][:, a:b].double().t()) * sx.double()[:, None] * sw
        return y
    if c["op"] in ("step", "prefill"):
        tokens = s["q"].shape[0]
        n = [c["n"]] * c["B"] if c["op"] == "step" else s["lengths"]
        if max(n) > 16384:
            return None
        r = c["Hv"] // c["Hk"]
        norm = lambda t: t.double() / (t.double().square().sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
        q = norm(s["q"]).repeat_interleave(r, 1) / math.sqrt(c["dk"])
        k = norm(s["k"]).repeat_interleave(r, 1)
        v, beta = s["v"].double(), s["beta"].double()
        a = s["g"].double().exp()
        a = a if c["decay"] == "channel" else a.unsqueeze(-1)
        out = torch.empty(tokens, c["Hv"], c["dv"], dtype=torch.float64, device=DEV)
        first = torch.tensor([sum(n[:i]) for i in range(len(n))], device=DEV)
        order = sorted(range(len(n)), key=lambda i: -n[i])  # longest first: the live ones are a leading part
        first, slots = first[order], s["slots"].long()[order]
        lengths = [n[i] for i in order]
        S = s["state"][slots].double()
        for t in range(lengths[0]):
            m = sum(1 for x in lengths if x > t)
            at = first[:m] + t
            X = S[:m] * a[at].unsqueeze(-1)
            e = beta[at].unsqueeze(-1) * (v[at] - torch.einsum("bhkv,bhk->bhv", X, k[at]))
            S[:m] = X + torch.einsum("bhk,bhv->bhkv", k[at], e)
            out[at] = torch.einsum("bhkv,bhk->bhv", S[:m], q[at])
        state = s["state"].double()
        state[slots] = S
        if c["op"] == "step":
            out = out.view(c["B"], c["n"], c["Hv"], c["dv"])
        return dict(out=out, state=state)
    if c["op"] == "select":
        G, W, V = c["G"], c["W"], c["V"]
        y = torch.log_softmax(s["logits"].double(), -1) + s["scores"].double().unsqueeze(-1)
        y[s["finished"]] = -math.inf
        f = s["finished"].nonzero()
        y[f[:, 0], f[:, 1], s["eos"]] = s["scores"].double()[f[:, 0], f[:, 1]]
        best = torch.stack([torch.sort(y[i].flatten(), descending=True)[0][:W] for i in range(G)])
        if best.shape[1] < W:
            best = torch.nn.functional.pad(best, (0, W - best.shape[1]), value=-math.inf)
        return dict(tokens=None, parents=None, scores=best, finished=None)
    G, W = s["parents"].shape
    got = []
    for t in s["states"]:
        t = t.view(G, W, -1).double()
        got.append(torch.stack([t[i][s["parents"][i].long()] for i in range(G)]).view(G * W, -1))
    return dict(enumerate(got))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        return dict(bytes=N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK) + 2 * T * K + (2 if c["out"] == "bf16" else 4) * T * N,
                    flops=2 * T * N * K)
    if c["op"] in ("step", "prefill"):
        seqs, tokens = (c["B"], c["B"] * c["n"]) if c["op"] == "step" else (c["S"], c["T"])
        state = c["Hv"] * c["dk"] * c["dv"]
        token = 4 * c["Hk"] * c["dk"] + 4 * c["Hv"] * c["dv"] + 4 * c["Hv"] * (1 + (c["dk"] if c["decay"] == "channel" else 1))
        return dict(bytes=8 * seqs * state + tokens * token, flops=7 * tokens * state)
    if c["op"] == "select":
        rows = c["G"] * (1 if c["first"] else c["W"] - c["finished"])
        return dict(bytes=rows * c["V"] * (4 if c["dtype"] == "fp32" else 2) + 18 * c["G"] * c["W"], flops=3 * rows * c["V"])
    reads = c["moved"] if c["cycle"] else min(c["moved"], c["W"] - c["moved"])
    return dict(bytes=c["G"] * ((reads + c["moved"]) * (c["row"] + c["small"]) + 4 * c["W"]), flops=0)
