"""Cases of the decayed linear attention (prompts and single tokens) and of the norms around a block.

``listed()`` and ``draw()`` name the cases, ``prepare()`` makes the tensors that a program holds
before the call, ``run()`` makes one call (the framework's entry points where ``own`` is true,
elementary torch operations in 32 bits otherwise), ``exact()`` is the definition in 64 bits and
``work()`` the bytes and operations that a call cannot do without.

Decayed linear attention, per sequence and value head (key head = value head // (hv / hk)), with
l = exp(log_decay) and a 128 x 128 fp32 state H:
    H_t = l H_{t-1} + k_t v_t^T,   o_t = scale * H_t^T q_t
Norms around a block, per row: u = x / rms(x) * w_post (or x), r = residual + alpha * gate * u,
y = r / rms(r) * w_pre.
"""
import math

import torch

own = False

D = 128          # head dimension
C = 128          # tokens of a chunk in the plain form
EPS = 1e-6


def listed():
    return [
        # one prompt of the layer's standard length and heads, a new request: zero state in, state out
        {"name": "prompt 4096", "op": "prefill", "lengths": "4096", "hk": 16, "hv": 48, "pool": 0, "start": False,
         "decay": "slopes"},
        # a long document
        {"name": "prompt 32768", "op": "prefill", "lengths": "32768", "hk": 16, "hv": 48, "pool": 0, "start": False,
         "decay": "slopes"},
        # prompts of several requests continued from their entries of the pool, ragged, one of a single token
        {"name": "prompts ragged pool", "op": "prefill", "lengths": "1711,4099,640,2953,1,7777,321,3000", "hk": 16,
         "hv": 48, "pool": 16, "start": True, "decay": "slopes"},
        # a short chat turn, where latency counts
        {"name": "prompt 37", "op": "prefill", "lengths": "37", "hk": 16, "hv": 48, "pool": 4, "start": True,
         "decay": "slopes"},
        # a batch of middling prompts on one of two head shards, with initial states
        {"name": "prompts shard", "op": "prefill",
         "lengths": "512,511,300,777,64,129,900,1025,450,333,610,256,711,95,402,150", "hk": 8, "hv": 24, "pool": 0,
         "start": True, "decay": "slopes"},
        # one decode step of a serving batch on a pool of cached states, two padding rows
        {"name": "tokens 64 pool", "op": "decode", "batch": 64, "hk": 16, "hv": 48, "pool": 128, "pad": 2,
         "decay": "slopes"},
        # a single request
        {"name": "tokens 1", "op": "decode", "batch": 1, "hk": 16, "hv": 48, "pool": 0, "pad": 0, "decay": "slopes"},
        # a large batch on one of two head shards, dense states
        {"name": "tokens 256 shard", "op": "decode", "batch": 256, "hk": 8, "hv": 24, "pool": 0, "pad": 0,
         "decay": "slopes"},
        # one token between two blocks
        {"name": "norm 1 row", "op": "norm", "rows": 1, "d": 5120, "wide": False, "post": False, "gate": "none"},
        # a decode batch: norm after the block, a channel gate, the residual stream kept in 32 bits
        {"name": "norm 64 rows", "op": "norm", "rows": 64, "d": 5120, "wide": True, "post": True, "gate": "channel"},
        # a prompt between two blocks: the ordinary residual + norm
        {"name": "norm 4096 rows", "op": "norm", "rows": 4096, "d": 5120, "wide": False, "post": False,
         "gate": "none"},
        # packed prompts with everything: both norms and a gate for each token, odd rows, another width
        {"name": "norm 9973 rows", "op": "norm", "rows": 9973, "d": 6144, "wide": False, "post": True, "gate": "row"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "norm"])
    if op == "norm":
        d = 8 * _log_int(rng, 16, 1024)
        rows = _log_int(rng, 1, 16384)
        return {"op": op, "rows": max(1, min(rows, 60_000_000 // d)), "d": d, "wide": rng.random() < 0.4,
                "post": rng.random() < 0.5, "gate": rng.choice(["none", "channel", "row"])}
    hk, hv = rng.choice([(16, 48), (8, 24), (4, 12), (16, 16), (8, 32), (1, 8), (5, 10), (2, 2)])
    decay = rng.choice(["slopes", "slopes", "none", "fast"])
    if op == "decode":
        batch = _log_int(rng, 1, 256)
        pool = rng.choice([0, batch + rng.randrange(1, 65)])
        return {"op": op, "batch": batch, "hk": hk, "hv": hv, "pool": pool,
                "pad": rng.randrange(0, batch // 8 + 1) if pool else 0, "decay": decay}
    n = rng.choice([1, 1, 2, 3, 5, 8, 13])
    total = max(n, _log_int(rng, 16, 24576))
    cuts = sorted(rng.randrange(0, total + 1) for _ in range(n - 1))
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    return {"op": op, "lengths": ",".join(str(x) for x in lengths), "hk": hk, "hv": hv,
            "pool": rng.choice([0, n + rng.randrange(0, 5)]), "start": rng.random() < 0.6, "decay": decay}


def _log_decay(kind, hv, dev):
    h = torch.arange(hv, dtype=torch.float64)
    if kind == "none":                  # plain linear attention: nothing is forgotten
        g = torch.zeros(hv, dtype=torch.float64)
    elif kind == "fast":                # a memory of a few tokens, down to less than one
        g = -0.25 * 2.0 ** (h % 6)
    else:                               # the usual geometric slopes, one half down to 2^-8
        g = -(2.0 ** (-8.0 * (h + 1) / hv))
    return g.to(torch.float32).to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        x = torch.empty(shape, dtype=torch.float32, device=dev)
        return (x.normal_(generator=gen) * std).to(dtype)

    s = dict(case)
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        s["x"] = normal(rows, d)
        s["residual"] = normal(rows, d, dtype=torch.float32 if case["wide"] else torch.bfloat16, std=3.0)
        s["gate"] = {"none": lambda: None, "channel": lambda: normal(d, std=0.5),
                     "row": lambda: normal(rows, d, std=0.5)}[case["gate"]]()
        s["w_post"] = 1.0 + normal(d, dtype=torch.float32, std=0.2) if case["post"] else None
        s["w_pre"] = 1.0 + normal(d, dtype=torch.float32, std=0.2)
        s["alpha"] = 0.70710678
        return s
    hk, hv = case["hk"], case["hv"]
    s["log_decay"] = _log_decay(case["decay"], hv, dev)
    s["scale"] = D ** -0.5
    lengths = [1] * case["batch"] if case["op"] == "decode" else [int(x) for x in case["lengths"].split(",")]
    n, total = len(lengths), sum(lengths)
    # q, k, v are views of the packed rows [q | k | v] that the projection writes
    packed = normal(total, (2 * hk + hv) * D)
    s["q"] = packed[:, : hk * D].view(total, hk, D)
    s["k"] = packed[:, hk * D: 2 * hk * D].view(total, hk, D)
    s["v"] = packed[:, 2 * hk * D:].view(total, hv, D)
    if case["pool"]:
        slot = torch.randperm(case["pool"], generator=gen, device=dev)[:n].to(torch.int32)
        if case["op"] == "decode" and case["pad"]:
            slot[-case["pad"]:] = -1
        s["slot"] = slot
        s["state"] = normal(case["pool"], hv, D, D, dtype=torch.float32)
    elif case["op"] == "decode" or case["start"]:
        s["state"] = normal(n, hv, D, D, dtype=torch.float32)
    if case["op"] == "prefill":
        cu = [0]
        for x in lengths:
            cu.append(cu[-1] + x)
        s["cu_host"] = torch.tensor(cu, dtype=torch.int32).numpy()
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["chunks"] = _chunk_table(lengths, dev)
    return s


def _chunk_table(lengths, dev):
    """Chunks of C tokens that restart with every sequence, laid out sequence by sequence: each chunk's
    sequence, its number in it and its length, and each sequence's first and last chunk."""
    seq = [i for i, x in enumerate(lengths) for _ in range(-(-x // C))]
    within = [j for x in lengths for j in range(-(-x // C))]
    count = [min(C, lengths[i] - j * C) for i, j in zip(seq, within)]
    nonempty = [i for i, x in enumerate(lengths) if x > 0]
    last = [len(seq) - 1 - seq[::-1].index(i) for i in nonempty]
    start = [sum(lengths[:i]) for i in range(len(lengths))]
    token = [[start[i] + min(j * C + r, lengths[i] - 1) for r in range(C)] for i, j in zip(seq, within)]
    row = [c * C + r for c, m in enumerate(count) for r in range(m)]
    table = {"seq": seq, "within": within, "count": count, "nonempty": nonempty, "last": last, "token": token,
             "row": row, "new": [c for c, j in enumerate(within) if j == 0]}
    return {k: torch.tensor(x, dtype=torch.int64, device=dev) for k, x in table.items()}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import gated_delta_rule_63_b200 as G
    if s["op"] == "norm":
        r, y = G.block_norm(s["x"], residual=s["residual"], gate=s["gate"], post_norm=s["post"], w_post=s["w_post"],
                            w_pre=s["w_pre"], alpha=s["alpha"], eps=EPS)
        return {"residual": r, "y": y}
    if s["op"] == "decode":
        if s["pool"]:
            o = G.decay_attn_decode_slots(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["slot"],
                                          scale=s["scale"])
        else:
            o = G.decay_attn_decode(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if s["pool"]:
        o = G.decay_attn_prefill_slots(s["q"], s["k"], s["v"], s["log_decay"], s["cu"], s["cu_host"], s["state"],
                                       s["slot"], init_from_pool=s["start"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    hT = torch.empty((len(s["cu_host"]) - 1, s["hv"], D, D), dtype=torch.float32, device=s["q"].device)
    o = G.decay_attn_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["cu"], s["cu_host"],
                             h0=s["state"] if s["start"] else None, hT=hT, scale=s["scale"])
    return {"o": o, "state": hT}


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _heads(x, hv):
    """[T, hk, D] -> fp32 [T, hv, D]: value head h reads key head h // (hv / hk)."""
    return x.float().repeat_interleave(hv // x.shape[1], dim=1)


def _plain_norm(s):
    u = s["x"].float()
    if s["post"]:
        u = u / (u.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w_post"]
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = s["residual"].float() + s["alpha"] * u
    y = r / (r.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w_pre"]
    return {"residual": r.to(s["residual"].dtype), "y": y.to(torch.bfloat16)}


def _plain_decode(s):
    hv, state = s["hv"], s["state"]
    live = torch.arange(s["batch"] - s["pad"], device=state.device)   # the padding rows are the last ones
    entry = s["slot"][: s["batch"] - s["pad"]].long() if s["pool"] else live
    q, k, v = _heads(s["q"], hv)[live], _heads(s["k"], hv)[live], s["v"].float()[live]
    H = state[entry] * s["log_decay"].exp()[:, None, None] + k[..., :, None] * v[..., None, :]
    state[entry] = H
    o = torch.zeros((s["batch"], hv, D), dtype=torch.bfloat16, device=state.device)
    o[live] = (s["scale"] * (q[..., :, None] * H).sum(-2)).to(torch.bfloat16)
    return {"o": o, "state": state}


def _plain_prefill(s):
    """Chunks of 128 tokens, padded with zero rows: products inside a chunk, and every chunk's
    starting state as the decayed sum of the chunks before it in its sequence."""
    dev, hv, g, tab = s["q"].device, s["hv"], s["log_decay"], s["chunks"]
    n, nc, seq, count = s["cu"].shape[0] - 1, tab["seq"].shape[0], tab["seq"], tab["count"]
    i, c = torch.arange(C, device=dev), torch.arange(nc, device=dev)
    there = i < count[:, None]                                        # [nc, C]

    def tiles(x):                                                     # -> [hv, nc, C, D], zero behind the end
        return (x[tab["token"]] * there[..., None, None]).permute(2, 0, 1, 3)

    q, k, v = tiles(_heads(s["q"], hv)), tiles(_heads(s["k"], hv)), tiles(s["v"].float())
    ahead = (i[:, None] - i).clamp(min=0)
    inside = (g[:, None, None] * ahead).exp() * (i[:, None] >= i)     # [hv, C, C]
    P = (q @ k.transpose(-1, -2)) * inside[:, None]
    left = (count[:, None] - 1 - i).clamp(min=0)                      # [nc, C] steps to the chunk's end
    K = k * (g[:, None, None] * left).exp()[..., None]
    add = (K.transpose(-1, -2) @ v).reshape(hv, nc, D * D)
    # the state after chunk c: what every chunk up to it in its sequence adds, decayed from its end to c's
    ends = torch.cumsum(count, 0)
    apart = (ends[:, None] - ends).clamp(min=0)
    same = (seq[:, None] == seq) & (c[:, None] >= c)
    after = ((g[:, None, None] * apart).exp() * same) @ add           # [hv, nc, D * D]
    entry = s["slot"].long() if s["pool"] else torch.arange(n, device=dev)
    if s["start"]:
        h0 = s["state"][entry].permute(1, 0, 2, 3).reshape(hv, n, D * D)
        after = after + (g[:, None] * (tab["within"] * C + count)).exp()[..., None] * h0[:, seq]
    else:
        h0 = torch.zeros((hv, n, D * D), device=dev)
    begin = after.roll(1, 1)                                          # the state before chunk c
    begin[:, tab["new"]] = h0[:, tab["nonempty"]]
    o = P @ v + (g[:, None] * (i + 1)).exp()[:, None, :, None] * (q @ begin.view(hv, nc, D, D))
    o = (s["scale"] * o).permute(1, 2, 0, 3).reshape(nc * C, hv, D)[tab["row"]].to(torch.bfloat16)
    final = h0.clone()
    final[:, tab["nonempty"]] = after[:, tab["last"]]
    final = final.view(hv, n, D, D).permute(1, 0, 2, 3)
    if s["pool"]:
        s["state"][entry] = final
        return {"o": o, "state": s["state"]}
    return {"o": o, "state": final.contiguous()}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "decode": _plain_decode, "prefill": _plain_prefill}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definition in 64 bits, token by token
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        f = torch.float64
        x = s["x"].to(f)
        rms = torch.sqrt(torch.sum(x * x, 1, keepdim=True) / case["d"] + EPS)
        u = x * s["w_post"].to(f) / rms if case["post"] else x
        gate = 1.0 if s["gate"] is None else s["gate"].to(f)
        r = s["residual"].to(f) + s["alpha"] * gate * u
        return {"residual": r, "y": r * s["w_pre"].to(f) / torch.sqrt(torch.sum(r * r, 1, keepdim=True) / case["d"]
                                                                     + EPS)}
    f, hv, group = torch.float64, case["hv"], case["hv"] // case["hk"]
    dev = s["q"].device
    cu = s["cu_host"].tolist() if case["op"] == "prefill" else list(range(case["batch"] + 1))
    n, total = len(cu) - 1, cu[-1]
    lam = torch.exp(s["log_decay"].to(f)).view(hv, 1, 1)
    entry = s["slot"].tolist() if case["pool"] else list(range(n))
    begins = case["op"] == "decode" or case["start"]
    H = torch.zeros((n, hv, D, D), dtype=f, device=dev)
    for i, e in enumerate(entry):
        if begins and e >= 0:
            H[i] = s["state"][e].to(f)
    o = torch.zeros((total, hv, D), dtype=f, device=dev)
    # the sequences that still have a token at step t take it together, longest first
    order = sorted(range(n), key=lambda i: cu[i] - cu[i + 1])
    H = H[order]
    starts = torch.tensor([cu[i] for i in order], device=dev)
    lens = [cu[i + 1] - cu[i] for i in order]
    live = n
    for t in range(max(lens)):
        while live and lens[live - 1] <= t:
            live -= 1
        at = starts[:live] + t
        q, k = (s[x][at].to(f).repeat_interleave(group, 1) for x in "qk")
        H[:live] *= lam
        H[:live] += k.unsqueeze(-1) * s["v"][at].to(f).unsqueeze(-2)
        o[at] = s["scale"] * torch.matmul(q.unsqueeze(-2), H[:live]).squeeze(-2)
    back = [order.index(i) for i in range(n)]
    H = H[back]
    if not case["pool"]:
        return {"o": o, "state": H}
    pool = s["state"].to(f)
    for i, e in enumerate(entry):
        if e >= 0:
            pool[e] = H[i]
        else:
            o[cu[i]:cu[i + 1]] = 0.0
    return {"o": o, "state": pool}


def work(case):
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        row = d * (2 + 2 * (4 if case["wide"] else 2) + 2 + (2 if case["gate"] == "row" else 0))
        vectors = d * (4 + (4 if case["post"] else 0) + (2 if case["gate"] == "channel" else 0))
        return {"bytes": rows * row + vectors, "flops": rows * d * (6 + (4 if case["post"] else 0))}
    hk, hv = case["hk"], case["hv"]
    one = hv * D * D * 4                                   # a sequence's state, one way
    if case["op"] == "decode":
        total, n = case["batch"] - case["pad"], case["batch"] - case["pad"]
        ways = 2
    else:
        lengths = [int(x) for x in case["lengths"].split(",")]
        total, n = sum(lengths), len(lengths)
        ways = 2 if case["start"] else 1
    return {"bytes": total * (2 * hk + 2 * hv) * D * 2 + ways * n * one + 4 * hv, "flops": 4 * D * D * hv * total}
