"""The steps of a decode layer around its matvecs: cases, plain forms and exact values.

Four operators that touch a matvec's fp32 input or output:

  lora      low-rank adapters of many requests beside shared projections
            (qmv.lora), added to the projections' outputs;
  heads     norms of the query and key heads and their rotation by one to
            three positions (qmv.head_norm_rope), before keys go to a cache;
  gate      routing to experts by softmax or sigmoid scores, a bias, groups and
            renormalised weights (qmv.router_gate), before the routed matvecs;
  logprobs  log probabilities of given tokens, entropy and the likeliest
            alternatives of the output head's logits (qmv.token_logprobs).

`run` computes them with elementary torch operations, or, where `own` is
true, with this package's entry points.
"""
import math

import torch

own = False

EPS = 1e-6  # the norms' epsilon
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def _lora(name, tokens, k, outs, rank, adapters, pattern, dtype):
    return {"name": name, "op": "lora", "tokens": tokens, "k": k, "outs": outs, "rank": rank, "adapters": adapters,
            "pattern": pattern, "dtype": dtype}


def _heads(name, tokens, heads, kv_heads, dim, rot, axes=1, interleaved=False, norm=True):
    return {"name": name, "op": "heads", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "axes": axes, "interleaved": interleaved, "norm": norm}


def _gate(name, tokens, k, experts, top_k, scoring, groups=1, top_groups=1, bias=False, renorm=True, scale=1.0):
    return {"name": name, "op": "gate", "tokens": tokens, "k": k, "experts": experts, "top_k": top_k,
            "scoring": scoring, "groups": groups, "top_groups": top_groups, "bias": bias, "renorm": renorm,
            "scale": scale}


def _logprobs(name, tokens, vocab, given, top, scale=1.0, masked=False):
    return {"name": name, "op": "logprobs", "tokens": tokens, "vocab": vocab, "given": given, "top": top,
            "scale": scale, "masked": masked}


def listed():
    return [
        # one request with an adapter on its q/k/v projections: latency alone
        _lora("lora 1 q/k/v rank 16", 1, 4096, "4096 1024 1024", 16, 8, "each", "f16"),
        # 16 requests, an adapter each, ranks from 5 to 64, on the gate and up projections: the adapters' bytes
        _lora("lora 16 gate/up rank 64", 16, 4096, "14336 14336", 64, 32, "each", "bf16"),
        # a batch that shares three adapters, a quarter of it without one, on the long down projection
        _lora("lora 64 down rank 32", 64, 14336, "4096", 32, 3, "mixed", "bf16"),
        # prompts of three requests, one after the other, behind a projection of the head's width
        _lora("lora 700 runs rank 16", 700, 5120, "5120", 16, 3, "runs", "f32"),
        # one decode token: latency alone
        _heads("heads 1x40", 1, 32, 8, 128, 128),
        # a verify batch of small heads, a part of each rotated in neighbouring pairs, no norm
        _heads("heads 16x36 of 80 dims", 16, 32, 4, 80, 32, interleaved=True, norm=False),
        # a prompt's chunk with images: time, height and width as positions
        _heads("heads 2000x32 three axes", 2000, 28, 4, 128, 128, axes=3),
        # many tokens: memory traffic alone
        _heads("heads 8192x72", 8192, 64, 8, 128, 128),
        # one token's routing, 128 experts: latency alone
        _gate("gate 1x128", 1, 4096, 128, 8, "softmax"),
        # the largest routed batch, sigmoid scores with a balance bias, half of eight groups
        _gate("gate 64x256 groups", 64, 5120, 256, 8, "sigmoid", 8, 4, bias=True, scale=2.5),
        # the verify batch of a draft behind the output head: the drafts' probabilities and 20 alternatives
        _logprobs("logprobs 6x152064 top 20", 6, 152064, 1, 20),
        # a prompt's log probabilities, an odd vocabulary: memory traffic
        _logprobs("logprobs 1000x50257 top 5", 1000, 50257, 1, 5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("lora", "heads", "gate", "logprobs"))
    if op == "lora":
        tokens = rng.choice((1, _log(rng, 1, 64), _log(rng, 1, 700)))
        # tokens x ranks x (inputs + outputs) of the largest case at most, and its adapters' bytes
        items, adapters = rng.randint(1, 3), _log(rng, 1, 32)
        most = int(min(9.5e7 / tokens, 1.5e7 / min(adapters, tokens)) / 8)
        k = 32 * _log(rng, 4, max(4, min(448, most // (64 * items))))
        width = max(1, min(14336, (most - items * k) // items))
        outs = " ".join(str(_log(rng, min(64, width), width)) for _ in range(items))
        wide = items * k + sum(int(n) for n in outs.split())
        rank = 8 * _log(rng, 1, max(1, min(8, most // wide)))
        return {"op": op, "tokens": tokens, "k": k, "outs": outs, "rank": rank, "adapters": adapters,
                "pattern": rng.choice(("each", "mixed", "runs") if tokens <= 64 else ("runs",)),
                "dtype": rng.choice(("f16", "bf16", "bf16", "f32"))}
    if op == "heads":
        dim = rng.choice((32, 64, 80, 96, 128, 128, 192, 256))
        heads, kv = rng.choice(((1, 1), (8, 1), (12, 12), (28, 4), (32, 8), (40, 8), (64, 8), (16, 0)))
        tokens = min(_log(rng, 1, 16000), (8192 * 72 * 128) // ((heads + kv) * dim))
        return {"op": op, "tokens": tokens, "heads": heads, "kv_heads": kv, "dim": dim,
                "rot": rng.choice((dim, dim, dim // 2, 16, dim // 4 * 2)), "axes": rng.choice((1, 1, 2, 3)),
                "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.7}
    if op == "gate":
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * rng.choice((8, 16, 20, 32, 48)) if groups > 1 else rng.choice((8, 60, 64, 128, 160, 256))
        top_groups = rng.randint(1, groups)
        return {"op": op, "tokens": rng.choice((1, 2, _log(rng, 1, 64), rng.randint(17, 64))),
                "k": min(4 * _log(rng, 64, 1280), 4 * (327680 // experts)), "experts": experts,
                "top_k": rng.choice((1, 2, 6, 8)), "scoring": rng.choice(("softmax", "sigmoid")), "groups": groups,
                "top_groups": top_groups, "bias": rng.random() < 0.5, "renorm": rng.random() < 0.7,
                "scale": rng.choice((1.0, 1.0, 2.5))}
    vocab = rng.choice((32000, 32003, 50257, 128256, 152064, _log(rng, 100, 160000)))
    return {"op": op, "tokens": rng.choice((1, rng.randint(1, 16), min(_log(rng, 1, 4000), 1000 * 50257 // vocab))),
            "vocab": vocab, "given": rng.choice((1, 1, 4)), "top": rng.choice((0, 1, 5, 20)),
            "scale": rng.choice((1.0, 1.0, 1.25)), "masked": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _outs(case):
    return [int(n) for n in case["outs"].split()]


def _ranks(case):
    """Rank of each adapter: the pool's largest, and smaller and odd ones among them."""
    top = case["rank"]
    return [max(1, r) for i in range(case["adapters"]) for r in ((top, top // 2, top, top // 3, top - 3)[i % 5],)]


def _adapters(case):
    """The adapter of each token (-1: none): part of the case, as its bytes go by it."""
    t, e = case["tokens"], case["adapters"]
    if case["pattern"] == "each":
        return [(5 * i + 1) % e for i in range(t)]
    if case["pattern"] == "mixed":
        return [-1 if i % 4 == 3 else (7 * i) % e for i in range(t)]
    return [i * e // t for i in range(t)]


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = case["tokens"]
    s = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "lora":
        k, e, rank, outs, kind = case["k"], case["adapters"], case["rank"], _outs(case), TYPES[case["dtype"]]
        s["x"] = normal(t, k)
        s["a"] = [(normal(e, rank, k) / math.sqrt(k)).to(kind) for _ in outs]
        s["b"] = [(normal(e, n, rank) * 0.1).to(kind) for n in outs]
        # the projections' outputs, as their columns lie beside each other
        whole = normal(t, sum(outs))
        s["base"] = list(whole.split(outs, 1))
        s["ids"] = torch.tensor(_adapters(case), dtype=torch.int32, device=dev)
        s["ranks"] = torch.tensor(_ranks(case), dtype=torch.int32, device=dev)
        s["scales"] = 0.5 + 1.5 * torch.rand(e, generator=g, device=dev)
    elif case["op"] == "heads":
        h, kv, dim, rot = case["heads"], case["kv_heads"], case["dim"], case["rot"]
        # columns of a q/k/v projection's output
        qkv = normal(t, (h + 2 * kv) * dim) * 1.3
        s["q"] = qkv[:, :h * dim].unflatten(1, (h, dim))
        s["k"] = qkv[:, h * dim:(h + kv) * dim].unflatten(1, (kv, dim)) if kv else None
        s["qw"] = 1.0 + 0.2 * normal(dim) if case["norm"] else None
        s["kw"] = 1.0 + 0.2 * normal(dim) if case["norm"] and kv else None
        i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
        s["freq"] = (1e6 ** (-2.0 * i / rot)).float()
        # tokens anywhere in a long context
        s["pos"] = torch.randint(0, 131072, (case["axes"], t), generator=g, device=dev, dtype=torch.int32)
        # the axes' sections of the pairs, as wide as each other
        s["axis"] = (torch.arange(rot // 2, device=dev) * case["axes"] // max(1, rot // 2)).int()
    elif case["op"] == "gate":
        s["x"] = normal(t, case["k"])
        s["w"] = normal(case["experts"], case["k"]) / math.sqrt(case["k"])
        s["bias"] = 0.1 * normal(case["experts"]) if case["bias"] else None
    else:
        v = case["vocab"]
        x = normal(t, v) * 3.0
        x[torch.arange(t, device=dev), torch.randint(0, v, (t,), generator=g, device=dev)] += 12.0
        if case["masked"]:  # tokens that a grammar forbids
            x.masked_fill_(torch.rand(t, v, generator=g, device=dev) < 0.3, -math.inf)
        s["x"] = x
        # a likely token first, as a draft proposes it, then any
        s["given"] = torch.randint(0, v, (t, case["given"]), generator=g, device=dev, dtype=torch.int32)
        s["given"][:, 0] = x.argmax(1).int()
    return s


# --------------------------------------------------------------- plain forms
def _lora_plain(s):
    case = s["case"]
    e, rank = case["adapters"], case["rank"]
    ids = s["ids"].long()
    if case["tokens"] < e:  # fewer tokens than adapters: each token's own one
        at = ids.clamp(min=0)
        mine = (ids[:, None] >= 0) & (torch.arange(rank, device=ids.device) < s["ranks"][at][:, None])
        by = torch.where(mine, s["scales"][at][:, None], torch.zeros_like(s["scales"][:1]))[..., None]
        return [base + torch.bmm(b[at].float(), torch.bmm(a[at].float(), s["x"][..., None]) * by)[..., 0]
                for a, b, base in zip(s["a"], s["b"], s["base"])]
    # every adapter's rows for every token, then the token's own ones
    mine = (ids[:, None] == torch.arange(e, device=ids.device))[:, :, None]
    mine = mine & (torch.arange(rank, device=ids.device) < s["ranks"][:, None])
    by = torch.where(mine, s["scales"][:, None].expand(e, rank), torch.zeros_like(s["scales"][:, None]))
    by = by.reshape(-1, e * rank)
    return [base + torch.matmul(torch.matmul(s["x"], a.float().view(e * rank, -1).t()) * by,
                                b.float().transpose(1, 2).reshape(e * rank, -1))
            for a, b, base in zip(s["a"], s["b"], s["base"])]


def _kept(s, name, make):
    """What a program keeps beside its inputs: outputs and workspaces."""
    if name not in s:
        s[name] = make()
    return s[name]


def _lora_own(s):
    import quantized_decode_gemv_qmv_amd as qmv

    case, x = s["case"], s["x"]
    outs = _kept(s, "out", lambda: [torch.empty_like(b) for b in s["base"]])
    ws = _kept(s, "ws", lambda: torch.empty(qmv.lora_workspace_bytes(len(outs), case["rank"], x.shape[0]),
                                            dtype=torch.uint8, device=x.device))
    return qmv.lora(x, s["ids"], list(zip(s["a"], s["b"], s["base"], outs)), ranks=s["ranks"], scales=s["scales"],
                    ws=ws)


def _heads_one(x, w, cos, sin, case):
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    rot = case["rot"]
    part = x[..., :rot]
    if case["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _heads_plain(s):
    case = s["case"]
    # angles in 64 bits: 32 lose the place in the circle of far positions
    angle = s["pos"].double()[s["axis"].long()].t() * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return {"q": _heads_one(s["q"], s["qw"], cos, sin, case),
            "k": None if s["k"] is None else _heads_one(s["k"], s["kw"], cos, sin, case)}


def _heads_own(s):
    import quantized_decode_gemv_qmv_amd as qmv

    q, k = s["q"], s["k"]
    qo = _kept(s, "qo", lambda: torch.empty(q.shape, device=q.device))
    ko = None if k is None else _kept(s, "ko", lambda: torch.empty(k.shape, device=q.device))
    q, k = qmv.head_norm_rope(q, k, s["pos"], s["freq"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                              pair_axis=s["axis"], interleaved=s["case"]["interleaved"], q_out=qo, k_out=ko)
    return {"q": q, "k": k}


def _gate_plain(s):
    case = s["case"]
    t, e, groups, k = case["tokens"], case["experts"], case["groups"], case["top_k"]
    # in 64 bits: which expert is chosen is decided at a border
    logits = torch.matmul(s["x"].double(), s["w"].double().t())
    if case["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if groups > 1:
        # a group counts by the sum of its two largest
        best = torch.sort(choice.view(t, groups, -1), dim=2, descending=True).values[:, :, :2].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        kept = torch.zeros(t, groups, dtype=torch.bool, device=choice.device).scatter_(1, order, True)
        choice = choice.view(t, groups, -1).masked_fill(~kept[:, :, None], -math.inf).view(t, e)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    weights = torch.gather(score, 1, ids)
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    return {"ids": ids.int(), "weights": (weights * case["scale"]).float()}


def _gate_own(s):
    import quantized_decode_gemv_qmv_amd as qmv

    case, x = s["case"], s["x"]
    ws = _kept(s, "ws", lambda: torch.zeros(qmv.router_gate_workspace_bytes(x.shape[0], case["experts"]),
                                            dtype=torch.uint8, device=x.device))
    ids, weights = qmv.router_gate(x, s["w"], case["top_k"], scoring=case["scoring"], bias=s["bias"],
                                   n_groups=case["groups"], top_groups=case["top_groups"], renorm=case["renorm"],
                                   scale=case["scale"], ws=ws)
    return {"ids": ids, "weights": weights}


def _logprobs_plain(s):
    case, x = s["case"], s["x"]
    z = x * case["scale"]
    top = z.amax(1, keepdim=True)
    d = z - top
    p = torch.exp(d)
    total = p.sum(1, keepdim=True)
    log = torch.log(total)
    # a forbidden token has no share in the entropy
    entropy = log - (p * torch.where(p > 0, d, torch.zeros_like(d))).sum(1, keepdim=True) / total
    out = {"logprobs": torch.gather(d, 1, s["given"].long()) - log, "entropy": entropy[:, 0]}
    if case["top"]:
        # whole numbers in the order of the logits, the lower index first among equal ones
        bits = x.view(torch.int32).long()
        key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * (1 << 32)
        key = key + torch.arange(x.shape[1] - 1, -1, -1, device=x.device)
        ids = x.shape[1] - 1 - (torch.topk(key, case["top"], dim=1).values & 0xFFFFFFFF)
        out["ids"], out["top"] = ids.int(), torch.gather(d, 1, ids) - log
    return out


def _logprobs_own(s):
    import quantized_decode_gemv_qmv_amd as qmv

    case, x = s["case"], s["x"]
    t, v = x.shape
    ws = _kept(s, "ws", lambda: torch.zeros(qmv.token_logprobs_workspace_bytes(t, v, case["top"]), dtype=torch.uint8,
                                            device=x.device))
    given, entropy, ids, top = qmv.token_logprobs(x, s["given"], top_n=case["top"], scale=case["scale"], ws=ws)
    out = {"logprobs": given, "entropy": entropy}
    if case["top"]:
        out["ids"], out["top"] = ids, top
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"lora": _lora_own, "heads": _heads_own, "gate": _gate_own, "logprobs": _logprobs_own}[op](state)
    return {"lora": _lora_plain, "heads": _heads_plain, "gate": _gate_plain, "logprobs": _logprobs_plain}[op](state)


# -------------------------------------------------------------------- work
def work(case):
    t = case["tokens"]
    if case["op"] == "lora":
        k, outs, ranks, ids = case["k"], _outs(case), _ranks(case), _adapters(case)
        size = 4 if case["dtype"] == "f32" else 2
        used = sum(ranks[i] for i in set(ids) if i >= 0)
        rows = sum(ranks[i] for i in ids if i >= 0)
        wide = len(outs) * k + sum(outs)
        return {"bytes": used * wide * size + 4 * t * k + 8 * t * sum(outs), "flops": 2 * rows * wide}
    if case["op"] == "heads":
        n = t * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 8 * n + 4 * t * case["axes"], "flops": n * (4 if case["norm"] else 0) + 3 * n * case["rot"] // case["dim"]}
    if case["op"] == "gate":
        return {"bytes": 4 * case["k"] * (t + case["experts"]) + 8 * t * case["top_k"],
                "flops": 2 * t * case["k"] * case["experts"]}
    n = t * case["vocab"]
    return {"bytes": 4 * n + t * (8 * case["given"] + 8 * case["top"] + 4), "flops": 6 * n}


# ----------------------------------------------------------- exact values
def exact(case, seed):
    s = prepare(case, seed)
    t = case["tokens"]
    if case["op"] == "lora":
        ids, ranks, x = s["ids"].tolist(), s["ranks"].tolist(), s["x"].double()
        outs = [b.double().clone() for b in s["base"]]
        for e in sorted(set(ids)):
            if e < 0:
                continue
            rows = torch.tensor([i for i, j in enumerate(ids) if j == e], device=x.device)
            r = ranks[e]
            for a, b, y in zip(s["a"], s["b"], outs):
                low = torch.matmul(x[rows], a[e, :r].double().t().contiguous())
                y[rows] += float(s["scales"][e]) * torch.matmul(low, b[e, :, :r].double().t().contiguous())
        return outs
    if case["op"] == "heads":
        rot, half = case["rot"], case["rot"] // 2
        result = {}
        for name, w in (("q", s["qw"]), ("k", s["kw"])):
            if s[name] is None:
                result[name] = None
                continue
            x = s[name].double()
            if w is not None:
                x = x / torch.sqrt((x * x).sum(2, keepdim=True) / case["dim"] + EPS) * w.double()
            y = x.clone()
            for i in range(half):
                angle = s["pos"][int(s["axis"][i])].double() * s["freq"][i].double()
                c, n = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
                u, v = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                y[:, :, u] = x[:, :, u] * c - x[:, :, v] * n
                y[:, :, v] = x[:, :, u] * n + x[:, :, v] * c
            result[name] = y
        return result
    if case["op"] == "gate":
        logits = (s["x"].double()[:, None, :] * s["w"].double()[None]).sum(2) if t <= 8 else \
            torch.stack([torch.mv(s["w"].double(), r) for r in s["x"].double()])
        score = torch.sigmoid(logits) if case["scoring"] == "sigmoid" else torch.softmax(logits, 1)
        bias = [0.0] * case["experts"] if s["bias"] is None else s["bias"].double().tolist()
        size = case["experts"] // case["groups"]
        ids, weights = [], []
        for row in score.tolist():
            choice = [p + q for p, q in zip(row, bias)]
            place = range(len(choice))
            if case["groups"] > 1:
                def worth(j):
                    return sum(sorted(choice[j * size:(j + 1) * size])[-2:])

                best = sorted(range(case["groups"]), key=lambda j: (-worth(j), j))[:case["top_groups"]]
                place = [i for j in best for i in range(j * size, (j + 1) * size)]
            picked = sorted(place, key=lambda i: (-choice[i], i))[:case["top_k"]]
            total = sum(row[i] for i in picked) if case["renorm"] else 1.0
            ids.append(picked)
            weights.append([row[i] / total * case["scale"] for i in picked])
        return {"ids": torch.tensor(ids, dtype=torch.int32), "weights": torch.tensor(weights, dtype=torch.float64)}
    n, v = case["top"], case["vocab"]
    result = {"logprobs": torch.empty(t, case["given"], dtype=torch.float64), "entropy": torch.empty(t, dtype=torch.float64)}
    if n:
        result["ids"] = torch.empty(t, n, dtype=torch.int32)
        result["top"] = torch.empty(t, n, dtype=torch.float64)
    for i in range(t):
        row = s["x"][i].double() * float(torch.tensor(case["scale"], dtype=torch.float32))
        log = row - torch.logsumexp(row, 0)
        result["logprobs"][i] = log[s["given"][i].long()].cpu()
        result["entropy"][i] = torch.special.entr(torch.exp(log)).sum().cpu()
        if n:
            order = torch.sort(s["x"][i], descending=True, stable=True).indices[:n]
            result["ids"][i], result["top"][i] = order.int().cpu(), log[order].cpu()
    return result
