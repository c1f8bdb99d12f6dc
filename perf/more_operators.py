"""The two ends of a serving step around the rotated cache, as measured cases.

A step begins with the projections' rows: heads are normalised, rotated by their position, transformed and
appended (``rope``).  It ends with logits: penalties, biases, a grammar's mask and the temperature make them the
probabilities that the drafts are checked against (``probs``), and the tokens that stay are counted (``counts``).

``own`` False: the operators in plain torch.  ``own`` True: the library's entry points.
"""

import math

import numpy as np
import torch

own = False

D = 128                       # head size of the cache
P = 16                        # tokens of a page
MOST = 32767                  # where counts stop


# ---- the cases -------------------------------------------------------------------------------
def _rope(name, batch, hq, hkv, lo, hi, new, transform, tv, layout="half", rot=128, scaling="none", factor=1.0, theta=1e6,
          norm=True, tree=False, sink=64, keep=256, flush=8):
    return {"name": name, "op": "rope", "batch": batch, "hq": hq, "hkv": hkv, "lo": lo, "hi": hi, "new": new, "transform": transform,
            "tv": tv, "layout": layout, "rot": rot, "scaling": scaling, "factor": factor, "theta": theta, "norm": norm, "tree": tree,
            "sink": sink, "keep": keep, "flush": flush}


def _probs(name, batch, nodes, vocab, dtype, hist, bias, allow, greedy):
    return {"name": name, "op": "probs", "batch": batch, "nodes": nodes, "vocab": vocab, "dtype": dtype, "hist": hist, "bias": bias,
            "allow": allow, "greedy": greedy}


def listed():
    return [
        # one user's next token behind a long prompt: latency alone
        _rope("rope-ctx32k-b1-n1", 1, 32, 8, 32760, 32760, 1, "orthogonal", True),
        # a served batch of ragged contexts, a token each
        _rope("rope-ctx4k8k-b64-n1", 64, 32, 8, 4096, 8192, 1, "orthogonal", True),
        # drafted trees at the longest contexts: positions by depth, Hadamard keys, adjacent pairs, half of the head
        _rope("rope-ctx128k-b4-tree16", 4, 64, 8, 131072, 131072, 16, "hadamard", False, "interleaved", 64, "yarn", 4.0, 1e4, False, True,
              0, 0, 128),
        # a prompt's odd remainder, one query head to a key head, no norm
        _rope("rope-ctx500-b3-n777", 3, 8, 8, 500, 777, 777, "invertible", True, "half", 96, "linear", 8.0, 1e4, False),
        # the prefill chunk of sixteen users
        _rope("rope-ctx16k-b16-n2048", 16, 32, 8, 16384, 16384, 2048, "invertible", False),
        # one user's next token, 32-bit logits, a small vocabulary: latency alone
        _probs("probs-b1-v32000", 1, 1, 32000, "float32", 900, 0, 0.0, 0.0),
        # a served batch: long histories, some biases, some rows greedy
        _probs("probs-b64-v151936", 64, 1, 151936, "bfloat16", 6000, 20, 0.0, 0.25),
        # constrained output: a grammar leaves two tokens in a hundred, an odd vocabulary
        _probs("probs-b48-grammar-v100003", 48, 1, 100003, "float16", 2000, 5, 0.02, 0.1),
        # drafted trees, every node with the penalties of its own path
        _probs("probs-b64-n16-v151936", 64, 16, 151936, "bfloat16", 4000, 8, 0.0, 0.0),
        # after a step of drafted trees: the kept paths and the tokens behind them
        {"name": "counts-step-b64-n16-v151936", "op": "counts", "batch": 64, "nodes": 16, "vocab": 151936, "lo": 0, "hi": 0, "made": 0},
        # one user's prompt is taken in
        {"name": "counts-admit-b1-ctx2k-v32000", "op": "counts", "batch": 1, "nodes": 0, "vocab": 32000, "lo": 2000, "hi": 2000, "made": 0},
        # stopped requests come back: long prompts, and what they had answered is counted again
        {"name": "counts-admit-b16-ctx128k-v151936", "op": "counts", "batch": 16, "nodes": 0, "vocab": 151936, "lo": 65536, "hi": 131072,
         "made": 4000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope"] * 4 + ["probs"] * 4 + ["counts"])
    if op == "rope":
        hkv, gqa = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        tree = rng.random() < 0.25
        batch = _log(rng, 1, 64)
        most = 32768 * 40 // (batch * hkv * (gqa + 1))                      # no dearer than the largest listed
        new = _log(rng, 1, max(1, min(128 if tree else 2048, most)))
        hi = _log(rng, 1, 131072)
        scaling = rng.choice(["none", "linear", "ntk", "bands", "yarn"])
        win = rng.choice([(16, 128, 8), (64, 256, 8), (0, 0, 128), (64, 256, 1), (5, 48, 16)])
        c = _rope("", batch, hkv * gqa, hkv, rng.randint(hi // 2, hi), hi, new, rng.choice(["orthogonal", "invertible", "hadamard"]),
                  rng.random() < 0.5, rng.choice(["half", "interleaved"]), rng.choice([128, 128, 64, 2 * rng.randint(2, 64)]), scaling,
                  1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]), rng.choice([1e4, 5e5, 1e6]), rng.random() < 0.5, tree, *win)
    elif op == "probs":
        vocab, nodes = _log(rng, 1000, 160000), rng.choice([1, 1, _log(rng, 2, 64)])
        batch = _log(rng, 1, max(1, min(64, 64 * 16 * 151936 // (vocab * nodes))))
        c = _probs("", batch, nodes, vocab, rng.choice(["float32", "bfloat16", "float16"]), rng.choice([0, _log(rng, 1, 20000)]),
                   rng.choice([0, _log(rng, 1, 300)]), rng.choice([0.0, 0.0, 0.02, 0.5]), rng.choice([0.0, 0.0, 0.25, 1.0]))
    else:
        step = rng.random() < 0.5
        hi = 0 if step else _log(rng, 100, 131072)
        c = {"name": "", "op": op, "batch": _log(rng, 1, 64 if step else 16), "nodes": _log(rng, 1, 64) if step else 0,
             "vocab": _log(rng, 1000, 160000), "lo": rng.randint(hi // 2, hi), "hi": hi, "made": 0 if step else rng.choice([0, _log(rng, 1, 4000)])}
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------------------------
# (the outputs' shapes belong to the case: lengths and counts are drawn from its sizes, values from the seed)
def _lengths(case):
    r = np.random.default_rng([case["batch"], case["lo"], case["hi"], 1])
    return r.integers(case["lo"], case["hi"] + 1, case["batch"])


def _counts(batch, n):
    r = np.random.default_rng([batch, n, 3])
    return r.integers((n + 1) // 2, n + 1, batch) if batch > 1 else np.array([n])


def _parents(counts, seed):
    r = np.random.default_rng([seed, 4])
    out = []
    for n in counts:
        i = np.arange(n)
        out.append(np.where(i == 0, -1, np.maximum(0, i - r.integers(1, 6, n))))
    return np.concatenate(out).astype(np.int32)


def _depths(counts, parent):
    out, at = np.zeros(len(parent), np.int64), 0
    for n in counts:
        for i in range(1, n):
            out[at + i] = out[at + parent[at + i]] + 1
        at += n
    return out


def _up(x, m):
    return -(-x // m) * m


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _cu(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _orthogonal(gen, hkv):
    q, r = torch.linalg.qr(torch.randn((hkv, D, D), generator=gen, device="cuda", dtype=torch.float64))
    return q * torch.sign(torch.diagonal(r, dim1=1, dim2=2)).unsqueeze(1)


def _matrices(case, gen):
    """T_K, T_K^-T and T_V in float32 (None where there is none)."""
    hkv, tk, tkit = case["hkv"], None, None
    if case["transform"] != "hadamard":
        t = _orthogonal(gen, hkv)
        if case["transform"] == "invertible":
            lam = torch.logspace(0, 2, D, dtype=torch.float64, device="cuda")
            a = (t * lam) @ t.transpose(1, 2)
            t = (torch.linalg.cholesky((a + a.transpose(1, 2)) / 2) * lam ** -0.25) @ t.transpose(1, 2)
        tk = t.float()
        tkit = torch.linalg.inv(tk.double()).transpose(1, 2).float().contiguous()
    return tk, tkit, _orthogonal(gen, hkv).float() if case["tv"] else None


def _turns(case):
    """Turns per token of every pair in 64 bits, and the factor of the rotated channels."""
    rot, theta, f, kind = case["rot"], case["theta"], case["factor"], case["scaling"]
    i = np.arange(rot // 2)
    if kind == "ntk":
        theta = theta * f ** (rot / (rot - 2))
    w, scale = theta ** (-2.0 * i / rot), 1.0
    if kind == "linear":
        w = w / f
    elif kind == "bands":                                                   # long waves stretched, short ones kept
        s = (8192.0 * w / (2 * np.pi) - 1.0) / (4.0 - 1.0)
        s = np.clip(s, 0.0, 1.0)
        w = w / f * (1 - s) + w * s
    elif kind == "yarn":
        at = lambda beta: rot * math.log(32768.0 / (beta * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        w, scale = w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1.0
    return w / (2 * np.pi), scale


def _prepare_rope(case, seed):
    dev, hq, hkv = "cuda", case["hq"], case["hkv"]
    gen = torch.Generator(dev).manual_seed(seed)
    ctx, n = _lengths(case), _counts(case["batch"], case["new"]) if case["tree"] else np.full(case["batch"], case["new"])
    seq = np.repeat(np.arange(case["batch"]), n)
    i = np.concatenate([np.arange(k) for k in n])
    pos = ctx[seq] + i
    far = ctx[seq] + _depths(n, _parents(n, seed)) if case["tree"] else pos
    edge = case["sink"] + np.maximum(0, ctx - case["sink"] - case["keep"]) // case["flush"] * case["flush"]
    cap = _up(case["keep"] + case["flush"] + int(n.max()) + P, P)
    rows = len(seq)
    qkv = torch.randn((rows, hq + 2 * hkv, D), generator=gen, device=dev)     # the fused projection's rows
    loud = torch.rand((hkv, D), generator=gen, device=dev).topk(2, dim=1).indices
    qkv[:, hq:hq + hkv] *= torch.ones((hkv, D), device=dev).scatter_(1, loud, 15.0)
    qkv = qkv.to(torch.bfloat16)
    w = lambda: 1.0 + 0.3 * torch.randn(D, generator=gen, device=dev)  # noqa: E731
    s = {"case": dict(case), "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:], "seq": _dev(seq.astype(np.int32)),
         "pos": _dev(pos.astype(np.int32)), "far": _dev(far.astype(np.int32)), "qw": w() if case["norm"] else None,
         "kw": w() if case["norm"] else None, "eps": 1e-6, "cap": cap}
    s["tk"], s["tkit"], s["tv"] = _matrices(case, gen)
    s["seq_len"], s["s_quant"] = _dev(ctx.astype(np.int32)), _dev(edge.astype(np.int32))
    # the rows that the program knows to go to the sink, and those for the ring
    s["first"], s["later"] = _dev(np.flatnonzero(pos < case["sink"])), _dev(np.flatnonzero(pos >= case["sink"]))
    for name, t in (("sink_k", max(1, case["sink"])), ("sink_v", max(1, case["sink"])), ("ring_k", cap), ("ring_v", cap)):
        s[name] = torch.zeros((case["batch"], hkv, t, D), dtype=torch.bfloat16, device=dev)
    turns, s["scale"] = _turns(case)
    s["turns"] = _dev(turns)
    if own:
        import bit_rotated_kv_gb300 as kvq
        s["kvq"] = kvq
        s["cfg"] = kvq.KVConfig(n_q_heads=hq, n_kv_heads=hkv, batch=case["batch"], max_pages_per_seq=1, num_pages=1, ring_cap=cap,
                                s_sink=case["sink"], s_keep=case["keep"], s_flush=case["flush"])
        c = kvq.KVCache(s["cfg"])
        for name in ("seq_len", "s_quant", "sink_k", "sink_v", "ring_k", "ring_v"):
            setattr(c, name, s[name])
        s["cache"] = c
        s["tr"] = kvq.Transform(kvq.KVQ_TRANSFORM_HADAMARD if case["transform"] == "hadamard" else kvq.KVQ_TRANSFORM_DENSE,
                                *(t if t is None else t.contiguous() for t in (s["tk"], s["tkit"], s["tv"])))
        kinds = {"none": kvq.KVQ_ROPE_PLAIN, "linear": kvq.KVQ_ROPE_LINEAR, "ntk": kvq.KVQ_ROPE_NTK, "bands": kvq.KVQ_ROPE_BANDS,
                 "yarn": kvq.KVQ_ROPE_YARN}
        context, a, b = {"bands": (8192.0, 1.0, 4.0), "yarn": (32768.0, 32.0, 1.0)}.get(case["scaling"], (0.0, 0.0, 0.0))
        s["rope"] = kvq.Rope.make(kvq.KVQ_ROPE_HALF if case["layout"] == "half" else kvq.KVQ_ROPE_INTERLEAVED, case["rot"], case["theta"],
                                  kinds[case["scaling"]], case["factor"], context, a, b, q_norm=s["qw"], k_norm=s["kw"], norm_eps=s["eps"])
        s["q_out"] = torch.empty((rows, hq, D), dtype=torch.bfloat16, device=dev)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return s


def _some_tokens(r, n, vocab):
    return np.minimum(vocab - 1, (vocab * r.random(n) ** 3)).astype(np.int32)   # few tokens often, most seldom


def _history(r, batch, vocab, hist):
    """Counts as the library keeps them: a bit for the prompt's tokens, the others' number below it."""
    c = np.zeros((batch, _up(vocab, 2)), np.int64)
    if hist:
        for b in range(batch):
            n = int(r.integers((hist + 1) // 2, hist + 1))
            c[b] += np.bincount(_some_tokens(r, n // 2, vocab), minlength=c.shape[1])
            c[b, _some_tokens(r, n - n // 2, vocab)] -= 1 << 15
    return c.astype(np.int16)


def _prepare_probs(case, seed):
    dev, batch, vocab = "cuda", case["batch"], case["vocab"]
    gen = torch.Generator(dev).manual_seed(seed)
    r = np.random.default_rng([seed, 2])
    n = _counts(batch, case["nodes"])
    rows = int(n.sum())
    logits = 2.5 * torch.randn((rows, vocab), generator=gen, device=dev)
    best = torch.randint(0, vocab, (rows, 24), generator=gen, device=dev)
    logits.scatter_add_(1, best, 4.0 + 11.0 * torch.rand((rows, 24), generator=gen, device=dev))
    s = {"case": dict(case), "logits": logits.to(getattr(torch, case["dtype"])), "cu": _dev(_cu(n)), "n_max": int(n.max()), "rows": rows}
    s["parent"] = _dev(_parents(n, seed)) if case["nodes"] > 1 else None
    s["token"] = _dev(_some_tokens(r, rows, vocab)) if case["nodes"] > 1 else None
    s["counts"] = _dev(_history(r, batch, vocab, case["hist"])) if case["hist"] else None
    f32 = lambda a: _dev(np.asarray(a, np.float32))  # noqa: E731
    temperature = r.uniform(0.5, 1.3, batch)
    temperature[r.random(batch) < case["greedy"]] = 0.0
    s["temperature"], s["repetition"] = f32(temperature), f32(r.choice([1.0, 1.1, 1.3], batch))
    s["presence"], s["frequency"] = f32(r.uniform(0, 1.0, batch)), f32(r.uniform(0, 0.5, batch))
    s["bias_cu"] = s["bias_token"] = s["bias"] = None
    if case["bias"]:
        k = _counts(batch, case["bias"])
        s["bias_cu"] = _dev(_cu(k))
        s["bias_token"] = _dev(np.concatenate([np.sort(r.choice(vocab, x, replace=False)) for x in k]).astype(np.int32))
        s["bias"] = f32(np.where(r.random(int(k.sum())) < 0.2, -100.0, r.normal(0, 3.0, int(k.sum()))))
    s["mask"] = s["mask_row"] = None
    if case["allow"]:
        words = -(-vocab // 32)
        bits = torch.rand((rows, words * 32), generator=gen, device=dev) < case["allow"]
        bits.scatter_(1, best[:, :4], True)
        weight = 1 << torch.arange(32, device=dev)
        s["mask"] = (bits.view(rows, words, 32) * weight).sum(-1).to(torch.int32)     # (the highest bit wraps to the sign)
        order = r.permutation(rows).astype(np.int32)
        s["mask_row"] = _dev(np.where(r.random(rows) < 0.1, -1, order).astype(np.int32))   # some rows are free
    if own:
        import bit_rotated_kv_gb300 as kvq
        s["kvq"] = kvq
        s["cfg"] = kvq.KVConfig(n_q_heads=1, n_kv_heads=1, batch=batch, max_pages_per_seq=1, num_pages=1, ring_cap=272)
        s["rules"] = kvq.LogitRules(temperature=s["temperature"], repetition=s["repetition"], presence=s["presence"],
                                    frequency=s["frequency"], counts=s["counts"], bias_cu=s["bias_cu"], bias_token=s["bias_token"],
                                    bias=s["bias"], mask=s["mask"], mask_row=s["mask_row"])
        s["p"] = torch.empty((rows, vocab), dtype=torch.float32, device=dev)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return s


def _prepare_counts(case, seed):
    r = np.random.default_rng([seed, 6])
    batch, vocab = case["batch"], case["vocab"]
    s = {"case": dict(case), "counts": torch.zeros((batch, _up(vocab, 2)), dtype=torch.int16, device="cuda")}
    if case["nodes"]:
        n = _counts(batch, case["nodes"])
        path, kept = np.full(int(n.sum()), -1, np.int32), np.zeros(batch, np.int32)
        for b, at in enumerate(_cu(n)[:-1]):
            kept[b] = r.integers(1, n[b] + 1)
            path[at:at + kept[b]] = np.concatenate([[0], np.sort(r.choice(np.arange(1, n[b]), kept[b] - 1, replace=False))])
        s |= {"cu": _dev(_cu(n)), "token": _dev(_some_tokens(r, len(path), vocab)), "path": _dev(path), "n_accept": _dev(kept),
              "next": _dev(_some_tokens(r, batch, vocab)), "before": _dev(_history(r, batch, vocab, 4000))}
    else:
        n, made = _lengths(case), np.full(batch, case["made"])
        s |= {"cu": _dev(_cu(n)), "token": _dev(_some_tokens(r, int(n.sum()), vocab)), "made_cu": _dev(_cu(made)),
              "made": _dev(_some_tokens(r, int(made.sum()), vocab)) if case["made"] else None}
    if own:
        import bit_rotated_kv_gb300 as kvq
        s["kvq"] = kvq
        s["cfg"] = kvq.KVConfig(n_q_heads=1, n_kv_heads=1, batch=batch, max_pages_per_seq=1, num_pages=1, ring_cap=272)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    return {"rope": _prepare_rope, "probs": _prepare_probs, "counts": _prepare_counts}[case["op"]](case, seed)


# ---- norm, rotation, transform and append in plain torch -------------------------------------------
def _hadamard(dev):
    h = torch.ones((1, 1), device=dev)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _headwise(x, matrices, gqa):
    """[n, H, D] by each head's matrix."""
    n, h, _ = x.shape
    if matrices is None:
        return (x @ _hadamard(x.device)) * (1.0 / math.sqrt(D))
    y = torch.einsum("nhgj,hij->nhgi", x.view(n, h // gqa, gqa, D), matrices)
    return y.reshape(n, h, D)


def _rope_plain(s):
    case, rot = s["case"], s["case"]["rot"]
    turn = s["far"].double().view(-1, 1) * s["turns"]
    angle = (turn - turn.floor()) * (2 * math.pi)
    cos, sin = (f(angle).float().unsqueeze(1) * s["scale"] for f in (torch.cos, torch.sin))

    def placed(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
        if case["layout"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([turned, x[..., rot:]], -1)

    q = _headwise(placed(s["q"], s["qw"]), s["tkit"], case["hq"] // case["hkv"]).to(torch.bfloat16)
    k = _headwise(placed(s["k"], s["kw"]), s["tk"], 1).to(torch.bfloat16)
    v = s["v"] if s["tv"] is None else _headwise(s["v"].float(), s["tv"], 1).to(torch.bfloat16)
    for rows, name, size in ((s["first"], "sink", max(1, case["sink"])), (s["later"], "ring", s["cap"])):
        at, slot = s["seq"][rows].long(), s["pos"][rows].long() % size
        s[name + "_k"][at, :, slot] = k[rows]
        s[name + "_v"][at, :, slot] = v[rows]
    s["seq_len"].scatter_reduce_(0, s["seq"].long(), s["pos"] + 1, "amax")
    return q


# ---- logits to probabilities in plain torch ----------------------------------------------------------
def _sequence_of(s):
    return torch.searchsorted(s["cu"].long(), torch.arange(s["rows"], device=s["cu"].device), right=True) - 1


def _probs_plain(s):
    case, dev, vocab = s["case"], s["logits"].device, s["case"]["vocab"]
    seq = _sequence_of(s)
    x = s["logits"].float()
    if s["bias"] is not None:
        at = torch.searchsorted(s["bias_cu"].long(), torch.arange(len(s["bias"]), device=dev), right=True) - 1
        dense = torch.zeros((case["batch"], vocab), device=dev)
        dense[at, s["bias_token"].long()] = s["bias"]
        x = x + dense[seq]
    known = s["counts"][:, :vocab].int() if s["counts"] is not None else torch.zeros((case["batch"], vocab), dtype=torch.int32, device=dev)
    made, seen = (known & MOST)[seq], (known != 0)[seq]
    if s["token"] is not None:                                              # the nodes above, the root (counted before) left out
        first = s["cu"].long()[seq]
        at = torch.arange(s["rows"], device=dev)
        for _ in range(s["n_max"]):
            up = s["parent"].long()[at]
            made.scatter_add_(1, s["token"].long()[at].view(-1, 1), (up >= 0).int().view(-1, 1))
            at = torch.where(up >= 0, first + up, at)
        seen = seen | (made > 0)
    each = lambda t: t[seq].view(-1, 1)  # noqa: E731
    rep = each(s["repetition"])
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - each(s["frequency"]) * made.float() - each(s["presence"]) * (made > 0).float()
    if s["mask"] is not None:
        bits = ((s["mask"].unsqueeze(-1) >> torch.arange(32, device=dev, dtype=torch.int32)) & 1).flatten(1)[:, :vocab] > 0
        free = (s["mask_row"] < 0).view(-1, 1)
        x = torch.where(free | bits[s["mask_row"].clamp(min=0).long()], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    token = torch.arange(vocab, device=dev)
    best = torch.where(x == top, token, vocab).amin(-1, keepdim=True)
    heat = each(s["temperature"])
    e = torch.exp((x - top) / torch.where(heat > 0, heat, 1.0))
    return torch.where(heat > 0, e / e.sum(-1, keepdim=True), (token == best).float())


# ---- counting in plain torch ---------------------------------------------------------------------------
def _tally(s, at, token, real):
    add = torch.zeros(s["counts"].shape, dtype=torch.int32, device=at.device)
    add.view(-1).scatter_add_(0, at * s["counts"].shape[1] + token.long(), real.int())
    c = s["counts"].int()
    s["counts"].copy_((c & ~MOST) | torch.clamp((c & MOST) + add, max=MOST))


def _rows_of(cu, n):
    return torch.searchsorted(cu.long(), torch.arange(n, device=cu.device), right=True) - 1


def _counts_plain(s):
    dev, batch = s["counts"].device, s["case"]["batch"]
    at = _rows_of(s["cu"], len(s["token"]))
    if s["case"]["nodes"]:
        i = torch.arange(len(s["token"]), device=dev) - s["cu"].long()[at]
        kept = (i > 0) & (i < s["n_accept"][at])
        token = s["token"][torch.where(kept, s["cu"].long()[at] + s["path"], 0).long()]
        _tally(s, torch.cat([at, torch.arange(batch, device=dev)]), torch.cat([token, s["next"]]),
               torch.cat([kept, torch.ones(batch, dtype=torch.bool, device=dev)]))
        return
    said = torch.zeros(s["counts"].shape, dtype=torch.int32, device=dev)
    said.view(-1).index_fill_(0, at * said.shape[1] + s["token"].long(), 1 << 15)
    s["counts"].copy_(s["counts"].int() | said)
    if s["made"] is not None:
        _tally(s, _rows_of(s["made_cu"], len(s["made"])), s["made"], torch.ones_like(s["made"]))


# ---- one pass ------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    kvq = s.get("kvq") if own else None
    if op == "rope":
        if own:
            kvq.kv_rope_qk(s["cfg"], s["tr"], s["rope"], s["q"], s["q_out"], s["far"], s["k"], s["v"], s["seq"], s["pos"], s["far"],
                           s["cache"], s["status"])
        q = s["q_out"] if own else _rope_plain(s)
        return q, s["sink_k"], s["sink_v"], s["ring_k"], s["ring_v"], s["seq_len"]
    if op == "probs":
        if not own:
            return _probs_plain(s)
        kvq.kv_logits_probs(s["cfg"], s["rules"], s["logits"], s["cu"], s["parent"], s["token"], s["p"], s["status"])
        return s["p"]
    if s["case"]["nodes"]:
        s["counts"].copy_(s["before"])                                       # (the step is taken again)
        if own:
            kvq.kv_token_counts(s["cfg"], s["counts"], s["case"]["vocab"], kvq.KVQ_COUNT_OUTPUT, s["cu"], s["token"], s["path"],
                                s["n_accept"], s["next"], s["status"])
        else:
            _counts_plain(s)
        return s["counts"]
    s["counts"].zero_()                                                      # (new sequences in old places)
    if own:
        kvq.kv_token_counts(s["cfg"], s["counts"], s["case"]["vocab"], kvq.KVQ_COUNT_PROMPT, s["cu"], s["token"], None, None, None,
                            s["status"])
        if s["made"] is not None:
            kvq.kv_token_counts(s["cfg"], s["counts"], s["case"]["vocab"], kvq.KVQ_COUNT_OUTPUT, s["made_cu"], s["made"], None, None, None,
                                s["status"])
    else:
        _counts_plain(s)
    return s["counts"]


# ---- what a pass cannot do without ---------------------------------------------------------------------
def work(case):
    op, b = case["op"], case["batch"]
    if op == "rope":
        rows = b * case["new"] * (0.75 if case["tree"] and b > 1 else 1.0)
        hq, hkv, dense = case["hq"], case["hkv"], case["transform"] != "hadamard"
        mats = hkv * (2 * dense + case["tv"])
        heads = rows * ((hq + hkv) * dense + hkv * case["tv"])
        adds = rows * (hq + hkv) * (not dense) * D * 7
        return {"bytes": rows * (hq + 2 * hkv) * D * 4 + mats * D * D * 4 + rows * 16, "flops": heads * 2.0 * D * D + adds}
    if op == "probs":
        rows = b * case["nodes"] * (0.75 if case["nodes"] > 1 and b > 1 else 1.0)
        v, a = case["vocab"], case["allow"]
        read = 4 if case["dtype"] == "float32" else 2
        share = 0.9 * a + 0.1 if a else 1.0                                  # of the logits: those that a mask lets through
        return {"bytes": rows * v * (read * share + 4 + (0.125 if a else 0)) + (b * v * 2 * share if case["hist"] else 0), "flops": rows * v * 4.0}
    if case["nodes"]:                                                        # the copy before it, and a kept path's tokens
        return {"bytes": b * case["vocab"] * 4 + b * case["nodes"] * 6, "flops": 0}
    return {"bytes": b * case["vocab"] * 2 + b * ((case["lo"] + case["hi"]) / 2 + case["made"]) * 4, "flops": 0}


# ---- from the definitions, in 64 bits --------------------------------------------------------------------
def _exact_rope(case, seed):
    s = prepare(case, seed)
    rot, hq, hkv = case["rot"], case["hq"], case["hkv"]
    phase = torch.polar(torch.full_like(s["turns"], s["scale"]).expand(len(s["far"]), -1).contiguous(),
                        2 * math.pi * torch.frac(s["far"].double().outer(s["turns"])))

    def butterflies(y):
        for h in (1, 2, 4, 8, 16, 32, 64):
            z = y.reshape(*y.shape[:-1], D // (2 * h), 2, h)
            y = torch.stack([z[..., 0, :] + z[..., 1, :], z[..., 0, :] - z[..., 1, :]], -2).reshape(y.shape)
        return y / math.sqrt(D)

    def head(x, w, t):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + s["eps"]) * w.double()
        c = torch.arange(rot // 2, device=x.device)
        a, b = (c, c + rot // 2) if case["layout"] == "half" else (2 * c, 2 * c + 1)
        z = torch.complex(x[:, a], x[:, b]) * phase
        x = x.clone()
        x[:, a], x[:, b] = z.real, z.imag
        return butterflies(x) if t is None else x @ t.double().T

    pick = lambda t, h: None if t is None else t[h]  # noqa: E731
    q = torch.stack([head(s["q"][:, h], s["qw"], pick(s["tkit"], h * hkv // hq)) for h in range(hq)], 1)
    out = {n: s[n].double() for n in ("sink_k", "sink_v", "ring_k", "ring_v")}
    ring, sink = (s["pos"] >= case["sink"]).nonzero().view(-1), (s["pos"] < case["sink"]).nonzero().view(-1)
    for h in range(hkv):
        k = head(s["k"][:, h], s["kw"], pick(s["tk"], h))
        v = s["v"][:, h].double() if s["tv"] is None else s["v"][:, h].double() @ s["tv"][h].double().T
        for x, end in ((k, "_k"), (v, "_v")):
            out["ring" + end][s["seq"][ring].long(), h, s["pos"][ring].long() % s["cap"]] = x[ring]
            out["sink" + end][s["seq"][sink].long(), h, s["pos"][sink].long()] = x[sink]
    n = torch.bincount(s["seq"], minlength=case["batch"]).int()
    return q, out["sink_k"], out["sink_v"], out["ring_k"], out["ring_v"], s["seq_len"] + n


def _exact_probs(case, seed):
    s = prepare(case, seed)
    vocab, out = case["vocab"], torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    parent, token = (t.tolist() if t is not None else None for t in (s["parent"], s["token"]))
    par = {n: s[n].double().tolist() for n in ("temperature", "repetition", "presence", "frequency")}
    bias_cu = s["bias_cu"].tolist() if s["bias"] is not None else None
    mask_row = s["mask_row"].tolist() if s["mask"] is not None else None
    column = torch.arange(vocab, device="cuda")
    for b in range(case["batch"]):
        c = s["counts"][b, :vocab].long() if s["counts"] is not None else torch.zeros(vocab, dtype=torch.int64, device="cuda")
        for r in range(cu[b], cu[b + 1]):
            x = s["logits"][r].double()
            if bias_cu is not None:
                at = slice(bias_cu[b], bias_cu[b + 1])
                x = x.index_add(0, s["bias_token"][at].long(), s["bias"][at].double())
            made, seen, i = c.remainder(1 << 15), c != 0, r
            if token is not None:
                above = []
                while parent[i] >= 0:
                    above.append(token[i])
                    i = cu[b] + parent[i]
                if above:
                    made = made + torch.bincount(torch.tensor(above, device="cuda"), minlength=vocab)
                    seen = seen | (made > 0)
            rep = par["repetition"][b]
            x = torch.where(seen, torch.maximum(x, torch.zeros_like(x)) / rep + torch.minimum(x, torch.zeros_like(x)) * rep, x)
            x = x - par["frequency"][b] * made - par["presence"][b] * made.clamp(max=1)
            if mask_row is not None and mask_row[r] >= 0:
                word = s["mask"][mask_row[r]][column // 32].long()
                x = x.masked_fill((word >> (column % 32)) % 2 == 0, -math.inf)
            if par["temperature"][b] > 0:
                out[r] = torch.softmax(x / par["temperature"][b], 0)
            else:
                out[r, int((x == x.max()).nonzero()[0])] = 1.0
    return out


def exact(case, seed):
    if case["op"] == "counts":
        return None                                                         # whole numbers
    return (_exact_rope if case["op"] == "rope" else _exact_probs)(case, seed)
