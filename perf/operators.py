"""Speculative decoding and page management over the rotated INT2 cache, as measured cases.

A serving step that drafts a tree of tokens reads the cache once for every node of the tree
(``tree``), checks the drafts against the target's probabilities (``verify``) and keeps the
accepted path's rows (``commit``).  Parallel samples share a prompt's pages (``fork``), and a pool
whose sequences come and go is kept dense (``compact``).

``own`` False: the operators in plain torch.  ``own`` True: the library's entry points.
"""

import math

import numpy as np
import torch

own = False

D = 128                       # head size of the cache
P = 16                        # tokens of a page
ONE = 1 << 60                 # probability 1 in the units of the verification


# ---- the cases -------------------------------------------------------------------------------
def _tree(name, batch, hq, hkv, lo, hi, nodes, group, l2=False, sink=64, keep=256, flush=8):
    return {"name": name, "op": "tree", "batch": batch, "hq": hq, "hkv": hkv, "lo": lo, "hi": hi, "nodes": nodes,
            "group": group, "l2": l2, "sink": sink, "keep": keep, "flush": flush}


def listed():
    return [
        # the oracle-sized layer: four drafted tokens on a short context -- latency alone
        _tree("tree-ctx512-b1-n4", 1, 4, 1, 504, 504, 4, 128, sink=16, keep=128),
        # one user, a long prompt, a wide tree of drafts: 64 nodes x 4 heads share each page
        _tree("tree-ctx32k-b1-n64", 1, 32, 8, 32760, 32760, 64, 128),
        # a served batch of ragged contexts, small trees of ragged size
        _tree("tree-ctx4k8k-b64-n8", 64, 32, 8, 4096, 8192, 8, 64),
        # the longest contexts, normalised keys, the finest groups and the widest heads-per-page
        _tree("tree-ctx128k-b4-n16", 4, 64, 8, 131072, 131072, 16, 32, l2=True, sink=0, keep=0, flush=128),
        # one user, eight drafts that were taken greedily (no draft distribution), a small vocabulary
        {"name": "verify-b1-n8-v32000", "op": "verify", "batch": 1, "nodes": 8, "vocab": 32000, "dist": False},
        # a served batch, sampled drafts with their distributions, a large vocabulary
        {"name": "verify-b64-n16-v151936", "op": "verify", "batch": 64, "nodes": 16, "vocab": 151936, "dist": True},
        # keeping the accepted path of one user's small tree
        {"name": "commit-b1-n8", "op": "commit", "batch": 1, "hkv": 8, "nodes": 8, "acc": 4, "lo": 600, "hi": 600,
         "sink": 64, "keep": 256, "flush": 8},
        # ... and of a batch of wide trees
        {"name": "commit-b64-n64", "op": "commit", "batch": 64, "hkv": 8, "nodes": 64, "acc": 9, "lo": 4096, "hi": 8192,
         "sink": 64, "keep": 256, "flush": 8},
        # four parallel samples of one long prompt, restarted
        {"name": "fork-ctx32k-1to4", "op": "fork", "prompts": 1, "samples": 4, "hkv": 8, "lo": 32760, "hi": 32760,
         "group": 128, "sink": 64, "keep": 256, "flush": 8},
        # a batch: eight prompts, seven samples each
        {"name": "fork-ctx4k8k-8to56", "op": "fork", "prompts": 8, "samples": 7, "hkv": 8, "lo": 4096, "hi": 8192,
         "group": 64, "sink": 64, "keep": 256, "flush": 8},
        # a small pool: one of eight sequences leaves, the pool is made dense, a new one is admitted
        {"name": "compact-b8-ctx2k", "op": "compact", "batch": 8, "leave": 1, "hkv": 8, "lo": 2048, "hi": 2048, "group": 128,
         "sink": 64, "keep": 256, "flush": 8},
        # a full pool: sixteen of 64 sequences leave at once
        {"name": "compact-b64-ctx8k", "op": "compact", "batch": 64, "leave": 16, "hkv": 8, "lo": 4096, "hi": 8192,
         "group": 64, "sink": 64, "keep": 256, "flush": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree"] * 5 + ["verify"] * 2 + ["commit", "fork", "compact"])
    hkv = rng.choice([1, 2, 4, 8])
    win = rng.choice([(16, 128, 8), (64, 256, 8), (0, 0, 128), (64, 256, 1), (5, 48, 16)])
    if op == "tree":
        gqa = rng.choice([1, 2, 4, 8])
        nodes = _log(rng, 1, 128)
        batch = _log(rng, 1, 64)
        most = 4 * 131072 * 8 * 128 // (batch * hkv * max(nodes * gqa, 128))     # no dearer than the largest listed
        hi = _log(rng, 64, max(65, min(131072, most)))
        c = _tree("", batch, hkv * gqa, hkv, rng.randint(hi // 2 + 1, hi), hi, nodes, rng.choice([32, 64, 128]),
                  rng.random() < 0.3, *win)
        del c["name"]
        return c
    if op == "verify":
        vocab, nodes = _log(rng, 1000, 160000), _log(rng, 1, 64)
        batch = _log(rng, 1, max(1, min(64, 64 * 16 * 151936 // (vocab * nodes))))
        return {"op": op, "batch": batch, "nodes": nodes, "vocab": vocab, "dist": rng.random() < 0.5}
    hi = _log(rng, 300, 8192)
    c = {"op": op, "hkv": hkv, "lo": rng.randint(hi // 2 + 1, hi), "hi": hi, "sink": win[0], "keep": win[1], "flush": win[2]}
    if op == "commit":
        nodes = _log(rng, 1, 64)
        return c | {"batch": _log(rng, 1, 64), "nodes": nodes, "acc": rng.randint(1, nodes)}
    c["group"] = rng.choice([32, 64, 128])
    if op == "fork":
        prompts = rng.randint(1, 8)
        return c | {"prompts": prompts, "samples": rng.randint(1, 7)}
    batch = rng.randint(2, 64)
    return c | {"batch": batch, "leave": rng.randint(1, max(1, batch // 4))}


# ---- inputs ------------------------------------------------------------------------------------
def _up(x, m):
    return -(-x // m) * m


def _head_bytes(group, l2):
    return _up(2 * 512 + 2 * P * (D // group) * 4 + (2 * P if l2 else 0), 32)


# (the outputs' shapes belong to the case: lengths and counts are drawn from its sizes, values from the seed)
def _lengths(case, batch):
    r = np.random.default_rng([batch, case["lo"], case["hi"], 1])
    return r.integers(case["lo"], case["hi"] + 1, batch)


def _edge(length, case):
    """Right edge of the INT2 region after the flush rule ran on `length` tokens."""
    over = np.maximum(0, length - case["sink"] - case["keep"])
    return case["sink"] + over // case["flush"] * case["flush"]


def _norms(shape, gen, dev):
    n = torch.exp(1.5 * torch.randn(shape, generator=gen, device=dev)) * math.sqrt(D)
    return torch.where(torch.rand(shape, generator=gen, device=dev) < 0.01, n * 0.03, n)


def _fill_pages(pages, group, l2, gen):
    """Codes and scales as the quantizer writes them: the inner two levels three times as often as
    the outer ones, value groups of unit variance, key groups a little wider than that (outlier
    channels spread by the rotation) or of unit norm with the norm kept apart."""
    ng, dev = D // group, pages.device
    n, hkv, _ = pages.shape
    step = max(1, (1 << 22) // hkv)
    for a in range(0, n, step):
        b = min(n, a + step)
        shape = (b - a, hkv)
        rnd = lambda: torch.randint(-2**31, 2**31, shape + (256,), dtype=torch.int32, generator=gen, device=dev)  # noqa: E731
        hi = rnd() & -0x55555556                                        # the upper bit of every code
        mid = (rnd() | rnd()) & 0x55555555                              # 1: an inner level (01 or 10)
        words = hi | (((hi >> 1) & 0x55555555) ^ mid)
        pages[a:b, :, :1024] = words.view(torch.uint8)
        o = 1024
        kd = (0.12 if l2 else 3.2) * torch.exp(0.12 * torch.randn(shape + (P, ng), generator=gen, device=dev))
        kz = 1.5 + 0.15 * torch.randn(shape + (P, ng), generator=gen, device=dev)
        pages[a:b, :, o:o + P * ng * 4] = torch.stack([kd, kz], -1).half().flatten(2).view(torch.uint8)
        o += P * ng * 4
        vd = 1.5 * torch.exp(0.12 * torch.randn(shape + (P * ng,), generator=gen, device=dev))
        vz = 1.5 + 0.15 * torch.randn(shape + (P * ng,), generator=gen, device=dev)
        pages[a:b, :, o:o + P * ng * 4] = torch.cat([vd, vz], -1).half().view(torch.uint8)
        o += P * ng * 4
        if l2:
            pages[a:b, :, o:o + 2 * P] = _norms(shape + (P,), gen, dev).half().view(torch.uint8)


def _cache(case, lens, extra, seed, owned=None, spare=0, hold=0):
    """A cache of sequences of `lens` tokens, the last `extra[b]` of them drafts that no flush has
    seen; physical pages in random order; one page behind the pool for the plain form's masked
    writes.  owned: whether a sequence holds pages of its own."""
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed)
    r = np.random.default_rng([seed, 2])
    batch, hkv, l2, group = len(lens), case["hkv"], case.get("l2", False), case.get("group", 128)
    edge = _edge(lens - extra, case)
    count = np.maximum(0, -(-(np.maximum(edge, lens if hold else 0) - case["sink"]) // P))
    count = count if owned is None else np.where(owned, count, 0)
    maxp = int(max(1, count.max())) + 1
    used = int(count.sum())
    total = max(1, used + spare)
    table = np.full((batch, maxp), -1, np.int32)
    ids = r.permutation(total)[:used].astype(np.int32)
    at = 0
    for b in range(batch):
        table[b, :count[b]] = ids[at:at + count[b]]
        at += count[b]
    ref = np.zeros(total + 1, np.int32)
    ref[ids] = 1
    cap = _up(case["keep"] + case["flush"] + int(np.max(extra)) + P, P)
    s = {"case": dict(case), "gqa": case.get("hq", hkv) // hkv, "hkv": hkv, "batch": batch, "maxp": maxp, "num_pages": total,
         "cap": cap, "group": group, "l2": l2, "sink": case["sink"], "max_ctx": int(max(lens.max(), case["hi"] + int(np.max(extra))))}
    s["pages"] = torch.zeros((total + 1, hkv, _head_bytes(group, l2)), dtype=torch.uint8, device=dev)
    _fill_pages(s["pages"], group, l2, gen)
    s["table"] = torch.from_numpy(table).to(dev)
    s["ref"] = torch.from_numpy(ref).to(dev)
    s["seq_len"] = torch.from_numpy(lens.astype(np.int32)).to(dev)
    s["s_quant"] = torch.from_numpy(edge.astype(np.int32)).to(dev)
    rows = max(1, case["sink"])
    for name, t in (("sink_k", rows), ("sink_v", rows), ("ring_k", cap), ("ring_v", cap)):
        x = torch.randn((batch, hkv, t, D), generator=gen, device=dev)
        if name.endswith("k"):
            x = x * (_norms((batch, hkv, t, 1), gen, dev) / math.sqrt(D) if l2 else 2.1)
            if name == "sink_k":
                x[:, :, :4] *= 0.05                                     # the low-norm sink tokens
        s[name] = x.to(torch.bfloat16)
    if own:
        import bit_rotated_kv_gb300 as kvq
        s["kvq"] = kvq
        s["cfg"] = kvq.KVConfig(n_q_heads=case.get("hq", hkv), n_kv_heads=hkv, batch=batch, max_pages_per_seq=maxp, num_pages=total,
                                ring_cap=cap, group_size=group, key_l2norm=l2, s_sink=case["sink"], s_keep=case["keep"],
                                s_flush=case["flush"])
        c = kvq.KVCache(s["cfg"])
        c.pages, c.page_table, c.seq_len, c.s_quant = s["pages"][:total], s["table"], s["seq_len"], s["s_quant"]
        c.sink_k, c.sink_v, c.ring_k, c.ring_v = s["sink_k"], s["sink_v"], s["ring_k"], s["ring_v"]
        s["cache"] = c
        s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return s


def _cu(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()


def _counts(case, batch):
    r = np.random.default_rng([batch, case["nodes"], 3])
    n = case["nodes"]
    return r.integers((n + 1) // 2, n + 1, batch) if batch > 1 else np.array([n])


def _parents(counts, seed):
    r = np.random.default_rng([seed, 4])
    out = []
    for n in counts:
        i = np.arange(n)
        out.append(np.where(i == 0, -1, np.maximum(0, i - r.integers(1, 6, n))))
    return np.concatenate(out).astype(np.int32)


def prepare(case, seed):
    dev = "cuda"
    op = case["op"]
    if op == "tree":
        lens = _lengths(case, case["batch"])
        n = _counts(case, case["batch"])
        s = _cache(case, lens + n, n, seed)
        s["cu"] = _cu(n)
        s["n_max"] = int(n.max())
        s["parent"] = torch.from_numpy(_parents(n, seed)).to(dev)
        gen = torch.Generator(dev).manual_seed(seed + 7)
        s["q"] = torch.randn((int(n.sum()), case["hq"], D), generator=gen, device=dev).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(D)
        if own:
            kvq = s["kvq"]
            s["out"] = torch.empty_like(s["q"])
            s["ws"] = torch.zeros(max(256, kvq.kv_attn_tree_workspace_bytes(s["cfg"], len(s["q"]), s["max_ctx"])),
                                  dtype=torch.uint8, device=dev)
        return s
    if op == "verify":
        n = _counts(case, case["batch"])
        rows, vocab = int(n.sum()), case["vocab"]
        gen = torch.Generator(dev).manual_seed(seed)
        cu = np.concatenate([[0], np.cumsum(n)])
        parent = _parents(n, seed)
        logits = 2.5 * torch.randn((rows, vocab), generator=gen, device=dev)
        p = torch.softmax(logits, -1)
        q = torch.softmax(logits.add_(torch.randn((rows, vocab), generator=gen, device=dev), alpha=0.7), -1)
        del logits
        base = np.repeat(cu[:-1], n)
        of = torch.from_numpy(base + np.maximum(parent, 0)).to(dev)          # the row that a node was drafted from
        if case["dist"]:                                                     # sampled drafts (exponential race)
            token = torch.empty(rows, dtype=torch.int64, device=dev)
            for a in range(0, rows, 64):
                e = torch.empty((min(64, rows - a), vocab), device=dev).exponential_(generator=gen)
                token[a:a + 64] = (q[of[a:a + 64]] / e).argmax(-1)
        else:                                                                # the draft's best ones, one for each sibling
            order = np.zeros(rows, np.int64)
            seen = {}
            for i, k in enumerate((base + np.maximum(parent, 0)).tolist()):
                order[i] = seen.get(k, 0)
                seen[k] = order[i] + 1
            best = torch.topk(q, min(vocab, int(order.max()) + 1), dim=-1).indices
            token = best[of, torch.from_numpy(order).to(dev)]
        s = {"case": dict(case), "batch": case["batch"], "cu": _cu(n), "n_max": int(n.max()), "p": p, "q": q if case["dist"] else None,
             "parent": torch.from_numpy(parent).to(dev), "token": token.to(torch.int32),
             "u": torch.rand(rows, generator=gen, device=dev)}
        if own:
            import bit_rotated_kv_gb300 as kvq
            s["kvq"] = kvq
            s["cfg"] = kvq.KVConfig(n_q_heads=1, n_kv_heads=1, batch=case["batch"], max_pages_per_seq=1, num_pages=1, ring_cap=272)
            s["path"] = torch.empty(rows, dtype=torch.int32, device=dev)
            s["n_accept"] = torch.empty(case["batch"], dtype=torch.int32, device=dev)
            s["next"] = torch.empty(case["batch"], dtype=torch.int32, device=dev)
            s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        return s
    if op == "commit":
        lens = _lengths(case, case["batch"])
        n = np.full(case["batch"], case["nodes"])
        s = _cache(case, lens + n, n, seed, owned=np.zeros(case["batch"], bool))
        r = np.random.default_rng([seed, 5])
        path = np.full((case["batch"], case["nodes"]), -1, np.int32)
        for b in range(case["batch"]):
            rest = r.choice(np.arange(1, case["nodes"]), case["acc"] - 1, replace=False) if case["acc"] > 1 else []
            path[b, :case["acc"]] = np.sort(np.concatenate([[0], rest]))
        s["path"] = torch.from_numpy(path.reshape(-1)).to(dev)
        s["n_accept"] = torch.full((case["batch"],), case["acc"], dtype=torch.int32, device=dev)
        s["cu"] = _cu(n)
        s["drafted"] = s["seq_len"].clone()
        return s
    if op == "fork":
        batch = case["prompts"] * (1 + case["samples"])
        lens = _lengths(case, batch)
        first = np.arange(batch) < case["prompts"]
        lens = np.where(first, lens, lens // 4 + 1)                          # samples that were stopped early
        s = _cache(case, lens, np.zeros(batch, np.int64), seed, spare=2 * batch)
        src = np.repeat(np.arange(case["prompts"]), case["samples"]).astype(np.int32)
        s["src"] = torch.from_numpy(src).to(dev)
        s["dst"] = torch.arange(case["prompts"], batch, dtype=torch.int32, device=dev)
        return s
    batch = case["batch"]
    lens = _lengths(case, batch)
    s = _cache(case, lens, np.zeros(batch, np.int64), seed, hold=1)
    k = case["leave"]
    groups = [(np.arange(k) + g * k) % batch for g in range(-(-batch // k))]
    s["leave"] = [torch.from_numpy(g.astype(np.int32)).to(dev) for g in groups]
    s["admit"] = []
    for g in groups:
        t = np.zeros(batch, np.int32)
        t[g] = lens[g]
        s["admit"].append(torch.from_numpy(t).to(dev))
    s["turn"] = 0
    s["n_live"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if own:
        kvq = s["kvq"]
        s["ws"] = torch.zeros(max(256, kvq.kv_pages_compact_workspace_bytes(s["cfg"])), dtype=torch.uint8, device=dev)
    return s


# ---- the tree's attention in plain torch -----------------------------------------------------------
def _code_places():
    """Where code [token][channel] of a page stands among the 128 words x 16 slots of its keys, and
    of its values (slot s + 8 e: bits 2 s + 16 e of the word)."""
    w = torch.arange(128).view(128, 1)
    slot = torch.arange(16).view(1, 16)
    lane, r, s, e = w // 4, w % 4, slot % 8, slot // 8
    kt, kc = (lane // 4 + 8 * (r % 2)).expand(128, 16), 16 * s + 2 * (lane % 4) + 8 * (r // 2) + e
    vt, vc = (2 * (lane % 4) + 8 * (r // 2)) + e, 16 * s + lane // 4 + 8 * (r % 2)
    places = torch.empty((2, P * D), dtype=torch.int64)
    places[0, (kt * D + kc).flatten()] = torch.arange(2048)
    places[1, (vt * D + vc).flatten()] = torch.arange(2048)
    return places


_PLACES = _code_places()


def _dequantized(s):
    """Keys and values of every page-table entry in 32 bits: two of [B, Hkv, entries * 16, 128]."""
    dev, ng, group = s["pages"].device, D // s["group"], s["group"]
    table = s["table"].clamp(min=0).long()
    got = s["pages"][table].transpose(1, 2)                                 # [B, Hkv, entries, bytes]
    lead = got.shape[:3]
    slots = (2 * (torch.arange(16, device=dev, dtype=torch.int32) % 8) + 16 * (torch.arange(16, device=dev, dtype=torch.int32) // 8))
    places = _PLACES.to(dev)

    def codes(part):
        w = got[..., 512 * part:512 * part + 512].contiguous().view(torch.int32)
        c = ((w.unsqueeze(-1) >> slots) & 3).to(torch.uint8).flatten(-2)
        return c[..., places[part]].view(*lead, P, ng, group).float()

    half = lambda a, n: got[..., a:a + 2 * n].contiguous().view(torch.float16).float()  # noqa: E731
    ks = half(1024, 2 * P * ng).view(*lead, P, ng, 2)
    k = (codes(0) - ks[..., 1:]) * ks[..., :1]
    o = 1024 + 4 * P * ng
    if s["l2"]:
        k = k * half(o + 4 * P * ng, P).view(*lead, P, 1, 1)
    vs = half(o, 2 * P * ng).view(*lead, 2, P // 2, ng, 2).transpose(-1, -2)   # [.., D/z, pair, token, group]
    vs = vs.reshape(*lead, 2, P, ng, 1)
    v = (codes(1) - vs[..., 1, :, :, :]) * vs[..., 0, :, :, :]
    b, h, n = lead
    return k.reshape(b, h, n * P, D), v.reshape(b, h, n * P, D)


def _tree_plain(s):
    dev, batch, hkv, g = s["pages"].device, s["batch"], s["hkv"], s["gqa"]
    k2, v2 = _dequantized(s)
    length, edge = s["seq_len"].long().view(-1, 1), s["s_quant"].long().view(-1, 1)
    cu = s["cu"].long()
    n = (cu[1:] - cu[:-1]).view(-1, 1)
    edge = torch.minimum(edge, length)
    # the three regions side by side, each with its tokens' positions
    j = torch.arange(s["cap"], device=dev).view(1, -1)
    recent = torch.maximum(edge, torch.full_like(edge, s["sink"])) + j
    slot = (recent % s["cap"]).view(batch, 1, -1, 1).expand(-1, hkv, -1, D)
    sink = torch.arange(s["sink"], device=dev).view(1, -1).expand(batch, -1)
    mid = s["sink"] + torch.arange(k2.shape[2], device=dev).view(1, -1).expand(batch, -1)
    k = torch.cat([s["sink_k"][:, :, :s["sink"]].float(), k2, s["ring_k"].gather(2, slot).float()], 2)
    v = torch.cat([s["sink_v"][:, :, :s["sink"]].float(), v2, s["ring_v"].gather(2, slot).float()], 2)
    pos = torch.cat([sink, mid, recent], 1)
    live = torch.cat([sink < length, mid < edge, recent < length], 1)
    v = torch.where(live.view(batch, 1, -1, 1), v, 0.0)
    # ancestors of every node, itself among them, by repeated squaring
    i = torch.arange(s["n_max"], device=dev)
    row = torch.minimum(cu[:-1].view(-1, 1) + i, cu[-1] - 1)
    real = i.view(1, -1) < n
    parent = torch.where(real, s["parent"].long()[row], -1)
    reach = ((parent.unsqueeze(-1) == i) | torch.eye(len(i), dtype=torch.bool, device=dev)).float()
    for _ in range(max(1, (len(i) - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    local = pos - (length - n)                                              # < 0: before the drafts
    seen = torch.gather(reach, 2, local.clamp(0, len(i) - 1).unsqueeze(1).expand(-1, len(i), -1)) > 0
    seen = live.unsqueeze(1) & ((local < 0).unsqueeze(1) | seen)            # [B, nodes, tokens]
    q = s["q"].float()[row].view(batch, len(i), hkv, g, D).permute(0, 2, 1, 3, 4).reshape(batch, hkv, len(i) * g, D)
    sc = (q @ k.transpose(2, 3)) * s["scale"]
    sc = sc.masked_fill(~seen.unsqueeze(1).repeat_interleave(g, 2), -math.inf)
    w = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=-1e30))
    out = (w @ v) / w.sum(-1, keepdim=True)
    out = out.view(batch, hkv, len(i), g, D).permute(0, 2, 1, 3, 4).reshape(batch, len(i), hkv * g, D)
    at = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(cu, at, right=True) - 1
    return out[b, at - cu[b]].to(torch.bfloat16)


# ---- verification in plain torch, in units of 2^-60 ---------------------------------------------------
def _units(x):
    return (x.double().clamp(0, 1) * float(ONE)).long()


def _mul(a, b):
    """floor(a b / 2^60) of two int64 in [0, 2^61)."""
    m = (1 << 30) - 1
    ah, al, bh, bl = a >> 30, a & m, b >> 30, b & m
    return ah * bh + ((ah * bl + al * bh + ((al * bl) >> 30)) >> 30)


def _verify_plain(s):
    dev, batch = s["p"].device, s["batch"]
    cu = s["cu"].long()
    n, first = cu[1:] - cu[:-1], cu[:-1]
    last = s["p"].shape[0] - 1
    pick = lambda w, x: w.gather(1, x.view(-1, 1)).view(-1)  # noqa: E731
    unit = _units(s["u"])
    cur = torch.zeros(batch, dtype=torch.int64, device=dev)
    left = _units(s["p"][first.clamp(max=last)])                        # weights of the current node
    mass = torch.full((batch,), ONE, dtype=torch.int64, device=dev)
    ended = torch.zeros(batch, dtype=torch.bool, device=dev)
    path = torch.full((s["p"].shape[0] + 1,), -1, dtype=torch.int32, device=dev)
    depth = (n > 0).long()
    path.scatter_(0, torch.where(n > 0, first, last + 1), 0)
    path[-1] = -1
    for c in range(1, s["n_max"]):
        row = (first + c).clamp(max=last)
        tried = (c < n) & (s["parent"].long()[row] == cur) & ~ended
        x = s["token"].long()[row]
        weight = pick(left, x)
        at = (first + cur).clamp(max=last)
        if s["q"] is None:
            want = mass
        else:
            want = _mul(mass, pick(_units(s["q"][at].gather(1, x.view(-1, 1))), torch.zeros_like(x)))
        taken = tried & (_mul(unit[row], want) < weight)
        missed = tried & ~taken
        if s["q"] is None:
            less = left.scatter(1, x.view(-1, 1), 0)
            less_mass = (mass - weight).clamp(min=0)
        else:
            less = (left - _mul(mass.view(-1, 1), _units(s["q"][at]))).clamp(min=0)
            less_mass = less.sum(1)
        gone = missed & (less_mass == 0)
        whole = _units(s["p"][at])
        fresh = _units(s["p"][row])
        left = torch.where(taken.view(-1, 1), fresh, torch.where(gone.view(-1, 1), whole, torch.where(missed.view(-1, 1), less, left)))
        mass = torch.where(taken, torch.full_like(mass, ONE), torch.where(missed, less_mass, mass))
        ended = (ended | gone) & ~taken
        cur = torch.where(taken, torch.full_like(cur, c), cur)
        path.scatter_(0, torch.where(taken, first + depth, last + 1), c)
        path[-1] = -1
        depth = depth + taken.long()
    total = left.sum(1)
    left = torch.where((total == 0).view(-1, 1), _units(s["p"][(first + cur).clamp(max=last)]), left)
    upto = left.cumsum(1)
    goal = _mul(unit[first.clamp(max=last)], upto[:, -1])
    token = torch.searchsorted(upto, goal.view(-1, 1), right=True).view(-1)
    return path[:-1], depth.to(torch.int32), torch.where(n > 0, token, -1).to(torch.int32)


# ---- the cache's rows and pages in plain torch ---------------------------------------------------------
def _commit_plain(s):
    dev, batch = s["seq_len"].device, s["batch"]
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    j = torch.arange(int(s["case"]["nodes"]), device=dev).view(1, -1)
    kept = j < s["n_accept"].long().view(-1, 1)
    path = torch.where(kept, s["path"].long()[(cu[:-1].view(-1, 1) + j).clamp(max=len(s["path"]) - 1)], j)
    start = (s["seq_len"].long() - n).view(-1, 1)
    b = torch.arange(batch, device=dev).view(-1, 1)
    read, write = (start + path) % s["cap"], (start + j) % s["cap"]
    for name in ("ring_k", "ring_v"):
        s[name][b, :, write] = s[name][b, :, read]
    s["seq_len"].copy_(s["seq_len"].long() - n + s["n_accept"].long())


def _count(at, by, size):
    return torch.zeros(size, dtype=torch.int32, device=at.device).index_add_(0, at.flatten(), by.flatten().to(torch.int32))


def _free_plain(s, seqs):
    seqs = seqs.long()
    rows = s["table"][seqs].long()
    s["ref"] -= _count(rows.clamp(min=0), rows >= 0, len(s["ref"]))
    s["table"][seqs] = -1
    s["seq_len"][seqs] = 0
    s["s_quant"][seqs] = s["sink"]


def _lowest_free(s):
    """How many of the pages up to each one are free: the k-th free page is where this reaches k + 1."""
    return (s["ref"][:s["num_pages"]] == 0).long().cumsum(0)


def _fork_plain(s):
    src, dst = s["src"].long(), s["dst"].long()
    _free_plain(s, dst)
    spare = s["num_pages"]
    tokens = s["s_quant"][src].long() - s["sink"]
    full, part = tokens // P, tokens % P > 0
    col = torch.arange(s["maxp"], device=src.device).view(1, -1)
    rows = torch.where(col < full.view(-1, 1), s["table"][src].long(), -1)
    s["ref"] += _count(rows.clamp(min=0), rows >= 0, len(s["ref"]))
    new = torch.searchsorted(_lowest_free(s), part.long().cumsum(0))        # the next free page for each that needs one
    new = torch.where(part, new, spare)
    old = torch.where(part, s["table"][src, full.clamp(max=s["maxp"] - 1)].long(), spare)
    s["pages"][new] = s["pages"][old]
    s["ref"][new] = 1
    s["table"][dst] = torch.where((col == full.view(-1, 1)) & part.view(-1, 1), new.view(-1, 1), rows).to(torch.int32)
    length, edge = s["seq_len"][src].long().view(-1, 1), s["s_quant"][src].long().view(-1, 1)
    slot = torch.arange(s["cap"], device=src.device).view(1, -1)
    live = (slot - edge) % s["cap"] < length - edge
    for name in ("ring_k", "ring_v"):
        s[name][dst] = torch.where(live.view(len(src), 1, -1, 1), s[name][src], s[name][dst])
    for name in ("sink_k", "sink_v"):
        live = torch.arange(s[name].shape[2], device=src.device).view(1, -1) < length.clamp(max=s["sink"])
        s[name][dst] = torch.where(live.view(len(src), 1, -1, 1), s[name][src], s[name][dst])
    s["seq_len"][dst] = s["seq_len"][src]
    s["s_quant"][dst] = s["s_quant"][src]


def _compact_plain(s, most):
    spare, n = s["num_pages"], s["num_pages"]
    ref = s["ref"][:n]
    page = torch.arange(n, device=ref.device)
    n_live = (ref > 0).sum()
    mover, hole = (ref > 0) & (page >= n_live), (ref == 0) & (page < n_live)
    k = torch.arange(most, device=ref.device)
    real = k < mover.sum()
    source = torch.searchsorted(mover.long().cumsum(0), k + 1)
    target = torch.searchsorted(hole.long().cumsum(0), k + 1)
    source, target = torch.where(real, source, spare), torch.where(real, target, spare)
    s["pages"][target] = s["pages"][source]
    where = torch.arange(n + 1, device=ref.device)
    where[source] = target
    s["table"].copy_(torch.where(s["table"] >= 0, where[s["table"].clamp(min=0).long()], -1))
    s["ref"][target] = s["ref"][source]
    s["ref"][source] = 0
    s["n_live"].copy_(n_live)


def _reserve_plain(s, tokens):
    spare = s["num_pages"]
    have = (s["table"] >= 0).sum(1)
    need = torch.where(tokens > 0, -(-(s["seq_len"].long() + tokens - s["sink"]) // P) - have, 0).clamp(min=0)
    end = need.cumsum(0)
    free = _lowest_free(s)
    need = torch.where(end <= free[-1], need, 0)
    col = torch.arange(s["maxp"], device=tokens.device).view(1, -1)
    i = col - have.view(-1, 1)
    mine = (i >= 0) & (i < need.view(-1, 1))
    page = torch.searchsorted(free, torch.where(mine, (end - need).view(-1, 1) + i + 1, 1))
    page = torch.where(mine, page, spare)
    s["table"].copy_(torch.where(mine, page, s["table"].long()))
    s["ref"][page.flatten()] = 1
    s["ref"][spare] = 0


# ---- one pass ------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    kvq = s.get("kvq") if own else None
    if op == "tree":
        if not own:
            return _tree_plain(s)
        kvq.kv_attn_tree(s["cfg"], s["cache"], s["q"], s["cu"], s["parent"], s["out"], s["scale"], s["max_ctx"], s["ws"], s["status"])
        return s["out"]
    if op == "verify":
        if not own:
            return _verify_plain(s)
        kvq.kv_verify_tree(s["cfg"], s["cu"], s["parent"], s["token"], s["p"], s["q"], s["u"], s["path"], s["n_accept"], s["next"],
                           s["status"])
        return s["path"], s["n_accept"], s["next"]
    if op == "commit":
        s["seq_len"].copy_(s["drafted"])                                    # (the drafts are appended again)
        if own:
            kvq.kv_tree_commit(s["cfg"], s["cache"], s["cu"], s["path"], s["n_accept"], s["status"])
        else:
            _commit_plain(s)
        return s["ring_k"].view(torch.int16), s["ring_v"].view(torch.int16), s["seq_len"]
    n = s["num_pages"]
    if op == "fork":
        if own:
            kvq.kv_seq_free(s["cfg"], s["cache"], s["ref"], s["dst"], s["status"])
            kvq.kv_seq_fork(s["cfg"], s["cache"], s["ref"], s["src"], s["dst"], s["status"])
        else:
            _fork_plain(s)
            s["ref"][n] = 0
        return (s["pages"][:n], s["table"], s["ref"][:n], s["seq_len"], s["s_quant"],
                *(s[k].view(torch.int16) for k in ("sink_k", "sink_v", "ring_k", "ring_v")))
    turn = s["turn"]
    s["turn"] = (turn + 1) % len(s["leave"])
    if own:
        kvq.kv_seq_free(s["cfg"], s["cache"], s["ref"], s["leave"][turn], s["status"])
        kvq.kv_pages_compact(s["cfg"], s["cache"], s["ref"], s["n_live"], s["ws"], s["status"])
        kvq.kv_pages_reserve(s["cfg"], s["cache"], s["ref"], s["admit"][turn], s["status"])
    else:
        _free_plain(s, s["leave"][turn])
        _compact_plain(s, s["maxp"] * len(s["leave"][turn]))
        s["ref"][n] = 0
        _reserve_plain(s, s["admit"][turn].long())
    return s["pages"][:n], s["table"], s["ref"][:n], s["seq_len"], s["s_quant"], s["n_live"]


# ---- what a pass cannot do without ---------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "verify":                       # the last node's target row, and its draft row where one was rejected
        return {"bytes": case["batch"] * case["vocab"] * 4 * (2 if case["dist"] else 1) + 16 * case["batch"] * case["nodes"], "flops": 0}
    if op == "commit":                       # the rows that move, read and written
        return {"bytes": case["batch"] * max(1, case["acc"] - 1) * case["hkv"] * D * 2 * 2 * 2 + 8 * case["batch"] * case["nodes"], "flops": 0}
    row = D * 2 * 2                          # a token's key and value in 16 bits
    mean = (case["lo"] + case["hi"]) / 2
    edge = float(_edge(np.int64(mean), case))
    head = _head_bytes(case.get("group", 128), case.get("l2", False))
    if op == "tree":
        n = case["nodes"] if case["batch"] == 1 else 0.75 * case["nodes"]
        b, hkv, hq = case["batch"], case["hkv"], case["hq"]
        window = min(mean, case["sink"]) + mean + n - edge
        cache = b * hkv * ((edge - case["sink"]) / P * head + window * row) + b * (edge - case["sink"]) / P * 4
        return {"bytes": cache + b * n * hq * D * 2 * 2, "flops": 4.0 * b * hq * n * (mean + n / 2) * D}
    if op == "fork":
        n = case["prompts"] * case["samples"]
        window = min(mean, case["sink"]) + mean - edge
        return {"bytes": n * (case["hkv"] * (2 * window * row + 2 * head) + 4 * 4 * edge / P), "flops": 0}
    gone = case["leave"] * (mean - case["sink"]) / P
    share = 1 - case["leave"] / case["batch"]
    return {"bytes": gone * share * 2 * head * case["hkv"] + 8 * case["batch"] * mean / P, "flops": 0}


# ---- the tree's attention from its definition, in 64 bits ------------------------------------------------
def exact(case, seed):
    if case["op"] != "tree":
        return None                                                         # whole numbers and copies
    s = prepare(case, seed)
    dev, ng, group = s["pages"].device, D // s["group"], s["group"]
    t, c = torch.arange(P, device=dev).view(P, 1), torch.arange(D, device=dev).view(1, D)
    # the word and the bit of key code (t, c) and of value code (t, c)
    kw = 4 * (4 * (t % 8) + (c % 8) // 2) + t // 8 + 2 * ((c % 16) // 8)
    kb = 2 * (c // 16) + 16 * (c % 2) + 0 * t
    vw = 4 * (4 * (c % 8) + (t % 8) // 2) + (c % 16) // 8 + 2 * (t // 8)
    vb = 2 * (c // 16) + 16 * (t % 2)
    lens, edges, cu = s["seq_len"].tolist(), s["s_quant"].tolist(), s["cu"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    for b in range(s["batch"]):
        lo, n = lens[b] - (cu[b + 1] - cu[b]), cu[b + 1] - cu[b]
        parent = s["parent"][cu[b]:cu[b + 1]].tolist()
        sees = torch.zeros((n, lens[b]), dtype=torch.bool)
        sees[:, :lo] = True
        for i in range(n):
            at = i
            while at >= 0:
                sees[i, lo + at] = True
                at = parent[at]
        sees = sees.to(dev)
        a, e = min(s["sink"], lens[b]), min(edges[b], lens[b])
        ids = s["table"][b, :-(-(e - a) // P)].long()
        recent = (torch.arange(e, lens[b], device=dev) % s["cap"])
        for h in range(s["hkv"]):
            page = s["pages"][ids, h]
            word = page[:, :1024].contiguous().view(torch.int32)
            f = page[:, 1024:].contiguous().view(torch.float16).double()
            kp = f[:, :2 * P * ng].view(-1, P, ng, 2)
            k = ((word[:, :128][:, kw] >> kb) & 3).double()
            k = kp[..., 0].repeat_interleave(group, 2) * (k - kp[..., 1].repeat_interleave(group, 2))
            if s["l2"]:
                k = k * f[:, 4 * P * ng:4 * P * ng + P].unsqueeze(-1)
            vp = f[:, 2 * P * ng:4 * P * ng].view(-1, 2, P // 2, ng, 2)
            v = ((word[:, 128:][:, vw] >> vb) & 3).double()
            dz = [vp[:, x].permute(0, 1, 3, 2).reshape(-1, P, ng).repeat_interleave(group, 2) for x in (0, 1)]
            v = dz[0] * (v - dz[1])
            k = torch.cat([s["sink_k"][b, h, :a].double(), k.reshape(-1, D)[:e - a], s["ring_k"][b, h, recent].double()])
            v = torch.cat([s["sink_v"][b, h, :a].double(), v.reshape(-1, D)[:e - a], s["ring_v"][b, h, recent].double()])
            q = s["q"][cu[b]:cu[b + 1], h * s["gqa"]:(h + 1) * s["gqa"]].double()
            x = torch.einsum("ngd,td->ngt", q, k) / math.sqrt(D)
            x = torch.where(sees.unsqueeze(1), x, -math.inf)
            out[cu[b]:cu[b + 1], h * s["gqa"]:(h + 1) * s["gqa"]] = torch.softmax(x, -1) @ v
    return out
