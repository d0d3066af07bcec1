"""A step over many requests at once, as cases with real sizes: keys and values appended to each request's
pages with the rotation applied on the way, attention for trees of drafted tokens over the cache, the
acceptance of a tree's path, and low-rank adapters of many requests beside a shared projection. What each
operator computes in its plain form, what the framework's calls compute, and the exact values in 64 bits.

The rows of request b are rows[b] .. rows[b + 1] - 1 of the row arrays. Row i of a request is a node of its
tree: parent[i] < i is the node before it, -1 stands for the cached positions. A node lies in the cache at
position start + i, is rotated by start + its depth and sees the cached positions, its ancestors and itself.
Without parents the rows are a chain. One cache (K or V) is [n_layers][nkv][slots][hd]; a paged cache's slot
of request b's position p is table[b][p / 128] * 128 + p % 128.
"""
import math
import random

import torch

own = False

PAGE = 128
N_LAYERS = 2
THETA, EPS = 1e6, 1e-6
VOCAB = 151936


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request's next token shortly after a 512-token prompt: the smallest call, latency counts
        attention("decode_1_at_512", "bf16", 32, 8, 128, 1, (1, 1), (512, 512), False),
        # the next token of 48 requests of very different lengths
        attention("decode_48_ragged", "bf16", 32, 8, 128, 48, (1, 1), (300, 8100), True),
        # one request's tree of 26 drafted tokens at an odd position
        attention("tree_26_at_8k", "f16", 32, 8, 128, 1, (26, 26), (8189, 8189), True),
        # ragged trees on a small model with one query head to each kv head
        attention("trees_5_mha64", "f16", 8, 8, 64, 5, (7, 40), (1, 1500), True),
        # trees of up to 64 nodes of eight requests late in long documents: the largest call
        attention("trees_8_at_32k", "bf16", 32, 8, 128, 8, (40, 64), (20000, 32700), True),
        # one decoded token's keys and values
        append("append_1", "bf16", 32, 8, 128, 1, (1, 1), (517, 517), False, True, True),
        # chunks of four requests' prompts at once, starting and ending inside pages
        append("append_prompts", "f16", 32, 8, 128, 4, (300, 512), (0, 3000), True, False, False),
        # the cache's part of one request's verified tree: its rows appended, the accepted path moved up
        accept("accept_1", "bf16", 32, 8, 128, 1, (26, 26), (1001, 1001), True),
        # the same for 16 requests
        accept("accept_16", "bf16", 32, 8, 128, 16, (31, 61), (100, 2000), True),
        # one request's adapter beside the output projection of one token
        adapters("adapter_1", 4096, 4096, 16, 1, (1, 1), 1),
        # next tokens of 24 requests with 16 adapters among them, beside the QKV projection
        adapters("adapters_24", 4096, 6144, 16, 24, (1, 1), 16),
        # chunks of four requests' prompts beside the down projection
        adapters("adapters_prompts", 12288, 4096, 64, 4, (300, 700), 3),
    ]


def attention(name, kv, nq, nkv, hd, seqs, rows, start, paged):
    return {"name": name, "op": "attention", "kv": kv, "nq": nq, "nkv": nkv, "hd": hd, "seqs": seqs, "rows_lo": rows[0],
            "rows_hi": rows[1], "start_lo": start[0], "start_hi": start[1], "paged": paged, "tree": True}


def append(name, kv, nq, nkv, hd, seqs, rows, start, paged, norm, tree):
    return {**attention(name, kv, nq, nkv, hd, seqs, rows, start, paged), "op": "append", "norm": norm, "tree": tree}


def accept(name, kv, nq, nkv, hd, seqs, rows, start, paged):
    return {**append(name, kv, nq, nkv, hd, seqs, rows, start, paged, True, True), "op": "accept"}


def adapters(name, k, n, rank, seqs, rows, count):
    return {"name": name, "op": "adapters", "k": k, "n": n, "rank": rank, "seqs": seqs, "rows_lo": rows[0], "rows_hi": rows[1], "count": count}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "accept", "adapters", "adapters"])
    if op == "adapters":
        seqs = _log(rng, 1, 64)
        hi = max(1, min(_log(rng, 1, 700), 2000 // seqs))
        lo = rng.randint(0 if seqs > 1 else 1, hi)
        k, n = (16 * _log(rng, 16, 768) for _ in "kn")
        c = adapters("", k, n, 8 * rng.choice([1, 2, 2, 3, 4, 8]), seqs, (lo, hi), rng.randint(1, 16))
    else:
        kv, paged = rng.choice(["bf16", "f16"]), rng.random() < 0.8
        nq, nkv, hd = rng.choice([(32, 8, 128), (32, 8, 128), (4, 2, 64), (8, 8, 64), (16, 1, 128), (32, 4, 128), (64, 8, 128)])
        seqs = _log(rng, 1, 48) if paged else 1
        hi = rng.choice([1, _log(rng, 2, 64), _log(rng, 2, 64)])
        lo = rng.randint(0 if seqs > 1 and hi > 1 else 1, hi)
        top = min(_log(rng, 1, 32700), 200000 // seqs, 8 * 50 * 25000 // (seqs * hi))
        start = (rng.randint(0, top), top)
        if op == "attention":
            c = attention("", kv, nq, nkv, hd, seqs, (lo, hi), start, paged)
        else:
            start = tuple(min(x, 4000) for x in start)
            c = {"append": append, "accept": lambda *a: accept(*a[:-2])}[op]("", kv, nq, nkv, hd, seqs, (lo, hi), start, paged, rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ what follows from a case alone
def _spread(lo, hi, i, seqs):
    """The i-th of `seqs` sizes between lo and hi, both of them taken, in no order."""
    if seqs == 1:
        return hi
    return lo + (hi - lo) * ((i * 7 + 3) % seqs if seqs % 7 else i) // (seqs - 1)


def _sizes(c):
    """(rows of each request, positions that the cache holds of each before)."""
    n = [_spread(c["rows_lo"], c["rows_hi"], b, c["seqs"]) for b in range(c["seqs"])]
    if "start_lo" not in c:
        return n, None
    return n, [_spread(c["start_lo"], c["start_hi"], c["seqs"] - 1 - b, c["seqs"]) for b in range(c["seqs"])]


def _geometry(c):
    """(positions of the longest request, pages of a request, pages of the pool, slots of a head)."""
    n, start = _sizes(c)
    max_seq = max(s + r for s, r in zip(start, n)) + 37
    pages = -(-max_seq // PAGE)
    if not c["paged"]:
        return max_seq, pages, 0, max_seq
    pool = sum(-(-(s + r) // PAGE) for s, r in zip(start, n)) + 3
    return max_seq, pages, pool, pool * PAGE


def _adapter_of(c):
    """The adapter of each request, -1 for one without."""
    return [-1 if b % 8 == 5 else (b * 5 + 1) % c["count"] for b in range(c["seqs"])]


def _dtype(c):
    return torch.bfloat16 if c["kv"] == "bf16" else torch.float16


# ------------------------------------------------------------------ inputs
def _tree(rng, n):
    """Parents of a drafted tree: the root, then nodes that hang on recent ones, several to one parent."""
    return [-1 if i == 0 else rng.randint(max(0, (i - 1) // 3 - 2), max(0, (i - 1) // 2)) for i in range(n)]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    rng = random.Random(seed * 7919 + 31)
    n, start = _sizes(c)
    begin = [0]
    for r in n:
        begin.append(begin[-1] + r)
    total = begin[-1]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    s = {"case": c, "n": n, "start": start, "begin": begin, "begin_dev": ints(begin)}
    if c["op"] == "adapters":
        s["x"] = normal(total, c["k"]).half()
        s["base"] = normal(total, c["n"])
        s["a"] = (normal(c["count"], c["rank"], c["k"]) * c["k"] ** -0.5).half()
        s["b"] = (normal(c["count"], c["n"], c["rank"]) * 0.1).half()
        s["scale"] = 0.5 + 2 * torch.rand(c["count"], device="cuda", generator=gen)
        s["adapter"] = _adapter_of(c)
        s["adapter_dev"] = ints(s["adapter"])
        return s
    max_seq, pages, pool, slots = _geometry(c)
    nq, nkv, hd, dt = c["nq"], c["nkv"], c["hd"], _dtype(c)
    s["start_dev"] = ints(start)
    s["parent"] = [p for r in n for p in (_tree(rng, r) if c["tree"] else range(-1, r - 1))]
    s["parent_dev"] = ints(s["parent"]) if c["tree"] else None
    s["table"] = None
    if c["paged"]:  # each request's pages anywhere in the pool, -1 where it has none
        order = torch.randperm(pool, device="cuda", generator=gen).int()
        s["table"] = torch.full((c["seqs"], pages), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b in range(c["seqs"]):
            own_pages = -(-(start[b] + n[b]) // PAGE)
            s["table"][b, :own_pages] = order[at:at + own_pages]
            at += own_pages
    for w in ("k", "v"):  # a few heavy channels in K; slots that nobody uses hold anything
        cache = torch.randn(N_LAYERS, nkv, slots, hd, device="cuda", generator=gen, dtype=dt)
        if w == "k":
            cache *= 1 + 5 * (torch.rand(nkv, 1, hd, device="cuda", generator=gen) > 0.96).to(dt)
        s[w + "_cache"] = cache
    if c["op"] == "attention":
        s["q"] = (normal(total, nq, hd) * (0.5 + 2 * torch.rand(nq, 1, device="cuda", generator=gen))).to(dt)
        return s
    s["qkv"] = [normal(total, (nq + 2 * nkv) * hd) * 2 for _ in range(N_LAYERS if c["op"] == "accept" else 1)]
    s["qn"], s["kn"] = (1 + 0.1 * normal(2, hd)) if c["norm"] else (None, None)
    freq = THETA ** (-torch.arange(0, hd, 2, device="cuda", dtype=torch.float64) / hd)
    angle = torch.arange(max_seq, device="cuda", dtype=torch.float64)[:, None] * freq
    s["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float()
    if c["op"] == "accept":
        # most predictions are the token of one of the node's children, the others anything
        tokens = [rng.randrange(VOCAB) for _ in range(total)]
        ids = [rng.randrange(VOCAB) for _ in range(total)]
        for b in range(c["seqs"]):
            kids = {}
            for i in range(n[b]):
                kids.setdefault(s["parent"][begin[b] + i], []).append(i)
            for i in range(n[b]):
                if i in kids and rng.random() < 0.85:
                    ids[begin[b] + i] = tokens[begin[b] + rng.choice(kids[i])]
        s["tokens"], s["ids"] = ints(tokens), ints(ids)
        s["root"] = ints([tokens[begin[b]] if n[b] else rng.randrange(VOCAB) for b in range(c["seqs"])])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    return {"attention": run_attention, "append": run_append, "accept": run_accept, "adapters": run_adapters}[c["op"]](c, state)


_plans = {}


def _plan(c, s):
    """What a user's program keeps: the configuration, the workspace and the status word of these sizes, and the batch."""
    from quantized_transformer_prefill_q1_gb300 import pf

    key = tuple(sorted((k, v) for k, v in c.items() if k != "name"))
    if key not in _plans:
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        if c["op"] == "adapters":
            _plans[key] = pf, None, None, status
        else:
            max_seq, _, pool, _ = _geometry(c)
            cfg = pf.pf_config(hidden=128, intermediate=128, n_q_heads=c["nq"], n_kv_heads=c["nkv"], head_dim=c["hd"], n_layers=N_LAYERS,
                               rope_theta=THETA, eps=EPS, final_eps=EPS, qk_norm=int(c.get("norm", False)),
                               kv_dtype=pf.KV_BF16 if c["kv"] == "bf16" else pf.KV_F16, max_seq=max_seq, max_chunk=512, kv_block_pool=pool)
            scratch = pf.attention_tree_scratch(cfg, c["seqs"], c["rows_hi"]) if c["op"] == "attention" else None
            _plans[key] = pf, cfg, scratch, status
    pf, cfg, scratch, status = _plans[key]
    if "batch" not in s:
        s["batch"] = pf.Batch(s["begin_dev"], n_rows=s["begin"][-1], max_rows=c["rows_hi"], start=s.get("start_dev"), parent=s.get("parent_dev"), blocks=s.get("table"))
    return pf, cfg, s["batch"], scratch, status


def _slots(s, b, lo, hi):
    p = torch.arange(lo, hi, device="cuda")
    return p if s["table"] is None else s["table"][b].long()[p // PAGE] * PAGE + p % PAGE


def _ancestors(parent):
    """[n, n] truth values on the GPU: whether node j is node i or before it."""
    n = len(parent)
    see = torch.zeros(n, n, dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
    return see.cuda()


def run_attention(c, s):
    nq, nkv, hd = c["nq"], c["nkv"], c["hd"]
    if own:
        pf, cfg, batch, scratch, status = _plan(c, s)
        out = torch.empty(s["begin"][-1], nq * hd, dtype=torch.float16, device="cuda")
        pf.pf_op_attention_tree(cfg, batch, s["q"], s["k_cache"], s["v_cache"], 1, out, scratch, status)
        return out
    out = []
    for b, n in enumerate(s["n"]):
        if n == 0:
            continue
        at, start = s["begin"][b], s["start"][b]
        i = _slots(s, b, 0, start + n)
        k, v = (s[w][1][:, i].float() for w in ("k_cache", "v_cache"))
        q = s["q"][at:at + n].float().view(n, nkv, nq // nkv, hd).permute(1, 0, 2, 3).reshape(nkv, -1, hd)
        x = (q @ k.transpose(1, 2)).view(nkv, n, nq // nkv, start + n) * hd ** -0.5
        see = torch.ones(n, start + n, dtype=torch.bool, device="cuda")
        see[:, start:] = _ancestors(s["parent"][at:at + n])
        x = torch.where(see[:, None], x, -math.inf)
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = (p / p.sum(-1, keepdim=True)).view(nkv, -1, start + n)
        out.append((p @ v).view(nkv, n, nq // nkv, hd).permute(1, 0, 2, 3).reshape(n, nq * hd))
    return torch.cat(out).half()


def _depths(c, s):
    """[rows] on the GPU: how many nodes lie before each one."""
    deep = []
    for at, end in zip(s["begin"], s["begin"][1:]):
        d = []
        for p in s["parent"][at:end]:
            d.append(0 if p < 0 else d[p] + 1)
        deep += d
    return torch.tensor(deep, device="cuda")


def _plain_append(c, s, layer, qkv):
    """Norm, rotation and store of one layer's rows; returns q."""
    nq, nkv, hd = c["nq"], c["nkv"], c["hd"]
    total = s["begin"][-1]
    x = qkv.view(total, nq + 2 * nkv, hd)
    first = torch.cat([torch.full((n,), p, device="cuda") for n, p in zip(s["n"], s["start"])])
    cs = s["rope"][first + _depths(c, s)][:, None]
    heads = []
    for part, w in ((x[:, :nq], s["qn"]), (x[:, nq:nq + nkv], s["kn"])):
        if w is not None:
            part = part * torch.rsqrt((part * part).mean(-1, keepdim=True) + EPS) * w
        lo, hi = part[..., :hd // 2], part[..., hd // 2:]
        heads.append(torch.cat((lo * cs[..., 0] - hi * cs[..., 1], hi * cs[..., 0] + lo * cs[..., 1]), -1).to(_dtype(c)))
    slot = torch.cat([_slots(s, b, p, p + n) for b, (n, p) in enumerate(zip(s["n"], s["start"]))])
    s["k_cache"][layer][:, slot] = heads[1].permute(1, 0, 2)
    s["v_cache"][layer][:, slot] = x[:, nq + nkv:].permute(1, 0, 2).to(_dtype(c))
    return heads[0]


def run_append(c, s):
    if own:
        pf, cfg, batch, _, status = _plan(c, s)
        q = torch.empty(s["begin"][-1], c["nq"], c["hd"], dtype=_dtype(c), device="cuda")
        pf.pf_op_batch_append(cfg, batch, s["qkv"][0], s["qn"], s["kn"], s["rope"], 1, q, s["k_cache"], s["v_cache"], status)
    else:
        q = _plain_append(c, s, 1, s["qkv"][0])
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def run_accept(c, s):
    """Every layer's rows appended, then the path that the predictions accept moved up in all layers."""
    total = s["begin"][-1]
    if own:
        pf, cfg, batch, _, status = _plan(c, s)
        q = torch.empty(total, c["nq"], c["hd"], dtype=_dtype(c), device="cuda")
        for layer in range(N_LAYERS):
            pf.pf_op_batch_append(cfg, batch, s["qkv"][layer], s["qn"], s["kn"], s["rope"], layer, q, s["k_cache"], s["v_cache"], status)
        path, count, after = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (total, c["seqs"], c["seqs"]))
        pf.pf_op_tree_accept(cfg, batch, s["tokens"], s["ids"], s["root"], path, count, after, s["k_cache"], s["v_cache"], status)
        return {"path": path, "count": count, "next": after, "k": s["k_cache"], "v": s["v_cache"]}
    for layer in range(N_LAYERS):
        _plain_append(c, s, layer, s["qkv"][layer])
    tokens, ids, root = (s[w].tolist() for w in ("tokens", "ids", "root"))
    paths, counts, after = [], [], []
    for b, n in enumerate(s["n"]):
        at = s["begin"][b]
        want, node, path = root[b], -1, []
        for i in range(n):  # children come after their parents: one walk in order of the nodes
            if s["parent"][at + i] == node and tokens[at + i] == want:
                path.append(i)
                node, want = i, ids[at + i]
        if path:
            slot = _slots(s, b, s["start"][b], s["start"][b] + n)
            for w in ("k_cache", "v_cache"):
                s[w][:, :, slot[:len(path)]] = s[w][:, :, slot[path]]
        paths += path + [-1] * (n - len(path))
        counts.append(len(path))
        after.append(want)
    got = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (paths, counts, after)]
    return {"path": got[0], "count": got[1], "next": got[2], "k": s["k_cache"], "v": s["v_cache"]}


def run_adapters(c, s):
    if own:
        pf, _, batch, _, status = _plan(c, s)
        out = torch.empty_like(s["base"])
        pf.pf_op_adapters(batch, s["x"], s["base"], out, s["adapter_dev"], s["a"], s["b"], s["scale"], status)
        return out
    out = s["base"].clone()
    for b, a in enumerate(s["adapter"]):
        rows = slice(s["begin"][b], s["begin"][b + 1])
        if a >= 0:
            out[rows] += s["scale"][a] * (s["x"][rows].float() @ s["a"][a].float().T) @ s["b"][a].float().T
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    n, start = _sizes(c)
    total = sum(n)
    if c["op"] == "adapters":
        m = sum(r for r, a in zip(n, _adapter_of(c)) if a >= 0)
        used = len({a for r, a in zip(n, _adapter_of(c)) if a >= 0 and r})
        return {"bytes": 2 * m * c["k"] + 8 * total * c["n"] + 2 * used * c["rank"] * (c["k"] + c["n"]), "flops": 2 * m * c["rank"] * (c["k"] + c["n"])}
    heads = (c["nq"] + 2 * c["nkv"]) * c["hd"]
    if c["op"] == "attention":
        keys = sum(s + r for s, r in zip(start, n) if r)
        pairs = sum(r * (s + 1) for s, r in zip(start, n))
        return {"bytes": 4 * c["nkv"] * c["hd"] * keys + 4 * total * c["nq"] * c["hd"], "flops": 4 * c["nq"] * c["hd"] * pairs}
    one = {"bytes": 6 * total * heads + 4 * total * c["hd"], "flops": 8 * total * heads}
    if c["op"] == "append":
        return one
    # what the accepted paths move depends on the tokens: at most 8 nkv hd bytes a node and layer, not counted
    return {"bytes": N_LAYERS * one["bytes"] + 16 * total, "flops": N_LAYERS * one["flops"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _place(s, b, p):
    return p if s["table"] is None else int(s["table"][b, p // PAGE]) * PAGE + p % PAGE


def _line(s, b, i):
    """Node i of request b and the nodes before it, the root's first."""
    line = []
    while i >= 0:
        line.append(i)
        i = s["parent"][s["begin"][b] + i]
    return line[::-1]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "adapters":
        out = s["base"].double()
        for b, a in enumerate(s["adapter"]):
            for r in range(s["begin"][b], s["begin"][b + 1]) if a >= 0 else ():
                out[r] += s["scale"][a].double() * torch.mv(s["b"][a].double(), torch.mv(s["a"][a].double(), s["x"][r].double()))
        return out
    nq, nkv, hd = c["nq"], c["nkv"], c["hd"]
    if c["op"] == "attention":
        out = torch.empty(s["begin"][-1], nq, hd, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["n"]):
            if n == 0:
                continue
            end = s["start"][b] + n
            hidden = torch.full((n, end), -math.inf, dtype=torch.float64)
            hidden[:, :s["start"][b]] = 0
            for i in range(n):
                hidden[i, [s["start"][b] + j for j in _line(s, b, i)]] = 0
            hidden = hidden.cuda()
            pages = [_place(s, b, p) for p in range(0, end, PAGE)]
            for g in range(nkv):
                k, v = (torch.cat([s[w][1, g, p:p + PAGE] for p in pages])[:end].double() for w in ("k_cache", "v_cache"))
                for h in range(g * (nq // nkv), (g + 1) * (nq // nkv)):
                    score = s["q"][s["begin"][b]:s["begin"][b] + n, h].double() @ k.T / math.sqrt(hd) + hidden
                    out[s["begin"][b]:s["begin"][b] + n, h] = torch.softmax(score, -1) @ v
        return out.view(-1, nq * hd)
    got = {w: s[w + "_cache"].double() for w in "kv"}
    qs = torch.empty(s["begin"][-1], nq, hd, dtype=torch.float64, device="cuda")
    half = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    for layer, qkv in zip(range(N_LAYERS) if c["op"] == "accept" else (1,), s["qkv"]):
        for b, n in enumerate(s["n"]):
            for i in range(n):
                r = s["begin"][b] + i
                x = qkv[r].double().view(nq + 2 * nkv, hd)
                qk = x[:nq + nkv]
                if c["norm"]:
                    w = torch.cat((s["qn"].double().expand(nq, hd), s["kn"].double().expand(nkv, hd)))
                    qk = qk / torch.sqrt(qk.square().mean(1, keepdim=True) + EPS) * w
                angle = (s["start"][b] + len(_line(s, b, i)) - 1) * torch.exp(-2 * half / hd * math.log(THETA))
                turn = torch.polar(torch.ones_like(angle), angle) * torch.complex(qk[:, :hd // 2].contiguous(), qk[:, hd // 2:].contiguous())
                qk = torch.cat((turn.real, turn.imag), 1)
                place = _place(s, b, s["start"][b] + i)
                qs[r], got["k"][layer, :, place], got["v"][layer, :, place] = qk[:nq], qk[nq:], x[nq + nkv:]
    if c["op"] == "append":
        return {"q": qs, **got}
    path, count, after = [], [], []
    for b, n in enumerate(s["n"]):
        at = s["begin"][b]
        tokens, ids = (s[w][at:at + n].tolist() for w in ("tokens", "ids"))
        want, line = int(s["root"][b]), []
        while True:
            before = line[-1] if line else -1
            fit = [i for i in range(n) if s["parent"][at + i] == before and tokens[i] == want]
            if not fit:
                break
            line.append(fit[0])
            want = ids[fit[0]]
        for j, i in enumerate(line):  # i >= j and both rise: no row is written before it is read
            for w in "kv":
                got[w][:, :, _place(s, b, s["start"][b] + j)] = got[w][:, :, _place(s, b, s["start"][b] + i)]
        path += line + [-1] * (n - len(line))
        count.append(len(line))
        after.append(want)
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (path, count, after)]
    return {"path": ints[0], "count": ints[1], "next": ints[2], **got}
