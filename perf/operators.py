"""The 8-bit KV cache (store, read-back, attention) and the log probabilities of given tokens, as
cases with real sizes: what each operator computes in its plain form, what the framework's calls
compute, and the exact values in 64 bits.

Layout of one 8-bit cache buffer (K or V): codes, one byte each, [n_layers][nkv][slots][hd]; then, from
the next multiple of 256 bytes, f32 scales [n_layers][nkv][ceil(slots / 32)], one for each block of 32
slots of a head. A paged cache's slot of position p is table[p / 128] * 128 + p % 128.
"""
import math

import torch

own = False

BLOCK = 32      # positions that share one scale
PAGE = 128      # positions of one block of a paged cache
CMAX = {"e4m3": 448.0, "int8": 127.0}
E_MIN = -32     # exponent of the scale of a block that holds only zeros
N_LAYERS, LAYER = 2, 1


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token shortly after a 512-token prompt: the smallest call, latency counts
        attention("decode_512", "e4m3", 32, 8, 128, 1, 512, False),
        # a drafted continuation of three tokens verified at an odd position, paged cache
        attention("verify3_8k_paged", "int8", 32, 8, 128, 3, 8189, True),
        # one decoded token at the end of a long document: the cache is all there is to read
        attention("decode_128k_paged", "e4m3", 32, 8, 128, 1, 131071, True),
        # a ragged chunk on a small model with one query head to each kv head
        attention("chunk77_mha64", "int8", 8, 8, 64, 77, 1000, False),
        # the last of a 2048-token prompt's four chunks
        attention("chunk512_at_1536", "e4m3", 32, 8, 128, 512, 1536, False),
        # a chunk late in a long document: the largest amount of arithmetic
        attention("chunk512_at_32k", "int8", 32, 8, 128, 512, 32256, True),
        # one decoded token's keys and values appended inside a block of 32
        store("append_1", "e4m3", 8, 128, 1, 517, True),
        # a chunk that starts and ends inside blocks
        store("append_512", "int8", 8, 128, 512, 1001, False),
        # the largest chunk a session takes
        store("append_8192", "e4m3", 8, 128, 8192, 0, False),
        # the next token's distribution after a prompt: one row of a 151936-token vocabulary
        logprobs("row_1", 1, 151936, 151936, 20, False),
        # a ragged batch of rows over an odd vocabulary with padded rows, some tokens ruled out
        logprobs("rows_37_odd", 37, 100003, 100008, 5, True),
        # every position of a 512-token chunk scored
        logprobs("rows_512", 512, 151936, 151936, 20, False),
    ]


def attention(name, kv, nq, nkv, hd, m, start, paged):
    return {"name": name, "op": "attention", "kv": kv, "nq": nq, "nkv": nkv, "hd": hd, "m": m, "start": start, "paged": paged}


def store(name, kv, nkv, hd, m, start, paged):
    return {"name": name, "op": "store", "kv": kv, "nkv": nkv, "hd": hd, "m": m, "start": start, "paged": paged}


def logprobs(name, rows, n, ld, top, masked):
    return {"name": name, "op": "logprobs", "rows": rows, "n": n, "ld": ld, "top": top, "masked": masked}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "store", "logprobs"])
    kv, paged = rng.choice(["e4m3", "int8"]), rng.random() < 0.5
    if op == "attention":
        nq, nkv, hd = rng.choice([(32, 8, 128), (32, 8, 128), (4, 2, 64), (8, 8, 64), (16, 1, 128), (32, 4, 128)])
        m = _log(rng, 1, 512)
        start = min(_log(rng, 1, 131072) - 1, 512 * 29000 // m)
        c = attention("", kv, nq, nkv, hd, m, start, paged)
    elif op == "store":
        c = store("", kv, rng.choice([1, 2, 8]), rng.choice([64, 128]), _log(rng, 1, 8000), _log(rng, 1, 16384) - 1, paged)
    else:
        n = _log(rng, 1000, 151936)
        rows = min(_log(rng, 1, 512), 512 * 151936 // n)
        c = logprobs("", rows, n, n + rng.choice([0, 0, 5, 64]), rng.randint(0, 32), rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ the cache's layout
def _geometry(c):
    length = c["start"] + c["m"]
    max_seq = length + 37  # room behind the sequence, ending inside a block
    pages = -(-max_seq // PAGE)
    pool = pages + 3 if c["paged"] else 0
    slots = pool * PAGE if c["paged"] else max_seq
    codes = N_LAYERS * c["nkv"] * slots * c["hd"]
    return length, max_seq, pages, pool, slots, codes, -(-codes // 256) * 256, -(-slots // BLOCK)


def _codes(c, buf):
    """The layer's codes [nkv, slots, hd] as a view of the buffer, in bytes."""
    _, _, _, _, slots, codes, _, _ = _geometry(c)
    return buf[:codes].view(N_LAYERS, c["nkv"], slots, c["hd"])[LAYER]


def _type(c):
    return torch.float8_e4m3fn if c["kv"] == "e4m3" else torch.int8


def _scales(c, buf):
    """The layer's scales [nkv, blocks] as a view of the buffer."""
    _, _, _, _, _, _, at, nblk = _geometry(c)
    return buf[at:].view(torch.float32).view(N_LAYERS, c["nkv"], nblk)[LAYER]


def _slots(c, table, lo, hi):
    p = torch.arange(lo, hi, device="cuda")
    return p if table is None else table.long()[p // PAGE] * PAGE + p % PAGE


def _exponent(c, amax):
    """Least integer e with amax <= CMAX 2^e, E_MIN for zero (exact: amax is an f16 value held in f32)."""
    mant, x = torch.frexp(amax)  # amax = mant 2^x, 0.5 <= mant < 1
    top, xt = math.frexp(CMAX[c["kv"]])
    return torch.where(amax > 0, x - xt + (mant > top).int(), E_MIN).int()


def _round(c, x):
    """The code of the nearest value of the 8-bit type, ties to even, in bytes."""
    return (x if c["kv"] == "e4m3" else torch.round(x)).to(_type(c)).view(torch.uint8)


def _power(e):
    """2^e in 32 bits, exact."""
    return ((e + 127) << 23).view(torch.float32)


# ------------------------------------------------------------------ inputs
def _kv_rows(c, gen, rows, which):
    """K or V rows as they leave the projections: normal values, a few heavy channels (K), a few heavy tokens (V)."""
    x = torch.randn(rows, c["nkv"], c["hd"], device="cuda", generator=gen)
    if which == "k":
        x *= 1 + 7 * (torch.rand(c["nkv"], c["hd"], device="cuda", generator=gen) > 0.96)
    else:
        x *= 0.4 * (1 + 3 * (torch.rand(rows, 1, 1, device="cuda", generator=gen) > 0.98))
    return x.half()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    c = dict(case)
    if c["op"] == "logprobs":
        x = torch.randn(c["rows"], c["ld"], device="cuda", generator=gen) * 2.5
        lead = torch.randint(c["n"], (c["rows"], 12), device="cuda", generator=gen)
        x.scatter_add_(1, lead, 6 * torch.rand(c["rows"], 12, device="cuda", generator=gen) + 6)
        tokens = torch.randint(c["n"], (c["rows"],), device="cuda", generator=gen, dtype=torch.int32)
        tokens[::2] = lead[::2, 0].int()  # half of them likely, half of them anything
        if c["masked"]:  # tokens that a grammar rules out, none of the given ones among them
            out = torch.rand(c["ld"], device="cuda", generator=gen) < 0.3
            out[tokens.long()] = False
            x[:, out] = -math.inf
        x[:, c["n"]:] = math.nan  # the padding behind a row
        return {"case": c, "logits": x, "tokens": tokens}
    length, _, pages, pool, slots, codes, at, nblk = _geometry(c)
    table = torch.randperm(pool, device="cuda", generator=gen)[:pages].int() if c["paged"] else None
    s = {"case": c, "table": table}
    held = length if c["op"] == "attention" else c["start"]
    for which in ("k", "v"):
        # slots that no position uses hold arbitrary bytes, their blocks' scales arbitrary values
        buf = torch.randint(256, (at + N_LAYERS * c["nkv"] * nblk * 4,), device="cuda", generator=gen, dtype=torch.uint8)
        if held:
            x = _kv_rows(c, gen, held, which).permute(1, 0, 2).float()
            nb = -(-held // BLOCK)
            x = torch.nn.functional.pad(x, (0, 0, 0, nb * BLOCK - held)).view(c["nkv"], nb, BLOCK, c["hd"])
            scale = _power(_exponent(c, x.abs().amax((2, 3))))
            i = _slots(c, table, 0, held)
            _codes(c, buf)[:, i] = _round(c, x / scale[:, :, None, None]).view(c["nkv"], nb * BLOCK, c["hd"])[:, :held]
            _scales(c, buf)[:, i[::BLOCK] // BLOCK] = scale
        s[which + "_cache"] = buf
    if c["op"] == "attention":
        q = torch.randn(c["m"], c["nq"], c["hd"], device="cuda", generator=gen)
        s["q"] = (q * (0.5 + 2 * torch.rand(c["nq"], 1, device="cuda", generator=gen))).half()
    else:
        s["k"], s["v"] = (_kv_rows(c, gen, c["m"], w) for w in ("k", "v"))
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    return {"attention": run_attention, "store": run_store, "logprobs": run_logprobs}[c["op"]](c, state)


_plans = {}


def _plan(c):
    """What a user's program keeps: the configuration, the workspace and the status word of these sizes."""
    from quantized_transformer_prefill_q1_gb300 import pf

    key = tuple(sorted((k, v) for k, v in c.items() if k != "name"))
    if key not in _plans:
        _, max_seq, _, pool, _, _, _, _ = _geometry(c)
        nq = c.get("nq", 2 * c["nkv"])
        cfg = pf.pf_config(hidden=128, intermediate=128, n_q_heads=nq, n_kv_heads=c["nkv"], head_dim=c["hd"], n_layers=N_LAYERS,
                           rope_theta=1e6, eps=1e-6, final_eps=1e-6, kv_dtype=pf.KV_E4M3 if c["kv"] == "e4m3" else pf.KV_INT8,
                           max_seq=max_seq, max_chunk=min(8192, c["m"]), kv_block_pool=pool)
        scratch = pf.attention_kv8_scratch(cfg, c["m"]) if c["op"] == "attention" else None
        _plans[key] = pf, cfg, scratch, torch.zeros(4, dtype=torch.int32, device="cuda")
    return _plans[key]


def run_attention(c, s):
    if own:
        pf, cfg, scratch, status = _plan(c)
        out = torch.empty(c["m"], c["nq"] * c["hd"], dtype=torch.float16, device="cuda")
        pf.pf_op_attention_kv8(cfg, s["q"], s["k_cache"], s["v_cache"], LAYER, c["start"], c["m"], out, scratch, s["table"], status)
        return out
    length = c["start"] + c["m"]
    i = _slots(c, s["table"], 0, length)
    k, v = (_codes(c, s[w])[:, i].view(_type(c)).float() * _scales(c, s[w])[:, i // BLOCK, None] for w in ("k_cache", "v_cache"))
    g = c["nq"] // c["nkv"]
    q = s["q"].float().view(c["m"], c["nkv"], g, c["hd"]).permute(1, 2, 0, 3).reshape(c["nkv"], g * c["m"], c["hd"])
    x = (q @ k.transpose(1, 2)).view(c["nkv"], g, c["m"], length) * c["hd"] ** -0.5
    pos = torch.arange(length, device="cuda")
    x = torch.where(pos[None, :] <= pos[c["start"]:, None], x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(c["nkv"], g * c["m"], length)
    o = (p @ v).view(c["nkv"], g, c["m"], c["hd"]).permute(2, 0, 1, 3)
    return o.reshape(c["m"], c["nq"] * c["hd"]).half()


def run_store(c, s):
    """Stores the chunk, then reads back every position of the blocks that it touches."""
    first = c["start"] // BLOCK * BLOCK
    end = c["start"] + c["m"]
    if own:
        pf, cfg, _, status = _plan(c)
        pf.pf_op_kv8_store(cfg, s["k"], s["v"], LAYER, c["start"], c["m"], s["k_cache"], s["v_cache"], s["table"], status)
        got = {}
        for w in ("k", "v"):
            got[w] = torch.empty(end - first, c["nkv"], c["hd"], device="cuda")
            pf.pf_op_kv8_load(cfg, s[w + "_cache"], LAYER, first, end - first, got[w], s["table"], status)
        return got
    i = _slots(c, s["table"], first, end)
    blk = i[::BLOCK] // BLOCK
    old = c["start"] - first  # positions of the first block that were there before
    got = {}
    for w in ("k", "v"):
        codes, scales = _codes(c, s[w + "_cache"]), _scales(c, s[w + "_cache"])
        x = torch.nn.functional.pad(s[w].float().permute(1, 0, 2), (0, 0, old, len(blk) * BLOCK - (end - first)))
        amax = x.reshape(c["nkv"], len(blk), BLOCK * c["hd"]).abs().amax(-1)
        scale = _power(_exponent(c, amax))
        if old:
            scale[:, 0] = torch.maximum(scale[:, 0], scales[:, blk[0]])
            x[:, :old] = codes[:, i[:old]].view(_type(c)).float() * scales[:, blk[0], None, None]
        x = x[:, :end - first]
        each = scale.repeat_interleave(BLOCK, 1)[:, :end - first, None]
        q = _round(c, x / each)
        codes[:, i] = q
        scales[:, blk] = scale
        got[w] = (q.view(_type(c)).float() * each).permute(1, 0, 2).contiguous()
    return got


def run_logprobs(c, s):
    rows, n, top = c["rows"], c["n"], c["top"]
    if own:
        from quantized_transformer_prefill_q1_gb300 import pf

        lp, ent = torch.empty(2, rows, device="cuda")
        got = {"logprob": lp, "entropy": ent}
        if top:
            got["top_ids"] = torch.empty(rows, top, dtype=torch.int32, device="cuda")
            got["top_logprob"] = torch.empty(rows, top, device="cuda")
        pf.pf_op_logprobs(s["logits"], rows, n, c["ld"], s["tokens"], lp, ent, top, got.get("top_ids"), got.get("top_logprob"))
        return got
    x = s["logits"][:, :n]
    d = x - x.amax(1, keepdim=True)
    e = torch.exp(d)
    z = e.sum(1)
    lz = torch.log(z)
    got = {"logprob": d.gather(1, s["tokens"].long()[:, None])[:, 0] - lz,
           "entropy": lz - torch.where(e > 0, d * e, 0).sum(1) / z}
    if top:
        # one whole number for each value, in the values' order and, among equals, lowest index first
        bits = x.contiguous().view(torch.int32).long()
        key = torch.where(bits < 0, -0x80000000 - bits, bits) * 2 ** 32 + torch.arange(n - 1, -1, -1, device="cuda")
        got["top_ids"] = (n - 1 - (key.topk(top, dim=1).values & 0xffffffff)).int()
        got["top_logprob"] = d.gather(1, got["top_ids"].long()) - lz[:, None]
    return got


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "logprobs":
        return {"bytes": 4 * c["rows"] * (c["n"] + 3 + 2 * c["top"]), "flops": 5 * c["rows"] * c["n"]}
    row = c["nkv"] * c["hd"]
    length = c["start"] + c["m"]
    if c["op"] == "store":
        back = c["m"] + c["start"] % BLOCK
        return {"bytes": 2 * row * (2 * c["m"] + c["m"] + back + 4 * back) + 8 * c["nkv"] * -(-back // BLOCK), "flops": 4 * row * c["m"]}
    pairs = c["m"] * c["start"] + c["m"] * (c["m"] + 1) // 2
    return {"bytes": 2 * row * length + 8 * c["nkv"] * -(-length // BLOCK) + 4 * c["m"] * c["nq"] * c["hd"],
            "flops": 4 * c["nq"] * c["hd"] * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def _power64(e):
    """2^e in 64 bits, exact (a library power may be off by its last bit, which would break ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _values64(c, s, w, positions):
    """What the cache holds at the given positions [nkv, P, hd]: the code read bit by bit, times its block's scale."""
    _, _, _, _, slots, codes, at, nblk = _geometry(c)
    buf = s[w]
    slot = positions if s["table"] is None else s["table"].long()[positions // PAGE] * PAGE + positions % PAGE
    u = buf[:codes].view(N_LAYERS, c["nkv"], slots, c["hd"])[LAYER].index_select(1, slot).int()
    scale = buf[at:].view(torch.float32).view(N_LAYERS, c["nkv"], nblk)[LAYER].index_select(1, slot // BLOCK).double()
    if c["kv"] == "int8":
        v = torch.where(u > 127, u - 256, u).double()
    else:
        field, frac = (u >> 3) & 15, (u & 7).double()
        v = torch.where(field > 0, (1 + frac / 8) * _power64(field - 7), frac / 512)
        v = torch.where(u > 127, -v, v)
    return v * scale[:, :, None]


def _nearest64(c, x):
    """x rounded to the 8-bit type's nearest value, ties to even, in 64 bits (|x| <= CMAX)."""
    if c["kv"] == "int8":
        return torch.round(x)
    step = _power64(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)  # three bits below the leading one; subnormals share 2^-9
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "logprobs":
        got = {k: [] for k in ("logprob", "entropy", "top_ids", "top_logprob")}
        for r in range(c["rows"]):
            x = s["logits"][r, :c["n"]].double()
            lse = torch.logsumexp(x, 0)
            lp = x - lse
            got["logprob"].append(lp[int(s["tokens"][r])])
            got["entropy"].append(-(lp.exp() * lp.clamp(min=-1e300)).sum())
            order = torch.sort(x, descending=True, stable=True).indices[:c["top"]]
            got["top_ids"].append(order.int())
            got["top_logprob"].append(lp[order])
        got = {k: torch.stack(v) for k, v in got.items()}
        return got if c["top"] else {k: got[k] for k in ("logprob", "entropy")}
    if c["op"] == "attention":
        length, g = c["start"] + c["m"], c["nq"] // c["nkv"]
        pos = torch.arange(length, device="cuda")
        k, v = (_values64(c, s, w, pos) for w in ("k_cache", "v_cache"))
        out = torch.empty(c["m"], c["nq"], c["hd"], dtype=torch.float64, device="cuda")
        see = pos[None, :] <= c["start"] + torch.arange(c["m"], device="cuda")[:, None]
        for h in range(c["nq"]):
            score = s["q"][:, h].double() @ k[h // g].T / math.sqrt(c["hd"])
            out[:, h] = torch.softmax(score.masked_fill(~see, -math.inf), -1) @ v[h // g]
        return out.view(c["m"], c["nq"] * c["hd"])
    first = c["start"] // BLOCK * BLOCK
    got = {}
    for w in ("k", "v"):
        new = s[w].double().permute(1, 0, 2)
        old = _values64(c, s, w + "_cache", torch.arange(first, c["start"], device="cuda"))
        was = s[w + "_cache"][_geometry(c)[6]:].view(torch.float32).view(N_LAYERS, c["nkv"], -1)[LAYER].double()
        rows = torch.cat([old, new], 1)
        for at in range(0, rows.shape[1], BLOCK):
            part = rows[:, at:at + BLOCK]
            skip = c["start"] - first if at == 0 else 0
            amax = part[:, skip:].abs().amax((1, 2))
            e = torch.ceil(torch.log2(amax / CMAX[c["kv"]])).clamp(min=E_MIN)
            e = torch.where(amax > CMAX[c["kv"]] * _power64(e), e + 1, e)  # where the logarithm fell on the wrong side
            e = torch.where((amax <= CMAX[c["kv"]] * _power64(e - 1)) & (e > E_MIN), e - 1, e)
            scale = _power64(e)
            if skip:
                p = torch.tensor(first, device="cuda")
                slot = p if s["table"] is None else s["table"].long()[p // PAGE] * PAGE + p % PAGE
                scale = torch.maximum(scale, was[:, slot // BLOCK])
            rows[:, at:at + BLOCK] = _nearest64(c, part / scale[:, None, None]) * scale[:, None, None]
        got[w] = rows.permute(1, 0, 2)
    return got
