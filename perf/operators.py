"""The operators of decoding several branches of one prompt: cases, inputs, plain forms, calls, exact values.

One prompt sits in a contiguous cache (the layout dec_get_kv returns); every branch keeps its own tokens in pages.
A step of all branches normalises and rotates queries and keys ("rope", or "append", which also puts keys and values
into the pages), attends over the shared prompt and the branch's own pages ("attend"), picks the next branches over
beams and vocabulary ("select") and gives every branch its parent's history ("reorder").

`run` computes an operator in elementary torch operations, or, where `own` is true, calls the framework's.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# Geometry of the repository's configurations: 16 query and 8 key/value heads of 128 (vocabulary 151,936, 28 layers),
# and 4 query and 2 key/value heads of 16 (vocabulary 512, 2 layers).
WIDE = {"n_q": 16, "n_kv": 8, "head_dim": 128}
TINY = {"n_q": 4, "n_kv": 2, "head_dim": 16}


def listed():
    return [
        # one new token of a single stream, straight after the projection (float32 in, bfloat16 for the next product)
        {"name": "rope 1 row", "op": "rope", "rows": 1, **WIDE, "rot": 128, "pairs": "half", "norm": True,
         "x": "f32", "y": "bf16", "scaled": False, "far": 4096},
        # a long prompt chunk with interleaved pairs, half of each head rotated, frequencies scaled for long contexts
        {"name": "rope 8191 rows partial", "op": "rope", "rows": 8191, **WIDE, "rot": 64, "pairs": "interleaved",
         "norm": True, "x": "bf16", "y": "bf16", "scaled": True, "far": 131072},
        # one token of each of 16 branches
        {"name": "append 16 branches", "op": "append", "seqs": 16, "rows": 16, **WIDE, "rot": 128, "pairs": "half",
         "norm": True, "x": "f32", "y": "bf16", "kv": "bf16", "page": 16, "scaled": False, "base": 4096},
        # ragged prompts of 37 sequences that go to pages together (padded rows among them), float32 cache
        {"name": "append 4099 ragged rows", "op": "append", "seqs": 37, "rows": 4099, **WIDE, "rot": 128,
         "pairs": "half", "norm": True, "x": "f32", "y": "f32", "kv": "f32", "page": 64, "scaled": True, "base": 0},
        # four branches just after a short prompt: latency
        {"name": "attend 4 x 512", "op": "attend", "batch": 4, **WIDE, "prefix": 512, "suffix": 33, "page": 16,
         "q": "bf16", "kv": "bf16", "idle": 0},
        # an ordinary beam search over a held-out document
        {"name": "attend 16 x 4096", "op": "attend", "batch": 16, **WIDE, "prefix": 4096, "suffix": 256, "page": 16,
         "q": "bf16", "kv": "bf16", "idle": 1},
        # many sampled answers to one very long prompt
        {"name": "attend 64 x 32768", "op": "attend", "batch": 64, **WIDE, "prefix": 32768, "suffix": 512, "page": 64,
         "q": "bf16", "kv": "bf16", "idle": 0},
        # the float32 cache, odd prefix length
        {"name": "attend 8 x 3001 f32", "op": "attend", "batch": 8, **WIDE, "prefix": 3001, "suffix": 100, "page": 16,
         "q": "f32", "kv": "f32", "idle": 0},
        # four beams over the whole vocabulary; twice as many candidates as beams, so that ended ones can be set aside
        {"name": "select 4 beams", "op": "select", "beams": 4, "vocab": 151936, "take": 8},
        # as many beams as the widest attention case has branches
        {"name": "select 64 beams", "op": "select", "beams": 64, "vocab": 151936, "take": 128},
        # a small model's pages
        {"name": "reorder 4 beams", "op": "reorder", "beams": 4, "layers": 2, **TINY, "suffix": 40, "page": 16,
         "kv": "f32"},
        # all layers of the wide model
        {"name": "reorder 64 beams", "op": "reorder", "beams": 64, "layers": 28, **WIDE, "suffix": 120, "page": 32,
         "kv": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, dims=(16, 64, 128, 128)):
    n_kv = rng.choice([1, 2, 4, 8])
    return {"n_q": n_kv * rng.choice([1, 2, 4, 8]), "n_kv": n_kv, "head_dim": rng.choice(dims)}


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "select", "reorder"])
    t = ["f32", "bf16"]
    if op in ("rope", "append"):
        h = _heads(rng, (16, 64, 80, 96, 128, 128))
        c = {"op": op, "rows": _log(rng, 1, 8192), **h, "rot": rng.choice([h["head_dim"], h["head_dim"] // 2]),
             "pairs": rng.choice(["half", "interleaved"]), "norm": rng.random() < 0.8, "x": rng.choice(t),
             "y": rng.choice(t), "scaled": rng.random() < 0.5}
        c["rows"] = max(1, min(c["rows"], 8191 * 24 // (h["n_q"] + h["n_kv"]) // (2 if op == "append" else 1)))
        if op == "rope":
            return {**c, "far": _log(rng, 1024, 1 << 20)}
        return {**c, "seqs": min(c["rows"], _log(rng, 1, 64)), "kv": rng.choice(t), "page": rng.choice([8, 16, 64, 128]),
                "base": rng.choice([0, 511, 4096, 32768])}
    if op == "attend":
        batch = _log(rng, 1, 64)
        c = {"op": op, "batch": batch, **_heads(rng), "prefix": _log(rng, 1, 32768) - 1, "suffix": _log(rng, 1, 512),
             "page": rng.choice([8, 16, 64, 128]), "q": rng.choice(t), "kv": rng.choice(t),
             "idle": rng.randrange(batch) if rng.random() < 0.2 else 0}
        most = work(listed()[6])
        while any(work(c)[k] > most[k] for k in most):
            c["prefix"] //= 2
            c["suffix"] = max(1, c["suffix"] // 2)
        return c
    if op == "select":
        beams = _log(rng, 1, 64)
        vocab = rng.choice([512, 32001, 50257, 151936, 151936])
        return {"op": op, "beams": beams, "vocab": vocab, "take": rng.randrange(1, min(2 * beams, vocab) + 1)}
    return {"op": op, "beams": _log(rng, 1, 64), "layers": rng.randrange(1, 29), **_heads(rng),
            "suffix": _log(rng, 1, 120), "page": rng.choice([8, 16, 32]), "kv": rng.choice(t)}


# ---- inputs -------------------------------------------------------------------------------------------------------

def _frequencies(rot, scaled):
    """Angular frequency of each pair (base 1e6), and the factor on cosine and sine. Scaled: frequencies that turn less
    than once in 32,768 positions are divided by 4, those that turn over 32 times stay, a ramp lies between."""
    w = 1e6 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if not scaled:
        return w, 1.0
    keep = np.clip((32768 * w / (2 * np.pi) - 1.0) / 31.0, 0.0, 1.0)
    return w * keep + w / 4.0 * (1.0 - keep), 0.1 * math.log(4.0) + 1.0


class _Make:
    """Seeded random tensors on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.n = np.random.default_rng(seed)

    def normal(self, shape, dtype, scale=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * scale).to(dtype)

    def ints(self, values):
        return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def _lengths(rng, count, most, idle):
    """Tokens that each branch holds: up to `most`, one branch at that; the last `idle` slots unused (-1)."""
    n = rng.integers(max(1, most // 2), most + 1, count)
    n[0] = most
    if idle:
        n[count - idle:] = -1
    return n


def _table(rng, need, width, pages):
    """A page table [branches][width] (-1 where a branch has no page) over a shuffled pool of `pages`."""
    ids, table, at = rng.permutation(pages), np.full((len(need), width), -1), 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at: at + k]
        at += k
    return table


def prepare(case, seed):
    c, mk = case, _Make(seed)
    s = {"case": c, "args": None}
    if c["op"] in ("rope", "append"):
        n, hq, hk, d, x = c["rows"], c["n_q"], c["n_kv"], c["head_dim"], DTYPES[c["x"]]
        qkv = mk.normal((n, (hq + 2 * hk) * d), x, 1.5)  # rows of the fused projection: q, k, v side by side
        s["q"], s["k"], s["v"] = qkv[:, : hq * d], qkv[:, hq * d: (hq + hk) * d], qkv[:, (hq + hk) * d:]
        s["gq"] = 1.0 + mk.normal((d,), torch.float32, 0.1) if c["norm"] else None
        s["gk"] = 1.0 + mk.normal((d,), torch.float32, 0.1) if c["norm"] else None
        w, s["factor"] = _frequencies(c["rot"], c["scaled"])
        s["w"] = torch.tensor(w, device="cuda")
        s["q_out"] = torch.zeros((n, hq * d), dtype=DTYPES[c["y"]], device="cuda")
        if c["op"] == "rope":
            first = int(mk.n.integers(0, c["far"]))
            s["pos"] = mk.ints(first + np.arange(n))
            s["k_out"] = torch.zeros((n, hk * d), dtype=DTYPES[c["y"]], device="cuda")
        else:
            m = c["seqs"]  # sequences of consecutive rows; the last rows pad the batch where there are more rows
            pad = (n - m) // 16
            cuts = np.sort(mk.n.choice(np.arange(1, n - pad), m - 1, replace=False)) if m > 1 else np.zeros(0, int)
            held = np.diff(np.concatenate([[0], cuts, [n - pad]]))
            before = mk.n.integers(0, 2 * c["page"], m)  # tokens that each sequence's pages hold already
            pos = np.concatenate([b + np.arange(k) for b, k in zip(before, held)] + [np.full(pad, -1 - c["base"])])
            s["pos"] = mk.ints(pos + c["base"])
            s["seq"] = mk.ints(np.concatenate([np.repeat(np.arange(m), held), np.zeros(pad, int)]))
            need = -(-(before + held) // c["page"])
            pages = n // c["page"] + 3 * m
            s["table"] = mk.ints(_table(mk.n, need, int(need.max()), pages))
            s["kp"] = mk.normal((pages, hk, c["page"], d), DTYPES[c["kv"]])
            s["vp"] = mk.normal((pages, hk, c["page"], d), DTYPES[c["kv"]])
    elif c["op"] == "attend":
        b, hq, hk, d, kv = c["batch"], c["n_q"], c["n_kv"], c["head_dim"], DTYPES[c["kv"]]
        s["q"] = mk.normal((b, hq * d), DTYPES[c["q"]], 1.2)
        s["pk"], s["pv"] = mk.normal((hk, c["prefix"], d), kv), mk.normal((hk, c["prefix"], d), kv)
        held = _lengths(mk.n, b, c["suffix"], c["idle"])
        width = -(-c["suffix"] // c["page"])
        pages = b * width
        s["len"] = mk.ints(held)
        s["table"] = mk.ints(_table(mk.n, -(-np.maximum(held, 0) // c["page"]), width, pages))
        s["kp"], s["vp"] = mk.normal((pages, hk, c["page"], d), kv), mk.normal((pages, hk, c["page"], d), kv)
        s["out"] = torch.zeros((b, hq * d), dtype=DTYPES[c["q"]], device="cuda")
        s["lse"] = torch.zeros((b, hq), dtype=torch.float32, device="cuda")
        s["scale"] = float(np.float32(d ** -0.5))
    elif c["op"] == "select":
        b = c["beams"]
        s["logits"] = mk.normal((b, c["vocab"]), torch.float32, 2.5)
        s["scores"] = mk.normal((b,), torch.float32, 1.0) - 12.0
        s["score"] = torch.zeros(c["take"], dtype=torch.float32, device="cuda")
        s["parent"] = torch.zeros(c["take"], dtype=torch.int32, device="cuda")
        s["token"] = torch.zeros(c["take"], dtype=torch.int32, device="cuda")
    else:
        b, hk, d, page = c["beams"], c["n_kv"], c["head_dim"], c["page"]
        held = np.full(b, c["suffix"])  # all beams of a search are equally long
        width = c["suffix"] // page + 1
        pages = b * width
        s["table"], s["len"] = mk.ints(_table(mk.n, np.full(b, width), width, pages)), mk.ints(held)
        s["spare"] = mk.ints(pages + mk.n.permutation(b))
        s["parent"] = mk.ints(mk.n.integers(0, b, b))
        shape = (c["layers"], pages + b, hk, page, d)
        s["kp"], s["vp"] = mk.normal(shape, DTYPES[c["kv"]]), mk.normal(shape, DTYPES[c["kv"]])
        s["new_table"] = torch.zeros((b, width), dtype=torch.int32, device="cuda")
        s["new_len"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    if own:
        s["args"] = _arguments(s)
    return s


def _arguments(s):
    """The argument block that a program fills once for its buffers, and the workspace beside it."""
    import weight_streaming_gemv_token_gb300 as W

    code = {"f32": W.DEC_F32, "bf16": W.DEC_BF16}
    c = s["case"]
    if c["op"] in ("rope", "append"):
        d = c["head_dim"]
        wide = (c["n_q"] + 2 * c["n_kv"]) * d
        both = dict(rows=c["rows"], n_q=c["n_q"], n_kv=c["n_kv"], head_dim=d, xdtype=code[c["x"]], ydtype=code[c["y"]],
                    q=s["q"], k=s["k"], q_out=s["q_out"], q_stride=wide, k_stride=wide, q_out_stride=c["n_q"] * d,
                    g_q=s["gq"], g_k=s["gk"], eps=1e-6, positions=s["pos"], rot_dim=c["rot"],
                    interleaved=int(c["pairs"] == "interleaved"), inv_freq=s["w"], rope_factor=s["factor"])
        if c["op"] == "rope":
            return W.qk_rope_args(k_out=s["k_out"], k_out_stride=c["n_kv"] * d, **both)
        return W.kv_append_args(v=s["v"], v_stride=wide, kvdtype=code[c["kv"]], seq=s["seq"], n_seq=c["seqs"],
                                k_pages=s["kp"], v_pages=s["vp"], num_pages=s["kp"].shape[0], page_size=c["page"],
                                page_table=s["table"], table_stride=s["table"].shape[1], base_pos=c["base"], **both)
    if c["op"] == "attend":
        a = W.attn_shared_args(batch=c["batch"], n_q=c["n_q"], n_kv=c["n_kv"], head_dim=c["head_dim"],
                               qdtype=code[c["q"]], kvdtype=code[c["kv"]], q=s["q"], out=s["out"], lse=s["lse"],
                               q_stride=s["q"].shape[1], out_stride=s["q"].shape[1], prefix_k=s["pk"],
                               prefix_v=s["pv"], prefix_len=c["prefix"], prefix_stride=c["prefix"], k_pages=s["kp"],
                               v_pages=s["vp"], num_pages=s["kp"].shape[0], page_size=c["page"],
                               page_table=s["table"], table_stride=s["table"].shape[1], seq_len=s["len"],
                               scale=s["scale"])
        return a.with_workspace(torch.empty(W.attn_shared_prefix_workspace(a), dtype=torch.uint8, device="cuda"))
    if c["op"] == "select":
        a = W.beam_select_args(beams=c["beams"], vocab=c["vocab"], n_out=c["take"], logits=s["logits"],
                               logits_stride=c["vocab"], scores=s["scores"], out_scores=s["score"],
                               out_parents=s["parent"], out_tokens=s["token"])
        return a.with_workspace(torch.empty(W.beam_select_workspace(a), dtype=torch.uint8, device="cuda"))
    return W.beam_reorder_args(beams=c["beams"], layers=c["layers"], n_kv=c["n_kv"], head_dim=c["head_dim"],
                               kvdtype=code[c["kv"]], k_pages=s["kp"], v_pages=s["vp"],
                               layer_stride=s["kp"].stride(0), num_pages=s["kp"].shape[1], page_size=c["page"],
                               parents=s["parent"], spare=s["spare"], old_table=s["table"], old_len=s["len"],
                               new_table=s["new_table"], new_len=s["new_len"], table_stride=s["table"].shape[1])


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import weight_streaming_gemv_token_gb300 as W

        call = {"rope": W.qk_norm_rope, "append": W.kv_append_paged, "attend": W.attn_shared_prefix,
                "select": W.beam_select, "reorder": W.beam_reorder_pages}[op]
        call(state["args"])
    else:
        {"rope": _rope, "append": _append, "attend": _attend, "select": _select, "reorder": _reorder}[op](state)
    return [state[k] for k in {"rope": ("q_out", "k_out"), "append": ("q_out", "kp", "vp"), "attend": ("out", "lse"),
                               "select": ("score", "parent", "token"),
                               "reorder": ("kp", "vp", "new_table", "new_len")}[op]]


def _turned(s, x, heads, gain):
    """float32 rows [n][heads][d]: RMS norm of each head, then the rotation of its first `rot` elements."""
    c = s["case"]
    x = x.float().reshape(c["rows"], heads, c["head_dim"])
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain
    angle = s["pos"].double()[:, None] * s["w"]  # 64 bits: far positions
    cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    rot = c["rot"]
    r = x[..., :rot]
    if c["pairs"] == "half":
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1) if rot < c["head_dim"] else r


def _rope(s):
    c = s["case"]
    s["q_out"].copy_(_turned(s, s["q"], c["n_q"], s["gq"]).reshape(c["rows"], -1))
    s["k_out"].copy_(_turned(s, s["k"], c["n_kv"], s["gk"]).reshape(c["rows"], -1))


def _append(s):
    c = s["case"]
    live = s["pos"] >= 0
    q = _turned(s, s["q"], c["n_q"], s["gq"]).reshape(c["rows"], -1).to(s["q_out"].dtype)
    s["q_out"].copy_(torch.where(live[:, None], q, s["q_out"]))
    at = torch.where(live, s["pos"] - c["base"], 0).long()
    page, slot = s["table"][s["seq"].long(), at // c["page"]].long(), at % c["page"]
    k = _turned(s, s["k"], c["n_kv"], s["gk"])
    v = s["v"].float().reshape(c["rows"], c["n_kv"], -1)
    n = c["rows"] - (c["rows"] - c["seqs"]) // 16  # padded rows are the last ones
    s["kp"][page[:n], :, slot[:n]] = k[:n].to(s["kp"].dtype)
    s["vp"][page[:n], :, slot[:n]] = v[:n].to(s["vp"].dtype)


def _attend(s):
    c = s["case"]
    b, hk, d = c["batch"], c["n_kv"], c["head_dim"]
    g = c["n_q"] // hk
    q = s["q"].float().reshape(b, hk, g, d)
    qp = q.transpose(0, 1).reshape(hk, b * g, d)  # all branches' rows of a head against the prefix at once
    sp = (qp @ s["pk"].float().transpose(1, 2) * s["scale"]).reshape(hk, b, g, -1).transpose(0, 1)
    own_k, own_v = (s[k][s["table"].clamp(min=0).long()].float().transpose(1, 2).reshape(b, hk, -1, d)
                    for k in ("kp", "vp"))
    hidden = torch.arange(own_k.shape[2], device="cuda") >= s["len"][:, None]
    ss = (q @ own_k.transpose(2, 3) * s["scale"]).masked_fill(hidden[:, None, None], -math.inf)
    top = torch.cat([sp, ss], -1).amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    pp, ps = torch.exp(sp - top), torch.exp(ss - top)
    total = pp.sum(-1, keepdim=True) + ps.sum(-1, keepdim=True)
    o = (pp.transpose(0, 1).reshape(hk, b * g, -1) @ s["pv"].float()).reshape(hk, b, g, d).transpose(0, 1)
    o = (o + ps @ own_v) / total
    used = (s["len"] >= 0)[:, None]
    s["out"].copy_(torch.where(used, o.reshape(b, -1).to(s["out"].dtype), s["out"]))
    s["lse"].copy_(torch.where(used, (top + torch.log(total)).reshape(b, -1), s["lse"]))


def _select(s):
    c = s["case"]
    x = s["logits"].double()  # 64 bits: neighbours in rank may differ in the last bits of 32
    top = x.amax(-1, keepdim=True)
    key = (x - (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))) + s["scores"].double()[:, None]).reshape(-1)
    # a few more than asked for, by index and then (stable) by key: of equal keys the lowest index comes first
    _, at = torch.topk(key, min(c["take"] + 32, key.numel()))
    at = torch.sort(at).values
    at = at[torch.sort(key[at], descending=True, stable=True).indices[: c["take"]]]
    s["score"].copy_(key[at])
    s["parent"].copy_(at // c["vocab"])
    s["token"].copy_(at % c["vocab"])


def _reorder(s):
    c = s["case"]
    p = s["parent"].long()
    held = s["len"][p]
    full, rest = (held // c["page"]).long(), held % c["page"]
    j = torch.arange(s["table"].shape[1], device="cuda")
    s["new_table"].copy_(torch.where(j < full[:, None], s["table"][p],
                                     torch.where(j == full[:, None], s["spare"][:, None], -1)))
    s["new_len"].copy_(held)
    src, dst = s["table"][p, full].long(), s["spare"].long()
    filled = (torch.arange(c["page"], device="cuda") < rest[:, None])[None, :, None, :, None]
    s["kp"][:, dst] = torch.where(filled, s["kp"][:, src], s["kp"][:, dst])
    s["vp"][:, dst] = torch.where(filled, s["vp"][:, src], s["vp"][:, dst])


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}
    if c["op"] in ("rope", "append"):
        n, hq, hk, d = c["rows"], c["n_q"], c["n_kv"], c["head_dim"]
        if c["op"] == "rope":
            return {"bytes": n * (hq + hk) * d * (size[c["x"]] + size[c["y"]]) + 4 * n, "flops": 8 * n * (hq + hk) * d}
        n -= (n - c["seqs"]) // 16
        return {"bytes": n * d * (size[c["x"]] * (hq + 2 * hk) + size[c["y"]] * hq + size[c["kv"]] * 2 * hk) + 8 * n,
                "flops": 8 * n * (hq + hk) * d}
    if c["op"] == "attend":
        b, hq, hk, d = c["batch"] - c["idle"], c["n_q"], c["n_kv"], c["head_dim"]
        held = b * c["suffix"] * 3 / 4  # lengths are uniform between half of the longest and the longest
        return {"bytes": 2 * hk * d * size[c["kv"]] * (c["prefix"] + held) + 2 * b * hq * d * size[c["q"]],
                "flops": 4 * hq * d * (b * c["prefix"] + held)}
    if c["op"] == "select":
        return {"bytes": 4 * c["beams"] * c["vocab"] + 12 * c["take"], "flops": 4 * c["beams"] * c["vocab"]}
    rest = c["suffix"] % c["page"]
    rows = c["beams"] * c["layers"] * c["n_kv"] * rest
    return {"bytes": 2 * 2 * rows * c["head_dim"] * size[c["kv"]] + 8 * c["beams"] * (c["suffix"] // c["page"] + 3),
            "flops": 0}


# ---- the definition in 64 bits --------------------------------------------------------------------------------------

def _np(t):
    return t.double().cpu().numpy()


def _exact_rows(s, x, heads, gain):
    c = s["case"]
    rot, d = c["rot"], c["head_dim"]
    x = _np(x).reshape(-1, heads, d).copy()
    if gain is not None:
        x = x / np.sqrt(np.mean(x ** 2, axis=-1, keepdims=True) + 1e-6) * _np(gain)
    z = np.exp(1j * (_np(s["pos"])[:, None, None] * _np(s["w"]))) * s["factor"]
    i = np.arange(rot // 2)
    a, b = (i, i + rot // 2) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
    z = z * (x[:, :, a] + 1j * x[:, :, b])
    x[:, :, a], x[:, :, b] = z.real, z.imag
    return x


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c = case
    if c["op"] == "rope":
        return [_exact_rows(s, s[k], h, s[g]).reshape(c["rows"], -1)
                for k, h, g in (("q", c["n_q"], "gq"), ("k", c["n_kv"], "gk"))]
    if c["op"] == "append":
        q, k = _exact_rows(s, s["q"], c["n_q"], s["gq"]), _exact_rows(s, s["k"], c["n_kv"], s["gk"])
        v, out, kp, vp = _np(s["v"]).reshape(k.shape), _np(s["q_out"]), _np(s["kp"]), _np(s["vp"])
        table = s["table"].cpu().numpy()
        for r, (pos, seq) in enumerate(zip(s["pos"].tolist(), s["seq"].tolist())):
            if pos >= 0:
                page, slot = divmod(pos - c["base"], c["page"])
                out[r] = q[r].reshape(-1)
                kp[table[seq, page], :, slot], vp[table[seq, page], :, slot] = k[r], v[r]
        return [out, kp, vp]
    if c["op"] == "attend":
        b, hk, d = c["batch"], c["n_kv"], c["head_dim"]
        g = c["n_q"] // hk
        out, lse = s["out"].double(), s["lse"].double()
        pk, pv, q = s["pk"].double(), s["pv"].double(), s["q"].double().reshape(b, hk, g, d)
        for i, n in enumerate(s["len"].tolist()):
            if n < 0:
                continue
            ids = s["table"][i, : -(-n // c["page"])].long()
            ks, vs = (s[k][ids].double().permute(1, 0, 2, 3).reshape(hk, -1, d)[:, :n] for k in ("kp", "vp"))
            score = torch.cat([q[i] @ pk.mT, q[i] @ ks.mT], -1) * s["scale"]
            lse[i] = torch.logsumexp(score, -1).reshape(-1)
            p = torch.exp(score - lse[i].reshape(hk, g, 1))
            out[i] = (p[..., : c["prefix"]] @ pv + p[..., c["prefix"]:] @ vs).reshape(-1)
        return [out, lse]
    if c["op"] == "select":
        x = _np(s["logits"])
        x -= np.max(x, axis=1, keepdims=True)
        x += (_np(s["scores"]) - np.log(np.sum(np.exp(x), axis=1)))[:, None]
        flat = x.reshape(-1)
        some = np.sort(np.argpartition(-flat, min(c["take"] + 64, flat.size - 1))[: c["take"] + 64])
        at = some[np.argsort(-flat[some], kind="stable")][: c["take"]]
        return [flat[at], at // c["vocab"], at % c["vocab"]]
    kp, vp, table, held = s["kp"].clone(), s["vp"].clone(), s["table"].tolist(), s["len"].tolist()
    new_table, new_len = np.full(np.shape(table), -1), np.zeros(c["beams"], int)
    for i, (p, spare) in enumerate(zip(s["parent"].tolist(), s["spare"].tolist())):
        full, rest = divmod(held[p], c["page"])
        new_table[i, :full], new_table[i, full], new_len[i] = table[p][:full], spare, held[p]
        for pool in (kp, vp):
            pool[:, spare, :, :rest] = pool[:, table[p][full], :, :rest]
    return [kp, vp, new_table, new_len]
