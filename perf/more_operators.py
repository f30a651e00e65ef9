"""The operators of a step that checks drafted trees of several requests: cases, inputs, plain forms, calls, exact values.

Each request holds tokens in pages and brings the rows of this step: its last known token and a tree of drafted ones
behind it (or a chain: a draft in one line, a prompt's rows). A step gives every request pages, positions, slots and
ancestor masks ("slots"), attends with all rows over cache and ancestors ("attend"), applies penalties, biases and grammar
masks to the logits and picks the greedy token after each row ("adjust"), and walks each tree along these tokens, moving
accepted keys and values to their places in all layers ("accept").

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
        # one stream with a small tree behind its last token: latency
        {"name": "slots 1 request", "op": "slots", "requests": 1, "drafts": 8, "ctx": 500, "page": 16, "tree": True,
         "done": 0, "tight": False},
        # a serving step: many requests with their trees, finished ones among them whose pages come back
        {"name": "slots 256 trees", "op": "slots", "requests": 256, "drafts": 32, "ctx": 8192, "page": 16, "tree": True,
         "done": 9, "tight": False},
        # ragged prompts that enter together, more than the pool has pages for
        {"name": "slots 37 prompts", "op": "slots", "requests": 37, "drafts": 450, "ctx": 100, "page": 64, "tree": False,
         "done": 3, "tight": True},
        # the tree of one stream over a decoder's own contiguous cache: latency
        {"name": "attend 1 x 8 over 512", "op": "attend", "batch": 1, "drafts": 8, "ctx": 33, "prefix": 512, **WIDE,
         "page": 16, "tree": True, "q": "bf16", "kv": "bf16", "idle": 0},
        # an ordinary serving step with trees
        {"name": "attend 8 x 16 over 4096", "op": "attend", "batch": 8, "drafts": 16, "ctx": 4096, "prefix": 0, **WIDE,
         "page": 16, "tree": True, "q": "bf16", "kv": "bf16", "idle": 0},
        # single new tokens of many requests of very different lengths, one slot unused
        {"name": "attend 48 single tokens", "op": "attend", "batch": 48, "drafts": 1, "ctx": 7000, "prefix": 0, **WIDE,
         "page": 64, "tree": False, "q": "bf16", "kv": "bf16", "idle": 1},
        # large trees over long documents
        {"name": "attend 32 x 64 over 16384", "op": "attend", "batch": 32, "drafts": 64, "ctx": 16384, "prefix": 0, **WIDE,
         "page": 64, "tree": True, "q": "bf16", "kv": "bf16", "idle": 0},
        # the float32 cache, odd sizes, small pages
        {"name": "attend 5 x 13 over 3001 f32", "op": "attend", "batch": 5, "drafts": 13, "ctx": 3001, "prefix": 0, **WIDE,
         "page": 8, "tree": True, "q": "f32", "kv": "f32", "idle": 0},
        # one stream's next token under every rule
        {"name": "adjust 1 row", "op": "adjust", "requests": 1, "drafts": 1, "vocab": 151936, "history": 700, "bias": 20,
         "masks": 1, "x": "f32", "y": "f32"},
        # the rows of 32 trees behind long histories, a grammar's mask for some
        {"name": "adjust 256 tree rows", "op": "adjust", "requests": 32, "drafts": 8, "vocab": 151936, "history": 4096,
         "bias": 100, "masks": 12, "x": "f32", "y": "f32"},
        # one small tree of a small model
        {"name": "accept 1 tree", "op": "accept", "batch": 1, "drafts": 12, "take": 4, "layers": 2, **TINY, "ctx": 40,
         "page": 16, "kv": "f32"},
        # all layers of the wide model
        {"name": "accept 32 trees", "op": "accept", "batch": 32, "drafts": 48, "take": 8, "layers": 28, **WIDE, "ctx": 90,
         "page": 32, "kv": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, dims=(16, 64, 128, 128)):
    n_kv = rng.choice([1, 2, 4, 8])
    return {"n_q": n_kv * rng.choice([1, 2, 4, 8]), "n_kv": n_kv, "head_dim": rng.choice(dims)}


def draw(rng):
    op = rng.choice(["slots", "attend", "attend", "attend", "adjust", "accept"])
    t = ["f32", "bf16"]
    if op == "slots":
        n, tree = _log(rng, 1, 256), rng.random() < 0.6
        return _within({"op": op, "requests": n, "drafts": _log(rng, 1, 64 if tree else max(2, min(2048, 16384 // n))),
                        "ctx": _log(rng, 1, 8192), "page": rng.choice([8, 16, 64, 128]), "tree": tree,
                        "done": rng.randrange(n) if rng.random() < 0.4 else 0, "tight": rng.random() < 0.3},
                       "ctx", "drafts")
    if op == "attend":
        batch = _log(rng, 1, 64)
        return _within({"op": op, "batch": batch, "drafts": _log(rng, 1, 64), "ctx": _log(rng, 1, 16384),
                        "prefix": rng.choice([0, 0, _log(rng, 1, 8192)]), **_heads(rng), "page": rng.choice([8, 16, 64, 128]),
                        "tree": rng.random() < 0.7, "q": rng.choice(t), "kv": rng.choice(t),
                        "idle": rng.randrange(batch) if rng.random() < 0.2 else 0}, "ctx", "prefix")
    if op == "adjust":
        vocab = rng.choice([512, 32001, 50257, 151936, 151936])
        n = _log(rng, 1, 64)
        return _within({"op": op, "requests": n, "drafts": _log(rng, 1, max(1, min(32, 256 // n))), "vocab": vocab,
                        "history": _log(rng, 1, 4096), "bias": rng.choice([0, _log(rng, 1, 300)]),
                        "masks": rng.choice([0, rng.randrange(1, n + 1)]), "x": rng.choice(t), "y": rng.choice(t)},
                       "drafts", "history")
    return _within({"op": op, "batch": _log(rng, 1, 32), "drafts": _log(rng, 1, 48), "take": rng.randrange(1, 9),
                    "layers": rng.randrange(1, 29), **_heads(rng), "ctx": _log(rng, 1, 90), "page": rng.choice([8, 16, 32]),
                    "kv": rng.choice(t)}, "layers")


def _within(c, *sizes):
    """The case with these sizes halved until it costs no more than the operator's largest listed one."""
    same = [work(k) for k in listed() if k["op"] == c["op"]]
    while any(work(c)[k] > max(w[k] for w in same) for k in work(c)) and any(c[k] > 1 for k in sizes):
        for k in sizes:
            c[k] = c[k] // 2 if k == "prefix" else max(1, c[k] // 2)
    return c


# ---- inputs -------------------------------------------------------------------------------------------------------

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

    def floats(self, values):
        return torch.tensor(np.asarray(values), dtype=torch.float32, device="cuda")


def _counts(rng, n, most):
    """Rows of each request: between half of `most` and that, in any order (their sum goes by the case alone)."""
    return rng.permutation(np.linspace(most, (most + 1) // 2, n).astype(int))


def _trees(rng, rows):
    """Parents within each request's rows: row 0 has none, a row hangs below any earlier one."""
    return np.concatenate([np.concatenate([[-1], (rng.random(k - 1) * np.arange(1, k)).astype(int)])[:k] for k in rows])


def _ancestors(parents, rows):
    """bool [rows][most rows of a request]: a row's ancestors and itself."""
    m, at = np.zeros((len(parents), max(rows)), bool), 0
    for k in rows:
        for i in range(k):
            p = parents[at + i]
            if p >= 0:
                m[at + i] = m[at + p]
            m[at + i, i] = True
        at += k
    return m


def _words(bits):
    """bool [rows][n] as words of 32 bits, int32 [rows][ceil(n / 32)]."""
    n = -(-bits.shape[1] // 32)
    b = np.zeros((bits.shape[0], 32 * n), np.uint8)
    b[:, : bits.shape[1]] = bits
    return np.packbits(b, axis=1, bitorder="little").view(np.uint32).view(np.int32)


def _table(rng, need, width, pages):
    """A page table [requests][width] (-1 where a request has no page) over a shuffled pool, and the pages left over."""
    ids, table, at = rng.permutation(pages), np.full((len(need), width), -1), 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at: at + k]
        at += k
    return table, ids[at:]


def prepare(case, seed):
    c, mk = case, _Make(seed)
    s = {"case": c, "args": None}
    if c["op"] == "slots":
        n, page = c["requests"], c["page"]
        fresh = _counts(mk.n, n, c["drafts"])
        held = mk.n.integers(0, c["ctx"] + 1, n)
        owned = -(-held // page) + mk.n.integers(0, 2, n)  # a page may be left over from a draft that was rejected
        width = -(-(c["ctx"] + c["drafts"]) // page) + 1
        more = np.maximum(-(-(held + fresh) // page) - owned, 0)
        if c["done"]:
            held[n - c["done"]:] = -1
        spare = int(more.sum() * (0.6 if c["tight"] else 1.2)) + 1
        s["pages"] = 2 * n * width  # those that are neither owned nor free are others'
        table, free = _table(mk.n, owned, width, s["pages"])
        free = free[:spare]
        ring, first = np.zeros(s["pages"], int), int(mk.n.integers(0, s["pages"]))
        ring[(first + np.arange(len(free))) % s["pages"]] = free
        s["held"], s["fresh"], s["owned"], s["table"] = mk.ints(held), mk.ints(fresh), mk.ints(owned), mk.ints(table)
        s["ring"], s["free"] = mk.ints(ring), mk.ints([first, len(free)])
        s["rows"] = int(fresh.sum()) + 3  # the batch is padded a little
        s["words"] = -(-c["drafts"] // 32) if c["tree"] else 0
        s["parents"] = None
        if c["tree"]:
            live = fresh[held >= 0]  # finished requests bring no rows
            s["parents"] = mk.ints(np.concatenate([_trees(mk.n, live), np.zeros(s["rows"] - int(live.sum()), int)]))
            s["mask"] = torch.zeros((s["rows"], s["words"]), dtype=torch.int32, device="cuda")
        s["new_table"] = torch.zeros_like(s["table"])
        s["new_owned"], s["ctx_len"] = torch.zeros_like(s["owned"]), torch.zeros_like(s["owned"])
        s["new_free"] = torch.zeros_like(s["free"])
        s["row_start"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        s["seq"] = torch.zeros(s["rows"], dtype=torch.int32, device="cuda")
        s["pos"] = torch.zeros(s["rows"], dtype=torch.int32, device="cuda")
        s["slots"] = torch.zeros(s["rows"], dtype=torch.int64, device="cuda")
    elif c["op"] == "attend":
        b, hq, hk, d, kv, page = c["batch"], c["n_q"], c["n_kv"], c["head_dim"], DTYPES[c["kv"]], c["page"]
        rows = _counts(mk.n, b, c["drafts"])
        held = mk.n.integers(c["ctx"] // 2, c["ctx"] + 1, b)
        held[0] = c["ctx"]
        width = -(-(c["ctx"] + c["drafts"]) // page)
        need = -(-(held + rows) // page)
        pages = b * width
        s["table"] = mk.ints(_table(mk.n, need, width, pages)[0])
        if c["idle"]:
            held[b - c["idle"]:] = -1
        n = int(rows.sum())
        s["row_start"], s["len"] = mk.ints(np.concatenate([[0], np.cumsum(rows)])), mk.ints(held)
        s["most"] = int(rows.max())
        s["mask"] = mk.ints(_words(_ancestors(_trees(mk.n, rows), rows))) if c["tree"] else None
        s["q"] = mk.normal((n, hq * d), DTYPES[c["q"]], 1.2)
        s["pk"], s["pv"] = (mk.normal((hk, c["prefix"], d), kv) for _ in range(2))
        s["kp"], s["vp"] = (mk.normal((pages, hk, page, d), kv) for _ in range(2))
        s["out"] = torch.zeros((n, hq * d), dtype=DTYPES[c["q"]], device="cuda")
        s["lse"] = torch.zeros((n, hq), dtype=torch.float32, device="cuda")
        s["scale"] = float(np.float32(d ** -0.5))
    elif c["op"] == "adjust":
        n, v = c["requests"], c["vocab"]
        rows = _counts(mk.n, n, c["drafts"])
        total = int(rows.sum())
        s["logits"] = mk.normal((total, v), torch.float32, 2.5).to(DTYPES[c["x"]])
        s["seq"] = mk.ints(np.repeat(np.arange(n), rows))
        s["row_start"] = mk.ints(np.concatenate([[0], np.cumsum(rows)]))
        # words of a text: few tokens come often
        s["tokens"] = mk.ints(np.minimum(mk.n.zipf(1.3, (n, c["history"])), v) - 1)
        length = mk.n.integers((c["history"] + 1) // 2, c["history"] + 1, n)
        s["tokens_len"], s["prompt_len"] = mk.ints(length), mk.ints(length * mk.n.random(n))
        s["draft"] = mk.ints(mk.n.integers(0, v, total))
        s["mask"] = mk.ints(_words(_ancestors(_trees(mk.n, rows), rows)))
        s["repetition"], s["frequency"], s["presence"] = (mk.floats(lo + mk.n.random(n) * w)
                                                          for lo, w in ((1.0, 0.5), (0.0, 0.3), (-0.2, 1.0)))
        nb = c["bias"]
        if nb:  # a token is biased once in a list; lists may be shorter than the longest
            s["bias_tokens"] = mk.ints([mk.n.choice(v, nb, replace=False) for _ in range(n)])
            s["bias"] = mk.floats(mk.n.standard_normal((n, nb)) * 3.0)
            s["bias_len"] = mk.ints(mk.n.integers((nb + 1) // 2, nb + 1, n))
        if c["masks"]:  # a row goes by one of the grammar's states, or by none
            s["allowed"] = mk.ints(_words(mk.n.random((c["masks"], v)) < mk.n.choice([0.01, 0.5, 0.95], c["masks"])[:, None]))
            s["allowed_row"] = mk.ints(mk.n.integers(-1, c["masks"], total))
        s["out"] = torch.zeros((total, v), dtype=DTYPES[c["y"]], device="cuda")
        s["next"] = torch.zeros(total, dtype=torch.int32, device="cuda")
    else:
        b, hk, d, page = c["batch"], c["n_kv"], c["head_dim"], c["page"]
        rows = _counts(mk.n, b, c["drafts"])
        parents, draft = _trees(mk.n, rows), mk.n.integers(0, 151936, int(rows.sum()))
        after, at = mk.n.integers(0, 151936, int(rows.sum())), 0
        for k in rows:
            # the path that is accepted lies behind the places it moves to, so that a pass can be repeated
            a = int(mk.n.integers(1, max(1, min(c["take"], (k + 1) // 2)) + 1))
            path = np.concatenate([[0], np.sort(mk.n.choice(np.arange(a, k), a - 1, replace=False))]).astype(int)
            parents[at + path[1:]] = path[:-1]
            after[at + path[:-1]] = draft[at + path[1:]]
            at += k
        held = mk.n.integers((c["ctx"] + 1) // 2, c["ctx"] + 1, b)
        width = -(-(c["ctx"] + c["drafts"]) // page)
        s["table"] = mk.ints(_table(mk.n, -(-(held + rows) // page), width, b * width)[0])
        s["parents"], s["draft"], s["next"] = mk.ints(parents), mk.ints(draft), mk.ints(after)
        s["row_start"], s["len"] = mk.ints(np.concatenate([[0], np.cumsum(rows)])), mk.ints(held)
        s["most"] = int(rows.max())
        shape = (c["layers"], b * width, hk, page, d)
        s["kp"], s["vp"] = mk.normal(shape, DTYPES[c["kv"]]), mk.normal(shape, DTYPES[c["kv"]])
        s["tokens"] = mk.ints(mk.n.integers(0, 151936, (b, c["ctx"] + c["drafts"])))
        s["count"], s["new_len"] = torch.zeros_like(s["len"]), torch.zeros_like(s["len"])
        s["path"] = torch.zeros((b, 8), dtype=torch.int32, device="cuda")
        s["accepted"] = torch.zeros((b, 8), dtype=torch.int32, device="cuda")
    if own:
        s["args"] = _arguments(s)
    return s


def _arguments(s):
    """The argument block that a program fills once for its buffers, and the workspace beside it."""
    import weight_streaming_gemv_token_gb300 as W

    code = {"f32": W.DEC_F32, "bf16": W.DEC_BF16}
    c = s["case"]
    if c["op"] == "slots":
        return W.step_slots_args(requests=c["requests"], rows=s["rows"], num_pages=s["pages"], page_size=c["page"],
                                 table_stride=s["table"].shape[1], base_pos=0, mask_words=s["words"], held=s["held"],
                                 fresh=s["fresh"], owned=s["owned"], parents=s["parents"], page_table=s["table"],
                                 free_ring=s["ring"], free_state=s["free"], new_table=s["new_table"],
                                 new_owned=s["new_owned"], new_free_state=s["new_free"], row_start=s["row_start"],
                                 ctx_len=s["ctx_len"], seq=s["seq"], positions=s["pos"], slots=s["slots"],
                                 mask=s.get("mask"))
    if c["op"] == "attend":
        a = W.attn_tree_args(batch=c["batch"], rows=s["q"].shape[0], n_q=c["n_q"], n_kv=c["n_kv"], head_dim=c["head_dim"],
                             qdtype=code[c["q"]], kvdtype=code[c["kv"]], q=s["q"], out=s["out"], lse=s["lse"],
                             q_stride=s["q"].shape[1], out_stride=s["q"].shape[1], row_start=s["row_start"],
                             mask=s["mask"], mask_words=s["mask"].shape[1] if c["tree"] else 0, prefix_k=s["pk"],
                             prefix_v=s["pv"], prefix_len=c["prefix"], prefix_stride=c["prefix"], k_pages=s["kp"],
                             v_pages=s["vp"], num_pages=s["kp"].shape[0], page_size=c["page"], page_table=s["table"],
                             table_stride=s["table"].shape[1], seq_len=s["len"], scale=s["scale"])
        return a.with_workspace(torch.empty(W.attn_tree_paged_workspace(a), dtype=torch.uint8, device="cuda"))
    if c["op"] == "adjust":
        nb, masks = c["bias"], c["masks"]
        return W.logits_adjust_args(rows=s["logits"].shape[0], vocab=c["vocab"], xdtype=code[c["x"]], ydtype=code[c["y"]],
                                    logits=s["logits"], logits_stride=c["vocab"], out=s["out"], out_stride=c["vocab"],
                                    next=s["next"], requests=c["requests"], seq=s["seq"], tokens=s["tokens"],
                                    tokens_stride=c["history"], tokens_len=s["tokens_len"], tokens_base=0,
                                    prompt_len=s["prompt_len"], draft_tokens=s["draft"], row_start=s["row_start"],
                                    mask=s["mask"], mask_words=s["mask"].shape[1], repetition=s["repetition"],
                                    frequency=s["frequency"], presence=s["presence"], bias_tokens=s.get("bias_tokens"),
                                    bias=s.get("bias"), bias_len=s.get("bias_len"), bias_stride=nb,
                                    allowed=s.get("allowed"), allowed_stride=s["allowed"].shape[1] if masks else 0,
                                    allowed_rows=masks, allowed_row=s.get("allowed_row"))
    return W.tree_accept_args(batch=c["batch"], rows=s["draft"].shape[0], path_stride=8, layers=c["layers"],
                              n_kv=c["n_kv"], head_dim=c["head_dim"], kvdtype=code[c["kv"]], row_start=s["row_start"],
                              parents=s["parents"], draft_tokens=s["draft"], next=s["next"], seq_len=s["len"],
                              k_pages=s["kp"], v_pages=s["vp"], layer_stride=s["kp"].stride(0),
                              num_pages=s["kp"].shape[1], page_size=c["page"], table_stride=s["table"].shape[1],
                              page_table=s["table"], tokens=s["tokens"], tokens_stride=s["tokens"].shape[1],
                              tokens_base=0, count=s["count"], new_len=s["new_len"], path=s["path"],
                              out_tokens=s["accepted"])


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import weight_streaming_gemv_token_gb300 as W

        call = {"slots": W.step_slots, "attend": W.attn_tree_paged, "adjust": W.logits_adjust,
                "accept": W.tree_accept_paged}[op]
        call(state["args"])
    else:
        {"slots": _slots, "attend": _attend, "adjust": _adjust, "accept": _accept}[op](state)
    keys = {"slots": ("new_table", "new_owned", "new_free", "ring", "row_start", "ctx_len", "seq", "pos", "slots")
            + (("mask",) if "mask" in state else ()), "attend": ("out", "lse"), "adjust": ("out", "next"),
            "accept": ("kp", "vp", "tokens", "count", "new_len", "path", "accepted")}[op]
    return [state[k] for k in keys]


def _slots(s):
    c = s["case"]
    page, n_pages, n = c["page"], s["pages"], s["rows"]
    held, fresh, owned = s["held"].long(), s["fresh"].long(), s["owned"].long()
    live = held >= 0
    fresh = torch.where(live, fresh, 0)
    need = torch.where(live, (held + fresh + page - 1) // page - owned, 0).clamp(min=0)
    ends = torch.cumsum(need, 0)
    served = live & ((need == 0) | (ends <= s["free"][1]))
    got = torch.where(served, need, 0)
    j = torch.arange(s["table"].shape[1], device="cuda")
    take = (s["free"][0] + (ends - need)[:, None] + j - owned[:, None]) % n_pages
    kept = (owned * live)[:, None]
    s["new_table"].copy_(torch.where(j < kept, s["table"],
                                     torch.where(live[:, None] & (j < kept + got[:, None]), s["ring"][take], -1)))
    s["new_owned"].copy_(kept[:, 0] + got)
    back = torch.where(live, 0, owned)
    to = (s["free"][0] + s["free"][1] + (torch.cumsum(back, 0) - back)[:, None] + j) % n_pages
    returned = j < back[:, None]
    s["ring"][to[returned]] = s["table"][returned]
    s["new_free"][0] = (s["free"][0] + got.sum()) % n_pages
    s["new_free"][1] = s["free"][1] - got.sum() + back.sum()
    s["row_start"][1:] = torch.cumsum(fresh, 0)
    s["ctx_len"].copy_(torch.where(served, held, -1))
    r = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["row_start"][1:].contiguous(), r.int(), right=True)
    inside = seq < c["requests"]
    seq = seq.clamp(max=c["requests"] - 1)
    used = inside & served[seq]
    i = r - s["row_start"][seq]
    at = held[seq] + i
    entry = s["new_table"][seq, (at // page).clamp(0, j.numel() - 1)].long()
    s["slots"].copy_(torch.where(used, entry * page + at % page, -1))
    s["seq"].copy_(torch.where(used, seq, -1))
    depth = i
    if c["tree"]:
        first = r - i
        up = torch.where(s["parents"] < 0, n, first + s["parents"])  # row n stands for none
        up = torch.cat([up, up.new_tensor([n])])
        bits = torch.zeros((n + 1, 32 * s["words"]), dtype=torch.bool, device="cuda")
        bits[r[used], i[used]] = True
        up[:n] = torch.where(used, up[:n], n)
        for _ in range(max(1, math.ceil(math.log2(c["drafts"])))):  # ancestors of twice the distance each time
            bits = bits | bits[up]
            up = up[up]
        depth = bits[:n].sum(1) - 1
        s["mask"].copy_((bits[:n].view(n, -1, 32).long() << torch.arange(32, device="cuda")).sum(2))
    s["pos"].copy_(torch.where(used, held[seq] + depth, -1))


def _padded(s, x, most):
    """Rows of all requests [rows][...] as [requests][most][...], and which of them there are."""
    start = s["row_start"].long()
    i = torch.arange(most, device="cuda")
    there = i < (start[1:] - start[:-1])[:, None]
    at = (start[:-1, None] + i).clamp(max=x.shape[0] - 1)
    return x[at], there, at


def _attend(s):
    c = s["case"]
    b, hk, d, most = c["batch"], c["n_kv"], c["head_dim"], s["most"]
    g = c["n_q"] // hk
    q, there, at = _padded(s, s["q"].float(), most)
    q = q.reshape(b, most, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, most * g, d)
    k, v = (s[n][s["table"].clamp(min=0).long()].float().transpose(1, 2).reshape(b, hk, -1, d) for n in ("kp", "vp"))
    j = torch.arange(k.shape[2], device="cuda") - s["len"][:, None].clamp(min=0)  # number of the drafted token
    j = j[:, None].expand(b, most, -1)
    if c["tree"]:
        word = s["mask"][at].gather(2, (j // 32).clamp(0, s["mask"].shape[1] - 1).long())
        seen = (j < 0) | ((j < 32 * s["mask"].shape[1]) & ((word >> (j % 32)) & 1 == 1))
    else:
        seen = j <= torch.arange(most, device="cuda")[:, None]
    seen = seen[:, None, :, None].expand(-1, -1, -1, g, -1).reshape(b, 1, most * g, -1)
    ss = (q @ k.transpose(2, 3) * s["scale"]).masked_fill(~seen, -math.inf)
    sp = q @ s["pk"].float().transpose(1, 2) * s["scale"]
    top = torch.cat([sp, ss], -1).amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    pp, ps = torch.exp(sp - top), torch.exp(ss - top)
    total = pp.sum(-1, keepdim=True) + ps.sum(-1, keepdim=True)
    o = (ps @ v + pp @ s["pv"].float()) / total
    o = o.reshape(b, hk, most, g, d).transpose(1, 2).reshape(b, most, -1)
    lse = (top + torch.log(total)).reshape(b, hk, most, g).transpose(1, 2).reshape(b, most, -1)
    used = there & (s["len"] >= 0)[:, None]
    s["out"][at[used]] = o[used].to(s["out"].dtype)
    s["lse"][at[used]] = lse[used]


def _adjust(s):
    c = s["case"]
    n, v, seq = c["requests"], c["vocab"], s["seq"].long()
    i = torch.arange(c["history"], device="cuda")
    inside, prompt = i < s["tokens_len"][:, None], i < s["prompt_len"][:, None]
    said = torch.zeros((n, v), device="cuda")
    said.scatter_add_(1, s["tokens"].long(), (inside & ~prompt).float())
    asked = torch.zeros((n, v), device="cuda")
    asked.scatter_add_(1, s["tokens"].long(), (inside & prompt).float())
    count = said[seq]
    most = 32 * s["mask"].shape[1]
    bits = ((s["mask"][:, :, None] >> torch.arange(32, device="cuda")) & 1).reshape(-1, most)
    at = (s["row_start"][seq].long()[:, None] + torch.arange(most, device="cuda")).clamp(max=s["draft"].numel() - 1)
    count.scatter_add_(1, s["draft"][at].long(), bits.float())  # drafted tokens on the way to the row
    x = s["logits"].float()
    rep, freq, pres = (s[k][seq][:, None] for k in ("repetition", "frequency", "presence"))
    x = torch.where((count > 0) | (asked[seq] > 0), torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * count
    x = x - torch.where(count > 0, pres, 0.0)
    if c["bias"]:
        bias = torch.zeros((n, v), device="cuda")
        listed_ = torch.arange(c["bias"], device="cuda") < s["bias_len"][:, None]
        bias.scatter_add_(1, s["bias_tokens"].long(), torch.where(listed_, s["bias"], 0.0))
        x = x + bias[seq]
    if c["masks"]:
        word = s["allowed"][s["allowed_row"].clamp(min=0).long()]
        ok = ((word[:, :, None] >> torch.arange(32, device="cuda")) & 1).reshape(x.shape[0], -1)[:, :v] == 1
        x = torch.where(ok | (s["allowed_row"] < 0)[:, None], x, -math.inf)
    s["out"].copy_(x)
    top = x.amax(1, keepdim=True)
    first = torch.where(x == top, torch.arange(v, device="cuda"), v).amin(1)
    s["next"].copy_(torch.where(top[:, 0] == -math.inf, -1, first))


def _accept(s):
    c = s["case"]
    b, most, page = c["batch"], s["most"], c["page"]
    parents, there, at = _padded(s, s["parents"].long(), most)
    draft, after = s["draft"].long()[at], s["next"].long()[at]
    i = torch.arange(most, device="cuda")
    cur, on = torch.zeros(b, dtype=torch.long, device="cuda"), torch.ones(b, dtype=torch.bool, device="cuda")
    path, out = torch.full((b, 8), -1, device="cuda"), torch.full((b, 8), -1, device="cuda")
    for step in range(8):
        token = after.gather(1, cur[:, None])
        path[:, step], out[:, step] = torch.where(on, cur, -1), torch.where(on, token[:, 0], -1)
        child = there & (parents == cur[:, None]) & (draft == token) & (i > 0)
        found = torch.where(child, i, most).amin(1)
        on = on & (found < most)
        cur = torch.where(on, found, cur)
    count = (path >= 0).sum(1)
    held = s["len"].long()
    s["path"].copy_(path)
    s["accepted"].copy_(out)
    s["count"].copy_(count)
    s["new_len"].copy_(held + count)
    q, step = torch.nonzero(path >= 0, as_tuple=True)
    src, dst = held[q] + path[q, step], held[q] + step
    s["tokens"][q, dst] = draft[q, path[q, step]].int()
    src_page, dst_page = s["table"][q, src // page].long(), s["table"][q, dst // page].long()
    for pool in (s["kp"], s["vp"]):
        pool[:, dst_page, :, dst % page] = pool[:, src_page, :, src % page]


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}
    if c["op"] == "slots":
        n, rows = c["requests"], (c["requests"] - c["done"]) * max(1, c["drafts"] * 3 // 4)
        words = -(-c["drafts"] // 32) if c["tree"] else 0
        width = -(-(c["ctx"] + c["drafts"]) // c["page"]) + 1
        return {"bytes": 24 * n + 4 * n * width + 2 * n * c["ctx"] // c["page"] + rows * (16 + (4 if c["tree"] else 0) + 4 * words),
                "flops": 0}
    if c["op"] == "attend":
        # lengths are uniform between half of the longest and the longest, rows too
        b, hq, hk, d = c["batch"] - c["idle"], c["n_q"], c["n_kv"], c["head_dim"]
        rows, own_keys = b * max(1.0, c["drafts"] * 0.75), c["ctx"] * 0.75 + max(1.0, c["drafts"] * 0.75)
        keys = c["prefix"] + b * own_keys
        return {"bytes": int(2 * hk * d * size[c["kv"]] * keys + 2 * rows * hq * d * size[c["q"]] + 4 * rows * hq),
                "flops": int(4 * hq * d * rows * (c["prefix"] + own_keys))}
    if c["op"] == "adjust":
        rows = int(c["requests"] * max(1.0, c["drafts"] * 0.75))
        once = c["vocab"] // 8 * c["masks"] + c["requests"] * (3 * c["history"] + 6 * c["bias"] + 24)
        return {"bytes": rows * c["vocab"] * (size[c["x"]] + size[c["y"]]) + once + 12 * rows, "flops": 2 * rows * c["vocab"]}
    # a path takes 1 to `take` rows, all but the first of which move
    moved = c["batch"] * (min(c["take"], (c["drafts"] * 3 // 4 + 1) // 2 + 1) - 1) / 2 * c["layers"] * c["n_kv"]
    return {"bytes": int(2 * 2 * moved * c["head_dim"] * size[c["kv"]]) + c["batch"] * (9 * c["drafts"] + 100), "flops": 0}


# ---- the definition in 64 bits --------------------------------------------------------------------------------------

def _np(t):
    return t.double().cpu().numpy()


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c = case
    if c["op"] == "slots":
        return _exact_slots(s)
    if c["op"] == "attend":
        return _exact_attend(s)
    if c["op"] == "adjust":
        return _exact_adjust(s)
    page, start, held = c["page"], s["row_start"].tolist(), s["len"].tolist()
    kp, vp, tokens, table = s["kp"].clone(), s["vp"].clone(), s["tokens"].cpu().numpy(), s["table"].tolist()
    parents, draft, after = (s[k].tolist() for k in ("parents", "draft", "next"))
    path, out = np.full((c["batch"], 8), -1), np.full((c["batch"], 8), -1)
    count = np.zeros(c["batch"], int)
    for b in range(c["batch"]):
        lo, hi = start[b], start[b + 1]
        cur = 0
        while cur is not None and count[b] < 8:
            step = count[b]
            path[b, step], out[b, step] = cur, after[lo + cur]
            tokens[b, held[b] + step] = draft[lo + cur]
            (p0, r0), (p1, r1) = divmod(held[b] + cur, page), divmod(held[b] + step, page)
            for pool in (kp, vp):
                pool[:, table[b][p1], :, r1] = pool[:, table[b][p0], :, r0]
            count[b] += 1
            cur = next((i for i in range(1, hi - lo) if parents[lo + i] == cur and draft[lo + i] == after[lo + cur]), None)
    return [kp, vp, tokens, count, np.array(held) + count, path, out]


def _exact_slots(s):
    c = s["case"]
    page, n = c["page"], s["rows"]
    held, fresh, owned, ring = (s[k].tolist() for k in ("held", "fresh", "owned", "ring"))
    old = s["table"].tolist()
    first, free = s["free"].tolist()
    parents = s["parents"].tolist() if c["tree"] else None
    table, new_owned, ctx = np.full(np.shape(old), -1), np.zeros(c["requests"], int), np.full(c["requests"], -1)
    start, seq, pos, slots = [0], np.full(n, -1), np.full(n, -1), np.full(n, -1)
    mask = np.zeros((n, 32 * max(1, s["words"])), bool)
    wanted, taken, returned = 0, 0, []
    for b in range(c["requests"]):
        if held[b] < 0:
            returned += old[b][: owned[b]]
            start.append(start[-1])
            continue
        total = held[b] + fresh[b]
        need = max(0, -(-total // page) - owned[b])
        wanted += need
        table[b, : owned[b]] = old[b][: owned[b]]
        new_owned[b] = owned[b]
        lo = start[-1]
        start.append(lo + fresh[b])
        if need and wanted > free:
            continue
        for j in range(need):
            table[b, owned[b] + j] = ring[(first + taken + j) % s["pages"]]
        taken += need
        new_owned[b] += need
        ctx[b] = held[b]
        for i in range(fresh[b]):
            t = held[b] + i
            seq[lo + i], slots[lo + i] = b, int(table[b, t // page]) * page + t % page
            depth = i
            if parents:
                up = i
                depth = -1
                while up >= 0:
                    mask[lo + i, up] = True
                    up, depth = parents[lo + up], depth + 1
            pos[lo + i] = held[b] + depth
    for k, p in enumerate(returned):
        ring[(first + free + k) % s["pages"]] = p
    r = [table, new_owned, np.array([(first + taken) % s["pages"], free - taken + len(returned)]), np.array(ring),
         np.array(start), ctx, seq, pos, slots]
    return r + ([_words(mask)] if c["tree"] else [])


def _exact_attend(s):
    c = s["case"]
    hk, d = c["n_kv"], c["head_dim"]
    g = c["n_q"] // hk
    out, lse = s["out"].double(), s["lse"].double()
    pk, pv, start = s["pk"].double(), s["pv"].double(), s["row_start"].tolist()
    for b, n in enumerate(s["len"].tolist()):
        lo, hi = start[b], start[b + 1]
        if n < 0 or hi == lo:
            continue
        r = hi - lo
        ids = s["table"][b, : -(-(n + r) // c["page"])].long()
        ks, vs = (s[k][ids].double().permute(1, 0, 2, 3).reshape(hk, -1, d)[:, : n + r] for k in ("kp", "vp"))
        seen = np.tril(np.ones((r, r), bool))
        if c["tree"]:
            m = s["mask"][lo:hi].cpu().numpy().view(np.uint32)
            seen = np.array([[bool(m[i, j // 32] >> np.uint32(j % 32) & np.uint32(1)) for j in range(r)] for i in range(r)])
        q = s["q"][lo:hi].double().reshape(r, hk, g, d).permute(1, 0, 2, 3)
        score = torch.cat([q @ pk.mT[:, None], q @ ks.mT[:, None]], -1) * s["scale"]
        score[..., c["prefix"] + n:] += torch.tensor(np.where(seen, 0.0, -np.inf), device="cuda")[None, :, None]
        z = torch.logsumexp(score, -1)
        p = torch.exp(score - z[..., None])
        o = p[..., : c["prefix"]] @ pv[:, None] + p[..., c["prefix"]:] @ vs[:, None]
        out[lo:hi], lse[lo:hi] = o.permute(1, 0, 2, 3).reshape(r, -1), z.permute(1, 0, 2).reshape(r, -1)
    return [out, lse]


def _exact_adjust(s):
    c = s["case"]
    v = c["vocab"]
    x, best = _np(s["logits"]), []
    tokens, length, prompt, draft, start = (s[k].cpu().numpy() for k in ("tokens", "tokens_len", "prompt_len", "draft", "row_start"))
    rep, freq, pres = (_np(s[k]) for k in ("repetition", "frequency", "presence"))
    mask = s["mask"].cpu().numpy().view(np.uint32)
    words = s["allowed"].cpu().numpy().view(np.uint8) if c["masks"] else None
    for r, b in enumerate(s["seq"].tolist()):
        mine = [draft[start[b] + j] for j in range(start[b + 1] - start[b]) if mask[r, j // 32] >> np.uint32(j % 32) & np.uint32(1)]
        ids, times = np.unique(np.concatenate([tokens[b, prompt[b]: length[b]], mine]).astype(int), return_counts=True)
        seen = np.union1d(ids, tokens[b, : min(prompt[b], length[b])])
        x[r, seen] = np.where(x[r, seen] > 0, x[r, seen] / rep[b], x[r, seen] * rep[b])
        x[r, ids] -= freq[b] * times + pres[b]
        if c["bias"]:
            k = int(s["bias_len"][b])
            x[r, s["bias_tokens"][b, :k].cpu().numpy()] += _np(s["bias"][b, :k])
        state = int(s["allowed_row"][r]) if c["masks"] else -1
        if state >= 0:
            x[r, np.unpackbits(words[state], bitorder="little")[:v] == 0] = -np.inf
        best.append(int(np.argmax(x[r])) if np.max(x[r]) > -np.inf else -1)
    return [x, np.array(best)]
