"""The operators that check drafted trees on the GPU against their float64 definitions.

Tolerances count roundings: u = 2^-24 is half a step of float32, 2^-8 of bfloat16 (relative to the value).
"""
import numpy as np
import pytest

import oracle.drafts as OD
from gpu_util import lib
from test_gpu_branches import HALF, TYPES, U, attn_tol, code, f64, inside, ints, rand, rope_case, tdt

pytestmark = pytest.mark.gpu


def random_tree(rng, n):
    """Parents of n rows: row 0 has none, the others hang below any earlier row."""
    return [-1] + [int(rng.integers(0, i)) for i in range(1, n)] if n else []


def words_of(bits, n=None):
    """bool [rows][n] as int32 words."""
    n = -(-bits.shape[1] // 32) if n is None else n
    b = np.zeros((bits.shape[0], 32 * n), np.uint8)
    b[:, : bits.shape[1]] = bits
    return np.packbits(b, axis=1, bitorder="little").view(np.int32).reshape(bits.shape[0], n)


def bits_of(words):
    w = np.ascontiguousarray(words.cpu().numpy()).view(np.uint8)
    return np.unpackbits(w, axis=1, bitorder="little").astype(bool)


# ---- tables and slots ----------------------------------------------------------------------------------------------------

def slots_case(W, held, fresh, owned, table, ring, state, page, rows, parents=None, words=0, base=0, num_pages=None):
    import torch

    n, width = table.shape
    o = {k: torch.full(shape, 77, dtype=torch.int32, device="cuda") for k, shape in (
        ("new_table", (n, width)), ("new_owned", (n,)), ("new_free_state", (2,)), ("row_start", (n + 1,)), ("ctx_len", (n,)),
        ("seq", (rows,)), ("positions", (rows,)))}
    o["slots"] = torch.full((rows,), 77, dtype=torch.int64, device="cuda")
    o["mask"] = torch.full((rows, words), 77, dtype=torch.int32, device="cuda") if words else None
    o["free_ring"] = ints(ring)
    a = W.step_slots_args(requests=n, rows=rows, num_pages=len(ring) if num_pages is None else num_pages, page_size=page,
                          table_stride=width, base_pos=base, mask_words=words, held=ints(held), fresh=ints(fresh),
                          owned=ints(owned), parents=None if parents is None else ints(parents), page_table=ints(table),
                          free_state=ints(state), **o)
    return a, o


def check_slots(o, want, words):
    for k in ("new_table", "new_owned", "new_free_state", "row_start", "ctx_len", "seq", "positions", "slots"):
        np.testing.assert_array_equal(o[k].cpu().numpy(), want[k], err_msg=k)
    np.testing.assert_array_equal(o["free_ring"].cpu().numpy(), want["ring"])
    if words:
        np.testing.assert_array_equal(bits_of(o["mask"]), want["mask"])


def state_of(rng, held, page, width, spare, extra=1):
    """Owned pages, their table and a ring with `spare` free pages that starts anywhere."""
    owned = np.array([-(-max(0, h) // page) if h >= 0 else int(rng.integers(0, width + 1)) for h in held])
    owned = np.minimum(owned + rng.integers(0, extra + 1, len(held)), width)
    pages = int(owned.sum()) + spare + 3
    ids = rng.permutation(pages)
    table, at = np.full((len(held), width), -1), 0
    for s, k in enumerate(owned):
        table[s, :k] = ids[at: at + k]
        at += k
    ring, first = np.full(pages, -5), int(rng.integers(0, pages))
    ring[(first + np.arange(spare)) % pages] = ids[at: at + spare]
    return owned, table, ring, (first, spare)


SLOT_CASES = [
    # requests, most rows, most tokens, page, tree, ended, spare pages (None: enough)
    (1, 1, 0, 16, True, 0, None),
    (1, 8, 40, 16, True, 0, None),
    (2, 1, 100, 1, False, 1, None),
    (7, 33, 65, 8, True, 2, None),       # masks of two words
    (40, 12, 300, 4, True, 5, 30),       # pages run out
    (5, 700, 10, 64, False, 0, None),    # prompts: chains of more rows than a block
    (300, 5, 64, 16, True, 40, 200),     # more requests than threads
    (3, 256, 20, 32, True, 1, None),     # the largest trees
    (4, 6, 30, 16, True, 4, None),       # every request ended
    (700, 1, 9, 1024, False, 9, 0),      # no page is free
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("c", SLOT_CASES, ids=str)
def test_step_slots(c, in_place):
    import torch

    W = lib()
    n, most, tokens, page, tree, ended, spare = c
    rng = np.random.default_rng(n * 1000 + most)
    fresh, held = rng.integers(0 if most > 1 else 1, most + 1, n), rng.integers(0, tokens + 1, n)
    fresh[0] = most
    held[rng.permutation(n)[:ended]] = -1
    live = [int(f) if h >= 0 else 0 for f, h in zip(fresh, held)]
    width = -(-(tokens + most) // page) + 1
    lack = sum(-(-(h + f) // page) for h, f in zip(held, live) if h >= 0)
    owned, table, ring, state = state_of(rng, held, page, width, lack if spare is None else spare)
    rows, words = sum(live) + 5, -(-most // 32) if tree else 0
    parents = np.concatenate([random_tree(rng, f) for f in live] + [[-9] * 5]).astype(int) if tree else None
    a, o = slots_case(W, held, fresh, owned, table, ring, state, page, rows, parents, words, base=11)
    if in_place:
        now = ints(table)
        a.set("page_table", now).set("new_table", now)
        o["new_table"] = now
    W.gemv_device_errors()
    W.step_slots(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    want = OD.step_slots(held, fresh, owned, table, ring, state, page, rows, parents, 11, words, in_place=in_place)
    check_slots(o, want, words)
    assert np.sum((want["ctx_len"] < 0) & (held >= 0)) == 0 or spare is not None
    if not in_place:
        W.step_slots(a)  # the same inputs again: the ring's returned pages are written where they were
        torch.cuda.synchronize()
        check_slots(o, want, words)


def test_step_slots_without_row_outputs():
    """Only tables and lengths; masks of chains without parents; rows without masks."""
    import torch

    W = lib()
    rng = np.random.default_rng(0)
    held, fresh = np.array([5, 0, -1, 30]), np.array([3, 40, 2, 1])
    owned, table, ring, state = state_of(rng, held, 4, 12, 20)
    for keep in ((), ("seq",), ("positions", "slots"), ("mask",)):
        a, o = slots_case(W, held, fresh, owned, table, ring, state, 4, 50, words=2 if "mask" in keep else 0)
        for k in ("seq", "positions", "slots", "mask"):
            if k not in keep:
                a.set(k, None)
        W.step_slots(a)
        torch.cuda.synchronize()
        want = OD.step_slots(held, fresh, owned, table, ring, state, 4, 50, None, 0, 2 if "mask" in keep else 0)
        for k in ("new_table", "new_owned", "new_free_state", "row_start", "ctx_len") + tuple(k for k in keep if k != "mask"):
            np.testing.assert_array_equal(o[k].cpu().numpy(), want[k], err_msg=k)
        if "mask" in keep:
            np.testing.assert_array_equal(bits_of(o["mask"]), want["mask"])
    assert W.gemv_device_errors() == 0


def test_step_slots_of_broken_trees():
    """Rows whose parent is no earlier row of their request, and rows below them, are left out and reported."""
    import torch

    W = lib()
    rng = np.random.default_rng(1)
    held, fresh = np.array([3, 9, 2]), np.array([6, 5, 4])
    parents = [7, 0, 2, -1, 1, 3] + [-1, 0, 5, 0, 3] + [0, 0, 2**31 - 1, -2**31]
    owned, table, ring, state = state_of(rng, held, 4, 6, 9)
    a, o = slots_case(W, held, fresh, owned, table, ring, state, 4, 15, parents, 1)
    W.gemv_device_errors()
    W.step_slots(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0x100
    want = OD.step_slots(held, fresh, owned, table, ring, state, 4, 15, parents, 0, 1)
    assert (want["seq"] == -1).sum() == 6
    check_slots(o, want, 1)


def test_step_slots_that_do_not_fit():
    """More rows than a mask has bits, tokens past the table's width, rows past the outputs: not served, reported."""
    import torch

    W = lib()
    rng = np.random.default_rng(2)
    held = np.array([3, 60, 2, 1])
    owned, table, ring, state = state_of(rng, held, 4, 16, 40)
    for fresh, rows, bits, limit in (([2, 3, 33, 1], 60, 0x100, 32), ([2, 9, 4, 1], 60, 0x80, 32), ([2, 3, 20, 2], 25, 0x80, 32)):
        parents = np.concatenate([random_tree(rng, f) for f in fresh] + [np.zeros(60, int)])[:rows]
        a, o = slots_case(W, held, np.array(fresh), owned, table, ring, state, 4, rows, parents, 1)
        W.gemv_device_errors()
        W.step_slots(a)
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == bits
        want = OD.step_slots(held, fresh, owned, table, ring, state, 4, rows, parents, 0, 1, limit)
        assert sorted(want["ctx_len"].tolist()) == sorted(-1 if i == (2 if fresh[2] == 33 else 1 if fresh[1] == 9 else 3) else int(h)
                                                          for i, h in enumerate(held))
        check_slots(o, want, 1)


def test_step_slots_with_a_broken_state():
    """A ring state outside the ring, owned counts outside the table, entries outside the pool, more returned pages than
    there is room for: reported, and nothing outside the arrays is written."""
    import torch

    W = lib()
    rng = np.random.default_rng(3)
    held, fresh = np.array([3, 5, -1]), np.array([2, 2, 0])
    owned, table, ring, state = state_of(rng, held, 4, 6, 9, extra=0)
    for kw in ({"state": (-1, 3)}, {"state": (0, len(ring) + 1)}, {"state": (len(ring), 1)}, {"owned": [1, 7, 1]},
               {"owned": [-1, 2, 1]}, {"ring": np.full(len(ring), len(ring)), "fresh": np.array([2, 9, 0])},
               {"table": np.full_like(table, -1)}, {"owned": [1, 2, 6], "state": (4, len(ring) - 2)}):
        c = {**dict(owned=owned, table=table, ring=ring, state=state, fresh=fresh), **kw}
        a, o = slots_case(W, held, c["fresh"], c["owned"], c["table"], c["ring"], c["state"], 4, 16)
        guard = torch.full((len(ring) + 64,), 5, dtype=torch.int32, device="cuda")
        guard[32: 32 + len(ring)] = ints(c["ring"])
        a.set("free_ring", guard[32: 32 + len(ring)])
        W.gemv_device_errors()
        W.step_slots(a)
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == 0x80, kw
        assert (guard[:32] == 5).all() and (guard[32 + len(ring):] == 5).all()
        s = o["slots"].cpu().numpy()
        assert ((s >= -1) & (s < 4 * len(ring))).all()


def test_step_slots_of_no_requests():
    import torch

    W = lib()
    a, o = slots_case(W, np.zeros(0), np.zeros(0), np.zeros(0), np.zeros((0, 2), int), [3, 1, 2, 0], (1, 2), 4, 7, words=1)
    W.step_slots(a)
    torch.cuda.synchronize()
    assert o["row_start"].tolist() == [0] and o["new_free_state"].tolist() == [1, 2] and W.gemv_device_errors() == 0
    assert (o["seq"] == -1).all() and (o["positions"] == -1).all() and (o["slots"] == -1).all() and (o["mask"] == 0).all()


# ---- append by slots -------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("c", [(9, 4, 2, 16, 16, 0, "f32", "f32", "bf16", 4), (70, 16, 8, 128, 128, 0, "bf16", "bf16", "bf16", 16),
                               (33, 0, 3, 80, 40, 1, "f32", "f32", "f32", 1), (5, 2, 1, 64, 64, 1, "bf16", "f32", "bf16", 64)], ids=str)
def test_kv_append_slots_is_the_append_by_tables(c):
    """The bits of kv_append_paged where a table leads to the same places; rows of slot -1 and padded rows store nothing."""
    import torch

    W = lib()
    rows, n_q, n_kv, d, rot, inter, x, y, kv, page = c
    rng = np.random.default_rng(rows)
    s, a, pos, _ = rope_case(W, rows, n_q, n_kv, d, rot, inter, x, y, pad=(2,), far=50)
    width = -(-rows // page)
    pages = width + 2
    table = rng.permutation(pages)[:width]
    v = rand((rows, n_kv * d), x, 9)
    both = dict(v=v, v_stride=n_kv * d, kvdtype=code(W, kv), num_pages=pages, page_size=page)
    idx = np.arange(rows)
    slots = table[idx // page].astype(np.int64) * page + idx % page
    got = []
    for by_slots in (False, True):
        pools = [torch.full((pages, n_kv, page, d), 3.0, device="cuda").to(tdt(kv)) for _ in range(2)]
        s["q_out"][0].fill_(7.0)
        if by_slots:
            W.kv_append_slots(W.kv_slots_args(k_pages=pools[0], v_pages=pools[1], **both, **a,
                                              slots=torch.tensor(slots, dtype=torch.int64, device="cuda")))
        else:
            W.kv_append_paged(W.kv_append_args(k_pages=pools[0], v_pages=pools[1], page_table=ints(table[None]),
                                               seq=ints(np.zeros(rows)), n_seq=1, table_stride=width, base_pos=50, **both, **a))
        torch.cuda.synchronize()
        got.append([s["q_out"][0].clone(), *pools])
    assert W.gemv_device_errors() == 0
    for p, q in zip(*got):
        assert torch.equal(p, q)
    # rows without a slot: every query is written, their places keep what they held
    slots[1::2] = -1
    pools = [torch.full((pages, n_kv, page, d), 3.0, device="cuda").to(tdt(kv)) for _ in range(2)]
    W.kv_append_slots(W.kv_slots_args(k_pages=pools[0], v_pages=pools[1], **both, **a,
                                      slots=torch.tensor(slots, dtype=torch.int64, device="cuda")))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0 and torch.equal(got[0][0], s["q_out"][0])
    at = torch.tensor([table[i // page] for i in range(1, rows, 2)], device="cuda"), torch.arange(1, rows, 2, device="cuda") % page
    for p, full in zip(pools, got[0][1:]):
        want = full.clone()
        want[at[0], :, at[1]] = 3.0
        assert torch.equal(p, want)


@pytest.mark.parametrize("x,kv,d", [("bf16", "bf16", 128), ("f32", "bf16", 40)])
def test_kv_append_slots_in_place_in_a_fused_buffer(x, kv, d):
    """Queries over themselves, keys and values the columns beside them: the bits of a call with buffers of its own."""
    import torch

    W = lib()
    rows, n_q, n_kv, page = 37, 4, 2, 16
    wide = (n_q + 2 * n_kv) * d
    qkv = rand((rows, wide), x, 1)
    freq, factor = W.rope_frequencies(d, 1e4)
    kw = dict(rows=rows, n_q=n_q, n_kv=n_kv, head_dim=d, xdtype=code(W, x), ydtype=code(W, x), kvdtype=code(W, kv), q_stride=wide,
              k_stride=wide, v_stride=wide, g_q=rand((d,), "f32", 2), g_k=rand((d,), "f32", 3), positions=ints(np.arange(rows) * 7),
              inv_freq=torch.tensor(freq, dtype=torch.float64, device="cuda"), eps=1e-6, rope_factor=factor, rot_dim=d, interleaved=0,
              slots=torch.arange(rows, device="cuda").flip(0) + 5, num_pages=4, page_size=page)
    pools, own = torch.zeros((2, 4, n_kv, page, d), device="cuda").to(tdt(kv)), torch.zeros((2, 4, n_kv, page, d), device="cuda").to(tdt(kv))
    q_out = torch.zeros((rows, n_q * d), dtype=tdt(x), device="cuda")
    cols = [qkv, qkv[:, n_q * d:], qkv[:, (n_q + n_kv) * d:]]
    W.kv_append_slots(W.kv_slots_args(q=cols[0], k=cols[1], v=cols[2], q_out=q_out, q_out_stride=n_q * d, k_pages=pools[0], v_pages=pools[1], **kw))
    keep = qkv.clone()
    W.kv_append_slots(W.kv_slots_args(q=cols[0], k=cols[1], v=cols[2], q_out=qkv, q_out_stride=wide, k_pages=own[0], v_pages=own[1], **kw))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    assert torch.equal(qkv[:, : n_q * d], q_out) and torch.equal(pools, own) and torch.equal(qkv[:, n_q * d:], keep[:, n_q * d:])


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_tree_accept_paged_of_keys_and_values_that_alternate(kv):
    """One buffer with every layer's keys in front of its values: the pools' layers lie between each other."""
    import torch

    W = lib()
    rows, lens, page = [9, 12], [5, 17], 4
    a, t = accept_case(W, rows, lens, 3, 2, 16, page, kv, 8, seed=2)
    both = torch.stack(t["pools"], 1).contiguous()  # [layer][keys, values][pages]..
    t["pools"] = [both[:, 0], both[:, 1]]
    a.set("k_pages", t["pools"][0]).set("v_pages", t["pools"][1])
    a.layer_stride = both.stride(0)
    W.gemv_device_errors()
    W.tree_accept_paged(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    assert check_accept(t, rows, lens, page, 8) > 1


def test_kv_append_slots_outside_the_pool():
    import torch

    W = lib()
    s, a, pos, _ = rope_case(W, 6, 2, 1, 16, 16, 0, "f32", "f32")
    v = rand((6, 16), "f32", 5)
    pools = torch.full((2, 8, 1, 4, 16), 3.0, device="cuda")  # the calls get pages 2 to 5 as their pool
    slots = torch.tensor([0, 15, 16, -2, 2**62, -2**62], dtype=torch.int64, device="cuda")
    W.gemv_device_errors()
    W.kv_append_slots(W.kv_slots_args(v=v, v_stride=16, kvdtype=W.DEC_F32, num_pages=4, page_size=4, k_pages=pools[0, 2:6],
                                      v_pages=pools[1, 2:6], slots=slots, **a))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0x80
    want = torch.full_like(pools[1], 3.0)
    want[2, 0, 0], want[5, 0, 3] = v[0], v[1]
    assert torch.equal(pools[1], want) and ((pools[0] != 3.0).any(-1) == (want != 3.0).any(-1)).all()


# ---- attention -------------------------------------------------------------------------------------------------------------

def tree_case(W, rows, n_q, n_kv, d, plen, lens, page, q, kv, mask="tree", seed=0, poison=True, lse=True, extra=0, width=None,
              scale=None, lead=0, tail=0, stride=None, words=None):
    """A call's arguments. rows: of each request; lead, tail: rows of no request in front and behind. mask: "tree", "chain"
    (none), "random" (any rows, none among them) or "none" (empty). poison: NaN and infinities in all of the caches that no
    row may use."""
    import torch

    rng = np.random.default_rng(seed)
    batch, total = len(rows), sum(rows) + lead + tail
    stride = plen if stride is None else stride
    need = [-(-(max(0, n) + r) // page) if n >= 0 else 0 for n, r in zip(lens, rows)]
    width = max(max(need), 1) if width is None else width
    pages = sum(need) + 2
    ids, table, at = rng.permutation(pages), np.full((batch, width), -1), 0
    for b, k in enumerate(need):
        table[b, : min(k, width)] = ids[at: at + min(k, width)]
        at += k
    seen = []
    for r in rows:
        if mask == "tree":
            seen.append(np.array([x[0] for x in OD.ancestors(random_tree(rng, r), r)], bool).reshape(r, r))
        elif mask == "chain":
            seen.append(np.tril(np.ones((r, r), bool)))
        else:
            seen.append(rng.random((r, r)) < (0.4 if mask == "random" else 0.0))
            if mask == "random" and r:
                seen[-1][rng.integers(0, r)] = False
    m = None
    if mask != "chain":
        words = max(1, -(-max(rows) // 32)) if words is None else words
        bits = np.zeros((total, 32 * words), bool)
        at = lead
        for s in seen:
            bits[at: at + len(s), : s.shape[1]] = s[:, : 32 * words]
            at += len(s)
        m = ints(words_of(bits, words))
        seen = [s & (np.arange(s.shape[1]) < 32 * words) for s in seen]
    pk, pv = rand((n_kv, stride, d), kv, seed + 1), rand((n_kv, stride, d), kv, seed + 2)
    kp, vp = rand((pages, n_kv, page, d), kv, seed + 3), rand((pages, n_kv, page, d), kv, seed + 4)
    if poison:
        used = np.zeros((pages, page), dtype=bool)
        for b, (n, r) in enumerate(zip(lens, rows)):
            for i in range(n + r if n >= 0 else 0):
                if i < width * page and (i < n or seen[b][:, i - n].any()):
                    used[table[b, i // page], i % page] = True
        u = torch.tensor(used, device="cuda")[:, None, :, None]
        for k, (t, pre) in enumerate(((kp, pk), (vp, pv))):
            t.masked_fill_(~u, float("nan") if k else float("inf"))
            pre[:, plen:] = float("nan")
    qq = rand((total, n_q * d + extra), q, seed + 5, 1.2)
    out = torch.full((total, n_q * d + extra), 7.0, dtype=tdt(q), device="cuda")
    ls = torch.full((total, n_q), 7.0, device="cuda") if lse else None
    a = W.attn_tree_args(
        batch=batch, rows=total, n_q=n_q, n_kv=n_kv, head_dim=d, qdtype=code(W, q), kvdtype=code(W, kv), q=qq, out=out, lse=ls,
        q_stride=n_q * d + extra, out_stride=n_q * d + extra, row_start=ints(lead + np.concatenate([[0], np.cumsum(rows)])),
        mask=m, mask_words=0 if m is None else m.shape[1], prefix_k=pk, prefix_v=pv, prefix_len=plen, prefix_stride=stride,
        k_pages=kp, v_pages=vp, page_table=ints(table), seq_len=ints(lens), num_pages=pages, page_size=page,
        table_stride=width, scale=d ** -0.5 if scale is None else scale)
    a.with_workspace(torch.full((W.attn_tree_paged_workspace(a),), 255, dtype=torch.uint8, device="cuda"))
    return a, dict(q=qq, out=out, lse=ls, pk=pk, pv=pv, kp=kp, vp=vp, table=table, seen=seen, lead=lead)


def check_tree(t, rows, n_q, n_kv, d, plen, lens, page, q, scale=None, skip=(), width=None):
    """Every row against the definition (skip: table entries that are left out); rows of no request unchanged."""
    group = n_q // n_kv
    width = t["table"].shape[1] if width is None else width
    scale = np.float64(np.float32(d ** -0.5 if scale is None else scale))
    total = t["q"].shape[0]
    Q, got = (f64(t[k])[:, : n_q * d].reshape(total, n_kv, group, d) for k in ("q", "out"))
    lse = f64(t["lse"]).reshape(total, n_kv, group) if t["lse"] is not None else None
    PK, PV, KP, VP = f64(t["pk"])[:, :plen], f64(t["pv"])[:, :plen], f64(t["kp"]), f64(t["vp"])
    at, written = t["lead"], np.zeros(total, bool)
    for b, (n, r) in enumerate(zip(lens, rows)):
        mine = slice(at, at + r)
        at += r
        if n < 0 or r == 0:
            continue
        written[mine] = True
        i = np.array([x for x in range(min(n + r, width * page)) if (b, x // page) not in skip], dtype=int)
        pg, sl = t["table"][b, i // page], i % page
        see = np.concatenate([np.ones((r, plen), bool), np.where(i < n, True, t["seen"][b][:, np.maximum(i - n, 0)])], 1)
        used = see.any(0)
        for g in range(n_kv):
            k, v = np.concatenate([PK[g], KP[pg, g, sl]])[used], np.concatenate([PV[g], VP[pg, g, sl]])[used]
            for j in range(r):
                kk, vv, qq = k[see[j][used]], v[see[j][used]], Q[mine][j, g]
                o, l, size = OD.attend(qq[None], kk, vv, [np.ones(len(kk), bool)], scale)
                if not len(kk):
                    assert (got[mine][j, g] == 0).all() and (lse is None or np.isneginf(lse[mine][j, g]).all())
                    continue
                tol, ltol = attn_tol(qq, kk, l[0], o[0], size[0], scale, q)
                inside(got[mine][j, g], o[0], tol, (b, j, g))
                if lse is not None:
                    inside(lse[mine][j, g], l[0], ltol, ("lse", b, j, g))
    assert (got[~written] == 7.0).all() and (lse is None or (lse[~written] == 7.0).all()), "a row of no request was written"


TREE_CASES = [
    # rows of each request, n_q, n_kv, d, prefix, lens, page, mask
    ([1], 1, 1, 8, 0, [0], 1, "chain"),
    ([1], 4, 2, 16, 0, [1], 16, "tree"),
    ([3], 4, 2, 16, 1, [0], 4, "tree"),
    ([2, 0, 5], 6, 2, 24, 5, [1, 7, -1], 8, "tree"),            # no rows, an unused request; group of 3
    ([3, 4], 4, 2, 16, 0, [0, 3], 4, "none"),                   # rows with nothing, rows with their request's tokens only
    ([7, 40, 1], 16, 1, 64, 63, [64, 1, 200], 64, "tree"),      # group of 16; masks of two words
    ([8], 16, 8, 128, 512, [33], 16, "tree"),
    ([16] * 4, 16, 8, 128, 0, [400, 1, 127, 128], 16, "tree"),
    ([1] * 9, 16, 8, 128, 0, [0, 1, 15, 16, 17, 700, -1, 128, 127], 8, "chain"),
    ([5, 9], 10, 2, 80, 129, [40, 31], 32, "random"),
    ([64, 33], 16, 8, 128, 0, [300, 1000], 64, "tree"),
    ([200], 8, 2, 128, 0, [77], 16, "chain"),                   # a prompt's rows behind others
    ([130, 3], 4, 4, 64, 100, [0, 260], 128, "chain"),
    ([90], 12, 4, 128, 30, [500], 1, "tree"),                   # group of 3, pages of one token; masks of three words
    ([21, 2], 5, 1, 96, 0, [140, 3], 2, "tree"),                # heads of a token in two row tiles
    ([13] * 5, 16, 8, 128, 0, [301, 255, 256, 257, 90], 8, "random"),
    ([2] * 33, 8, 4, 128, 257, [(i * 29) % 300 for i in range(33)], 16, "tree"),
    ([6, 250, 3], 16, 2, 128, 40, [10, 300, 2000], 32, "tree"),
    ([4], 2, 2, 128, 3000, [2500], 64, "tree"),                 # long for few rows
    ([70], 32, 2, 64, 0, [900], 16, "random"),
    ([300, 20], 4, 2, 64, 0, [5, 640], 8, "tree"),              # masks of ten words
    ([40, 9], 4, 1, 40, 20, [100, 700], 16, "tree"),            # a request's rows in row tiles of 64, one of them nearly empty
]


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("c", TREE_CASES, ids=lambda c: f"b{len(c[0])}x{max(c[0])}_q{c[1]}_kv{c[2]}_d{c[3]}_p{c[4]}_page{c[6]}_{c[7]}")
def test_attn_tree_paged(c, types):
    import torch

    W = lib()
    rows, n_q, n_kv, d, plen, lens, page, mask = c
    a, t = tree_case(W, rows, n_q, n_kv, d, plen, lens, page, *types, mask=mask, lead=2, tail=3, stride=plen + 37)
    W.gemv_device_errors()
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    check_tree(t, rows, n_q, n_kv, d, plen, lens, page, types[0])
    first = [t["out"].clone(), t["lse"].clone()]
    W.attn_tree_paged(a)  # the same bits again, on a used workspace
    torch.cuda.synchronize()
    assert torch.equal(first[0], t["out"]) and torch.equal(first[1], t["lse"])


def wide(batch, n_kv, page):
    """Entries of tables wide enough that few rows too go to the tensor cores."""
    return max(49 * 153 * 128 // (batch * n_kv * page), 1024 // page) + 1


@pytest.mark.parametrize("c", [c for c in TREE_CASES if c[3] == 128 and c[4] == 0 and c[6] >= 8] + [
    ([1], 2, 1, 128, 0, [0], 8, "chain"), ([2, 0, 5], 6, 2, 128, 0, [1, 7, -1], 8, "tree"), ([3, 4], 4, 2, 128, 0, [0, 3], 8, "none"),
    ([4, 1, 3], 4, 2, 128, 0, [2500, 128, 127], 64, "tree"), ([5], 3, 1, 128, 0, [255], 16, "random")], ids=str)
def test_attn_tree_paged_few_rows_of_wide_tables(c):
    import torch

    W = lib()
    rows, n_q, n_kv, d, plen, lens, page, mask = c
    a, t = tree_case(W, rows, n_q, n_kv, d, plen, lens, page, "bf16", "bf16", mask=mask, lead=2, tail=3, width=wide(len(rows), n_kv, page))
    W.gemv_device_errors()
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    check_tree(t, rows, n_q, n_kv, d, plen, lens, page, "bf16")


@pytest.mark.parametrize("types,d", [(t, d) for t in TYPES for d in (64, 128)], ids=str)
def test_attn_tree_paged_drafts_that_are_not_finite(types, d):
    """Keys and values of drafted rows that are NaN or infinite reach the rows that see them and no others: a chain of 40
    rows whose rows from 25 on see them, and trees of two branches of which one does."""
    import torch

    W = lib()
    n_q, n_kv, page = 4, 2, 16
    for mask, R, odd in (("chain", 40, 25), ("tree", 12, 7)):
        a, t = tree_case(W, [R, 3], n_q, n_kv, d, 20, [90, 200], page, *types, mask=mask, seed=3)
        if mask == "tree":
            par = [-1, 0, 1, 2, 3, 4, 0, 6, 7, 8, 9, 10]  # rows 7 to 11 hang below row 7
            bits = np.array([x[0] for x in OD.ancestors(par, R)])
            t["seen"][0] = bits
            m = t["seen"]
            a.set("mask", ints(words_of(np.concatenate([np.pad(m[0], ((0, 0), (0, 20))), np.pad(m[1], ((0, 0), (0, 29)))]))))
            for pool in (t["kp"], t["vp"]):
                for i in range(90, 90 + R):  # (the drawn tree left some rows unseen)
                    pool[t["table"][0, i // page], :, i % page] = rand((n_kv, d), types[1], 100 + i)
        W.attn_tree_paged(a)
        torch.cuda.synchronize()
        clean = t["out"].clone()
        hit = torch.tensor(np.concatenate([t["seen"][0][:, odd], [False] * 3]), device="cuda")
        assert 0 < hit.sum() < R
        for pool, value in (("vp", float("nan")), ("vp", float("inf")), ("vp", -float("inf")), ("kp", float("nan")), ("kp", float("inf"))):
            keep = t[pool].clone()
            at = t["table"][0, (90 + odd) // page], slice(None), (90 + odd) % page
            t[pool][at][:, d // 2] = value
            t["out"].fill_(7.0)
            W.attn_tree_paged(a)
            torch.cuda.synchronize()
            assert torch.equal(t["out"][~hit], clean[~hit]), (mask, pool, value)
            bad = ~torch.isfinite(t["out"][hit].float().reshape(-1, n_q, d))
            assert bad[..., d // 2].all() or pool == "kp", (mask, pool, value)
            if pool == "kp" and value != value:
                assert bad.all()
            t[pool].copy_(keep)
    assert W.gemv_device_errors() == 0


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16")], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_attn_tree_paged_drafts_that_are_not_finite_in_every_request(types, d):
    """Several hundred short requests without a prefix, each with a drafted value that is not finite in every head: a CTA has
    one such piece after the other, each of one tile. Rows that see it are not finite, the others hold the bits they have
    without it."""
    import torch

    W = lib()
    n_q, n_kv, page, B, R, odd = 16, 8, 16, 300, 16, 3
    lens = [(7 * i) % 90 for i in range(B)]
    a, t = tree_case(W, [R] * B, n_q, n_kv, d, 0, lens, page, *types, seed=11, poison=False)
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    clean = t["out"].clone()
    hit = torch.tensor(np.concatenate([s[:, odd] for s in t["seen"]]), device="cuda")
    assert B <= hit.sum() < B * R
    i = np.array(lens) + odd
    at = torch.tensor(t["table"][np.arange(B), i // page], device="cuda").long(), slice(None), torch.tensor(i % page, device="cuda")
    t["vp"][at + (d - 1,)] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").repeat(100)[:, None].to(t["vp"].dtype)
    for _ in range(10):
        t["out"].fill_(7.0)
        W.attn_tree_paged(a)
        torch.cuda.synchronize()
        assert torch.equal(t["out"][~hit], clean[~hit])
        assert not torch.isfinite(t["out"][hit].view(-1, n_q, d)[..., d - 1]).any()
        assert torch.equal(t["out"][hit].view(-1, n_q, d)[..., : d - 1], clean[hit].view(-1, n_q, d)[..., : d - 1])
    assert W.gemv_device_errors() == 0


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_attn_tree_paged_strides_and_no_lse(types, d):
    import torch

    W = lib()
    rows, lens = [9, 1, 0, 30], [40, 300, 5, 129]
    a, t = tree_case(W, rows, 4, 2, d, 70, lens, 16, *types, extra=5, lse=False, scale=0.3, width=40, words=2)
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    check_tree(t, rows, 4, 2, d, 70, lens, 16, types[0], scale=0.3)
    assert (f64(t["out"])[:, 4 * d:] == 7.0).all()


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_attn_tree_paged_negative_scale(types, scale):
    import torch

    W = lib()
    rows, lens = [9, 20], [140, 33]
    a, t = tree_case(W, rows, 4, 2, 128, 200, lens, 16, *types, scale=scale)
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    t2 = {**t, "q": -t["q"]} if scale < 0 else t
    check_tree(t2, rows, 4, 2, 128, 200, lens, 16, types[0], scale=abs(scale))


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("q", ["bf16", "f32"])
def test_attn_tree_paged_large_scores(q, kv):
    """Scores of hundreds in rising and falling order: the running maximum moves often and far."""
    import torch

    W = lib()
    rows, lens = [5, 17], [700, 650]
    a, t = tree_case(W, rows, 4, 2, 128, 300, lens, 64, q, kv, seed=2, poison=False)
    ramp = torch.linspace(0, 30, 300, device="cuda")
    t["pk"][0] *= ramp[:, None].to(t["pk"].dtype)
    t["pk"][1] *= ramp.flip(0)[:, None].to(t["pk"].dtype)
    t["kp"][:, 0] *= torch.linspace(0, 30, 64, device="cuda")[:, None].to(t["kp"].dtype)
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    check_tree(t, rows, 4, 2, 128, 300, lens, 64, q)


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 64])
def test_attn_tree_paged_long_sums_are_not_cut_off(R, kv):
    """Float32 results over thousands of values of one sign. A matrix instruction cuts its sums off instead of rounding them:
    a block's three lose up to 2 u each, whatever the number of blocks; that of all blocks is rounded, as are reciprocal and
    product (one u each; the errors of probabilities enter numerator and denominator alike, those of rounded sums have no
    sign). So the mean relative error of the results lies within 6 u + 2 u, and 8 u for what is left of the errors without a
    sign. Sums that are cut off block by block lose some 1.5 u a block: 100 to 500 u here."""
    import torch

    W = lib()
    batch, n_q, n_kv, d, ctx, page = 24, 16, 8, 128, 4096, 64
    a, t = tree_case(W, [R] * batch, n_q, n_kv, d, 0, [ctx] * batch, page, "f32", kv, mask="chain", poison=False)
    for b in range(len(t["vp"])):
        t["vp"][b].uniform_(1, 2)
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    errors = []
    for b in (0, 11, 23):
        pages = torch.tensor(t["table"][b], device="cuda").long()
        k, v = (t[x][pages].transpose(0, 1).reshape(n_kv, -1, d)[:, : ctx + R].double() for x in ("kp", "vp"))
        q = t["q"].double().view(batch, R, n_kv, n_q // n_kv, d)[b]
        s = torch.einsum("rghd,gkd->ghrk", q, k) * d ** -0.5
        s.masked_fill_(torch.arange(ctx + R, device="cuda") > ctx + torch.arange(R, device="cuda")[:, None], -float("inf"))
        want = torch.einsum("ghrk,gkd->rghd", torch.softmax(s, -1), v)
        errors.append((t["out"].double().view(batch, R, n_kv, n_q // n_kv, d)[b] / want - 1).mean().item())
    assert max(map(abs, errors)) <= 16 * U, [e / U for e in errors]


@pytest.mark.parametrize("kv,d,R,batch,ctx", [("bf16", 128, 64, 24, 1 << 17), ("bf16", 64, 64, 24, 1 << 17), ("bf16", 96, 64, 24, 1 << 18),
                                              ("bf16", 96, 1, 96, 1 << 20), ("f32", 128, 64, 24, 1 << 17), ("f32", 128, 1, 24, 1 << 19)], ids=str)
def test_attn_tree_paged_bfloat16_results_of_long_sums_round_as_they_should(kv, d, R, batch, ctx):
    """Bfloat16 results next to a border: values are 1 or 1 + 2^-7, chosen so that a result is 1 + 2^-8 (a border) and 2^-14
    (1024 u) more in even elements, less in odd ones; the choice leaves out at most the largest of 2^14 probabilities (2^-13
    of 2^-7: 16 u). Matrix instructions cut up to 256 sums of a result off before these are added up rounded, by up to 2 u
    each of a sum that grows evenly: 256 u. Weights enter by 2^-7: 2^-24 of each. What rounded sums of some thousand terms
    lose has no sign: 64 u are more than what the root of their number gives. So 340 u are enough. Cut off all along, a
    result loses a quarter of u for every instruction: 3,800 u and more here. (One request's pages serve all, over and
    over.)"""
    import torch

    W = lib()
    n_q, n_kv, page, own = 16, 8, 64, 1 << 14
    a, t = tree_case(W, [R] * batch, n_q, n_kv, d, 0, [0] * batch, page, "bf16", kv, mask="none", poison=False, lse=False)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((own // page, n_kv, page, d), generator=g, device="cuda").to(tdt(kv))
    q = torch.randn((n_kv, d), generator=g, device="cuda").bfloat16()
    scale = float(np.float32(0.1 * d ** -0.5))
    s = torch.einsum("gd,gkd->gk", q.double(), k.transpose(0, 1).reshape(n_kv, own, d).double()) * scale
    p = torch.softmax(s, -1)
    assert p.max() < 2.0 ** -13
    order = torch.rand((n_kv, d, own), generator=g, device="cuda").argsort(-1)
    weight = torch.gather(p[:, None].expand(-1, d, -1), -1, order).cumsum(-1)
    target = torch.tensor([0.5 + 2.0 ** -7, 0.5 - 2.0 ** -7], dtype=torch.float64, device="cuda").repeat(d // 2)
    high = torch.zeros_like(order, dtype=torch.bool).scatter_(-1, order, weight <= target[:, None])
    v = (1 + high.transpose(1, 2).double() / 128).view(n_kv, own // page, page, d).transpose(0, 1).contiguous().to(tdt(kv))
    t["q"].copy_(q.repeat_interleave(n_q // n_kv, 0).reshape(1, -1).expand(batch * R, -1))
    table = torch.arange(own // page, dtype=torch.int32, device="cuda").repeat(batch, (ctx + R) // own + 1)
    a.set("k_pages", k).set("v_pages", v).set("page_table", table).set("seq_len", ints([ctx] * batch))
    a.num_pages, a.table_stride, a.scale = own // page, table.shape[1], scale
    a.with_workspace(torch.empty(W.attn_tree_paged_workspace(a), dtype=torch.uint8, device="cuda"))
    W.gemv_device_errors()
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    out = t["out"].view(batch * R * n_q, d).float()
    assert (out[:, ::2] == 1 + 2.0 ** -7).all() and (out[:, 1::2] == 1.0).all(), [x.unique(return_counts=True) for x in (out[:, ::2], out[:, 1::2])]


@pytest.mark.parametrize("types,d,plen", [(("bf16", "bf16"), 128, 0), (("bf16", "bf16"), 128, 300), (("bf16", "bf16"), 64, 0),
                                          (("f32", "f32"), 128, 0), (("f32", "bf16"), 96, 50)], ids=str)
@pytest.mark.parametrize("full", [False, True])
def test_attn_tree_paged_in_place(types, d, plen, full):
    """The output over the queries, unused requests left as they are: the bits of a call with buffers of its own."""
    import torch

    W = lib()
    rows = [(3 * i) % 11 for i in range(20)]
    lens = [(37 * i) % 400 - 1 for i in range(20)]
    a, t = tree_case(W, rows, 8, 4, d, plen, lens, 16, *types, tail=2, width=wide(20, 4, 16) if full else None)
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    live = torch.tensor(np.repeat(np.array(lens) >= 0, rows).tolist() + [False] * 2, device="cuda")
    want = torch.where(live[:, None], t["out"], t["q"])
    for _ in range(5):
        q = t["q"].clone()
        a.set("q", q).set("out", q)
        W.attn_tree_paged(a)
        torch.cuda.synchronize()
        assert torch.equal(q, want)


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_attn_tree_paged_bad_pages(types, d):
    """Entries outside the pool are left out and reported; so are tokens and rows past the table's width."""
    import torch

    W = lib()
    rows, lens, page = [3, 5, 2, 6], [40, 180, 40, 60], 16
    a, t = tree_case(W, rows, 4, 2, d, 30, lens, page, *types, poison=False)
    bad = t["table"].copy()
    bad[0, 1], bad[1, 0], bad[1, 9], bad[2, 2] = -1, a.num_pages, -2**31, 2**31 - 1
    a.set("page_table", ints(bad))
    W.gemv_device_errors()
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0x80
    check_tree(t, rows, 4, 2, d, 30, lens, page, types[0], skip={(0, 1), (1, 0), (1, 9), (2, 2)})
    for width, held in ((3, [40, 2**31 - 1, 40, 45]), (0, [0, 0, 0, 0])):
        a, t = tree_case(W, rows, 4, 2, d, 30 if width else 0, [40, 48, 40, 45] if width else held, page, *types, width=max(width, 1))
        a.set("seq_len", ints(held))
        a.table_stride = width
        if width:
            a.set("page_table", ints(t["table"][:, :3]))
        W.attn_tree_paged(a)
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == 0x80
        if width:
            check_tree(t, rows, 4, 2, d, 30, [40, 48, 40, 45], page, types[0], width=3)
        else:
            assert (t["out"] == 0).all() and torch.isneginf(t["lse"]).all()


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")], ids=str)
@pytest.mark.parametrize("full", [False, True])
def test_attn_tree_paged_row_starts_that_fall(types, full):
    """Starts outside the rows or falling are taken as the highest start so far: rows and workspace stay inside."""
    import torch

    W = lib()
    a, t = tree_case(W, [4, 4, 4, 4], 4, 2, 128, 0, [20, 30, 40, 50], 16, *types, mask="chain", width=wide(4, 2, 16) if full else None)
    good = t["out"].clone()
    for starts in ([0, 16, 0, 16, 16], [-5, 4, 2, 8, 99], [16, 0, 16, 0, 16], [2**31 - 1, -2**31, 3, 3, 3]):
        a.set("row_start", ints(starts))
        t["out"].fill_(7.0)
        W.attn_tree_paged(a)
        torch.cuda.synchronize()
        top = np.maximum.accumulate(np.clip(np.array(starts), 0, 16))
        live = np.zeros(16, bool)
        for b in range(4):
            live[top[b]: top[b + 1]] = True
        assert ((t["out"] != 7.0).any(1).cpu().numpy() == live).all(), starts
    assert good is not None


@pytest.mark.parametrize("types,d,plen", [(("bf16", "bf16"), 128, 0), (("bf16", "bf16"), 128, 40), (("bf16", "bf16"), 96, 0), (("f32", "f32"), 64, 0),
                                          (("f32", "bf16"), 128, 300)], ids=str)
@pytest.mark.parametrize("batch,R", [(3, 40), (33, 6), (70, 9), (300, 3)])
def test_attn_tree_paged_row_starts_that_fall_are_the_highest_so_far(batch, R, types, d, plen):
    """Starts that fall or lie outside the rows: the bits of a call whose starts are the highest so far."""
    import torch

    W = lib()
    rng = np.random.default_rng(batch + plen)
    lens = rng.integers(-1, 200, batch).tolist()
    a, t = tree_case(W, [R] * batch, 4, 2, d, plen, lens, 16, *types, mask="random", poison=False, seed=batch)
    total = batch * R
    rises = np.arange(batch + 1) * R
    for k in range(4):
        starts = rises.copy()
        at = rng.permutation(batch + 1)[: max(1, (batch + 1) // (1, 2, 4, 12)[k])]
        starts[at] = rng.integers(-R, total + R, len(at)) if k % 2 else rng.choice([-2**31, 2**31 - 1, 0, total, 5], len(at), p=[0.4, 0.1, 0.2, 0.1, 0.2])
        got = []
        for x in (starts, np.maximum.accumulate(np.clip(starts, 0, total))):
            a.set("row_start", ints(x))
            t["out"].fill_(7.0), t["lse"].fill_(7.0)
            W.gemv_device_errors()
            W.attn_tree_paged(a)
            torch.cuda.synchronize()
            got.append([t["out"].clone(), t["lse"].clone(), W.gemv_device_errors()])
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and got[0][2] == got[1][2], (k, starts)


def test_attn_tree_paged_many_requests():
    """More requests than threads of a CTA, most of them without rows."""
    import torch

    W = lib()
    rng = np.random.default_rng(5)
    rows = (rng.random(4096) < 0.02).astype(int) * rng.integers(1, 4, 4096)
    rows[[0, 4095]] = 2
    lens = rng.integers(-1, 60, 4096)
    lens[[0, 4095]] = 30, 45
    for types, width in ((("bf16", "bf16"), None), (("bf16", "bf16"), wide(4096, 1, 8)), (("f32", "f32"), None)):
        a, t = tree_case(W, rows.tolist(), 2, 1, 128, 0, lens.tolist(), 8, *types, poison=False, width=width)
        W.gemv_device_errors()
        W.attn_tree_paged(a)
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == 0
        check_tree(t, rows.tolist(), 2, 1, 128, 0, lens.tolist(), 8, types[0])


@pytest.mark.parametrize("page", [4, 64])
def test_attn_tree_paged_pools_past_32_bits(page):
    """Pages whose first element lies past 2^31 elements and 2^32 bytes."""
    import torch

    W = lib()
    n_kv, d, pages = 8, 128, 33000 * 64 // page
    a, t = tree_case(W, [5, 2], 16, n_kv, d, 0, [70, 64], page, "bf16", "bf16", poison=False)
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    small = t["out"].clone()
    far = torch.zeros((2, pages, n_kv, page, d), dtype=torch.bfloat16, device="cuda")
    have = t["table"] >= 0
    table = np.where(have, pages - 1 - np.cumsum(have).reshape(have.shape), -1).astype(np.int32)
    for k, name in enumerate(("kp", "vp")):
        far[k, torch.tensor(table[have], device="cuda").long()] = t[name][torch.tensor(t["table"][have], device="cuda").long()]
    a.set("k_pages", far[0]).set("v_pages", far[1]).set("page_table", ints(table))
    a.num_pages = pages
    t["out"].fill_(7.0)
    W.attn_tree_paged(a)
    torch.cuda.synchronize()
    assert torch.equal(small, t["out"]) and W.gemv_device_errors() == 0


def test_attn_tree_paged_of_single_rows_is_the_branches_attention():
    """One row a request over prefix and pages: the values of attn_shared_prefix, whose last own token is the row's."""
    import torch

    W = lib()
    lens, page, d = [33, 0, 5, 250, -1], 16, 128
    a, t = tree_case(W, [1] * 5, 16, 8, d, 300, lens, page, "bf16", "bf16", mask="chain")
    W.attn_tree_paged(a)
    out = torch.full_like(t["out"], 7.0)
    b = W.attn_shared_args(batch=5, n_q=16, n_kv=8, head_dim=d, qdtype=W.DEC_BF16, kvdtype=W.DEC_BF16, q=t["q"], out=out,
                           q_stride=16 * d, out_stride=16 * d, prefix_k=t["pk"], prefix_v=t["pv"], prefix_len=300,
                           prefix_stride=300, k_pages=t["kp"], v_pages=t["vp"], page_table=ints(t["table"]),
                           seq_len=ints([n + 1 if n >= 0 else -1 for n in lens]), num_pages=t["kp"].shape[0], page_size=page,
                           table_stride=t["table"].shape[1], scale=d ** -0.5)
    b.with_workspace(torch.empty(W.attn_shared_prefix_workspace(b), dtype=torch.uint8, device="cuda"))
    W.attn_shared_prefix(b)
    torch.cuda.synchronize()
    # both round to bfloat16 once, of values that differ by the products' roundings
    assert (t["out"].float() - out.float()).abs().max() <= 2 * 2.0 ** -8 * out.float().abs().max()
    check_tree(t, [1] * 5, 16, 8, d, 300, lens, page, "bf16")


# ---- logits ------------------------------------------------------------------------------------------------------------------

def adjust_case(W, rows, vocab, x, y, seed=0, history=50, drafts=True, bias=4, masks=2, penalties=True, extra=0, offset=0,
                mask=True, in_place=False, prompt=True, base=0, far=False):
    """rows: of each request; far: text and drafts over the whole vocabulary. Returns arguments and what the definition takes."""
    import torch

    rng = np.random.default_rng(seed)
    n, total = len(rows), sum(rows)

    def buffer(dtype, fill=None):
        t = rand((total * (vocab + extra) + offset,), dtype, seed + 1, 3.0) if fill is None else torch.full(
            (total * (vocab + extra) + offset,), fill, dtype=tdt(dtype), device="cuda")
        return t, t[offset:].view(total, vocab + extra)[:, :vocab]

    xs, ys = buffer(x), buffer(y, 7.0)
    if in_place:
        ys = xs
    p = dict(logits=f64(xs[1]), rows=rows, seq=np.repeat(np.arange(n), rows), start=np.concatenate([[0], np.cumsum(rows)]))
    p["tokens"] = rng.integers(-1, vocab + 2 if far else max(2, min(vocab + 2, 40)), (n, history + 3))  # out of range ones too
    p["len"] = np.full(n, history) if far else rng.integers(0, history + 1, n)
    p["prompt"] = (p["len"] * rng.random(n)).astype(int) if prompt else np.zeros(n, int)
    p["draft"] = rng.integers(0, vocab if far else min(vocab, 30), total)
    p["trees"] = [random_tree(rng, r) if mask else None for r in rows]
    p["rep"], p["freq"], p["pres"] = (rng.random(n).astype(np.float32) + np.float32(lo) for lo in (0.7, -0.2, -0.3))
    p["bias_tokens"] = rng.integers(-1, min(vocab, 50) + 1, (n, max(1, bias)))
    p["bias"] = rng.standard_normal((n, max(1, bias))).astype(np.float32)
    p["bias_len"] = rng.integers(0, bias + 1, n)
    p["allowed"] = rng.random((max(1, masks), vocab)) < rng.choice([0.0, 0.02, 0.7], (max(1, masks), 1))
    p["allowed_row"] = rng.integers(-1, max(1, masks), total)
    seen = [[x[0] for x in OD.ancestors(t, r)] for t, r in zip(p["trees"], rows)]
    bits = np.zeros((total, max(1, max(rows))), bool)
    for s, lo in zip(seen, p["start"]):
        for i, b in enumerate(s):
            bits[lo + i, : len(b)] = b
    p["next"] = torch.full((total,), -9, dtype=torch.int32, device="cuda")
    p["out"], p["whole"] = ys[1], ys[0]
    kw = dict(rows=total, vocab=vocab, requests=n, xdtype=code(W, x), ydtype=code(W, y), logits=xs[1],
              logits_stride=vocab + extra, out=ys[1], out_stride=vocab + extra, next=p["next"], seq=ints(p["seq"]),
              tokens=ints(p["tokens"]), tokens_stride=history + 3, tokens_len=ints(p["len"] - base), tokens_base=base,
              prompt_len=ints(p["prompt"]) if prompt else None)
    if drafts:
        kw.update(draft_tokens=ints(p["draft"]), row_start=ints(p["start"]))
        if mask:
            kw.update(mask=ints(words_of(bits)), mask_words=-(-bits.shape[1] // 32))
    if penalties:
        kw.update({k: torch.tensor(p[s], device="cuda") for k, s in (("repetition", "rep"), ("frequency", "freq"), ("presence", "pres"))})
    if bias:
        kw.update(bias_tokens=ints(p["bias_tokens"]), bias=torch.tensor(p["bias"], device="cuda"), bias_len=ints(p["bias_len"]),
                  bias_stride=bias)
    if masks:
        w = words_of(p["allowed"])
        kw.update(allowed=ints(w), allowed_stride=w.shape[1], allowed_rows=masks, allowed_row=ints(p["allowed_row"]))
    p.update(drafts=drafts, has_bias=bool(bias), masks=masks, penalties=penalties)
    return W.logits_adjust_args(**kw), p


def check_adjust(p, y, x_rows=None):
    """Each of at most five float32 steps (factor, product, two differences, bias) is off by half a step of its result,
    which is not above |x| (1 + 1/0.7) + |freq| n + |pres| + |bias|; a rounding to y follows."""
    out, nxt = f64(p["out"]), p["next"].cpu().numpy()
    for r, s in enumerate(p["seq"]):
        lo = p["start"][s]
        see = OD.ancestors(p["trees"][s], p["rows"][s])[r - lo][0]
        drafted = p["draft"][lo: lo + len(see)][see] if p["drafts"] else []
        text = p["tokens"][s, : p["len"][s]]
        f = (float(p["rep"][s]), float(p["freq"][s]), float(p["pres"][s])) if p["penalties"] else (1.0, 0.0, 0.0)
        k = p["bias_len"][s] if p["has_bias"] else 0
        pairs = [(int(t), float(b)) for t, b in zip(p["bias_tokens"][s, :k], p["bias"][s, :k])]
        m = p["allowed_row"][r] if p["masks"] else -1
        want, token = OD.adjust(p["logits"][r], text, int(p["prompt"][s]), drafted, *f, pairs, p["allowed"][m] if m >= 0 else None)
        size = np.abs(np.where(np.isfinite(p["logits"][r]), p["logits"][r], 0)) * 2.5 + abs(f[1]) * (len(text) + len(drafted)) + abs(f[2]) + max(
            [0.0] + [abs(b) for _, b in pairs])
        fin = np.isfinite(want)
        np.testing.assert_array_equal(out[r][~fin], want[~fin])
        inside(out[r][fin], want[fin], (5 * U * size + HALF[y] * (np.abs(np.where(fin, want, 0)) + 5 * U * size))[fin], r)
        if nxt[r] != token:  # only where two values lie closer than the roundings
            assert token >= 0 and nxt[r] >= 0 and want[token] - want[nxt[r]] <= 10 * U * size[token], (r, nxt[r], token)


ADJUST_CASES = [
    # rows of each request, vocabulary, options
    ([1], 1, {}),
    ([1], 33, {"drafts": False}),
    ([3, 1, 0, 7], 512, {}),
    ([1] * 40, 1000, {"drafts": False, "masks": 0}),
    ([9, 40], 4097, {"history": 400}),                       # masks of two words
    ([2, 5], 32001, {"bias": 0, "extra": 3}),                # rows off 16 bytes
    ([1, 2], 50257, {"penalties": False, "offset": 1}),
    ([4, 4], 151936, {"history": 3000, "prompt": False}),
    ([3], 151936, {"mask": False, "base": 7}),               # chains
    ([2], 300000, {}),                                       # two passes over the vocabulary
    ([1] * 90, 20000, {"in_place": True, "history": 5}),
    ([400, 2, 290], 700, {"mask": False, "far": True}),      # more drafted tokens before a row than are listed
    ([270, 9], 1500, {"far": True}),                         # masks of nine words
    ([1], 40000, {"history": 24000, "far": True}),           # more tokens with a rule than are listed
]


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("c", ADJUST_CASES, ids=str)
def test_logits_adjust(c, types):
    import torch

    W = lib()
    rows, vocab, o = c
    if o.get("in_place") and types[0] != types[1]:
        pytest.skip("in place means one type")
    a, p = adjust_case(W, rows, vocab, *types, **o)
    W.gemv_device_errors()
    W.logits_adjust(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    check_adjust(p, types[1])
    if o.get("extra") or o.get("offset"):
        gap = torch.ones_like(p["whole"], dtype=torch.bool)
        gap[o.get("offset", 0):].view(sum(rows), -1)[:, :vocab] = False
        assert (p["whole"][gap] == 7.0).all()
    if not o.get("in_place"):
        first = [p["out"].clone(), p["next"].clone()]
        a.set("out", None)  # the token alone
        p["next"].fill_(-9)
        W.logits_adjust(a)
        torch.cuda.synchronize()
        assert torch.equal(first[1], p["next"])
        a.set("out", p["out"]).set("next", None)
        p["out"].fill_(7.0)
        W.logits_adjust(a)
        torch.cuda.synchronize()
        assert torch.equal(first[0], p["out"])


def test_logits_adjust_special_values():
    """NaN, infinities, ties, rows that a mask leaves empty, rows of no request."""
    import torch

    W = lib()
    v = 5000
    x = rand((8, v), "f32", 1)
    x[0, 17] = x[0, 4000] = x[0, 2500] = 50.0                # a tie across CTAs
    x[1, 3], x[1, 4] = float("nan"), float("inf")
    x[2] = float("nan")
    x[3] = -float("inf")
    x[4, 100] = -float("inf")
    allowed = torch.zeros((2, 157), dtype=torch.int32, device="cuda")
    allowed[1, 3] = 1 << 4                                    # only token 100
    seq = ints([0, 0, 0, 0, 1, 1, -1, 2])
    out, nxt = torch.full_like(x, 7.0), torch.full((8,), -9, dtype=torch.int32, device="cuda")
    tok = ints([[3, 4, -7, v, 2**31 - 1, -2**31]] * 2)
    a = W.logits_adjust_args(rows=8, vocab=v, requests=2, xdtype=0, ydtype=0, logits=x, logits_stride=v, out=out, out_stride=v,
                             next=nxt, seq=seq, tokens=tok, tokens_stride=6, tokens_len=ints([6, 2**31 - 1]),
                             repetition=torch.tensor([2.0, 1.0], device="cuda"), allowed=allowed, allowed_stride=157,
                             allowed_rows=2, allowed_row=ints([-1, -1, -1, -1, 1, 0, 1, 1]))
    W.gemv_device_errors()
    W.logits_adjust(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    assert nxt.tolist() == [17, 4, -1, -1, -1, -1, -9, -9]
    assert torch.isnan(out[1, 3]) and out[1, 4] == float("inf") and torch.isnan(out[2]).all() and torch.isneginf(out[3:6]).all()
    assert (out[6:] == 7.0).all()
    a.set("allowed_row", ints([2, -1, -1, -1, -1, -1, -1, -1]))  # a mask there is not
    W.logits_adjust(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0x4 and nxt[0] == 17 and torch.isfinite(out[0]).all()


@pytest.mark.parametrize("c", [([1], 40, {}), ([3, 1, 0, 7], 512, {}), ([9, 40, 33], 4097, {"history": 400}), ([40, 64], 5000, {"mask": False, "base": 7}),
                               ([400, 2, 290], 700, {"mask": False, "far": True}), ([270, 9], 1500, {"far": True}),
                               ([33, 5], 300000, {"far": True, "mask": False}), ([50, 300, 20], 900, {"text": False, "mask": False})], ids=str)
def test_logits_adjust_of_a_prompts_rows(c):
    """A prompt that ends among the drafted rows, behind them, or where the text ends: its tokens count as the prompt's, in
    the list of a row's drafted tokens, in the words (more than a list holds) and without a text."""
    import torch

    W = lib()
    rows, vocab, o = c
    o = dict(o)
    text = o.pop("text", True)
    rng = np.random.default_rng(sum(rows))
    a, p = adjust_case(W, rows, vocab, "f32", "f32", **o)
    if not text:
        p["len"][:] = 0
        a.set("tokens", None).set("tokens_len", None)
    for k in range(3):
        more = [0, max(rows) + 5, rng.integers(0, np.array(rows) + 2)][k]
        p["prompt"] = p["len"] + more
        a.set("prompt_len", ints(p["prompt"]))
        p["out"].fill_(7.0)
        W.gemv_device_errors()
        W.logits_adjust(a)
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == 0
        check_adjust(p, "f32")


@pytest.mark.parametrize("n,at", [(30, 0), (30, 29), (300, 17), (2000, 1000)])
def test_logits_of_a_prompts_last_row_are_those_of_the_prompt_as_text(n, at):
    """A prompt whose rows from `at` on are this step's: its last row's logits hold the bits of a call that has the whole
    prompt as text, and so do those of a tree's rows behind it, drafted tokens counting as said."""
    import torch

    W = lib()
    v, more = 1200, 3
    rng = np.random.default_rng(n)
    text = rng.integers(0, 60, n + more)
    x = rand((1, v), "f32", 1, 3.0).expand(n + more - at, v).contiguous()
    kw = dict(vocab=v, requests=1, xdtype=0, ydtype=0, logits_stride=v, out_stride=v, prompt_len=ints([n]),
              repetition=torch.tensor([1.3], device="cuda"), frequency=torch.tensor([0.4], device="cuda"),
              presence=torch.tensor([0.7], device="cuda"))
    R = n + more - at
    out, nxt = torch.empty_like(x), torch.empty(R, dtype=torch.int32, device="cuda")
    W.logits_adjust(W.logits_adjust_args(rows=R, logits=x, out=out, next=nxt, seq=ints([0] * R), tokens=ints(text[None]), tokens_stride=n + more,
                                         tokens_len=ints([at]), draft_tokens=ints(text[at:]), row_start=ints([0, R]), **kw))
    for k in range(more + 1):
        o, t = torch.empty_like(x[:1]), torch.empty(1, dtype=torch.int32, device="cuda")
        W.logits_adjust(W.logits_adjust_args(rows=1, logits=x[:1], out=o, next=t, tokens=ints(text[None]), tokens_stride=n + more,
                                             tokens_len=ints([n + k]), **kw))
        torch.cuda.synchronize()
        assert torch.equal(o[0], out[n - at - 1 + k]) and t[0] == nxt[n - at - 1 + k], k
    assert W.gemv_device_errors() == 0


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("v,pairs", [(1000, [(5, 9), (5, 600), (130, 999)]), (40000, [(5, 6), (100, 300), (511, 512), (3, 39999), (20000, 20001)]),
                                     (300000, [(7, 299999), (4096, 8192)])], ids=str)
def test_logits_adjust_zeros_of_both_signs_tie(v, pairs, x):
    """A row whose greatest logits are -0.0 and, at a higher token, 0.0: of equal ones the lowest token is the greedy one,
    whether one thread, warp or CTA has both or several do; tokens with a rule and without one."""
    import torch

    W = lib()
    rows = 4 * len(pairs)
    logits = -1 - rand((rows, v), x, 3).abs()
    text = np.full((rows, 2), -1)
    for r, (lo, hi) in enumerate(pairs * 4):
        logits[r, lo], logits[r, hi] = -0.0, 0.0
        text[r] = [(-1, -1), (lo, -1), (-1, hi), (lo, hi)][r // len(pairs)]
    out, nxt = torch.empty_like(logits), torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    W.logits_adjust(W.logits_adjust_args(
        rows=rows, vocab=v, requests=rows, xdtype=code(W, x), ydtype=code(W, x), logits=logits, logits_stride=v, out=out, out_stride=v,
        next=nxt, tokens=ints(text), tokens_stride=2, tokens_len=ints([2] * rows), repetition=torch.full((rows,), 1.5, device="cuda")))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    assert nxt.tolist() == [lo for lo, _ in pairs] * 4
    at = torch.arange(rows, device="cuda"), torch.tensor([lo for lo, _ in pairs] * 4, device="cuda")
    assert torch.signbit(out[at]).all()  # the logit itself stays -0.0


def test_logits_adjust_long_texts_and_lists():
    """One token many times, its biases listed many times: counts are exact, the last bias counts, every pass the same bits."""
    import torch

    W = lib()
    v, n = 40000, 30000
    rng = np.random.default_rng(0)
    x = rand((2, v), "f32", 2)
    text = np.where(rng.random(n) < 0.5, 77, rng.integers(0, v, n))
    bt = np.where(rng.random(1023) < 0.5, 78, rng.integers(0, v, 1023))
    bv = rng.standard_normal(1023).astype(np.float32)
    outs = []
    for _ in range(3):
        out, nxt = torch.empty_like(x), torch.empty(2, dtype=torch.int32, device="cuda")
        W.logits_adjust(W.logits_adjust_args(
            rows=2, vocab=v, requests=1, xdtype=0, ydtype=0, logits=x, logits_stride=v, out=out, out_stride=v, next=nxt,
            seq=ints([0, 0]), tokens=ints(text[None]), tokens_stride=n, tokens_len=ints([n]), prompt_len=ints([1000]),
            frequency=torch.tensor([0.125], device="cuda"), bias_tokens=ints(bt[None]), bias=torch.tensor(bv[None], device="cuda"),
            bias_len=ints([1023]), bias_stride=1023))
        torch.cuda.synchronize()
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    want, _ = OD.adjust(f64(x[1]), text, 1000, [], 1.0, 0.125, 0.0, list(zip(bt.tolist(), bv.tolist())), None)
    inside(f64(outs[0][1]), want, 4 * U * (np.abs(want) + 0.125 * n + 5.0), "row 1")


# ---- acceptance ----------------------------------------------------------------------------------------------------------------

def accept_case(W, rows, lens, layers, n_kv, d, page, kv, most, seed=0, chain=False, tokens=True, base=0, lead=0, apart=0):
    import torch

    rng = np.random.default_rng(seed)
    b, total = len(rows), sum(rows) + lead
    trees = [None if chain else random_tree(rng, r) for r in rows]
    draft, after = rng.integers(0, 5, total), rng.integers(-1, 5, total)  # few tokens: paths come by themselves, siblings of one token
    need = [-(-(max(0, n) + r) // page) if n >= 0 else 0 for n, r in zip(lens, rows)]
    width, pages = max(max(need), 1), sum(need) + 1
    table, at = np.full((b, width), -1), 0
    ids = rng.permutation(pages)
    for s, k in enumerate(need):
        table[s, :k] = ids[at: at + k]
        at += k
    pools = [rand((layers, pages + apart, n_kv, page, d), kv, seed + k)[:, :pages] for k in range(2)]
    hist = max(max(lens) + max(rows) + base, 1)
    text = rng.integers(0, 9, (b, hist))
    o = {k: torch.full(s, 77, dtype=torch.int32, device="cuda") for k, s in (("count", (b,)), ("new_len", (b,)), ("path", (b, most)), ("out_tokens", (b, most)))}
    t = dict(trees=trees, draft=draft, after=after, table=table, pools=pools, before=[f64(p) for p in pools], text=text, lead=lead,
             tokens=ints(text) if tokens else None, **o)
    parents = None if chain else ints([-1] * lead + [x for p in trees for x in p])
    a = W.tree_accept_args(batch=b, rows=total, path_stride=most, layers=layers, n_kv=n_kv, head_dim=d, kvdtype=code(W, kv),
                           row_start=ints(lead + np.concatenate([[0], np.cumsum(rows)])), parents=parents, draft_tokens=ints(draft),
                           next=ints(after), seq_len=ints(lens), k_pages=pools[0], v_pages=pools[1],
                           layer_stride=(pages + apart) * n_kv * page * d, num_pages=pages, page_size=page, table_stride=width,
                           page_table=ints(table), tokens=t["tokens"], tokens_stride=hist, tokens_base=base, **o)
    return a, t


def check_accept(t, rows, lens, page, most, base=0):
    at, table = t["lead"], t["table"]
    pools, text = [p.copy() for p in t["before"]], t["text"].copy()
    longest = 0
    for s, (r, n) in enumerate(zip(rows, lens)):
        draft, after = t["draft"][at: at + r], t["after"][at: at + r]
        at += r
        path = OD.accept(t["trees"][s], draft, after, most) if n >= 0 and r > 0 else []
        longest = max(longest, len(path))
        assert t["count"][s] == len(path) and t["new_len"][s] == (-1 if n < 0 else n + len(path))
        assert t["path"][s].tolist() == path + [-1] * (most - len(path))
        assert t["out_tokens"][s].tolist() == [int(after[p]) for p in path] + [-1] * (most - len(path))
        for k, p in enumerate(path):
            (p0, i0), (p1, i1) = divmod(n + p, page), divmod(n + k, page)
            for pool, old in zip(pools, t["before"]):
                pool[:, table[s, p1], :, i1] = old[:, table[s, p0], :, i0]
            text[s, n + base + k] = draft[p]
    for got, want in zip(t["pools"], pools):
        np.testing.assert_array_equal(f64(got), want)
    if t["tokens"] is not None:
        np.testing.assert_array_equal(t["tokens"].cpu().numpy(), text)
    return longest


ACCEPT_CASES = [
    # rows of each request, lens, layers, n_kv, d, page, longest path, options
    ([1], [0], 1, 1, 8, 1, 1, {}),
    ([12], [40], 2, 2, 16, 16, 8, {}),
    ([40, 3, 0, 9], [0, 17, 5, -1], 3, 2, 24, 4, 16, {"lead": 3}),
    ([256, 100], [33, 1], 2, 8, 128, 32, 256, {}),
    ([30, 30], [7, 9], 2, 1, 64, 8, 3, {"chain": True}),          # paths that are cut
    ([2000], [5], 1, 2, 16, 16, 20, {"chain": True, "tokens": False}),  # more rows than fit shared memory
    ([1500], [5], 1, 2, 16, 16, 64, {}),
    ([64] * 20, [i * 5 for i in range(20)], 28, 8, 128, 16, 12, {"base": 11}),
    ([6, 7], [3, 4], 2, 2, 16, 4, 8, {"apart": 3}),               # layers with gaps between them
]


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("c", ACCEPT_CASES, ids=lambda c: f"b{len(c[0])}x{max(c[0])}_l{c[2]}_kv{c[3]}_d{c[4]}_page{c[5]}_{c[6]}")
def test_tree_accept_paged(c, kv):
    import torch

    W = lib()
    rows, lens, layers, n_kv, d, page, most, o = c
    longest = 0
    for seed in range(3):
        a, t = accept_case(W, rows, lens, layers, n_kv, d, page, kv, most, seed=seed, **o)
        W.gemv_device_errors()
        W.tree_accept_paged(a)
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == 0
        longest = max(longest, check_accept(t, rows, lens, page, most, o.get("base", 0)))
    assert longest > 1 or max(rows) == 1


def test_tree_accept_paged_moves_that_overlap():
    """A path whose rows are each other's places: 0, 2, 3, 4, .. to 0, 1, 2, 3, .., more than one batch of moves."""
    import torch

    W = lib()
    n, R, page = 5, 30, 4
    a, t = accept_case(W, [R], [n], 2, 2, 16, page, "f32", 32)
    par = [-1, 0, 0] + list(range(2, R - 1))
    draft, after = np.arange(R), np.full(R, -1)
    after[0], after[2: R - 1] = 2, np.arange(3, R)
    t.update(trees=[par], draft=draft, after=after)
    a.set("parents", ints(par)).set("draft_tokens", ints(draft)).set("next", ints(after))
    W.tree_accept_paged(a)
    torch.cuda.synchronize()
    assert check_accept(t, [R], [n], page, 32) == R - 1


def test_tree_accept_paged_without_pools_and_bad_places():
    """Tokens alone (no layers); pages outside the pool are not moved, places behind the texts not written, both reported."""
    import torch

    W = lib()
    a, t = accept_case(W, [12, 9], [3, 4], 1, 2, 16, 4, "f32", 8, seed=1)
    a.layers = 0
    a.set("k_pages", None).set("v_pages", None).set("page_table", None)
    W.gemv_device_errors()
    W.tree_accept_paged(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    t["before"] = [f64(p) for p in t["pools"]]
    for s in range(2):
        lo = (0, 12)[s]
        path = OD.accept(t["trees"][s], t["draft"][lo: lo + (12, 9)[s]], t["after"][lo: lo + (12, 9)[s]], 8)
        assert t["path"][s].tolist()[: len(path)] == path
    par, draft = [-1, 0, 0, 2, 3], np.arange(5)
    after = np.array([2, -1, 3, 4, 9])  # the path 0, 2, 3, 4
    a, t = accept_case(W, [5], [6], 2, 2, 16, 4, "f32", 8)
    t.update(trees=[par], draft=draft, after=after)
    a.set("parents", ints(par)).set("draft_tokens", ints(draft)).set("next", ints(after))
    bad = t["table"].copy()
    bad[0, 2] = a.num_pages  # tokens 8 to 11: the places of rows 2, 3, 4
    a.set("page_table", ints(bad))
    text = t["tokens"][:, :8].contiguous()
    a.set("tokens", text)
    a.tokens_stride = 8
    W.tree_accept_paged(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0x80 | 0x8
    for got, old in zip(t["pools"], t["before"]):
        np.testing.assert_array_equal(f64(got), old)
    assert t["path"][0].tolist() == [0, 2, 3, 4, -1, -1, -1, -1] and text[0, 6:].tolist() == [0, 2]


# ---- streams and graphs --------------------------------------------------------------------------------------------------------

def test_attentions_of_two_streams_at_once():
    """Calls on three streams, each with its own workspace, give the bits that they give alone."""
    import torch

    W = lib()
    cases = [([16] * 6, 16, 8, 128, 0, [900, 1, 127, 128, 2000, 40], 16, "tree", "bf16", "bf16"),
             ([5, 9, 30], 10, 2, 80, 129, [400, 31, 77], 32, "random", "f32", "bf16"),
             ([64, 33], 16, 8, 128, 300, [300, 1000], 64, "tree", "bf16", "bf16"),
             ([13, 1], 16, 8, 128, 0, [301, 2000], 8, "tree", "f32", "f32")]
    made, want = [], []
    for i, (rows, n_q, n_kv, d, plen, lens, page, mask, q, kv) in enumerate(cases):
        a, t = tree_case(W, rows, n_q, n_kv, d, plen, lens, page, q, kv, mask=mask, seed=i)
        W.attn_tree_paged(a)
        torch.cuda.synchronize()
        check_tree(t, rows, n_q, n_kv, d, plen, lens, page, q)
        want.append([t["out"].clone(), t["lse"].clone()])
        t["out"].fill_(3), t["lse"].fill_(3)
        made.append((a, t))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(30):
        for (a, _), st in zip(made, streams):
            W.attn_tree_paged(a, st)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    for (_, t), w in zip(made, want):
        assert torch.equal(t["out"], w[0]) and torch.equal(t["lse"], w[1])


class Step:
    """A step of trees over one layer, its state kept on the device from step to step."""

    def __init__(self, W, B, R, n_q, n_kv, d, page, width, vocab, q, kv, plen, seed=0):
        import torch

        total, num = B * R, 2 * B + 2  # (enough for all at the start, not later)
        i32 = dict(dtype=torch.int32, device="cuda")
        z = lambda *shape: torch.zeros(shape, **i32)
        self.fresh, self.parents, self.draft = z(B), z(total), z(total)
        self.qkv = torch.zeros((total, (n_q + 2 * n_kv) * d), device="cuda")
        self.logits = torch.zeros((total, vocab), device="cuda")
        self.held, self.owned, self.state = z(B), z(B), ints([0, num])
        self.table, self.ring = torch.full((B, width), -1, **i32), ints(np.random.default_rng(seed).permutation(num))
        self.text = z(B, width * page + R)
        new_owned, new_state, row_start, ctx, seq, pos, mask = z(B), z(2), z(B + 1), z(B), z(total), z(total), z(total, 1)
        slots = torch.zeros(total, dtype=torch.int64, device="cuda")
        self.back = [(self.owned, new_owned), (self.state, new_state)]
        self.pools = torch.zeros((2, 1, num, n_kv, page, d), device="cuda").to(tdt(kv))
        pk, pv = (rand((n_kv, max(plen, 1), d), kv, seed + k) for k in (1, 2))
        q_out = torch.zeros((total, n_q * d), dtype=tdt(q), device="cuda")
        self.out, self.adjusted, self.next = torch.zeros_like(q_out), torch.zeros_like(self.logits), z(total)
        self.count, self.path, self.acc = z(B), z(B, R), z(B, R)
        new_len = z(B)
        self.back.append((self.held, new_len))
        freq, factor = W.rope_frequencies(d, 1e4)
        wide = (n_q + 2 * n_kv) * d
        self.calls = [
            (W.step_slots, W.step_slots_args(
                requests=B, rows=total, num_pages=num, page_size=page, table_stride=width, base_pos=plen, mask_words=1,
                held=self.held, fresh=self.fresh, owned=self.owned, parents=self.parents, page_table=self.table,
                free_ring=self.ring, free_state=self.state, new_table=self.table, new_owned=new_owned, new_free_state=new_state,
                row_start=row_start, ctx_len=ctx, seq=seq, positions=pos, slots=slots, mask=mask)),
            (W.kv_append_slots, W.kv_slots_args(
                rows=total, n_q=n_q, n_kv=n_kv, head_dim=d, xdtype=W.DEC_F32, ydtype=code(W, q), kvdtype=code(W, kv), q=self.qkv,
                k=self.qkv[:, n_q * d:], v=self.qkv[:, (n_q + n_kv) * d:], q_out=q_out, q_stride=wide, k_stride=wide,
                v_stride=wide, q_out_stride=n_q * d, g_q=None, g_k=None, positions=pos, inv_freq=torch.tensor(freq, dtype=torch.float64, device="cuda"),
                eps=1e-6, rope_factor=factor, rot_dim=d, interleaved=0, k_pages=self.pools[0], v_pages=self.pools[1],
                slots=slots, num_pages=num, page_size=page))]
        a = W.attn_tree_args(
            batch=B, rows=total, n_q=n_q, n_kv=n_kv, head_dim=d, qdtype=code(W, q), kvdtype=code(W, kv), q=q_out, out=self.out,
            q_stride=n_q * d, out_stride=n_q * d, row_start=row_start, mask=mask, mask_words=1, prefix_k=pk, prefix_v=pv,
            prefix_len=plen, prefix_stride=max(plen, 1), k_pages=self.pools[0], v_pages=self.pools[1], page_table=self.table,
            seq_len=ctx, num_pages=num, page_size=page, table_stride=width, scale=d ** -0.5)
        a.with_workspace(torch.empty(W.attn_tree_paged_workspace(a), dtype=torch.uint8, device="cuda"))
        self.calls += [
            (W.attn_tree_paged, a),
            (W.logits_adjust, W.logits_adjust_args(
                rows=total, vocab=vocab, requests=B, xdtype=0, ydtype=0, logits=self.logits, logits_stride=vocab,
                out=self.adjusted, out_stride=vocab, next=self.next, seq=seq, tokens=self.text, tokens_stride=self.text.shape[1],
                tokens_len=self.held, draft_tokens=self.draft, row_start=row_start, mask=mask, mask_words=1,
                repetition=torch.full((B,), 1.25, device="cuda"), frequency=torch.full((B,), 0.5, device="cuda"))),
            (W.tree_accept_paged, W.tree_accept_args(
                batch=B, rows=total, path_stride=R, layers=1, n_kv=n_kv, head_dim=d, kvdtype=code(W, kv), row_start=row_start,
                parents=self.parents, draft_tokens=self.draft, next=self.next, seq_len=ctx, held=self.held, k_pages=self.pools[0],
                v_pages=self.pools[1], layer_stride=self.pools[0].numel(), num_pages=num, page_size=page, table_stride=width,
                page_table=self.table, tokens=self.text, tokens_stride=self.text.shape[1], count=self.count, new_len=new_len,
                path=self.path, out_tokens=self.acc))]
        self.ctx = ctx
        self.seen = [ctx, self.out, self.adjusted, self.next, self.count, self.path, self.acc, self.held, self.owned, self.state,
                     self.table, self.ring, self.text, self.pools, q_out, pos, slots, mask]

    def run(self, stream=None):
        for call, a in self.calls:
            call(a, stream)
        for to, new in self.back:
            to.copy_(new)


@pytest.mark.parametrize("q,kv,d,plen", [("bf16", "bf16", 128, 0), ("bf16", "bf16", 64, 70), ("f32", "f32", 128, 0),
                                         ("f32", "bf16", 80, 33)], ids=str)
def test_a_captured_step_of_trees_follows_its_inputs(q, kv, d, plen):
    """A graph of a step's calls is captured once and replayed on its own state, requests growing, ending and starting again;
    an equal state is driven by eager calls on another stream. Both hold the same bits after every step."""
    import torch

    W = lib()
    B, R, width, page, vocab = 5, 9, 12, 8, 900
    eager, graph = (Step(W, B, R, 8, 4, d, page, width, vocab, q, kv, plen) for _ in range(2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        graph.run(side)
    W.gemv_device_errors()
    rng = np.random.default_rng(3)
    moved = waited = 0
    for step in range(20):
        held = eager.held.cpu().numpy()
        held[held > width * page - 2 * R] = -1
        if step % 4 == 3:
            held[step % B] = -1
        start = eager.held.cpu().numpy() < 0
        held[start] = 0  # an ended request's place is taken again
        before = held.copy()
        fresh = rng.integers(0, R + 1, B)
        fresh[step % B] = R
        total = np.clip(fresh, 0, None)
        total[held < 0] = 0
        parents, drafts = np.zeros(B * R, int), rng.integers(0, 3, B * R)
        at = 0
        for r in total:
            parents[at: at + r] = random_tree(rng, int(r))
            at += r
        logits = rng.standard_normal((B * R, vocab)).astype(np.float32)
        logits[:, :3] += 4  # (drafted tokens come often)
        qkv = rng.standard_normal((B * R, graph.qkv.shape[1])).astype(np.float32)
        for s in (eager, graph):
            for x, y in ((s.fresh, fresh), (s.parents, parents), (s.draft, drafts), (s.held, held)):
                x.copy_(ints(y))
            s.logits.copy_(torch.tensor(logits)), s.qkv.copy_(torch.tensor(qkv))
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side if step % 2 else torch.cuda.default_stream()):
            eager.run(side if step % 2 else None)
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == 0
        for i, (x, y) in enumerate(zip(eager.seen, graph.seen)):
            assert torch.equal(x, y), (step, i)
        moved += int((eager.count - 1).clamp(min=0).sum())
        wait = (before >= 0) & (eager.ctx.cpu().numpy() < 0)  # not served: they keep what they have
        waited += int(wait.sum())
        np.testing.assert_array_equal(eager.held.cpu().numpy()[wait], before[wait])
        assert (eager.held.cpu().numpy()[before < 0] == -1).all()
    assert moved > 0 and waited > 0  # rows were accepted behind the first ones; some requests had to wait


# ---- together ------------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("shape,kv,y", [("TINY", "f32", "f32"), ("TINY", "bf16", "f32"), ("Q4_SMALL", "bf16", "bf16")], ids=str)
def test_trees_continue_a_decoders_prompt(shape, kv, y):
    """Two requests continue a prompt that the decoder prefilled, by trees of drafted tokens: slots, append, attention over
    the decoder's own cache, logits by the requests' rules, acceptance, step after step, pages coming from one ring and going
    back at the end. The first request has no rules: its tokens are those that the decoder generates alone; the second has a
    repetition penalty and a mask: its tokens are those of the oracle's logits under these rules. Keys and values in the
    pages are the oracle's of the accepted tokens. (What lies between the operators, products with the weights and the
    SwiGLU, is computed on the host.)"""
    import torch

    import oracle as O
    import workloads as Wl
    from gpu_util import FP32_TOL, LOW_TOL, close
    from oracle import primitives as P
    from weight_streaming_gemv_token_gb300.decoder import Decoder

    W = lib()
    s = getattr(Wl, shape)
    tol = FP32_TOL if kv == y == "f32" else LOW_TOL
    weights = Wl.decoder_weights(s, seed=1, wdtype="f32" if kv == "f32" else "bf16")
    prompt = [int(x) for x in Wl.prompt_uniform(21, s.vocab, seed=0)]
    d, n, page, width, R, steps, B = s.head_dim, len(prompt), 4, 12, 7, 5, 2
    total, most = B * R, R
    dec = Decoder(s, weights, kv_dtype=kv, max_seq=n + 64)
    first = dec.prefill(prompt, is_last=True)
    alone = [first] + [int(x) for x in dec.generate(first, steps * R)]
    dec.rewind(n)
    # the second request by the oracle's logits and the rules: penalty 1.3, only even tokens
    even = np.arange(s.vocab) % 2 == 0

    def rule(logits, text):
        return OD.adjust(logits, text, 0, [], float(np.float32(1.3)), 0.0, 0.0, [], even)

    ora = O.OracleDecoder(s, weights, kv_dtype=kv, max_seq=n + 64)
    ora.prefill(prompt)
    ruled = [int(x) for x in [first]]
    for _ in range(steps * R):
        ruled.append(rule(ora.step(ruled[-1]), prompt + ruled)[1])
    truth = [alone, ruled]
    freq, factor = W.rope_frequencies(d, s.rope_theta)
    wd = torch.tensor(freq, dtype=torch.float64, device="cuda")
    num = B * width + 3
    pools = torch.full((2, s.layers, num, s.n_kv, page, d), float("nan"), device="cuda").to(tdt(kv))
    rng = np.random.default_rng(2)
    ring = ints(rng.permutation(num))
    i32 = dict(dtype=torch.int32, device="cuda")
    tables = [torch.full((B, width), -1, **i32) for _ in range(2)]
    owned = [torch.zeros(B, **i32) for _ in range(2)]
    state = [ints([0, num]), torch.zeros(2, **i32)]
    held = [torch.zeros(B, **i32) for _ in range(2)]
    row_start, ctx = torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
    seq, pos, mask = torch.zeros(total, **i32), torch.zeros(total, **i32), torch.zeros((total, 1), **i32)
    slots = torch.zeros(total, dtype=torch.int64, device="cuda")
    fresh, draft_d, par_d = ints([R] * B), torch.zeros(total, **i32), torch.zeros(total, **i32)
    text = torch.zeros((B, n + width * page), **i32)
    text[:, :n] = ints(prompt)
    nxt, count, path, acc = torch.zeros(total, **i32), torch.zeros(B, **i32), torch.zeros((B, most), **i32), torch.zeros((B, most), **i32)
    gains = [[torch.tensor(P.widen(w[g]).astype(np.float32), device="cuda") for g in ("g_q", "g_k")] for w in weights["layers"]]
    wide = (s.n_q + 2 * s.n_kv) * d
    done = [[first], [first]]  # tokens known so far, the last one not in the cache
    W.gemv_device_errors()
    for step in range(steps):
        cur, nex = step % 2, 1 - step % 2
        parents, drafts, deep = [], [], 0
        for b in range(B):  # a branch that is right for a while, wrong ones beside it
            at = len(done[b]) - 1
            par = [-1, 0, 0, 2, 2, 4, 1]
            tok = [done[b][-1]] + [int(rng.integers(0, s.vocab)) for _ in range(R - 1)]
            if step != 1:  # (one step in which nothing is right)
                tok[2], tok[4], tok[5] = truth[b][at + 1], truth[b][at + 2], truth[b][at + 3]
            if step == 2:
                tok[4] = (tok[4] + 1) % s.vocab
            parents, drafts = parents + par, drafts + tok
        par_d.copy_(ints(parents)), draft_d.copy_(ints(drafts))
        W.step_slots(W.step_slots_args(
            requests=B, rows=total, num_pages=num, page_size=page, table_stride=width, base_pos=n, mask_words=1,
            held=held[cur], fresh=fresh, owned=owned[cur], parents=par_d, page_table=tables[cur], free_ring=ring,
            free_state=state[cur], new_table=tables[nex], new_owned=owned[nex], new_free_state=state[nex],
            row_start=row_start, ctx_len=ctx, seq=seq, positions=pos, slots=slots, mask=mask))
        h = ora.E[np.array(drafts)].copy()
        for l, w in enumerate(ora.layers):
            x = P.rmsnorm(h, w["g_in"], s.eps)
            qkv = torch.tensor(np.concatenate([x @ w[m].T for m in ("w_q", "w_k", "w_v")], 1).astype(np.float32), device="cuda")
            q_out = torch.empty((total, s.n_q * d), dtype=tdt(y), device="cuda")
            W.kv_append_slots(W.kv_slots_args(
                rows=total, n_q=s.n_q, n_kv=s.n_kv, head_dim=d, xdtype=W.DEC_F32, ydtype=code(W, y), kvdtype=code(W, kv),
                q=qkv, k=qkv[:, s.n_q * d:], v=qkv[:, (s.n_q + s.n_kv) * d:], q_out=q_out, q_stride=wide, k_stride=wide,
                v_stride=wide, q_out_stride=s.n_q * d, g_q=gains[l][0], g_k=gains[l][1], positions=pos, inv_freq=wd,
                eps=s.eps, rope_factor=factor, rot_dim=d, interleaved=0, k_pages=pools[0, l], v_pages=pools[1, l], slots=slots,
                num_pages=num, page_size=page))
            K, V, valid = dec.kv(l)
            assert valid == n
            out = torch.empty_like(q_out)
            a = W.attn_tree_args(
                batch=B, rows=total, n_q=s.n_q, n_kv=s.n_kv, head_dim=d, qdtype=code(W, y), kvdtype=code(W, kv), q=q_out,
                out=out, q_stride=s.n_q * d, out_stride=s.n_q * d, row_start=row_start, mask=mask, mask_words=1, prefix_k=K,
                prefix_v=V, prefix_len=n, prefix_stride=K.shape[1], k_pages=pools[0, l], v_pages=pools[1, l],
                page_table=tables[nex], seq_len=ctx, num_pages=num, page_size=page, table_stride=width, scale=d ** -0.5)
            a.with_workspace(torch.empty(W.attn_tree_paged_workspace(a), dtype=torch.uint8, device="cuda"))
            W.attn_tree_paged(a)
            h = h + f64(out) @ w["w_o"].T
            x = P.rmsnorm(h, w["g_post"], s.eps)
            h = h + P.swiglu(x @ w["w_gate"].T, x @ w["w_up"].T) @ w["w_down"].T
        logits = torch.tensor((P.rmsnorm(h, ora.g_final, s.eps) @ ora.E.T).astype(np.float32), device="cuda")
        allowed = words_of(even[None])
        W.logits_adjust(W.logits_adjust_args(
            rows=total, vocab=s.vocab, requests=B, xdtype=0, ydtype=0, logits=logits, logits_stride=s.vocab, out=logits,
            out_stride=s.vocab, next=nxt, seq=seq, tokens=text, tokens_stride=text.shape[1], tokens_len=held[cur], tokens_base=n,
            draft_tokens=draft_d, row_start=row_start, mask=mask, mask_words=1, repetition=torch.tensor([1.0, 1.3], device="cuda"),
            allowed=ints(allowed), allowed_stride=allowed.shape[1], allowed_rows=1, allowed_row=ints([-1] * R + [0] * R)))
        W.tree_accept_paged(W.tree_accept_args(
            batch=B, rows=total, path_stride=most, layers=s.layers, n_kv=s.n_kv, head_dim=d, kvdtype=code(W, kv),
            row_start=row_start, parents=par_d, draft_tokens=draft_d, next=nxt, seq_len=ctx, k_pages=pools[0], v_pages=pools[1],
            layer_stride=pools.stride(1), num_pages=num, page_size=page, table_stride=width, page_table=tables[nex],
            tokens=text, tokens_stride=text.shape[1], tokens_base=n, count=count, new_len=held[nex], path=path, out_tokens=acc))
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == 0
        for b in range(B):
            k = int(count[b])
            assert k == {1: 1, 2: 2}.get(step, 4), (step, b, k)
            done[b] += acc[b, :k].tolist()
            assert done[b] == truth[b][: len(done[b])], (step, b)
            assert int(held[nex][b]) == len(done[b]) - 1
            assert text[b, n: n + len(done[b]) - 1].tolist() == done[b][:-1]
    end, tab = steps % 2, tables[steps % 2].cpu().numpy()
    for b in range(B):
        ref = O.OracleDecoder(s, weights, kv_dtype=kv, max_seq=n + 64)
        ref.prefill(prompt)
        for t in done[b][:-1]:
            ref.step(int(t))
        i = np.arange(len(done[b]) - 1)
        for l in range(s.layers):
            for pool, theirs in zip(pools[:, l], ref.kv(l)):
                close(f64(pool)[tab[b, i // page], :, i % page].transpose(1, 0, 2), theirs[:, n:], tol, f"cache of request {b}, layer {l}")
    # both requests end: every page is free again
    W.step_slots(W.step_slots_args(
        requests=B, rows=0, num_pages=num, page_size=page, table_stride=width, held=ints([-1] * B), fresh=fresh, owned=owned[end],
        page_table=tables[end], free_ring=ring, free_state=state[end], new_table=tables[1 - end], new_owned=owned[1 - end],
        new_free_state=state[1 - end], row_start=row_start, ctx_len=ctx))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0 and state[1 - end][1] == num and (tables[1 - end] == -1).all()
    assert sorted(ring.tolist()) == list(range(num))
    dec.close()
