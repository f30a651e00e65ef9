"""Host side of the calls for drafted trees: how the attention is cut up, refusals (no GPU)."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

import oracle.drafts as OD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def W():
    from weight_streaming_gemv_token_gb300 import build as bld

    bld.build()
    import weight_streaming_gemv_token_gb300 as W

    return W


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """csrc/attn_tree_plan.h and csrc/spans.h compiled as plain C++."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("tree")
    src = d / "p.cpp"
    src.write_text('#include "attn_tree_plan.h"\n#include "spans.h"\nusing namespace wsg;\nextern "C" {\n'
                   "int plan(const attn_tree_args* a, long long* o) {\n"
                   "  if (!attn_tree_sizes_ok(a)) return 0;\n  const AtPlan p = attn_tree_plan(a, 152);\n"
                   "  const long long v[] = {1 << p.cut.mshift, p.prefix_row_tiles, p.prefix_tiles, p.pieces, p.ctas, (long long)p.o,\n"
                   "    (long long)p.ml, (long long)p.rec, (long long)p.line, (long long)p.total,\n"
                   "    (long long)(a->prefix_len ? a->rows * sizeof(AtRow) : p.ctas * sizeof(AtSeam))};\n"
                   "  for (int i = 0; i < 11; ++i) o[i] = v[i];\n  return 1;\n}\n"
                   "AtCut cut(int group, int mt, int chain, int cap) { return AtCut{group, 1, __builtin_ctz(mt), chain, cap}; }\n"
                   "int keys(int group, int mt, int chain, int cap, int n, int rows, int t) {\n"
                   "  return at_keys(cut(group, mt, chain, cap), n, rows, t); }\n"
                   "int tiles(int group, int mt, int chain, int cap, int n, int rows, int t) {\n"
                   "  return at_tiles(cut(group, mt, chain, cap), n, rows, t); }\n"
                   "int extra() { return kAtExtra; }\n"
                   "long long head(int group, int mt, int chain, int cap, int n, int rows) {\n"
                   "  return at_head_units(cut(group, mt, chain, cap), n, rows); }\n"
                   "long long first(long long W, int C, int c) { return at_first(at_shares(W, C), c); }\n"
                   "int owner(long long W, int C, long long p) { return at_owner(at_shares(W, C), p); }\n"
                   "int meet(size_t p, size_t a, size_t q, size_t b) {\n"
                   "  return spans_meet(Span{(void*)p, a}, Span{(void*)q, b}); }\n}\n")
    lib = d / "p.so"
    inc = os.path.join(ROOT, "weight_streaming_gemv_token_gb300", "csrc")
    cmd = [cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o", str(lib)]
    checked = ["-fsanitize=undefined", "-fno-sanitize-recover=undefined"]  # where the toolchain has its library
    if subprocess.run(cmd + checked, capture_output=True).returncode != 0:
        subprocess.run(cmd, check=True)
    L, q, i, z = ctypes.CDLL(str(lib)), ctypes.c_longlong, ctypes.c_int, ctypes.c_size_t
    L.plan.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    L.keys.argtypes = L.tiles.argtypes = [i] * 7
    L.head.argtypes, L.head.restype = [i] * 6, q
    L.first.argtypes, L.first.restype = [q, i, i], q
    L.owner.argtypes = [q, i, q]
    L.meet.argtypes = [z] * 4
    return L


NAMES = "mt prefix_row_tiles prefix_tiles pieces ctas o ml rec line total rec_bytes".split()


def test_keys_of_row_tiles(host):
    """A row tile looks at the request's tokens and its own rows: all of them, or in a chain up to its last token."""
    big = 1 << 30
    for group, mt, n, rows in ((1, 16, 0, 1), (2, 16, 100, 20), (3, 16, 5, 11), (16, 16, 7, 3), (2, 128, 1000, 200),
                               (5, 128, 129, 77)):
        T = -(-rows * group // mt)
        for t in range(T):
            assert host.keys(group, mt, 0, big, n, rows, t) == n + rows
            last = min(rows, ((t + 1) * mt - 1) // group + 1)  # the token of the tile's last row
            assert host.keys(group, mt, 1, big, n, rows, t) == n + last
            assert host.tiles(group, mt, 1, big, n, rows, t) == max(1, -(-(n + last) // 128))
            assert host.keys(group, mt, 0, n + 1, n, rows, t) == n + 1  # the table ends there
            assert host.tiles(group, mt, 0, 0, n, rows, t) == 1  # no table: still a tile, for the rows' zeros
        for chain in (0, 1):
            assert host.head(group, mt, chain, big, n, rows) == sum(host.tiles(group, mt, chain, big, n, rows, t) + host.extra() for t in range(T))
    assert host.keys(2, 16, 0, 1 << 30, 2**31 - 1, 2**20, 0) == 1 << 30


def test_shares_cover_the_line_once(host):
    for W, C in ((1, 1), (5, 5), (151, 151), (152, 152), (153, 152), (1000, 152), (10**9 + 7, 152), (2**40, 152)):
        ends = [host.first(W, C, c) for c in range(C + 1)]
        assert ends[0] == 0 and ends[-1] == W and all(a < b for a, b in zip(ends, ends[1:]))
        for c in range(C):
            for p in {ends[c], ends[c + 1] - 1, (ends[c] + ends[c + 1]) // 2}:
                assert host.owner(W, C, p) == c


def test_pieces_have_numbers_of_their_own_inside_the_workspace(W, host):
    """The pieces of random steps, walked as the kernel does: tiles are covered once, no two pieces share a number, and
    every number lies inside the workspace."""
    rng = np.random.default_rng(0)
    for trial in range(300):
        n_kv, group = int(rng.choice([1, 2, 8])), int(rng.integers(1, 17))
        batch = int(rng.integers(1, 40))
        rows = rng.integers(0, int(rng.choice([2, 9, 70, 400])), batch)
        lens = np.where(rng.random(batch) < 0.15, -1, rng.integers(0, int(rng.choice([1, 300, 5000])), batch))
        total, chain = int(rows.sum()) + int(rng.integers(0, 3)), int(rng.integers(0, 2))
        if total == 0:
            continue
        plen, width, d = int(rng.choice([0, 0, 1, 700])), int(rng.integers(0, 400)), int(rng.choice([16, 64, 128]))
        t = int(rng.integers(0, 2))
        a = W.attn_tree_args(batch=batch, rows=total, n_q=n_kv * group, n_kv=n_kv, head_dim=d, qdtype=t, kvdtype=t, q=P,
                             out=P, q_stride=0, out_stride=0, row_start=P, mask=None if chain else P, mask_words=1,
                             prefix_len=plen, prefix_stride=plen, k_pages=P, v_pages=P, page_table=P, seq_len=P,
                             num_pages=1, page_size=16, table_stride=width, scale=1.0)
        out = (ctypes.c_longlong * len(NAMES))()
        assert host.plan(ctypes.byref(a), out) == 1
        p = dict(zip(NAMES, out))
        cap, mt = 16 * width, p["mt"]
        E = host.extra()
        segs = [p["prefix_tiles"]] * (n_kv * p["prefix_row_tiles"])
        for R, n in zip(rows.tolist(), lens.tolist()):
            if n >= 0 and R > 0:
                segs += [host.tiles(group, mt, chain, cap, n, R, i) for i in range(-(-R * group // mt))] * n_kv
        if not segs:
            continue
        starts, seen = np.concatenate([[0], np.cumsum(np.array(segs) + E)]), {}
        line = int(starts[-1])
        assert p["ctas"] in (152, 304, 608)
        C = min(p["ctas"], line)
        for c in range(C):
            lo, hi = host.first(line, C, c), host.first(line, C, c + 1)
            j = int(np.searchsorted(starts, lo, side="right")) - 1
            while lo < hi:
                end = min(hi, int(starts[j + 1]))
                t0, t1 = (max(0, x - int(starts[j]) - E) for x in (lo, end))
                if t1 > t0:
                    assert c + j not in seen and c + j < p["pieces"], trial
                    seen[c + j] = (j, t0, t1)
                lo, j = end, j + 1
        for j, kt in enumerate(segs):  # the pieces that a join looks at are those there are, and cover the segment
            c0, c1 = host.owner(line, C, int(starts[j]) + E), host.owner(line, C, int(starts[j]) + E + kt - 1)
            parts = [seen[c + j] for c in range(c0, c1 + 1)]
            assert [x[0] for x in parts] == [j] * len(parts)
            assert [x[1] for x in parts] == [0] + [x[2] for x in parts[:-1]] and parts[-1][2] == kt
        assert len(seen) == sum(host.owner(line, C, int(starts[j]) + E + kt - 1) - host.owner(line, C, int(starts[j]) + E) + 1
                                for j, kt in enumerate(segs))
        slots = p["pieces"] * mt
        assert p["o"] == 0 and slots * d * 4 <= p["ml"] and p["ml"] + slots * 8 <= p["rec"]
        assert p["rec"] + p["rec_bytes"] <= p["line"] and p["line"] + 8 <= p["total"]
        assert p["ml"] % 256 == p["rec"] % 256 == p["line"] % 256 == 0


def test_sizes_whose_work_cannot_be_counted(W, host):
    """Sizes under which requests could have 2^37 units of work (a tile of 128 keys against a row tile of 16) are refused; under
    all others their number fits, however rows and tokens fall on the requests."""
    good = dict(batch=1, rows=1, n_q=1, n_kv=1, head_dim=64, qdtype=0, kvdtype=0, q=P, out=P, q_stride=64, out_stride=64, row_start=P,
                k_pages=P, v_pages=P, page_table=P, seq_len=P, num_pages=1, page_size=1024, table_stride=1, scale=1.0,
                d_workspace=P << 8, workspace_bytes=1 << 60)
    out = (ctypes.c_longlong * len(NAMES))()

    def ok(**kw):
        return host.plan(ctypes.byref(W.attn_tree_args(**{**good, **kw})), out) == 1

    full = dict(table_stride=1 << 20)  # 2^30 tokens, 2^23 tiles
    assert ok(rows=1, **full) and ok(rows=(1 << 18) - 64, **full) and not ok(rows=(1 << 18), **full)
    assert ok(batch=4096, rows=4096, n_q=3, n_kv=3, **full) and not ok(batch=4096, rows=4096, n_q=4, n_kv=4, **full)
    assert ok(batch=4096, rows=(1 << 20) - 1, n_q=16, n_kv=16, table_stride=8) and not ok(batch=4096, rows=(1 << 20) - 1, n_q=16, table_stride=1 << 20)
    kw = {**good, "batch": 4096, "rows": 4096, "n_q": 4, "n_kv": 4, "q_stride": 256, "out_stride": 256, **full}
    with pytest.raises(W.WsgError, match="attn_tree_paged") as e:
        W.attn_tree_paged(W.attn_tree_args(**kw))
    assert e.value.status == 1
    rng = np.random.default_rng(1)
    most = 0
    for _ in range(3000):
        n_kv, group = 1 << int(rng.integers(0, 8)), int(rng.integers(1, 17))
        rows, batch = int(2 ** rng.uniform(0, 24)), int(2 ** rng.uniform(0, 12))
        width = int(2 ** rng.uniform(0, 20))
        if rows * n_kv * group >= 1 << 24 or not ok(batch=batch, rows=rows, n_q=n_kv * group, n_kv=n_kv, table_stride=width):
            continue
        tiles = lambda r: -(-r * group // 16)
        k = min(batch, rows)  # requests of one row and the rest in one, or shared out
        for shares in ([1] * (k - 1) + [rows - k + 1], [rows // k + (i < rows % k) for i in range(k)]):
            units = n_kv * sum(tiles(r) for r in shares) * (-(-width * 1024 // 128) + host.extra())
            most = max(most, units)
            assert units < 1 << 37
    assert most > 1 << 36


def test_spans(host):
    assert host.meet(100, 10, 109, 5) and host.meet(109, 5, 100, 10) and host.meet(100, 10, 100, 1)
    assert not host.meet(100, 10, 110, 5) and not host.meet(110, 5, 100, 10)
    assert not host.meet(0, 10, 0, 10) and not host.meet(100, 0, 100, 10)


# ---- the definitions themselves ----------------------------------------------------------------------------------------

def test_definition_of_ancestors():
    r = OD.ancestors([-1, 0, 0, 1, 5, 4, 3], 7)
    assert [x and x[1] for x in r] == [0, 1, 1, 2, None, None, 3]
    assert np.flatnonzero(r[6][0]).tolist() == [0, 1, 3, 6]
    assert [x[1] for x in OD.ancestors(None, 3)] == [0, 1, 2]


def test_definition_of_slots():
    """Two requests and an ended one: 3 tokens and 4 rows, pages of 4; 0 tokens and 1 row."""
    o = OD.step_slots([3, -1, 0], [4, 9, 1], [1, 2, 0], np.array([[5, -1], [7, 8], [-1, -1]]), np.array([1, 2, 3, 0, 4, 6, 9, 9, 9, 9]),
                      (0, 3), 4, 6)
    assert o["new_table"].tolist() == [[5, 1], [-1, -1], [2, -1]] and o["new_owned"].tolist() == [2, 0, 1]
    assert o["row_start"].tolist() == [0, 4, 4, 5] and o["ctx_len"].tolist() == [3, -1, 0]
    assert o["slots"].tolist() == [23, 4, 5, 6, 8, -1] and o["positions"].tolist() == [3, 4, 5, 6, 0, -1]
    assert o["ring"].tolist()[:6] == [1, 2, 3, 7, 8, 6] and o["new_free_state"].tolist() == [2, 3]


def test_definition_of_adjusted_logits():
    x, t = OD.adjust([2.0, -2.0, 4.0, 1.0, 0.5], [0, 1, 0], 1, [3], 2.0, 0.25, 0.5, [(4, 9.0), (4, 2.0)],
                     np.array([True, True, False, True, True]))
    # token 0: prompt and once after it; 1 and 3: once; 2: masked; 4: the later bias
    assert x.tolist() == [0.25, -4.75, -math.inf, -0.25, 2.5] and t == 4
    assert OD.adjust([math.nan, -math.inf], [], 0, [], 1.0, 0.0, 0.0, [], None)[1] == -1


def test_definition_of_logits_of_a_prompts_rows():
    """Tokens of the prompt that are still drafted rows do not count as said."""
    one = OD.adjust([3.0, 3.0, 3.0, 3.0], [0], 3, [1, 2, 1, 3], 2.0, 0.25, 0.5, [], None)[0]
    assert one.tolist() == [1.5, 0.75, 1.5, 0.75]  # 0, 2: prompt only; 1: prompt and once behind it; 3: once
    for k in range(4):  # wherever the text ends
        two = OD.adjust([3.0, 3.0, 3.0, 3.0], [0, 1, 2, 1, 3][:k], 3, [0, 1, 2, 1, 3][k:], 2.0, 0.25, 0.5, [], None)[0]
        assert (one == two).all()
    assert OD.adjust([3.0, 3.0], [], 9, [1], 2.0, 0.25, 0.5, [], None)[0].tolist() == [3.0, 1.5]


def test_definition_of_acceptance():
    assert OD.accept([-1, 0, 0, 2, 2], [9, 5, 6, 7, 8], [6, 0, 8, 0, 3], 8) == [0, 2, 4]
    assert OD.accept([-1, 0, 0, 2, 2], [9, 5, 6, 7, 8], [6, 0, 8, 0, 3], 2) == [0, 2]
    assert OD.accept(None, [1, 2, 3, 4], [2, 3, 5, 4], 8) == [0, 1, 2]
    assert OD.accept([-1, 0], [1, -1], [-1, -1], 8) == [0]


# ---- refusals ------------------------------------------------------------------------------------------------------------

P = 4096  # an address that is never used: every call below is refused before any kernel


def places(*names, start=1):
    """Addresses far apart."""
    return {n: (i + start) << 32 for i, n in enumerate(names)}


SLOTS = dict(requests=4, rows=16, num_pages=8, page_size=16, table_stride=2, base_pos=0, mask_words=1,
             **places("held", "fresh", "owned", "parents", "page_table", "free_ring", "free_state", "new_table", "new_owned",
                      "new_free_state", "row_start", "ctx_len", "seq", "positions", "slots", "mask"))
APPEND = dict(rows=4, n_q=4, n_kv=2, head_dim=16, xdtype=0, ydtype=0, kvdtype=1, q=P, k=P, v=P, q_out=P, q_stride=64,
              k_stride=32, v_stride=32, q_out_stride=64, g_q=P, g_k=P, positions=P, inv_freq=P, eps=1e-6, rope_factor=1.0,
              rot_dim=16, interleaved=0, k_pages=P, v_pages=P, slots=P, num_pages=8, page_size=16)
ATTN = dict(batch=4, rows=9, n_q=4, n_kv=2, head_dim=16, qdtype=0, kvdtype=1, q_stride=64, out_stride=64, mask_words=1,
            prefix_len=8, prefix_stride=8, num_pages=8, page_size=16, table_stride=2, scale=0.25, workspace_bytes=1 << 30,
            **places("q", "out", "lse", "row_start", "mask", "prefix_k", "prefix_v", "k_pages", "v_pages", "page_table",
                     "seq_len", "d_workspace"))
ADJUST = dict(rows=4, vocab=100, requests=3, xdtype=0, ydtype=0, logits_stride=100, out_stride=104, tokens_stride=50,
              tokens_base=0, mask_words=1, bias_stride=5, allowed_stride=4, allowed_rows=2,
              **places("logits", "out", "next", "seq", "tokens", "tokens_len", "prompt_len", "draft_tokens", "row_start",
                       "mask", "repetition", "frequency", "presence", "bias_tokens", "bias", "bias_len", "allowed",
                       "allowed_row"))
ACCEPT = dict(batch=3, rows=9, path_stride=4, layers=2, n_kv=2, head_dim=16, kvdtype=1, layer_stride=8 * 2 * 16 * 16,
              num_pages=8, page_size=16, table_stride=2, tokens_stride=40, tokens_base=0,
              **places("row_start", "parents", "draft_tokens", "next", "seq_len", "k_pages", "v_pages", "page_table",
                       "tokens", "count", "new_len", "path", "out_tokens", "held"))
CALLS = {"step_slots": ("step_slots_args", SLOTS), "kv_append_slots": ("kv_slots_args", APPEND),
         "attn_tree_paged": ("attn_tree_args", ATTN), "logits_adjust": ("logits_adjust_args", ADJUST),
         "tree_accept_paged": ("tree_accept_args", ACCEPT)}
HEADS = [{"head_dim": 4}, {"head_dim": 20}, {"head_dim": 136}, {"head_dim": 0}, {"head_dim": -8}]
PAGES = [{"page_size": 0}, {"page_size": 3}, {"page_size": 2048}, {"page_size": -16}, {"num_pages": -1}]
POOLS = [{"k_pages": P + 2}, {"v_pages": P + 8}, {"k_pages": None}, {"v_pages": None}]


def nulls(*names):
    return [{n: None} for n in names]


BAD = {
    "step_slots": PAGES + [{"requests": -1}, {"requests": 4097}, {"rows": -1}, {"table_stride": -1}, {"base_pos": -1},
                           {"base_pos": (1 << 30) + 1}, {"table_stride": 1 << 27}, {"mask_words": 9}, {"mask_words": -1},
                           {"mask_words": 0}] + nulls(
        "held", "fresh", "owned", "page_table", "free_ring", "free_state", "new_table", "new_owned", "new_free_state",
        "row_start", "ctx_len"),
    "kv_append_slots": HEADS + PAGES + POOLS + [
        {"rows": -1}, {"n_q": -1}, {"n_kv": 0}, {"xdtype": 2}, {"ydtype": 5}, {"kvdtype": 2}, {"rot_dim": 3}, {"rot_dim": 18},
        {"eps": -1.0}, {"q_stride": -1}, {"v_stride": -1}, {"q_out_stride": 63}] + nulls("q", "k", "v", "q_out", "positions",
                                                                                         "inv_freq", "slots"),
    "attn_tree_paged": HEADS + PAGES + POOLS + [
        {"batch": -1}, {"batch": 4097}, {"rows": -1}, {"rows": 1 << 22}, {"n_q": 3}, {"n_q": 0}, {"n_kv": 0}, {"n_q": 34, "n_kv": 2},
        {"qdtype": 2}, {"kvdtype": 2}, {"prefix_len": -1}, {"prefix_stride": 7}, {"out_stride": 63}, {"q_stride": -1},
        {"table_stride": -1}, {"table_stride": 1 << 30}, {"mask_words": -1}, {"mask_words": (1 << 20) + 1},
        {"prefix_len": (1 << 30) - 31, "prefix_stride": 1 << 30}, {"prefix_k": P + 4}, {"d_workspace": P + 16}] + nulls(
        "q", "out", "row_start", "seq_len", "prefix_k", "prefix_v", "page_table", "d_workspace"),
    "logits_adjust": [{"rows": -1}, {"vocab": 0}, {"vocab": (1 << 20) + 1}, {"requests": -1}, {"xdtype": 2}, {"ydtype": 2},
                      {"mask_words": -1}, {"mask_words": 0}, {"bias_stride": -1}, {"allowed_rows": -1}, {"tokens_base": -1},
                      {"out": None, "next": None}, {"logits_stride": 99}, {"out_stride": 99}, {"logits_stride": -100},
                      {"tokens_stride": -1}, {"allowed_stride": 3}] + nulls("logits", "tokens_len", "row_start", "bias",
                                                                            "bias_len"),
    "tree_accept_paged": HEADS + PAGES + POOLS + [
        {"batch": -1}, {"batch": 65536}, {"rows": -1}, {"path_stride": 0}, {"path_stride": 257}, {"layers": -1},
        {"layers": 65536}, {"n_kv": 0}, {"n_kv": 16385}, {"kvdtype": 2}, {"table_stride": -1}, {"layer_stride": -4096},
        {"layer_stride": 4097}, {"layer_stride": 8 * 2 * 16 * 16 - 8}, {"layer_stride": 0}, {"tokens_base": -1},
        {"tokens_stride": -1}] + nulls("row_start", "draft_tokens", "next", "seq_len", "page_table", "count", "new_len", "path",
                                       "out_tokens"),
}


@pytest.mark.parametrize("call,change", [(c, b) for c, bs in BAD.items() for b in bs], ids=str)
def test_refusals(W, call, change):
    args, good = CALLS[call]
    with pytest.raises(W.WsgError) as e:
        getattr(W, call)(getattr(W, args)(**{**good, **change}))
    assert e.value.status == 1, str(e.value)
    assert call in str(e.value)


OFF = {  # bytes of an element behind each pointer, with the codes that decide it
    "step_slots": {**{n: 4 for n in places("held", "fresh", "owned", "parents", "page_table", "free_ring", "free_state",
                                           "new_table", "new_owned", "new_free_state", "row_start", "ctx_len", "seq",
                                           "positions", "mask")}, "slots": 8},
    "kv_append_slots": {"g_q": 4, "g_k": 4, "positions": 4, "inv_freq": 8, "q": "xdtype", "k": "xdtype", "v": "xdtype",
                        "q_out": "ydtype", "slots": 8},
    "attn_tree_paged": {"q": "qdtype", "out": "qdtype", "lse": 4, "row_start": 4, "mask": 4, "page_table": 4, "seq_len": 4},
    "logits_adjust": {"logits": "xdtype", "out": "ydtype", **{n: 4 for n in places(
        "next", "seq", "tokens", "tokens_len", "prompt_len", "draft_tokens", "row_start", "mask", "repetition", "frequency",
        "presence", "bias_tokens", "bias", "bias_len", "allowed", "allowed_row")}},
    "tree_accept_paged": {n: 4 for n in places("row_start", "parents", "draft_tokens", "next", "seq_len", "page_table", "tokens",
                                               "count", "new_len", "path", "out_tokens", "held")},
}


@pytest.mark.parametrize("call,name", [(c, n) for c, names in OFF.items() for n in names], ids=str)
def test_refusals_of_addresses_off_their_elements(W, call, name):
    """An address that no element of the field's type can have: the kernel's access would fault."""
    args, good = CALLS[call]
    size = OFF[call][name]
    for code, width in ((0, 4), (1, 2)) if isinstance(size, str) else ((None, size),):
        kw = {**good, **({size: code} if code is not None else {})}
        for off in [o for o in (1, 2, 4) if o < width]:
            with pytest.raises(W.WsgError) as e:
                getattr(W, call)(getattr(W, args)(**{**kw, name: (99 << 32) + off}))
            assert e.value.status == 1 and call in str(e.value) and "aligned to its elements" in str(e.value)


OVER = {  # outputs, and the arguments that they must not lie over
    "step_slots": (("new_table", "new_owned", "new_free_state", "row_start", "ctx_len", "seq", "positions", "slots", "mask", "free_ring"),
                   ("held", "fresh", "owned", "parents", "page_table", "free_state")),
    "attn_tree_paged": (("out", "lse", "d_workspace"), ("q", "row_start", "mask", "page_table", "seq_len")),
    "logits_adjust": (("out", "next"), ("logits", "seq", "tokens", "tokens_len", "prompt_len", "draft_tokens", "row_start", "mask",
                                        "repetition", "frequency", "presence", "bias_tokens", "bias", "bias_len", "allowed",
                                        "allowed_row")),
    "tree_accept_paged": (("count", "new_len", "path", "out_tokens", "tokens"),
                          ("row_start", "parents", "draft_tokens", "next", "seq_len", "held", "page_table")),
}
IN_PLACE = {("step_slots", "new_table", "page_table"), ("attn_tree_paged", "out", "q"), ("logits_adjust", "out", "logits")}


@pytest.mark.parametrize("call", list(OVER))
def test_refusals_of_outputs_over_other_arguments(W, call):
    """Other CTAs would have yet to read what one writes over."""
    args, good = CALLS[call]
    outs, ins = OVER[call]
    for o in outs:
        for other in ins + tuple(x for x in outs if x != o):
            # the first word of the other, and the last word of `o` on its first
            for at in (good[other] + (0 if (call, o, other) not in IN_PLACE else 16),):
                if o == "d_workspace":
                    at = good[other]
                with pytest.raises(W.WsgError, match="overlap") as e:
                    getattr(W, call)(getattr(W, args)(**{**good, o: at}))
                assert e.value.status == 1 and call in str(e.value), (o, other)


@pytest.fixture(scope="module")
def series(tmp_path_factory):
    """csrc/spans.h compiled as plain C++: whether two series of spans meet."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("spans")
    (d / "s.cpp").write_text('#include "spans.h"\nusing namespace wsg;\nextern "C" {\n'
                             "int meet(size_t p, size_t a, long long n, long long s, size_t q, size_t b, long long m, long long t) {\n"
                             "  return series_meet(Spans{{(void*)p, a}, n, s}, Spans{{(void*)q, b}, m, t}); }\n"
                             "size_t pool(long long pages, long long page) { return span_pool((void*)16, pages, page).bytes; }\n}\n")
    inc = os.path.join(ROOT, "weight_streaming_gemv_token_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(d / "s.cpp"), "-o", str(d / "s.so")], check=True)
    L, q, z = ctypes.CDLL(str(d / "s.so")), ctypes.c_longlong, ctypes.c_size_t
    L.meet.argtypes, L.pool.argtypes, L.pool.restype = [z, z, q, q, z, z, q, q], [q, q], z
    return L


def test_series_of_spans(series):
    """Against the bytes themselves: equal strides exactly, other strides by what each covers as a whole."""
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(4000):
        n, m = (int(x) for x in rng.integers(1, 6, 2))
        s = int(rng.integers(1, 40))
        t = s if rng.random() < 0.7 else int(rng.integers(1, 40))
        a, b = int(rng.integers(1, s + 6)), int(rng.integers(1, t + 6))
        p, q = (int(x) for x in rng.integers(1000, 1300, 2))
        x, y = ({p0 + i * st + k for i in range(c) for k in range(w)} for p0, w, c, st in ((p, a, n, s), (q, b, m, t)))
        got = bool(series.meet(p, a, n, s, q, b, m, t))
        if s == t or n == 1 or m == 1:
            assert got == bool(x & y), (p, a, n, s, q, b, m, t)
        else:
            assert got == (p <= max(y) and q <= max(x))
        seen.add((got, s == t))
    assert len(seen) == 4
    assert not series.meet(0, 8, 2, 8, 0, 8, 2, 8) and not series.meet(100, 0, 2, 8, 100, 8, 1, 8)
    assert series.meet(100, 8, 4, 0, 104, 8, 1, 0)
    big = 1 << 62
    assert series.pool(2**31 - 1, 16384 * 1024 * 128 * 4) == big and series.pool(3, 10) == 30 and series.pool(0, 10) == 0
    assert series.meet(1 << 40, big, 1, 0, 3 << 50, 4, 1, 0) and not series.meet(1 << 40, big, 1, 0, (1 << 40) - 4, 4, 1, 0)


def test_refusals_of_outputs_over_caches(W):
    """An output over the prefix or a pool; a pool over another argument of the calls that write it."""
    bf, pool = 2 * 16 * 16 * 2, 8 * 2 * 16 * 16 * 2  # a page, a pool
    for o in ("out", "lse", "d_workspace"):
        for name, size in (("prefix_k", 2 * 8 * 16 * 2), ("prefix_v", 2 * 8 * 16 * 2), ("k_pages", pool), ("v_pages", pool)):
            for at in (0, (size - 1) // 256 * 256):
                with pytest.raises(W.WsgError, match="attn_tree_paged: an output overlaps") as e:
                    W.attn_tree_paged(W.attn_tree_args(**{**ATTN, o: ATTN[name] + at}))
                assert e.value.status == 1
    apart = places(*[n for n in APPEND if APPEND[n] == P])
    good = {**APPEND, **apart}
    inputs = ("q", "k", "v", "g_q", "g_k", "positions", "inv_freq", "slots")
    for o, size in (("k_pages", pool), ("v_pages", pool), ("q_out", 64 * 4 * 4)):
        for other in inputs + tuple(x for x in ("k_pages", "v_pages", "q_out") if x != o):
            kw = {**good, other: good[o] + size - 16}  # its first bytes are the output's last
            if o == "q_out" and other.endswith("pages"):
                kw = {**good, "q_out": good[other] + pool - 16}
            with pytest.raises(W.WsgError, match="kv_append_slots: an output overlaps") as e:
                W.kv_append_slots(W.kv_slots_args(**kw))
            assert e.value.status == 1, (o, other)
    # one row of queries in place reaches into the keys beside it
    with pytest.raises(W.WsgError, match="kv_append_slots: an output overlaps"):
        W.kv_append_slots(W.kv_slots_args(**{**good, "q_out": good["q"], "k": good["q"] + 63 * 4, "q_stride": 96, "k_stride": 96, "q_out_stride": 96}))
    layers = 2 * pool
    for o in ("count", "new_len", "path", "out_tokens", "tokens", "row_start", "parents", "draft_tokens", "next", "seq_len", "held", "page_table"):
        for name in ("k_pages", "v_pages"):
            for at in (0, pool, layers - 4):
                with pytest.raises(W.WsgError, match="tree_accept_paged: a pool overlaps") as e:
                    W.tree_accept_paged(W.tree_accept_args(**{**ACCEPT, o: ACCEPT[name] + at}))
                assert e.value.status == 1, (o, name, at)
    for at in (0, pool, layers - bf):
        with pytest.raises(W.WsgError, match="tree_accept_paged: a pool overlaps"):
            W.tree_accept_paged(W.tree_accept_args(**{**ACCEPT, "v_pages": ACCEPT["k_pages"] + at}))


def test_refusals_of_rows_that_move_in_place(W):
    for change in ({"out_stride": 72}, {"q_stride": 0}, {"q_stride": 128}):
        with pytest.raises(W.WsgError, match="attn_tree_paged: out over q needs") as e:
            W.attn_tree_paged(W.attn_tree_args(**{**ATTN, "out": ATTN["q"], **change}))
        assert e.value.status == 1
    for change in ({"out_stride": 108}, {"ydtype": 1}, {"xdtype": 1}):
        with pytest.raises(W.WsgError, match="logits_adjust: out over logits needs") as e:
            W.logits_adjust(W.logits_adjust_args(**{**ADJUST, "out": ADJUST["logits"], "out_stride": 100, **change}))
        assert e.value.status == 1
    for change in ({"q_out_stride": 72}, {"q_stride": 0}, {"ydtype": 1}):
        with pytest.raises(W.WsgError, match="kv_append_slots: q_out over q needs") as e:
            W.kv_append_slots(W.kv_slots_args(**{**APPEND, "k": 2 * P, **change}))
        assert e.value.status == 1


def test_empty_calls_do_nothing(W):
    W.attn_tree_paged(W.attn_tree_args(**{**ATTN, "batch": 0}))
    W.attn_tree_paged(W.attn_tree_args(**{**ATTN, "rows": 0}))
    W.logits_adjust(W.logits_adjust_args(**{**ADJUST, "rows": 0}))
    W.tree_accept_paged(W.tree_accept_args(**{**ACCEPT, "batch": 0}))
    W.kv_append_slots(W.kv_slots_args(**{**APPEND, "rows": 0}))


def test_null_argument_blocks(W):
    for call in CALLS:
        assert getattr(W.library(), call)(None, None) == 1
    assert W.library().attn_tree_paged_workspace(None) == 0


def test_argument_blocks_refuse_other_tensors(W):
    import torch

    f, i, l = torch.zeros(4), torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    for call, name, t in (("step_slots", "slots", i), ("step_slots", "held", l), ("step_slots", "mask", f),
                          ("kv_append_slots", "slots", i), ("attn_tree_paged", "mask", l), ("attn_tree_paged", "row_start", l),
                          ("logits_adjust", "allowed", f), ("logits_adjust", "next", l), ("logits_adjust", "repetition", i),
                          ("logits_adjust", "logits", i), ("tree_accept_paged", "count", l), ("tree_accept_paged", "tokens", l)):
        args, good = CALLS[call]

        class OnDevice:  # what the block looks at of a tensor
            is_cuda, dtype, shape = True, t.dtype, t.shape

            def __getattr__(self, n):
                return getattr(t, n)

        with pytest.raises(W.WsgError, match=f"{args}.{name}: the tensor is"):
            getattr(W, call)(getattr(W, args)(**{**good, name: OnDevice()}))
        with pytest.raises(W.WsgError, match="not on a CUDA device"):
            getattr(W, args)(**{**good, name: t})


def test_argument_blocks_refuse_masks_that_are_not_contiguous(W):
    import torch

    t = torch.zeros((4, 6), dtype=torch.int32)[:, ::2]

    class OnDevice:
        is_cuda, dtype, shape = True, t.dtype, t.shape

        def __getattr__(self, n):
            return getattr(t, n)

    for call in ("step_slots", "attn_tree_paged", "logits_adjust"):
        args, good = CALLS[call]
        with pytest.raises(W.WsgError, match=f"{args}.mask"):
            getattr(W, call)(getattr(W, args)(**{**good, "mask": OnDevice()}))
