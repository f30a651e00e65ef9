"""Host side of the calls for several branches: index arithmetic, rotation frequencies, refusals (no GPU)."""
import ctypes
import itertools
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import oracle.branches as OB

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def W():
    from weight_streaming_gemv_token_gb300 import build as bld

    bld.build()
    import weight_streaming_gemv_token_gb300 as W

    return W


@pytest.fixture(scope="module")
def paging(tmp_path_factory):
    """csrc/paging.h compiled as plain C++."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("paging")
    src = d / "p.cpp"
    src.write_text('#include "paging.h"\nusing namespace wsg;\nextern "C" {\n'
                   "int shift_of(int n) { return page_shift(n); }\n"
                   "int page(int pages, int n_kv, int shift, int width, const int32_t* row, int64_t i) {\n"
                   "  return page_of(PagePool{pages, n_kv, shift, width}, row, i); }\n"
                   "int64_t row(int pages, int n_kv, int shift, int page, int g, int64_t i) {\n"
                   "  return pool_row(PagePool{pages, n_kv, shift, 0}, page, g, i); }\n}\n")
    lib = d / "p.so"
    inc = os.path.join(ROOT, "weight_streaming_gemv_token_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    L.page.argtypes = [ctypes.c_int] * 4 + [ctypes.c_void_p, ctypes.c_int64]
    L.row.argtypes = [ctypes.c_int] * 5 + [ctypes.c_int64]
    L.row.restype = ctypes.c_int64
    return L


def test_page_sizes(paging):
    for n in range(-2, 1100):
        ok = 1 <= n <= 1024 and n & (n - 1) == 0
        assert paging.shift_of(n) == (int(math.log2(n)) if ok else -1), n


def test_every_page_lookup_stays_inside(paging):
    """Indexes around both ends of a table, entries around both ends of the pool."""
    for pages, width, shift in itertools.product((0, 1, 3), (0, 1, 2, 5), (0, 1, 4)):
        row = np.array([2, -1, 0, 3, 2**31 - 1][:width] + [77], dtype=np.int32)  # 77: behind the row, never to be read
        for i in list(range(-3, (width + 1) << shift)) + [-2**31, 2**31 - 1, 2**31, 2**40, -2**40]:
            p = paging.page(pages, 2, shift, width, row.ctypes.data, i)
            want = -1
            if 0 <= i < width << shift and 0 <= row[i >> shift] < pages:
                want = row[i >> shift]
            assert p == want, (pages, width, shift, i)


def test_pool_rows_are_64_bit_and_distinct(paging):
    seen = set()
    for page, g, i in itertools.product(range(3), range(4), range(8)):
        r = paging.row(3, 4, 3, page, g, i)
        assert r == (page * 4 + g) * 8 + i
        seen.add(r)
    assert len(seen) == 96
    # token indexes of later pages use their place inside the page
    assert paging.row(3, 4, 3, 1, 2, 8 * 7 + 5) == (1 * 4 + 2) * 8 + 5
    assert paging.row(2**31 - 1, 64, 10, 2**31 - 2, 63, 1023) == ((2**31 - 2) * 64 + 63) * 1024 + 1023


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """csrc/attn_plan.h compiled as plain C++: the plan of an attention call on 152 SMs."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    src = d / "p.cpp"
    src.write_text('#include "attn_plan.h"\nextern "C" int plan(const attn_shared_args* a, long long* o) {\n'
                   "  if (!wsg::attn_sizes_ok(a)) return 0;\n"
                   "  const wsg::AsPlan p = wsg::attn_plan(a, 152);\n"
                   "  const long long v[] = {p.tc, p.own_joins, p.na, p.row_groups, p.prefix_slots, p.prefix_chunk,\n"
                   "    p.own_slots, p.own_block, p.own_seg, p.own_per, p.prefix_items, p.own_items,\n"
                   "    (long long)p.o, (long long)p.ml, (long long)p.total};\n"
                   "  for (int i = 0; i < 15; ++i) o[i] = v[i];\n  return 1;\n}\n")
    lib = d / "p.so"
    inc = os.path.join(ROOT, "weight_streaming_gemv_token_gb300", "csrc")
    cmd = [cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o", str(lib)]
    checked = ["-fsanitize=undefined", "-fno-sanitize-recover=undefined"]  # where the toolchain has its library
    if subprocess.run(cmd + checked, capture_output=True).returncode != 0:
        subprocess.run(cmd, check=True)
    return ctypes.CDLL(str(lib)).plan


NAMES = ("tc own_joins na row_groups prefix_slots prefix_chunk own_slots own_block own_seg own_per prefix_items own_items "
         "o ml total").split()


def test_attention_plans_cover_every_key_once(W, plan):
    """Prefix splits and own pieces cover their axes; every slot that is written or joined lies inside the workspace."""
    rng = np.random.default_rng(0)
    for n in range(3000):
        n_kv = int(rng.choice([1, 2, 3, 8, 16]))
        group = int(rng.choice([1, 2, 3, 8, 9, 16]))
        batch = int(np.exp(rng.uniform(0, np.log(300))))
        page = int(2 ** rng.integers(0, 8))
        width = int(rng.choice([0, 1, 2, 7, int(np.exp(rng.uniform(0, np.log(5000))))]))
        plen = int(rng.choice([0, 1, 127, 128, 129, int(np.exp(rng.uniform(0, np.log(300000))))]))
        d = int(rng.choice([8, 16, 64, 96, 128]))
        a = W.attn_shared_args(**{**ATTN, "batch": batch, "n_q": n_kv * group, "n_kv": n_kv, "head_dim": d,
                                  "qdtype": int(rng.integers(0, 2)), "kvdtype": int(rng.integers(0, 2)), "prefix_len": plen,
                                  "prefix_stride": plen, "page_size": page, "table_stride": width})
        out = (ctypes.c_longlong * 15)()
        assert plan(ctypes.byref(a), out) == 1
        p = dict(zip(NAMES, out))
        rows, capacity, segs = batch * group, page * width, batch * n_kv
        block = 128 if p["tc"] else p["na"] or 128
        assert p["row_groups"] * block >= rows > (p["row_groups"] - 1) * block
        assert p["prefix_slots"] * p["prefix_chunk"] >= plen and (p["prefix_slots"] - 1) * p["prefix_chunk"] < max(1, plen)
        assert p["prefix_items"] == p["prefix_slots"] * n_kv * p["row_groups"]
        assert p["tc"] == (plen > 0 and d == 128 and a.qdtype == 1 and a.kvdtype == 1)
        assert p["tc"] <= (p["prefix_chunk"] % 128 == 0)
        slots = p["prefix_slots"] + p["own_slots"]
        assert p["ml"] >= slots * batch * n_kv * group * d * 4 and p["total"] >= p["ml"] + 8 * slots * batch * n_kv * group
        if p["own_joins"]:
            assert p["own_items"] == segs and p["own_slots"] == 0 and a.kvdtype == 1
            continue
        assert p["own_seg"] * p["own_block"] >= capacity
        warps = 1 if a.kvdtype == 0 else 4 if d == 128 and a.qdtype == 1 else 8
        assert p["own_items"] * warps * p["own_per"] >= p["own_seg"] * segs
        if capacity:  # the slots that the pieces of a segment take, whatever it holds
            seg = np.unique(np.clip([0, 1, segs // 2, segs - 1], 0, segs - 1))
            first, last = seg * p["own_seg"] // p["own_per"], ((seg + 1) * p["own_seg"] - 1) // p["own_per"]
            assert (last - first < p["own_slots"]).all()


def test_attention_plan_of_an_empty_call(W, tmp_path):
    """No branch is a call with nothing to do, whose workspace can be asked for like any other's. (A process of its own:
    a division by zero would end it.)"""
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    src = tmp_path / "e.cpp"
    src.write_text('#include "attn_plan.h"\nint main() {\n  for (int i = 0; i < 32; ++i) {\n    attn_shared_args a{};\n'
                   "    a.n_q = 16, a.n_kv = 8, a.head_dim = i & 1 ? 128 : 64, a.qdtype = i >> 1 & 1, a.kvdtype = i >> 2 & 1;\n"
                   "    a.prefix_len = a.prefix_stride = i & 8 ? 512 : 0, a.page_size = 16, a.table_stride = i & 16 ? 4 : 0;\n"
                   "    if (!wsg::attn_sizes_ok(&a)) return 1;\n    const wsg::AsPlan p = wsg::attn_plan(&a, 152);\n"
                   "    if (p.total == 0 || p.prefix_items || p.own_items) return 2;\n  }\n  return 0;\n}\n")
    inc = os.path.join(ROOT, "weight_streaming_gemv_token_gb300", "csrc")
    # (an integer division by zero has no trap on every machine: the compiler's own check finds it there)
    cmd = [cxx, "-std=c++17", "-O1", "-I", inc, str(src), "-o", str(tmp_path / "e")]
    checked = ["-fsanitize=integer-divide-by-zero", "-fsanitize-undefined-trap-on-error"]
    subprocess.run(cmd + checked, check=True)
    assert subprocess.run([str(tmp_path / "e")]).returncode == 0


def test_frequencies(W):
    w, f = W.rope_frequencies(128, 1e6)
    np.testing.assert_allclose(w, 1e6 ** (-np.arange(0, 128, 2) / 128), rtol=1e-14)
    assert f == 1.0
    lin, f = W.rope_frequencies(64, 1e4, W.ROPE_LINEAR, factor=8.0)
    np.testing.assert_allclose(lin, 1e4 ** (-np.arange(0, 64, 2) / 64) / 8, rtol=1e-14)
    assert f == 1.0
    base, f = W.rope_frequencies(64, 1e4, W.ROPE_BASE, factor=8.0)
    plain = 1e4 ** (-np.arange(0, 64, 2) / 64)
    assert base[0] == 1.0 and f == 1.0
    np.testing.assert_allclose(base[-1], plain[-1] / 8, rtol=1e-12)  # the slowest pair takes the whole factor
    ramp, f = W.rope_frequencies(128, 1e6, W.ROPE_RAMP, factor=4.0, orig_context=32768)
    plain = 1e6 ** (-np.arange(0, 128, 2) / 128)
    turns = 32768 * plain / (2 * np.pi)
    fast, slow = turns >= 32, turns <= 1
    assert fast.any() and slow.any() and not (fast | slow).all()
    np.testing.assert_allclose(np.array(ramp)[fast], plain[fast], rtol=1e-13)
    np.testing.assert_allclose(np.array(ramp)[slow], plain[slow] / 4, rtol=1e-13)
    mid = ~(fast | slow)
    assert ((np.array(ramp)[mid] < plain[mid]) & (np.array(ramp)[mid] > plain[mid] / 4)).all()
    assert abs(f - (0.1 * math.log(4.0) + 1.0)) < 1e-6


def test_frequency_refusals(W):
    for kw in ({"rot_dim": 3}, {"rot_dim": 0}, {"rot_dim": 130}, {"theta": 0.0}, {"theta": -1.0}, {"theta": math.nan},
               {"theta": math.inf}, {"kind": 4}, {"kind": -1}, {"kind": 1, "factor": 0.5}, {"kind": 1, "factor": math.nan},
               {"kind": 2, "factor": 2.0, "rot_dim": 2}, {"kind": 3, "factor": 2.0, "orig_context": 0.0},
               {"kind": 3, "factor": 2.0, "orig_context": 10.0, "beta_slow": 4.0, "beta_fast": 4.0},
               {"kind": 3, "factor": 2.0, "orig_context": 10.0, "beta_slow": 0.0}):
        with pytest.raises(W.WsgError) as e:
            W.rope_frequencies(**{"rot_dim": 64, "theta": 1e4, **kw})
        assert e.value.status == 1, kw
    assert W.library().rope_frequencies(None, None, None) == 1


P = 4096  # an address that is never used: every call below is refused before any kernel

ROPE = dict(rows=4, n_q=4, n_kv=2, head_dim=16, xdtype=0, ydtype=0, q=P, k=P, q_out=P, k_out=P, q_stride=64, k_stride=32,
            q_out_stride=64, k_out_stride=32, g_q=P, g_k=P, positions=P, inv_freq=P, eps=1e-6, rope_factor=1.0,
            rot_dim=16, interleaved=0)
APPEND = dict(rows=4, n_q=4, n_kv=2, head_dim=16, xdtype=0, ydtype=0, kvdtype=1, q=P, k=P, v=P, q_out=P, q_stride=64,
              k_stride=32, v_stride=32, q_out_stride=64, g_q=P, g_k=P, positions=P, inv_freq=P, eps=1e-6,
              rope_factor=1.0, rot_dim=16, interleaved=0, k_pages=P, v_pages=P, page_table=P, seq=P, n_seq=4,
              num_pages=8, page_size=16, table_stride=2, base_pos=0)
ATTN = dict(batch=4, n_q=4, n_kv=2, head_dim=16, qdtype=0, kvdtype=1, q=P, out=P, lse=P, q_stride=64, out_stride=64,
            prefix_k=P, prefix_v=P, prefix_len=8, prefix_stride=8, k_pages=P, v_pages=P, page_table=P, seq_len=P,
            num_pages=8, page_size=16, table_stride=2, scale=0.25, d_workspace=P, workspace_bytes=1 << 30)
SELECT = dict(beams=4, vocab=100, n_out=8, logits=P, logits_stride=100, scores=P, out_scores=P, out_parents=P,
              out_tokens=P, d_workspace=P, workspace_bytes=1 << 30)
REORDER = dict(beams=4, layers=2, n_kv=2, head_dim=16, kvdtype=1, k_pages=P, v_pages=P, layer_stride=1024, num_pages=8,
               page_size=16, table_stride=2, parents=P, spare=P, old_table=P, old_len=P, new_table=2 * P, new_len=2 * P)
CALLS = {"qk_norm_rope": ("qk_rope_args", ROPE), "kv_append_paged": ("kv_append_args", APPEND),
         "attn_shared_prefix": ("attn_shared_args", ATTN), "beam_select": ("beam_select_args", SELECT),
         "beam_reorder_pages": ("beam_reorder_args", REORDER)}
HEADS = [{"head_dim": 4}, {"head_dim": 20}, {"head_dim": 136}, {"head_dim": 0}, {"head_dim": -8}]
ROWS = HEADS + [{"rows": -1}, {"n_q": -1}, {"n_kv": -1}, {"xdtype": 2}, {"ydtype": 5}, {"rot_dim": 3}, {"rot_dim": 18},
                {"rot_dim": -2}, {"eps": -1.0}, {"eps": math.nan}, {"q": None}, {"k": None}, {"q_out": None},
                {"positions": None}, {"inv_freq": None}, {"q_stride": -1}, {"k_stride": -1}, {"q_out_stride": 63}]
PAGES = [{"page_size": 0}, {"page_size": 3}, {"page_size": 2048}, {"page_size": -16}, {"num_pages": -1},
         {"k_pages": P + 2}, {"v_pages": P + 8}, {"k_pages": None}, {"v_pages": None}]
BAD = {
    "qk_norm_rope": ROWS + [{"k_out": None}, {"k_out_stride": 31}],
    "kv_append_paged": ROWS + PAGES + [{"n_kv": 0}, {"kvdtype": 2}, {"v": None}, {"page_table": None}, {"n_seq": -1},
                                       {"table_stride": -1}, {"base_pos": -1}, {"v_stride": -1}],
    "attn_shared_prefix": HEADS + PAGES + [
        {"batch": -1}, {"batch": 65536}, {"batch": 4096, "n_q": 4096, "n_kv": 4096, "out_stride": 1 << 20}, {"n_q": 3}, {"n_q": 0}, {"n_kv": 0}, {"n_q": 34, "n_kv": 2}, {"qdtype": 2},
        {"kvdtype": 2}, {"q": None}, {"out": None}, {"seq_len": None}, {"prefix_k": None}, {"prefix_v": None},
        {"prefix_len": -1}, {"prefix_stride": 7}, {"page_table": None}, {"out_stride": 63}, {"q_stride": -1},
        {"table_stride": -1}, {"table_stride": 1 << 30},
        {"prefix_len": (1 << 30) - 31, "prefix_stride": 1 << 30}, {"prefix_k": P + 4}, {"d_workspace": None},
        {"d_workspace": P + 16}],
    "beam_select": [{"beams": 0}, {"beams": 1025}, {"vocab": 0}, {"n_out": 0}, {"n_out": 1025},
                    {"beams": 1024, "vocab": 1 << 21, "logits_stride": 1 << 21}, {"logits": None}, {"scores": None},
                    {"out_scores": None}, {"out_parents": None}, {"out_tokens": None}, {"logits_stride": 99},
                    {"logits_stride": -100}, {"d_workspace": None}, {"d_workspace": P + 16}],
    "beam_reorder_pages": HEADS + PAGES + [
        {"beams": -1}, {"layers": 0}, {"layers": 65536}, {"n_kv": 0}, {"kvdtype": 2}, {"table_stride": 0},
        {"layer_stride": -1024}, {"layer_stride": 1025}, {"parents": None}, {"spare": None}, {"old_table": None},
        {"old_len": None}, {"new_table": None}, {"new_len": None}, {"new_table": P}, {"new_len": P},
        {"new_table": P + 28}, {"new_table": P - 28}, {"new_len": P + 12}, {"n_kv": 16385}],
}


@pytest.mark.parametrize("call,change", [(c, b) for c, bs in BAD.items() for b in bs], ids=str)
def test_refusals(W, call, change):
    args, good = CALLS[call]
    with pytest.raises(W.WsgError) as e:
        getattr(W, call)(getattr(W, args)(**{**good, **change}))
    assert e.value.status == 1, str(e.value)
    assert call in str(e.value)


OFF = {  # bytes of an element behind each pointer, with the codes that decide it
    "qk_norm_rope": {"g_q": 4, "g_k": 4, "positions": 4, "inv_freq": 8, "q": "xdtype", "k": "xdtype", "q_out": "ydtype",
                     "k_out": "ydtype"},
    "kv_append_paged": {"g_q": 4, "g_k": 4, "positions": 4, "inv_freq": 8, "q": "xdtype", "k": "xdtype", "v": "xdtype",
                        "q_out": "ydtype", "page_table": 4, "seq": 4},
    "attn_shared_prefix": {"q": "qdtype", "out": "qdtype", "lse": 4, "page_table": 4, "seq_len": 4},
    "beam_select": {"logits": 4, "scores": 4, "out_scores": 4, "out_parents": 4, "out_tokens": 4},
    "beam_reorder_pages": {"parents": 4, "spare": 4, "old_table": 4, "old_len": 4, "new_table": 4, "new_len": 4},
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
                getattr(W, call)(getattr(W, args)(**{**kw, name: 8 * P + off}))
            assert e.value.status == 1 and call in str(e.value) and "aligned to its elements" in str(e.value)


APART = {**REORDER, "layer_stride": 8 * 2 * 16 * 16}  # layers side by side


@pytest.mark.parametrize("change", [{"layer_stride": 0}, {"layer_stride": 8 * 2 * 16 * 16 - 8}, {"num_pages": 9},
                                    {"kvdtype": 0, "layer_stride": 8 * 2 * 16 * 16 - 4}], ids=str)
def test_refusals_of_layers_that_overlap(W, change):
    """One layer's copies would be another's sources."""
    with pytest.raises(W.WsgError, match="beam_reorder_pages: layers of") as e:
        W.beam_reorder_pages(W.beam_reorder_args(**{**APART, **change}))
    assert e.value.status == 1


@pytest.mark.parametrize("change", [{"new_len": "parents"}, {"new_len": "spare"}, {"new_len": "old_table"},
                                    {"new_len": "new_table"}, {"new_table": "parents"}, {"new_table": "spare"},
                                    {"new_table": "old_len"}], ids=str)
def test_refusals_of_outputs_over_inputs(W, change):
    """A slot's parent or spare page would be written over while its other layers have yet to read it."""
    at = {n: 8 * P * (i + 1) for i, n in enumerate(("parents", "spare", "old_table", "old_len", "new_table", "new_len"))}
    entries = {"old_table": 8, "new_table": 8}
    (out, over), = change.items()
    mine, theirs = 4 * entries.get(out, 4), 4 * entries.get(over, 4)
    for off in (0, theirs - 4, 4 - mine):  # the same place, the last word of the other, its first
        with pytest.raises(W.WsgError, match="overlap") as e:
            W.beam_reorder_pages(W.beam_reorder_args(**{**APART, **at, out: at[over] + off}))
        assert e.value.status == 1


@pytest.mark.parametrize("call,out", [("qk_norm_rope", "q"), ("qk_norm_rope", "k"), ("kv_append_paged", "q")], ids=str)
def test_refusals_of_rows_that_move_in_place(W, call, out):
    """Outputs over their own inputs with another stride or type would be written over rows that are still to be read."""
    args, good = CALLS[call]
    base = {**good, **{n: 8 * P * (i + 1) for i, n in enumerate(("q", "k", "v", "q_out", "k_out")) if n in good}}
    for change in ({f"{out}_out_stride": base[f"{out}_stride"] + 8}, {f"{out}_stride": 0}, {"ydtype": 1}, {"xdtype": 1},
                   {"rows": 1, "ydtype": 1}):
        with pytest.raises(W.WsgError, match=f"{call}: {out}_out over {out} needs") as e:
            getattr(W, call)(getattr(W, args)(**{**base, f"{out}_out": base[out], **change}))
        assert e.value.status == 1


def test_refusals_of_attention_over_queries_that_move(W):
    """A branch's output is written while others have yet to read their queries."""
    for change in ({"out_stride": 72}, {"q_stride": 0}, {"q_stride": 128}):
        with pytest.raises(W.WsgError, match="attn_shared_prefix: out over q needs") as e:
            W.attn_shared_prefix(W.attn_shared_args(**{**ATTN, "q": 8 * P, "out": 8 * P, **change}))
        assert e.value.status == 1


def test_null_arguments_and_empty_calls(W):
    lib = W.library()
    for call in CALLS:
        assert getattr(lib, call)(None, None) == 1, call
    assert lib.attn_shared_prefix_workspace(None) == 0 and lib.beam_select_workspace(None) == 0
    W.qk_norm_rope(W.qk_rope_args(**{**ROPE, "rows": 0}))
    W.qk_norm_rope(W.qk_rope_args(**{**ROPE, "n_q": 0, "n_kv": 0}))
    W.kv_append_paged(W.kv_append_args(**{**APPEND, "rows": 0}))
    W.attn_shared_prefix(W.attn_shared_args(**{**ATTN, "batch": 0}))
    W.beam_reorder_pages(W.beam_reorder_args(**{**REORDER, "beams": 0}))


def test_argument_blocks(W):
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError, match="missing rows"):
        W.qk_rope_args(**{k: v for k, v in ROPE.items() if k != "rows"})
    with pytest.raises(TypeError, match="no field"):
        W.beam_select_args(**SELECT, speed=1)
    with pytest.raises(W.WsgError, match="not on a CUDA device"):
        W.qk_rope_args(**{**ROPE, "q": torch.zeros(4)})


class OnDevice:
    """A CPU tensor that says it is on the GPU (its address is never used: every call with it is refused)."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, i):
        return OnDevice(self.t[i])


def test_argument_blocks_refuse_tensors_of_another_type(W):
    """What a call would read as something else, torch's default types first: int64 indexes, float32 frequencies (half as
    long as what is read of them), float16 for bfloat16."""
    torch = pytest.importorskip("torch")

    def t(shape, dtype):
        return OnDevice(torch.zeros(shape, dtype=getattr(torch, dtype)))

    fixed = {"int32": "positions seq page_table seq_len parents spare old_table old_len new_table new_len out_parents "
                      "out_tokens".split(),
             "float32": "g_q g_k lse logits scores out_scores".split(), "float64": ["inv_freq"]}
    coded = {"q": "xdtype", "k": "xdtype", "v": "xdtype", "q_out": "ydtype", "k_out": "ydtype", "out": "qdtype",
             "prefix_k": "kvdtype", "prefix_v": "kvdtype", "k_pages": "kvdtype", "v_pages": "kvdtype"}
    types = ("int32", "int64", "float32", "float64", "float16", "bfloat16")
    seen = set()
    for call, (args, good) in CALLS.items():
        block = getattr(W, args)
        for name in good:
            for want, names in fixed.items():
                if name not in names:
                    continue
                seen.add(name)
                block(**{**good, name: t(4, want)})
                for other in set(types) - {want}:
                    with pytest.raises(W.WsgError, match=f"{args}.{name}: the tensor is {other}") as e:
                        block(**{**good, name: t(4, other)})
                    assert e.value.status == 1
            code = coded.get(name)
            if code and call == "attn_shared_prefix" and name == "q":
                code = "qdtype"
            if code is None:
                continue
            seen.add(name)
            for value, ok in ((0, {"float32"}), (1, {"bfloat16"})):
                for dtype in types:
                    kw = {**good, code: value, name: t(4, dtype)}
                    if dtype in ok:
                        block(**kw)
                        continue
                    with pytest.raises(W.WsgError, match=f"{args}.{name}: the tensor is {dtype}") as e:
                        block(**kw)
                    assert e.value.status == 1
                # the same by a later change, in either order: at the call
                a = block(**{**good, code: 1 - value})
                a.set(name, t(4, "bfloat16" if value else "float32")).set(code, value).verify()
                setattr(a, code, 1 - value)
                with pytest.raises(W.WsgError, match=f"{args}.{name}: the tensor is"):
                    getattr(W, call)(a)
    assert seen == set(coded) | {n for names in fixed.values() for n in names}
    for dtype in ("uint8", "uint16", "int16"):  # bytes, or bfloat16 by its bits
        W.attn_shared_args(**{**ATTN, "kvdtype": 1, **{n: t(4, dtype) for n in ("prefix_k", "prefix_v", "k_pages", "v_pages")}})


def test_argument_blocks_refuse_tensors_with_gaps(W):
    """Elements that are not side by side; rows and layers may lie apart."""
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    wide, pool = torch.zeros((4, 8), **i32), torch.zeros((3, 2, 8, 2, 16, 16), dtype=torch.bfloat16)
    W.kv_append_args(**{**APPEND, "page_table": OnDevice(wide[:, :2]), "k_pages": OnDevice(pool[0, 1])})
    W.beam_reorder_args(**{**REORDER, "k_pages": OnDevice(pool[:, 1]), "old_table": OnDevice(wide[:, 4:])})
    W.qk_rope_args(**{**ROPE, "q": OnDevice(torch.zeros(4, 200)[:, 7:71])})
    none = torch.zeros(2, 16, 0, dtype=torch.bfloat16).transpose(1, 2)  # nothing in it, whatever its strides
    W.attn_shared_args(**{**ATTN, "prefix_len": 0, "prefix_k": OnDevice(none), "k_pages": OnDevice(none)})
    for call, args, change in ((W.kv_append_args, APPEND, {"page_table": wide.t()}),
                               (W.kv_append_args, APPEND, {"positions": wide[:, 1]}),
                               (W.kv_append_args, APPEND, {"v_pages": pool[:, 0, 0]}),
                               (W.beam_reorder_args, REORDER, {"k_pages": pool[:, :, :, 0]}),
                               (W.beam_reorder_args, REORDER, {"spare": wide[:, 0]}),
                               (W.qk_rope_args, ROPE, {"q": torch.zeros(64, 4).t()}),
                               (W.attn_shared_args, ATTN, {"seq_len": wide[:, 3]}),
                               (W.beam_select_args, SELECT, {"logits": torch.zeros(100, 4).t()})):
        call(**{**args, **{k: OnDevice(v.contiguous()) for k, v in change.items()}})
        with pytest.raises(W.WsgError, match="not contiguous") as e:
            call(**{**args, **{k: OnDevice(v) for k, v in change.items()}})
        assert e.value.status == 1


def test_argument_blocks_refuse_numbers_that_do_not_fit(W):
    """A size beyond its field would be taken by its low bits: 2^32 + 4 rows as 4."""
    for call, (args, good) in CALLS.items():
        block = getattr(W, args)
        for name, kind in block._kind.items():
            if kind not in (ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t):
                continue
            bits = 8 * ctypes.sizeof(kind)
            for value in (2**bits + 4, 2 ** (bits - 1 if kind is not ctypes.c_size_t else bits), -2**bits + 4):
                with pytest.raises(W.WsgError, match=f"{args}.{name}: .* outside") as e:
                    block(**{**good, name: value})
                assert e.value.status == 1
                a = block(**good)
                with pytest.raises(W.WsgError, match=f"{args}.{name}: .* outside"):
                    setattr(a, name, value)
                assert getattr(a, name) == good[name]


def test_oracle_rotation_layouts():
    """Both layouts turn each pair by its angle and leave lengths as they are; position 0 turns nothing."""
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((3, 16)), np.array([1.0, 0.3, 0.01])
    for inter in (0, 1):
        y = OB.rotate(x, 7, w, 6, inter)
        a, b = (slice(0, 6, 2), slice(1, 6, 2)) if inter else (slice(0, 3), slice(3, 6))
        z = (x[:, a] + 1j * x[:, b]) * np.exp(7j * w)
        np.testing.assert_allclose(y[:, a] + 1j * y[:, b], z)
        np.testing.assert_array_equal(y[:, 6:], x[:, 6:])
        np.testing.assert_array_equal(OB.rotate(x, 0, w, 6, inter), x)


def test_oracle_attention_joins_and_selects():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 8)), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    o, lse, _ = OB.attend(q, k, v, 0.5)
    parts = [OB.attend(q, k[s], v[s], 0.5) for s in (slice(0, 2), slice(2, 5))]
    wts = np.exp(np.array([p[1] for p in parts]) - lse)
    np.testing.assert_allclose(sum(w[:, None] * p[0] for w, p in zip(wts, parts)), o)
    sc, pa, to = OB.beam_select(np.zeros((2, 3)), np.array([0.0, 0.0]), 4)
    assert pa.tolist() == [0, 0, 0, 1] and to.tolist() == [0, 1, 2, 0]
    np.testing.assert_allclose(sc, -np.log(3.0))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    """csrc/beam_plan.h compiled as plain C++: every place that a CTA's threads load of a selection's lists, with the
    places that the workspace has. Returns how many are loaded; -1: one outside the workspace, -2: one past its list's
    count, -3: not each once, -4: another place handed on than loaded."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("walk")
    src = d / "w.cpp"
    src.write_text('#include "beam_plan.h"\n#include <vector>\nusing namespace wsg;\n'
                   'extern "C" long long layout(int beams, int vocab, int n_out, long long* o) {\n'
                   "  const BeamLayout L = beam_layout(beams, vocab, n_out);\n"
                   "  o[0] = L.chunk, o[1] = L.per_row, o[2] = L.chunks, o[3] = L.slots, o[4] = L.list;\n"
                   "  return (long long)L.total; }\n"
                   'extern "C" long long walk(int beams, int vocab, int n_out, const uint32_t* count) {\n'
                   "  const BeamLayout L = beam_layout(beams, vocab, n_out);\n"
                   "  const size_t places = (L.total - L.flat) / 4, listed = (size_t)L.slots * L.list;\n"
                   "  if (listed > places || L.key + 8 * listed > L.flat) return -1;\n"
                   "  std::vector<char> seen(listed);\n  long long n = 0, handed = 0, bad = 0;\n"
                   "  for (int t = 0; t < kBeamThreads; ++t)\n"
                   "    beam_walk(L.slots, L.list, t, [&](int q) { return count[q]; },\n"
                   "              [&](size_t p) -> uint32_t {\n"
                   "                if (p >= listed) { bad = -1; return 0; }\n"
                   "                if (p % L.list >= count[p / L.list]) bad = -2;\n"
                   "                if (seen[p]++) bad = -3;\n                ++n;\n                return p * 7 + 1; },\n"
                   "              [&](uint32_t k, size_t p) { if (k && k != (uint32_t)(p * 7 + 1)) bad = -4; handed += k != 0; });\n"
                   "  return bad ? bad : handed == n ? n : -4;\n}\n")
    lib = d / "w.so"
    inc = os.path.join(ROOT, "weight_streaming_gemv_token_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    L.layout.restype = L.walk.restype = ctypes.c_longlong
    return L


def test_selection_reads_no_place_behind_its_lists(walk):
    """Lists that are full and lists that are not, of lengths that no number of threads divides."""
    rng = np.random.default_rng(0)
    cases = [(64, 100, 64), (64, 75, 64), (1, 1, 1), (1000, 40, 1000), (4, 151936, 8), (1, 151936, 1024), (1024, 129, 1024),
             (3, 9000, 1000), (513, 33, 700)]
    cases += [(int(np.exp(rng.uniform(0, np.log(1024)))), int(np.exp(rng.uniform(0, np.log(9000)))),
               int(np.exp(rng.uniform(0, np.log(1024))))) for _ in range(60)]
    for beams, vocab, n_out in cases:
        o = (ctypes.c_longlong * 5)()
        walk.layout(beams, vocab, n_out, o)
        chunk, per_row, chunks, slots, width = o
        assert per_row * chunk >= vocab and chunks == beams * per_row <= 4096 and slots == min(n_out, chunks)
        assert width == min(chunk, vocab)
        for count in (np.full(slots, width), rng.integers(0, width + 1, slots), np.zeros(slots)):
            count = np.ascontiguousarray(count, dtype=np.uint32)
            assert walk.walk(beams, vocab, n_out, count.ctypes.data_as(ctypes.c_void_p)) == count.sum(), (beams, vocab, n_out)


def test_prefix_kernel_has_no_wait_without_a_limit():
    """Warps of the tensor-core prefix kernel that wait for some others, not for the whole CTA, do so on mbarriers, whose
    waits give up, or at a barrier that each of them comes to whatever it has given up: one behind a condition of its own
    would keep a warp for good whose partner has given up before it."""
    with open(os.path.join(ROOT, "weight_streaming_gemv_token_gb300", "csrc", "attn_prefix_tc.cuh")) as f:
        code = "\n".join(line.split("//")[0] for line in f)
    assert not re.search(r"barrier\.(cta\.)?(sync|red|arrive)|bar\.(red|arrive)|__barrier_sync|__syncthreads_", code)
    blocks, found = [], 0  # the openings of the blocks around each place
    for m in re.finditer(r"[{}]|\bbar\.sync", code):
        if m[0] == "{":
            blocks.append(code[max(code.rfind(c, 0, m.start()) for c in ";{}") + 1: m.start()].strip())
        elif m[0] == "}":
            blocks.pop()
        else:
            found += 1
            inner = [b for b in blocks if "namespace" not in b and "__global__" not in b]
            assert inner == ["else if (works)"], inner  # (the same for all warps that the barrier counts)
    assert found == 1 and not blocks
