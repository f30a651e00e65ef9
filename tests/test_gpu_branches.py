"""The operators for several branches of one prompt on the GPU against their float64 definitions.

Tolerances count roundings: u = 2^-24 is half a step of float32, 2^-8 of bfloat16 (relative to the value).
"""
import itertools

import numpy as np
import pytest

import oracle.branches as OB

from gpu_util import lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}


def tdt(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def code(W, name):
    return {"f32": W.DEC_F32, "bf16": W.DEC_BF16}[name]


def rand(shape, dtype, seed, scale=1.0):
    """Seeded device tensor of `dtype` (drawn on the host)."""
    import torch

    a = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * np.float32(scale)
    return torch.from_numpy(a).to("cuda").to(tdt(dtype))


def ints(a):
    import torch

    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


def inside(got, ref, tol, what):
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], ref[bad][:3], np.broadcast_to(tol, ref.shape)[bad][:3])


# ---- rotation, append ----------------------------------------------------------------------------------------------

# Float32 roundings between an input and an output of the rotation, relative to |a| + |b| of the pair: the sum of 128
# squares (8 in a chain, then 4 levels: 12) halves to 6 under the root, mean, eps, root and reciprocal add 3.5; two
# products with 1/rms and gain; the angle in half turns is off by 2^-25 (1.6 u in radians), sincospi by 2 ulp (4 u),
# the factor 1; product and fma 2. Together under 21.
ROPE_U = 24 * U


def rope_case(W, rows, n_q, n_kv, d, rot, inter, x, y, norm=True, far=0, pad=(), extra=0, offset=0, scaled=False, seed=0):
    """Inputs of a rotation call: row strides have `extra` elements more than the heads, data starts at `offset`."""
    import torch

    def rows_of(width, dtype, seed=None):
        n = rows * (width + extra) + offset
        t = rand((n,), dtype, seed, 1.5) if seed is not None else torch.full((n,), 7.0, dtype=tdt(dtype), device="cuda")
        return t, t[offset:].view(rows, width + extra)[:, :width]

    s = {"q": rows_of(n_q * d, x, seed + 1), "k": rows_of(n_kv * d, x, seed + 2), "q_out": rows_of(n_q * d, y),
         "k_out": rows_of(n_kv * d, y)}
    gq = 1.0 + rand((d,), "f32", seed + 3, 0.1) if norm else None
    gk = 1.0 + rand((d,), "f32", seed + 4, 0.1) if norm else None
    w, f = (W.rope_frequencies(rot, 1e6, W.ROPE_RAMP, 4.0, 32768) if scaled else W.rope_frequencies(rot, 1e6)) if rot else ([], 1.0)
    pos = far + np.arange(rows)
    pos[list(pad)] = -1
    wd = torch.tensor(w, dtype=torch.float64, device="cuda") if rot else None
    args = dict(rows=rows, n_q=n_q, n_kv=n_kv, head_dim=d, xdtype=code(W, x), ydtype=code(W, y), q=s["q"][1],
                k=s["k"][1], q_out=s["q_out"][1], q_stride=n_q * d + extra, k_stride=n_kv * d + extra,
                q_out_stride=n_q * d + extra, g_q=gq, g_k=gk, positions=ints(pos), inv_freq=wd, eps=1e-6,
                rope_factor=f, rot_dim=rot, interleaved=inter)
    return s, args, pos, (gq, gk, w, f)


def rope_ref(x, gain, eps, pos, w, rot, inter, f, y):
    """One row's heads and their tolerance."""
    r = OB.norm_rope(x, gain, eps, pos, w, rot, inter, f)
    n = OB.norm_rope(x, gain, eps, 0, w, 0, inter)  # normalised, not rotated
    size = np.abs(n).copy()
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    size[..., a] = size[..., b] = (np.abs(n[..., a]) + np.abs(n[..., b])) * max(1.0, f)
    return r, ROPE_U * size + HALF[y] * (np.abs(r) + ROPE_U * size) + 1e-37


def check_rope(W, s, pos, extra, rows, n_q, n_kv, d, rot, inter, y, norm, which=("q", "k")):
    gq, gk, w, f = extra
    for name, heads, g in (("q", n_q, gq), ("k", n_kv, gk)):
        if name not in which or heads == 0:
            continue
        x, got = f64(s[name][1]).reshape(rows, heads, d), f64(s[name + "_out"][1]).reshape(rows, heads, d)
        for r in range(rows):
            if pos[r] < 0:
                assert (got[r] == 7.0).all(), "a padded row was written"
                continue
            ref, tol = rope_ref(x[r], f64(g) if norm else None, 1e-6, pos[r], w, rot, inter, f, y)
            inside(got[r], ref, tol, (name, r))


ROPE_CASES = [
    # rows, n_q, n_kv, d, rot, interleaved, x, y, options
    (1, 16, 8, 128, 128, 0, "f32", "bf16", {}),
    (1, 1, 1, 8, 8, 0, "f32", "f32", {}),              # rot / 2 is half a lane's elements
    (3, 4, 2, 16, 16, 1, "bf16", "f32", {"far": 130000}),
    (7, 5, 0, 24, 20, 0, "f32", "f32", {"pad": (0, 6)}),   # no keys; pairs that straddle lanes; padded ends
    (7, 0, 3, 64, 32, 1, "bf16", "bf16", {"pad": (3,)}),   # no queries
    (33, 3, 1, 80, 40, 0, "bf16", "f32", {"scaled": True, "far": 2**31 - 40}),  # the last positions there are
    (33, 6, 2, 96, 96, 0, "f32", "bf16", {"extra": 8}),
    (5, 4, 4, 120, 22, 1, "f32", "f32", {"extra": 3, "offset": 1}),  # rows that start off 16 bytes
    (5, 2, 2, 128, 64, 0, "bf16", "bf16", {"extra": 1, "offset": 3}),
    (9, 4, 2, 64, 0, 0, "f32", "f32", {}),              # norm alone
    (9, 4, 2, 128, 128, 0, "f32", "f32", {"norm": False, "far": 1 << 20}),  # rotation alone
    (1500, 16, 8, 128, 128, 0, "f32", "bf16", {"pad": tuple(range(1490, 1500)), "scaled": True}),  # several heads a unit
    (1500, 9, 3, 128, 64, 1, "bf16", "f32", {"far": 131072}),
]


@pytest.mark.parametrize("c", ROPE_CASES, ids=str)
def test_qk_norm_rope(c):
    import torch

    W = lib()
    rows, n_q, n_kv, d, rot, inter, x, y, o = c
    norm = o.get("norm", True)
    s, a, pos, extra = rope_case(W, rows, n_q, n_kv, d, rot, inter, x, y, **o)
    W.qk_norm_rope(W.qk_rope_args(k_out=s["k_out"][1], k_out_stride=n_kv * d + o.get("extra", 0), **a))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    check_rope(W, s, pos, extra, rows, n_q, n_kv, d, rot, inter, y, norm)
    for name, width in (("q_out", n_q * d), ("k_out", n_kv * d)):  # nothing between the rows
        whole = f64(s[name][0])
        gap = whole[o.get("offset", 0):].reshape(rows, -1)[:, width:]
        assert (gap == 7.0).all() and (whole[: o.get("offset", 0)] == 7.0).all()


def test_qk_norm_rope_in_place():
    import torch

    W = lib()
    s, a, pos, extra = rope_case(W, 37, 4, 2, 128, 128, 0, "bf16", "bf16", seed=5)
    W.qk_norm_rope(W.qk_rope_args(k_out=s["k_out"][1], k_out_stride=2 * 128, **a))
    a.update(q_out=s["q"][1])
    W.qk_norm_rope(W.qk_rope_args(k_out=s["k"][1], k_out_stride=2 * 128, **a))
    torch.cuda.synchronize()
    assert torch.equal(s["q"][1], s["q_out"][1]) and torch.equal(s["k"][1], s["k_out"][1])


def test_qk_norm_rope_special_values():
    """A zero row stays zero; infinities and NaN outside the rotated part stay where they are without a norm."""
    import torch

    W = lib()
    s, a, pos, extra = rope_case(W, 2, 2, 1, 32, 16, 0, "f32", "f32", norm=False)
    s["q"][1].zero_()
    s["q"][1][0, 20], s["q"][1][0, 21], s["q"][1][1, 40] = float("inf"), float("nan"), float("-inf")
    W.qk_norm_rope(W.qk_rope_args(k_out=s["k_out"][1], k_out_stride=32, **a))
    torch.cuda.synchronize()
    want = f64(s["q"][1])
    want[1, 32 + 0], want[1, 32 + 8] = 0, 0
    got = f64(s["q_out"][1])
    # the -inf sits in a rotated pair (element 8 of head 1): only that pair is not finite
    assert not np.isfinite(got[1, [32, 40]]).all()
    got[1, [32, 40]] = 0
    want[1, [32, 40]] = 0
    np.testing.assert_array_equal(got, want)


def page_case(rng, n_seq, lengths, page, width=None, spare=0):
    """A shuffled page table for sequences of the given lengths; -1 where a sequence has no page."""
    need = [-(-max(0, n) // page) for n in lengths]
    width = max(need + [1]) if width is None else width
    total = sum(need) + spare
    ids = rng.permutation(total)
    table, at = np.full((n_seq, width), -1, dtype=np.int32), 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at: at + k]
        at += k
    return table, total, ids[at:]


APPEND_CASES = [
    # rows per sequence (0: none), first index of each, n_q, n_kv, d, x, y, kv, page, base
    ([1], [0], 4, 2, 16, "f32", "bf16", "f32", 1, 0),
    ([1] * 16, [15, 16, 17, 0, 31, 32, 33, 63] * 2, 16, 8, 128, "f32", "bf16", "bf16", 16, 4096),
    ([7, 0, 1, 30], [5, 0, 8, 1], 3, 1, 24, "bf16", "f32", "f32", 8, 100),
    ([64, 65, 63], [0, 0, 0], 0, 2, 64, "bf16", "bf16", "bf16", 64, 0),  # no queries
    ([300, 1, 411], [100, 0, 7], 4, 4, 128, "f32", "f32", "bf16", 128, 32768),
]


@pytest.mark.parametrize("c", APPEND_CASES, ids=str)
@pytest.mark.parametrize("pads", [0, 3])
def test_kv_append_paged(c, pads):
    import torch

    W = lib()
    held, first, n_q, n_kv, d, x, y, kv, page, base = c
    rng = np.random.default_rng(3)
    rows = sum(held) + pads
    table, pages, _ = page_case(rng, len(held), [f + h for f, h in zip(first, held)], page, spare=1)
    seq = np.concatenate([np.repeat(np.arange(len(held)), held), np.full(pads, 99)])  # never looked at behind padding
    pos = np.concatenate([base + f + np.arange(h) for f, h in zip(first, held)] + [np.full(pads, -5)]).astype(int)
    s, a, _, extra = rope_case(W, rows, n_q, n_kv, d, d, 0, x, y, seed=9)
    a["positions"] = ints(pos)
    v = rand((rows, n_kv * d), x, 77)
    kp = rand((pages, n_kv, page, d), kv, 78)
    vp = rand((pages, n_kv, page, d), kv, 79)
    k0, v0 = f64(kp), f64(vp)
    W.kv_append_paged(W.kv_append_args(
        v=v, v_stride=n_kv * d, kvdtype=code(W, kv), k_pages=kp, v_pages=vp, page_table=ints(table), seq=ints(seq),
        n_seq=len(held), num_pages=pages, page_size=page, table_stride=table.shape[1], base_pos=base, **a))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    check_rope(W, s, pos, extra, rows, n_q, n_kv, d, d, 0, y, True, which=("q",))
    gk, vv, ktol = f64(a["g_k"]), f64(v).reshape(rows, n_kv, d), np.zeros_like(k0)
    for r in range(rows):
        if pos[r] < 0:
            continue
        p, slot = divmod(pos[r] - base, page)
        ref, tol = rope_ref(f64(s["k"][1]).reshape(rows, n_kv, d)[r], gk, 1e-6, pos[r], extra[2], d, 0, 1.0, kv)
        k0[table[seq[r], p], :, slot], ktol[table[seq[r], p], :, slot] = ref, tol
        v0[table[seq[r], p], :, slot] = f64(torch.tensor(vv[r]).to(tdt(kv)))
    inside(f64(kp), k0, ktol, "key pages (untouched rows exactly)")
    np.testing.assert_array_equal(f64(vp), v0)


def test_kv_append_paged_bad_pages():
    """Rows whose sequence, index or page is out of range are not stored; the others and every query are."""
    import torch

    W = lib()
    n_q, n_kv, d, page, pages = 2, 1, 16, 4, 4
    table = ints([[0, 1], [4, 2], [-1, 3], [2**31 - 1, -2**31]])
    seq = np.array([0, 1, 2, 3, 3, 4, -1, 0, 0, 2], dtype=np.int32)
    idx = np.array([1, 0, 3, 0, 4, 0, 0, 8, -2, 4])  # only rows 0 and 9 have a page
    base = 10
    s, a, _, extra = rope_case(W, 10, n_q, n_kv, d, d, 1, "f32", "f32", seed=4)
    a["positions"] = ints(idx + base)
    v = rand((10, d), "f32", 5)
    kp, vp = (torch.full((pages, n_kv, page, d), 3.0, device="cuda") for _ in range(2))
    W.gemv_device_errors()
    W.kv_append_paged(W.kv_append_args(v=v, v_stride=d, kvdtype=W.DEC_F32, k_pages=kp, v_pages=vp, page_table=table,
                                       seq=ints(seq), n_seq=4, num_pages=pages, page_size=page, table_stride=2,
                                       base_pos=base, **a))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0x80
    check_rope(W, s, idx + base, extra, 10, n_q, n_kv, d, d, 1, "f32", True, which=("q",))
    want = torch.full_like(vp, 3.0)
    want[0, 0, 1], want[3, 0, 0] = v[0], v[9]
    assert torch.equal(vp, want)
    changed = (kp != 3.0).any(-1)
    assert changed.sum() == 2 and changed[0, 0, 1] and changed[3, 0, 0]


# ---- attention -----------------------------------------------------------------------------------------------------

def attn_case(W, batch, n_q, n_kv, d, plen, lens, page, q, kv, stride=None, seed=0, poison=True, lse=True, extra=0,
              width=None, scale=None):
    """A call's arguments; `poison` puts NaN and infinities in every cache row that no branch may use."""
    import torch

    rng = np.random.default_rng(seed)
    stride = plen if stride is None else stride
    table, pages, _ = page_case(rng, batch, lens, page, width, spare=1)
    pk, pv = rand((n_kv, stride, d), kv, seed + 1), rand((n_kv, stride, d), kv, seed + 2)
    kp, vp = rand((pages, n_kv, page, d), kv, seed + 3), rand((pages, n_kv, page, d), kv, seed + 4)
    if poison:
        used = np.zeros((pages, page), dtype=bool)
        for b, n in enumerate(lens):
            for i in range(max(0, n)):
                used[table[b, i // page], i % page] = True
        u = torch.tensor(used, device="cuda")[:, None, :, None]
        for k, (t, pre) in enumerate(((kp, pk), (vp, pv))):
            t.masked_fill_(~u, float("nan") if k else float("inf"))
            pre[:, plen:] = float("nan")
    qq = rand((batch, n_q * d + extra), q, seed + 5, 1.2)
    out = torch.full((batch, n_q * d + extra), 7.0, dtype=tdt(q), device="cuda")
    ls = torch.full((batch, n_q), 7.0, device="cuda") if lse else None
    a = W.attn_shared_args(
        batch=batch, n_q=n_q, n_kv=n_kv, head_dim=d, qdtype=code(W, q), kvdtype=code(W, kv), q=qq, out=out, lse=ls,
        q_stride=n_q * d + extra, out_stride=n_q * d + extra, prefix_k=pk, prefix_v=pv, prefix_len=plen,
        prefix_stride=stride, k_pages=kp, v_pages=vp, page_table=ints(table), seq_len=ints(lens), num_pages=pages,
        page_size=page, table_stride=table.shape[1], scale=d ** -0.5 if scale is None else scale)
    a.with_workspace(torch.full((W.attn_shared_prefix_workspace(a),), 255, dtype=torch.uint8, device="cuda"))
    return a, dict(q=qq, out=out, lse=ls, pk=pk, pv=pv, kp=kp, vp=vp, table=table)


def attn_tol(q, k, lse, o, size, scale, dtype):
    """Tolerances of outputs and lse. A score q.k (d products, float32 accumulation, at most one step per term) is off by
    at most 2 (d + 4) u scale sum |q k|; a probability relatively by that twice (its own score and the maximum's), 8 u for
    the exponential, its argument and the rescaling, and 2^-16 where it enters a product as a bfloat16 pair; the sums over
    n keys by 2 n u of size = sum p |v|; the output's rounding follows."""
    n, d = k.shape
    ds = 2 * (d + 4) * U * scale * np.max(np.abs(q) @ np.abs(k).T, axis=1)[:, None] + 2 * U * np.abs(lse)[:, None]
    rel = 2 * ds + 8 * U + 2.0 ** -16 * (dtype == "bf16") + 2 * n * U
    return rel * size + HALF[dtype] * (np.abs(o) + rel * size) + 1e-30, 2 * ds[:, 0] + (8 + 2 * n) * U + 2 * U * np.abs(lse)


def check_attn(t, batch, n_q, n_kv, d, plen, lens, page, q, scale=None, skip=()):
    """Every branch against the definition (skip: table entries that are left out); unused slots unchanged."""
    group = n_q // n_kv
    scale = np.float64(np.float32(d ** -0.5 if scale is None else scale))
    Q, got = f64(t["q"])[:, : n_q * d].reshape(batch, n_kv, group, d), f64(t["out"])[:, : n_q * d].reshape(batch, n_kv, group, d)
    lse = f64(t["lse"]).reshape(batch, n_kv, group) if t["lse"] is not None else None
    PK, PV, KP, VP = f64(t["pk"])[:, :plen], f64(t["pv"])[:, :plen], f64(t["kp"]), f64(t["vp"])
    for b, n in enumerate(lens):
        if n < 0:
            assert (got[b] == 7.0).all() and (lse is None or (lse[b] == 7.0).all()), "an unused slot was written"
            continue
        i = np.array([x for x in range(n) if (b, x // page) not in skip], dtype=int)
        pg, sl = t["table"][b, i // page], i % page
        for g in range(n_kv):
            k = np.concatenate([PK[g], KP[pg, g, sl]])
            v = np.concatenate([PV[g], VP[pg, g, sl]])
            o, l, size = OB.attend(Q[b, g], k, v, scale)
            if len(k) == 0:
                assert (got[b, g] == 0).all() and (lse is None or np.isneginf(lse[b, g]).all())
                continue
            tol, ltol = attn_tol(Q[b, g], k, l, o, size, scale, q)
            inside(got[b, g], o, tol, (b, g))
            if lse is not None:
                inside(lse[b, g], l, ltol, ("lse", b, g))


ATTN_CASES = [
    # batch, n_q, n_kv, d, prefix, lens, page
    (1, 1, 1, 8, 0, [1], 1),
    (1, 4, 2, 16, 1, [0], 16),
    (2, 4, 2, 16, 0, [0, 3], 4),                     # a branch with nothing at all
    (3, 6, 2, 24, 5, [1, -1, 17], 8),                # an unused slot; group of 3
    (5, 16, 1, 64, 63, [64, 1, 65, 0, 128], 64),     # group of 16
    (4, 16, 8, 128, 64, [15, 16, 17, 33], 16),
    (4, 16, 8, 128, 127, [1, 2, 3, 4], 1),
    (7, 10, 2, 80, 129, [40, 31, 32, 33, 0, 63, 64], 32),
    (8, 16, 8, 128, 257, [5] * 8, 8),
    (9, 8, 8, 128, 511, [100, 3, -1, 7, 0, 1, 250, 64, 9], 128),   # group of 1
    (17, 8, 2, 96, 640, [i * 3 for i in range(17)], 16),
    (33, 16, 8, 128, 1000, [i for i in range(33)], 16),            # 66 rows a key/value head
    (64, 16, 8, 128, 1025, [(i * 7) % 90 for i in range(64)], 32),  # 128 rows
    (70, 8, 2, 128, 385, [3] * 70, 16),                            # 280 rows
    (3, 4, 2, 128, 5000, [700, 20, 1], 64),                        # long for few rows
    (3, 8, 2, 128, 0, [5, 0, 70], 16),                             # no prefix
    (2, 4, 2, 128, 0, [1500, 3], 32),                              # ... and long own keys
    (5, 16, 1, 128, 300, [40, 0, -1, 1, 100], 16),                 # group of 16
    (2, 16, 1, 128, 100, [900, 10], 8),                            # ... long, pages shorter than a block
    (4, 12, 4, 128, 2000, [33, 7, 64, 0], 4),                      # group of 3
    (2, 8, 2, 64, 3000, [1200, 1], 16),                            # both axes cut, a shorter head
    (40, 32, 8, 128, 1500, [64 - i for i in range(40)], 64),       # 160 rows: two blocks of rows
]
TYPES = [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")]


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("c", ATTN_CASES, ids=lambda c: f"b{c[0]}_q{c[1]}_kv{c[2]}_d{c[3]}_p{c[4]}_page{c[6]}")
def test_attn_shared_prefix(c, types):
    import torch

    W = lib()
    batch, n_q, n_kv, d, plen, lens, page = c
    a, t = attn_case(W, batch, n_q, n_kv, d, plen, lens, page, *types, stride=plen + 37)
    W.gemv_device_errors()
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    check_attn(t, batch, n_q, n_kv, d, plen, lens, page, types[0])
    first = t["out"].clone()
    W.attn_shared_prefix(a)  # the same bits again, on a used workspace
    torch.cuda.synchronize()
    assert torch.equal(first, t["out"])


@pytest.mark.parametrize("types", TYPES, ids=str)
def test_attn_shared_prefix_without_branches(types):
    """A step in which every branch has ended: a workspace can be asked for, the call does nothing."""
    import torch

    W = lib()
    for d, plen, width in ((128, 512, 4), (128, 0, 4), (64, 512, 0), (64, 0, 4)):
        a, t = attn_case(W, 1, 4, 2, d, plen, [min(1, width)], 16, *types, width=width)
        a.batch = 0
        a.with_workspace(torch.empty(W.attn_shared_prefix_workspace(a), dtype=torch.uint8, device="cuda"))
        W.attn_shared_prefix(a)
        torch.cuda.synchronize()
        assert (t["out"] == 7.0).all() and W.gemv_device_errors() == 0


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32")], ids=str)
def test_attn_shared_prefix_strides_and_no_lse(types):
    import torch

    W = lib()
    lens = [3, 40, 0, -1, 19]
    a, t = attn_case(W, 5, 4, 2, 128, 70, lens, 16, *types, extra=5, lse=False, scale=0.3, width=9)
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    check_attn(t, 5, 4, 2, 128, 70, lens, 16, types[0], scale=0.3)
    assert (f64(t["out"])[:, 4 * 128:] == 7.0).all()


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_attn_shared_prefix_large_scores(kv):
    """Scores of hundreds, of both signs, in rising and falling order: the running maximum moves often and far."""
    import torch

    W = lib()
    lens = [130, 1]
    a, t = attn_case(W, 2, 4, 2, 128, 700, lens, 64, "f32", kv, seed=2)
    ramp = torch.linspace(0, 30, 700, device="cuda")
    t["pk"][0] *= ramp[:, None].to(t["pk"].dtype)
    t["pk"][1] *= ramp.flip(0)[:, None].to(t["pk"].dtype)
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    check_attn(t, 2, 4, 2, 128, 700, lens, 64, "f32")


@pytest.mark.parametrize("types,batch", [(("bf16", "bf16"), 2), (("bf16", "bf16"), 20), (("f32", "f32"), 2)], ids=str)
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_attn_shared_prefix_negative_scale(types, batch, scale):
    import torch

    W = lib()
    lens = [33] * batch
    a, t = attn_case(W, batch, 4, 2, 128, 200, lens, 16, *types, scale=scale)
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    group, k = 2, None
    Q, got = f64(t["q"]).reshape(batch, 2, group, 128), f64(t["out"]).reshape(batch, 2, group, 128)
    for b in range(batch):
        for g in range(2):
            i = np.arange(33)
            at = t["table"][b, i // 16], g, i % 16
            k = np.concatenate([f64(t["pk"])[g], f64(t["kp"])[at]])
            v = np.concatenate([f64(t["pv"])[g], f64(t["vp"])[at]])
            o, l, size = OB.attend(Q[b, g], k, v, float(np.float32(scale)))
            inside(got[b, g], o, attn_tol(Q[b, g], k, l, o, size, abs(scale), types[0])[0], (b, g))


@pytest.mark.parametrize("types,d", [(("bf16", "bf16"), 128), (("bf16", "bf16"), 64), (("f32", "f32"), 128)], ids=str)
@pytest.mark.parametrize("width", [8, 80])
def test_attn_shared_prefix_in_place(types, d, width):
    """The output over the queries, unused slots left as they are: the bits of a call with buffers of its own."""
    import torch

    W = lib()
    batch, n_q, n_kv = 33, 8, 4
    lens = [(5 * i) % 97 - 1 for i in range(batch)]
    a, t = attn_case(W, batch, n_q, n_kv, d, 700, lens, 16, *types, width=width)
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    want = torch.where((ints(lens) < 0)[:, None], t["q"], t["out"])
    for _ in range(5):
        q = t["q"].clone()
        a.set("q", q).set("out", q)
        W.attn_shared_prefix(a)
        torch.cuda.synchronize()
        assert torch.equal(q, want)


def test_attn_shared_prefix_bad_pages():
    """Entries outside the pool are left out and reported; so are tokens past the table's width."""
    import torch

    W = lib()
    lens, page = [40, 40, 40, 64], 16
    a, t = attn_case(W, 4, 4, 2, 128, 30, lens, page, "bf16", "bf16", poison=False)
    bad = t["table"].copy()
    bad[0, 1], bad[1, 0], bad[2, 2] = -1, a.num_pages, 2**31 - 1
    a.set("page_table", ints(bad)).set("seq_len", ints([40, 40, 40, 65]))
    W.gemv_device_errors()
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0x80
    check_attn(t, 4, 4, 2, 128, 30, lens, page, "bf16", skip={(0, 1), (1, 0), (2, 2)})


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("plen,width,lens,bad", [
    (30, 0, [1, 0, -1], True), (0, 0, [3, 0, -1], True), (30, 0, [0, -1, 0], False), (30, 2, [33, 32, -1], True),
    (30, 2, [32, 5, -1], False), (30, 70, [70 * 16 + 1, 9, -1], True), (300, 70, [70 * 16, 9, 2**31 - 1], True)])
def test_attn_shared_prefix_reports_tokens_without_a_page(types, d, plen, width, lens, bad):
    """Tokens past the table's width are reported by every form of the call, with a table of no pages too; they are left
    out and the others attended to."""
    import torch

    W = lib()
    held = [min(n, 16 * width) for n in lens]
    a, t = attn_case(W, 3, 4, 2, d, plen, held, 16, *types, width=width)
    a.set("seq_len", ints(lens))
    W.gemv_device_errors()
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == (0x80 if bad else 0)
    check_attn(t, 3, 4, 2, d, plen, held, 16, types[0])


def test_attn_shared_prefix_reads_a_decoders_cache():
    """The prefix may be a decoder's own cache: one branch without tokens of its own, whose query repeats over the
    prefix, agrees with the definition on that cache."""
    import torch

    import workloads as Wl
    from weight_streaming_gemv_token_gb300.decoder import Decoder

    W = lib()
    s = Wl.TINY
    dec = Decoder(s, Wl.decoder_weights(s, seed=1), kv_dtype="bf16", max_seq=40)
    dec.prefill([int(x) for x in Wl.prompt_uniform(21, s.vocab, seed=0)], is_last=True)
    K, V, n = dec.kv(1)
    lens = [0, 5]
    a, t = attn_case(W, 2, s.n_q, s.n_kv, s.head_dim, n, lens, 8, "f32", "bf16")
    a.set("prefix_k", K).set("prefix_v", V)
    a.prefix_stride = K.shape[1]
    t["pk"], t["pv"] = K, V
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    check_attn(t, 2, s.n_q, s.n_kv, s.head_dim, n, lens, 8, "f32")
    dec.close()


def test_attn_shared_prefix_pools_past_32_bits():
    """Pages whose first element lies past 2^31 elements and 2^32 bytes."""
    import torch

    W = lib()
    n_kv, d, page, pages = 8, 128, 64, 33000  # 2.16e9 elements a pool
    a, t = attn_case(W, 2, 16, n_kv, d, 10, [70, 64], page, "bf16", "bf16")
    far = torch.zeros((2, pages, n_kv, page, d), dtype=torch.bfloat16, device="cuda")
    ids = np.array([pages - 1, pages - 2, pages - 3])
    for k, name in enumerate(("kp", "vp")):
        far[k, ids] = t[name][t["table"][t["table"] >= 0]]
    table = np.array([[pages - 1, pages - 2], [pages - 3, -1]], dtype=np.int32)
    small = t["out"].clone()
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    small = t["out"].clone()
    a.set("k_pages", far[0]).set("v_pages", far[1]).set("page_table", ints(table))
    a.num_pages = pages
    t["out"].fill_(7.0)
    W.attn_shared_prefix(a)
    torch.cuda.synchronize()
    assert torch.equal(small, t["out"])
    # and an append there
    s, b, _, extra = rope_case(W, 1, 16, n_kv, d, d, 0, "f32", "bf16", far=9)
    v = rand((1, n_kv * d), "f32", 5)
    W.kv_append_paged(W.kv_append_args(v=v, v_stride=n_kv * d, kvdtype=W.DEC_BF16, k_pages=far[0], v_pages=far[1],
                                       page_table=ints(table), seq=None, n_seq=2, num_pages=pages, page_size=page,
                                       table_stride=2, base_pos=9, **b))
    torch.cuda.synchronize()
    assert torch.equal(far[1, pages - 1, :, 0], v.view(n_kv, d).bfloat16())


# ---- selection -----------------------------------------------------------------------------------------------------

def run_select(W, logits, scores, n_out, stride=None, offset=0):
    import torch

    beams, vocab = logits.shape
    stride = stride or vocab
    buf = torch.full((offset + beams * stride,), float("inf"), device="cuda")  # what lies between rows is not read
    buf[offset:].view(beams, stride)[:, :vocab] = torch.tensor(logits, device="cuda")
    x = buf[offset:]
    sc = torch.tensor(np.asarray(scores, dtype=np.float32), device="cuda")
    outs = [torch.full((n_out,), 7, dtype=dt, device="cuda") for dt in (torch.float32, torch.int32, torch.int32)]
    a = W.beam_select_args(beams=beams, vocab=vocab, n_out=n_out, logits=x, logits_stride=stride, scores=sc,
                           out_scores=outs[0], out_parents=outs[1], out_tokens=outs[2])
    a.with_workspace(torch.full((W.beam_select_workspace(a),), 255, dtype=torch.uint8, device="cuda"))
    W.beam_select(a)
    W.beam_select(a)  # a used workspace
    torch.cuda.synchronize()
    return [o.cpu().numpy() for o in outs]


def check_select(got, logits, scores, n_out):
    """Scores: the sum of exponentials is float32 (each term 3 u with its argument, at most 64 in a chain, then joins:
    under 96 u relative, so absolute in the logarithm); one rounding of the score."""
    s, p, t = OB.beam_select(np.asarray(logits, dtype=np.float32), np.asarray(scores, dtype=np.float32), n_out)
    np.testing.assert_array_equal(got[1], p)
    np.testing.assert_array_equal(got[2], t)
    some = p >= 0
    assert np.isneginf(got[0][~some]).all()
    inside(got[0][some].astype(np.float64), s[some], 96 * U + U * np.abs(s[some]), "scores")


@pytest.mark.parametrize("c", [(1, 1, 1), (1, 2, 5), (2, 7, 14), (3, 512, 6), (1, 1024, 1024), (5, 1025, 10),
                               (4, 151936, 8), (31, 50257, 62), (64, 151936, 128), (1, 151936, 2), (1000, 40, 1000),
                               (2, 32001, 1000)], ids=str)
def test_beam_select(c):
    W = lib()
    beams, vocab, n_out = c
    rng = np.random.default_rng(beams + vocab)
    logits = (rng.standard_normal((beams, vocab)) * 2.5).astype(np.float32)
    scores = (rng.standard_normal(beams) - 12).astype(np.float32)
    check_select(run_select(W, logits, scores, n_out), logits, scores, n_out)


@pytest.mark.parametrize("c", [(64, 100, 64), (64, 75, 64), (64, 100, 200), (47, 129, 33), (3, 9017, 1000)], ids=str)
@pytest.mark.parametrize("kind", ["normal", "levels", "equal"])
def test_beam_select_lists_of_odd_lengths(c, kind):
    """Over 4,096 listed candidates in lists whose lengths no number of threads divides, masked logits among them."""
    W = lib()
    beams, vocab, n_out = c
    rng = np.random.default_rng(vocab)
    x = {"normal": lambda: rng.standard_normal((beams, vocab)), "levels": lambda: rng.integers(0, 2, (beams, vocab)),
         "equal": lambda: np.zeros((beams, vocab))}[kind]().astype(np.float32)
    if kind != "equal":
        x[rng.random((beams, vocab)) < 0.05] = -np.inf
    if kind == "levels":
        x[:] = x[0]  # (equal rows: their float32 sums tie as the definition's do)
    check_select(run_select(W, x, [-1.0] * beams, n_out), x, [-1.0] * beams, n_out)


@pytest.mark.parametrize("beams,n_out", [(8, 8), (3, 200), (200, 3)])
def test_beam_select_scores_in_place(beams, n_out):
    """New scores over the old ones, as a search keeps them."""
    import torch

    W = lib()
    logits, scores = rand((beams, 30000), "f32", 1, 2.0), rand((max(beams, n_out),), "f32", 2)
    want = run_select(W, logits.cpu().numpy(), scores[:beams].cpu().numpy(), n_out)
    parents, tokens = ints(np.zeros(n_out)), ints(np.zeros(n_out))
    for _ in range(5):
        sc = scores.clone()
        a = W.beam_select_args(beams=beams, vocab=30000, n_out=n_out, logits=logits, logits_stride=30000, scores=sc,
                               out_scores=sc, out_parents=parents, out_tokens=tokens)
        a.with_workspace(torch.empty(W.beam_select_workspace(a), dtype=torch.uint8, device="cuda"))
        W.beam_select(a)
        torch.cuda.synchronize()
        for got, w in zip((sc[:n_out], parents, tokens), want):
            np.testing.assert_array_equal(got.cpu().numpy(), w)
        assert torch.equal(sc[n_out:], scores[n_out:])


def test_beam_select_strided_rows():
    W = lib()
    rng = np.random.default_rng(1)
    logits = rng.standard_normal((3, 5001)).astype(np.float32)
    check_select(run_select(W, logits, [0, -1, -2], 9, stride=5007, offset=1), logits, [0, -1, -2], 9)


@pytest.mark.parametrize("n_out", [1, 3, 200, 1000])
def test_beam_select_ties(n_out):
    """All logits equal, and equal beams: the lowest flat indexes in order, through every narrowing step."""
    W = lib()
    logits = np.zeros((3, 9000), dtype=np.float32)
    got = run_select(W, logits, [-1.0, -1.0, -1.0], n_out)
    assert got[1].tolist() == [0] * n_out and got[2].tolist() == list(range(n_out))
    logits[1, 8000:8003] = 1.0  # three ahead of the tie (of row 1, whose others fall behind)
    check_select(run_select(W, logits, [-1.0, -1.0, -1.0], n_out), logits, [-1.0] * 3, n_out)


def test_beam_select_few_levels():
    """Logits of a few values only: ties across chunks and beams at every rank."""
    W = lib()
    rng = np.random.default_rng(5)
    logits = rng.integers(0, 3, (2, 12345)).astype(np.float32)
    logits[1] = logits[0, ::-1]
    check_select(run_select(W, logits, [-2.0, -2.0], 777), logits, [-2.0, -2.0], 777)


def test_beam_select_masks():
    W = lib()
    rng = np.random.default_rng(7)
    x = rng.standard_normal((6, 3000)).astype(np.float32)
    x[0, 5:] = -np.inf                     # five tokens left
    x[1] = -np.inf                         # nothing left
    x[2, ::2] = np.nan                     # masked by NaN
    x[3, 17] = np.inf                      # no distribution
    x[4, 1:] = np.finfo(np.float32).min    # the type's lowest value: finite, chosen last
    scores = [0.0, 0.0, -1.0, 0.0, -3.0, -np.inf]
    for n in (1, 4, 40, 1000):
        got = run_select(W, x, scores, n)
        check_select(got, np.where(np.isposinf(x).any(1, keepdims=True), -np.inf, x), scores, n)
    # fewer candidates than asked for
    got = run_select(W, x[:2], scores[:2], 9)
    assert got[1].tolist() == [0] * 5 + [-1] * 4 and got[2].tolist()[5:] == [-1] * 4
    got = run_select(W, x[1:2], [0.0], 3)
    assert got[1].tolist() == [-1] * 3 and np.isneginf(got[0]).all()
    got = run_select(W, x[:1], [np.nan], 3)
    assert got[1].tolist() == [-1] * 3


@pytest.mark.parametrize("beams", [2, 4, 40])
@pytest.mark.parametrize("shift", [0.0, 1000.0, -30000.0])
def test_beam_select_sure_beams(beams, shift):
    """Beams that are sure of their next token, in equal pairs, so that the best keys are near 0 and the bar is exactly one
    of them while logits and log-sums are large: what reaches the bar by less than the log-sum's last place is listed."""
    W = lib()
    rng = np.random.default_rng(beams)
    for n_out in (1, 3, beams - 1):
        logits = (rng.standard_normal((beams, 3000)) * 0.5).astype(np.float32)
        logits[np.arange(beams), rng.integers(0, 3000, beams)] = rng.uniform(9, 30, beams)
        logits = (logits + shift).astype(np.float32)
        logits[1::2] = logits[::2]
        scores = -np.floor(np.arange(beams) / 2).astype(np.float32)
        check_select(run_select(W, logits, scores, n_out), logits, scores, n_out)


def test_beam_select_lowest_scores():
    """Beams at the type's lowest score, whose lowest logits overflow the sum: such a candidate counts as the lowest finite
    score and comes behind every other."""
    W = lib()
    rng = np.random.default_rng(3)
    low = np.finfo(np.float32).min
    x = rng.standard_normal((3, 2500)).astype(np.float32)
    x[:, 40:] = low
    got = run_select(W, x, [low, -1.0, low], 50)
    s, p, t = OB.beam_select(x[1:2], np.array([-1.0], dtype=np.float32), 40)
    assert got[1][:40].tolist() == [1] * 40 and got[2][:40].tolist() == t.tolist()
    inside(got[0][:40].astype(np.float64), s, 96 * U + U * np.abs(s), "scores")
    assert (got[0][40:] == low).all()
    got = run_select(W, x, [low, -1.0, low], 1000)
    assert np.isfinite(got[0]).all() and (got[1] >= 0).all() and len(set(zip(got[1].tolist(), got[2].tolist()))) == 1000
    x = np.full((1, 2000), low, dtype=np.float32)
    x[0, 700] = 0.0
    got = run_select(W, x, [low], 3)
    assert got[2].tolist() == [700, 0, 1] and (got[0] == low).all()
    # rows of nothing but the lowest value are even distributions, whatever its size
    x = np.full((3, 5), low, dtype=np.float32)
    x[2, 3] = 0.0
    check_select(run_select(W, x, [-2.0, -1.5, -4.0], 11), x, [-2.0, -1.5, -4.0], 11)
    # score and log-sum together beyond float32, on either side: nothing to offer
    got = run_select(W, np.array([[1e38, 3e38], [low, low], [0.0, 1.0]], dtype=np.float32), [low, -low, -5.0], 6)
    assert got[1].tolist() == [2, 2, -1, -1, -1, -1] and got[2].tolist() == [1, 0, -1, -1, -1, -1]


@pytest.mark.parametrize("score", [0.0, -3.0, -1e6, -1e9])
def test_beam_select_masked_rows_of_beams_far_behind(score):
    """Rows of nothing but the type's lowest value are even distributions over what is not masked: their log-sums decide,
    and equal ones tie, whatever the beams' common score and the logits' level take up of the sum. (All rows' sums of
    exponentials are exact or apart: keys differ by 0.2 or tie.)"""
    W = lib()
    low, top = np.finfo(np.float32).min, np.finfo(np.float32).max
    x = np.full((8, 5), low, dtype=np.float32)
    x[1, 2:] = -np.inf
    x[2, 1:] = -np.inf
    x[3] = [0.0, 1.0, 2.0, -3.0, low]
    x[4, :2] = -np.inf
    x[5], x[6], x[7] = -7.0, top, 12345.67
    for n_out in (1, 4, 9, 17, 40):
        check_select(run_select(W, x, [score] * 8, n_out), x, [score] * 8, n_out)


# ---- reorder -------------------------------------------------------------------------------------------------------

REORDER_CASES = [
    # beams, layers, n_kv, d, page, kv, lengths
    (1, 1, 1, 8, 1, "bf16", [0]),
    (3, 2, 2, 16, 16, "f32", [16, 32, 31]),
    (4, 3, 2, 24, 8, "bf16", [7, -1, 9, 30]),
    (8, 28, 8, 128, 32, "bf16", [33, 64, 95, 1, 0, 31, 40, 41]),
    (64, 2, 8, 128, 16, "f32", [(i * 5) % 47 for i in range(64)]),
]


@pytest.mark.parametrize("c", REORDER_CASES, ids=lambda c: f"b{c[0]}_l{c[1]}_kv{c[2]}_d{c[3]}_page{c[4]}")
def test_beam_reorder_pages(c):
    import torch

    W = lib()
    beams, layers, n_kv, d, page, kv, lens = c
    rng = np.random.default_rng(beams)
    width = max(lens) // page + 2
    table, pages, spare = page_case(rng, beams, [n + (n >= 0) for n in lens], page, width, spare=beams)
    parents = rng.integers(0, beams, beams)
    parents[-1] = parents[0]  # one parent twice
    if beams > 2:
        parents[1] = -1
    pools = [rand((layers, pages, n_kv, page, d), kv, seed) for seed in (1, 2)]
    want, wt, wl = OB.beam_reorder([p.cpu().float().numpy() for p in pools], table, np.array(lens), parents, spare, page)
    nt, nl = ints(np.full((beams, width), 55)), ints(np.full(beams, 55))
    W.gemv_device_errors()
    W.beam_reorder_pages(W.beam_reorder_args(
        beams=beams, layers=layers, n_kv=n_kv, head_dim=d, kvdtype=code(W, kv), k_pages=pools[0], v_pages=pools[1],
        layer_stride=pools[0].stride(0), num_pages=pages, page_size=page, table_stride=width, parents=ints(parents),
        spare=ints(spare), old_table=ints(table), old_len=ints(lens), new_table=nt, new_len=nl))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    for p, w in zip(pools, want):
        np.testing.assert_array_equal(p.cpu().float().numpy(), w)
    np.testing.assert_array_equal(nt.cpu().numpy(), wt)
    np.testing.assert_array_equal(nl.cpu().numpy(), wl)


def test_beam_reorder_pages_bad_indexes():
    """A parent, page, spare page or length out of range makes its slot unused and is reported; nothing else changes."""
    import torch

    W = lib()
    page, pages, width = 4, 8, 2
    table = ints([[0, 1], [2, 8], [3, -1], [4, 5], [4, 5], [4, 5]])
    lens = ints([5, 6, 7, 8, 2, 3])
    for parents, spare, ok in (([6, 2**31 - 1, 0], [6, 7, 6], [False, False, True]),   # parents outside
                               ([1, 2, 0], [6, 7, 6], [False, False, True]),           # their tail pages outside
                               ([3, 0, 0], [6, 8, -1], [False, False, False]),         # full table; spare pages outside
                               ([4, 5, -7], [6, 7, 99], [True, True, None])):          # None: unused, not an error
        kp, vp = (torch.arange(pages * page * 8, device="cuda", dtype=torch.float32).view(1, pages, 1, page, 8) for _ in range(2))
        kp, vp = kp.clone(), vp.clone() + 0.5
        k0 = kp.clone()
        W.gemv_device_errors()
        pt, ptl = ints(np.full((6, width), 55)), ints([55] * 6)
        W.beam_reorder_pages(W.beam_reorder_args(
            beams=6, layers=1, n_kv=1, head_dim=8, kvdtype=W.DEC_F32, k_pages=kp, v_pages=vp, layer_stride=0,
            num_pages=pages, page_size=page, table_stride=width, parents=ints(parents + [-1] * 3),
            spare=ints(spare + [7] * 3), old_table=table, old_len=lens, new_table=pt, new_len=ptl))
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == (0x80 if False in ok else 0)
        n = ptl.cpu().numpy()
        assert (n[3:] == -1).all() and (pt.cpu().numpy()[3:] == -1).all()
        touched = set()
        for i, good in enumerate(ok):
            if good:
                assert n[i] == lens[parents[i]].item()
                touched.add(spare[i])
            else:
                assert n[i] == -1 and (pt.cpu().numpy()[i] == -1).all()
        for p in range(pages):
            if p not in touched:
                assert torch.equal(kp[:, p], k0[:, p])


def test_beam_reorder_pages_bad_filled_pages():
    """A filled page outside the pool, the first, one in the middle or the last of many, makes the slot unused in every
    layer, whether its tail page is good or empty."""
    import torch

    W = lib()
    page, width, beams, layers = 4, 300, 6, 3
    pages = beams * width + beams
    table = np.arange(beams * width, dtype=np.int32).reshape(beams, width)
    lens = [4 * 299, 4 * 299 + 3, 4 * 290 + 1, 8, 5, 3]
    table[0, 298], table[1, 0], table[2, 150], table[3, 1] = -1, pages, 2**31 - 1, -2**31
    table[4, 2] = -1  # behind the tail: not needed
    spare = beams * width + np.arange(beams)
    pools = [rand((layers, pages, 1, page, 8), "f32", seed) for seed in (1, 2)]
    before = [p.clone() for p in pools]
    nt, nl = ints(np.full((beams, width), 55)), ints(np.full(beams, 55))
    W.gemv_device_errors()
    W.beam_reorder_pages(W.beam_reorder_args(
        beams=beams, layers=layers, n_kv=1, head_dim=8, kvdtype=W.DEC_F32, k_pages=pools[0], v_pages=pools[1],
        layer_stride=pools[0].stride(0), num_pages=pages, page_size=page, table_stride=width,
        parents=ints(np.arange(beams)), spare=ints(spare), old_table=ints(table), old_len=ints(lens), new_table=nt,
        new_len=nl))
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0x80
    assert nl.tolist() == [-1] * 4 + lens[4:]
    want = np.full((beams, width), -1)
    want[4, 0], want[4, 1], want[5, 0] = table[4, 0], spare[4], spare[5]
    np.testing.assert_array_equal(nt.cpu().numpy(), want)
    for p, b in zip(pools, before):
        b[:, spare[4], :, :1] = b[:, table[4, 1], :, :1]
        b[:, spare[5], :, :3] = b[:, table[5, 0], :, :3]
        assert torch.equal(p, b)


# ---- together --------------------------------------------------------------------------------------------------------

def test_operators_on_another_stream_and_in_a_graph():
    """One captured graph holds a step of all operators (sharing one workspace); its replays give what eager calls give."""
    import torch

    W = lib()
    batch, n_q, n_kv, d, plen, page, vocab = 6, 8, 4, 128, 333, 16, 5000
    lens = [20, 5, 0, 33, 17, -1]
    a, t = attn_case(W, batch, n_q, n_kv, d, plen, lens, page, "bf16", "bf16", poison=False, width=4)
    a2, t2 = attn_case(W, batch, n_q, n_kv, d, plen + 64, lens, page, "bf16", "bf16", poison=False, width=4, seed=50)
    n = max(a.workspace_bytes, a2.workspace_bytes)
    shared = torch.empty(n, dtype=torch.uint8, device="cuda")
    a.with_workspace(shared), a2.with_workspace(shared)
    logits, scores = rand((batch, vocab), "f32", 8, 2.0), rand((batch,), "f32", 9)
    outs = [torch.zeros(12, dtype=dt, device="cuda") for dt in (torch.float32, torch.int32, torch.int32)]
    b = W.beam_select_args(beams=batch, vocab=vocab, n_out=12, logits=logits, logits_stride=vocab, scores=scores,
                           out_scores=outs[0], out_parents=outs[1], out_tokens=outs[2])
    b.with_workspace(torch.empty(W.beam_select_workspace(b), dtype=torch.uint8, device="cuda"))
    s, ra, pos, extra = rope_case(W, batch, n_q, n_kv, d, d, 0, "f32", "bf16", far=plen)
    r = W.qk_rope_args(k_out=s["k_out"][1], k_out_stride=n_kv * d, **ra)

    def step(stream):
        W.qk_norm_rope(r, stream)
        W.attn_shared_prefix(a, stream)
        W.attn_shared_prefix(a2, stream)
        W.beam_select(b, stream)

    step(None)
    torch.cuda.synchronize()
    want = [x.clone() for x in (s["q_out"][1], t["out"], t2["out"], *outs)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for x in (s["q_out"][1], t["out"], t2["out"], *outs):
            x.fill_(7)
    step(side)
    side.synchronize()
    keep = lens.index(-1)
    for x, w in zip((s["q_out"][1], t["out"], t2["out"], *outs), want):
        same = torch.equal(x, w)
        assert same, "another stream"
    g = torch.cuda.CUDAGraph()
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(side)
    with torch.cuda.graph(g2, stream=side):  # a second graph on the same workspace
        W.attn_shared_prefix(a2, side)
        W.attn_shared_prefix(a, side)
    for k in range(3):
        for x in (s["q_out"][1], t["out"], t2["out"], *outs):
            x.fill_(7)
        (g.replay(), g2.replay()) if k % 2 else (g2.replay(), g.replay())
        torch.cuda.synchronize()
        for x, w in zip((s["q_out"][1], t["out"], t2["out"], *outs), want):
            assert torch.equal(x, w)
    assert keep == 5 and W.gemv_device_errors() == 0


def test_beam_search_over_a_shared_prompt():
    """Several steps as a beam search makes them: append (norm, rotation, pages), attention over the shared prompt and
    the pages, a projection to logits (gemm_bf16), selection, reorder. Every beam's attention after each step equals the
    definition over its own history, kept on the host token by token."""
    import torch

    W = lib()
    beams, n_q, n_kv, d, plen, page, vocab, steps = 4, 4, 2, 128, 150, 4, 1000, 11
    rng = np.random.default_rng(12)
    pk, pv = rand((n_kv, plen + 5, d), "bf16", 1), rand((n_kv, plen + 5, d), "bf16", 2)
    head = rand((vocab, n_q * d), "bf16", 3, 0.2)
    emb = rand((vocab, (n_q + 2 * n_kv) * d), "f32", 4, 1.5)  # stands for embedding and projections of a token
    gq, gk = 1.0 + rand((d,), "f32", 5, 0.1), 1.0 + rand((d,), "f32", 6, 0.1)
    w, factor = W.rope_frequencies(d, 1e6)
    wd = torch.tensor(w, dtype=torch.float64, device="cuda")
    width = -(-(steps + 1) // page) + 1
    pages = beams * (width + steps)
    free = list(range(pages))
    kp, vp = (torch.full((1, pages, n_kv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = np.full((beams, width), -1)
    table[:, 0] = [free.pop() for _ in range(beams)]
    table, length = ints(table), ints([0] * beams)
    tokens, scores = ints(rng.integers(0, vocab, beams)), torch.tensor([0.0, -1.0, -2.0, -3.0], device="cuda")
    history = [[] for _ in range(beams)]  # (k, v) rows of each beam
    out = torch.empty((beams, n_q * d), dtype=torch.bfloat16, device="cuda")
    q_out, logits = torch.empty_like(out), torch.empty((beams, vocab), device="cuda")
    sc, pa, to = (torch.empty(beams, dtype=dt, device="cuda") for dt in (torch.float32, torch.int32, torch.int32))
    W.gemv_device_errors()
    for step in range(steps):
        rows = emb[tokens.long()].contiguous()
        q, k, v = rows, rows[:, n_q * d:], rows[:, (n_q + n_kv) * d:]
        wide = rows.shape[1]
        W.kv_append_paged(W.kv_append_args(
            rows=beams, n_q=n_q, n_kv=n_kv, head_dim=d, xdtype=W.DEC_F32, ydtype=W.DEC_BF16, kvdtype=W.DEC_BF16, q=q,
            k=k, v=v, q_out=q_out, q_stride=wide, k_stride=wide, v_stride=wide, q_out_stride=n_q * d, g_q=gq, g_k=gk,
            positions=ints([plen + step] * beams), inv_freq=wd, eps=1e-6, rope_factor=factor, rot_dim=d, interleaved=0,
            k_pages=kp, v_pages=vp, page_table=table, seq=None, n_seq=beams, num_pages=pages, page_size=page,
            table_stride=width, base_pos=plen))
        length = length + 1
        a = W.attn_shared_args(
            batch=beams, n_q=n_q, n_kv=n_kv, head_dim=d, qdtype=W.DEC_BF16, kvdtype=W.DEC_BF16, q=q_out, out=out,
            q_stride=n_q * d, out_stride=n_q * d, prefix_k=pk, prefix_v=pv, prefix_len=plen, prefix_stride=plen + 5,
            k_pages=kp, v_pages=vp, page_table=table, seq_len=length, num_pages=pages, page_size=page,
            table_stride=width, scale=d ** -0.5)
        a.with_workspace(torch.empty(W.attn_shared_prefix_workspace(a), dtype=torch.uint8, device="cuda"))
        W.attn_shared_prefix(a)
        W.gemm_bf16(out, head, logits, beams, vocab, n_q * d)
        b = W.beam_select_args(beams=beams, vocab=vocab, n_out=beams, logits=logits, logits_stride=vocab, scores=scores,
                               out_scores=sc, out_parents=pa, out_tokens=to)
        b.with_workspace(torch.empty(W.beam_select_workspace(b), dtype=torch.uint8, device="cuda"))
        W.beam_select(b)
        spare = [free.pop() for _ in range(beams)]
        nt, nl = torch.empty_like(table), torch.empty_like(length)
        W.beam_reorder_pages(W.beam_reorder_args(
            beams=beams, layers=1, n_kv=n_kv, head_dim=d, kvdtype=W.DEC_BF16, k_pages=kp, v_pages=vp, layer_stride=0,
            num_pages=pages, page_size=page, table_stride=width, parents=pa, spare=ints(spare), old_table=table,
            old_len=length, new_table=nt, new_len=nl))
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == 0
        # the host's account of the same step: the stored rows, then attention over each beam's own history
        tab = table.cpu().numpy()
        for i in range(beams):
            at = tab[i, step // page], slice(None), step % page
            kr, vr = f64(kp[0])[at], f64(vp[0])[at]
            ref, tol = rope_ref(f64(k[i, : n_kv * d]).reshape(n_kv, d), f64(gk), 1e-6, plen + step, w, d, 0, factor, "bf16")
            inside(kr, ref, tol, "stored key")
            np.testing.assert_array_equal(vr, f64(v[i, : n_kv * d].bfloat16()).reshape(n_kv, d))
            history[i] = history[i] + [(kr, vr)]
            for g in range(n_kv):
                kk = np.concatenate([f64(pk)[g, :plen], [h[0][g] for h in history[i]]])
                vv = np.concatenate([f64(pv)[g, :plen], [h[1][g] for h in history[i]]])
                qq = f64(q_out[i]).reshape(n_kv, n_q // n_kv, d)[g]
                ref, l, size = OB.attend(qq, kk, vv, float(np.float32(d ** -0.5)))
                tol = attn_tol(qq, kk, l, ref, size, float(np.float32(d ** -0.5)), "bf16")[0]
                inside(f64(out[i]).reshape(n_kv, n_q // n_kv, d)[g], ref, tol, (step, i, g))
        check_select([x.cpu().numpy() for x in (sc, pa, to)], logits.cpu().numpy(), scores.cpu().numpy(), beams)
        parents = pa.cpu().numpy()
        history = [history[p] for p in parents]
        assert nl.tolist() == [step + 1] * beams
        table, length, scores, tokens = nt, nl, sc.clone(), to.clone()


@pytest.mark.parametrize("shape,kv,y", [("TINY", "f32", "f32"), ("TINY", "bf16", "f32"), ("Q4_SMALL", "bf16", "bf16")], ids=str)
def test_branches_continue_a_decoders_prompt(shape, kv, y):
    """Branches of a prompt that the decoder prefilled: appended keys carry on the rotation and norm of the prompt's,
    attention reads the decoder's own cache. Keys, values and logits of every branch are those of the decoder and of the
    oracle on the branch's whole token sequence, within the tolerances that the decoder itself is held to. (What lies
    between the operators, products with the weights and the SwiGLU, is computed on the host.)"""
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
    d, n, page, width, steps = s.head_dim, len(prompt), 4, 3, 6
    rng = np.random.default_rng(3)
    rows = rng.integers(0, s.vocab, (3, steps))  # the branches' tokens; the last two differ from their second on
    rows[2, 0] = rows[1, 0]
    B = len(rows)
    dec = Decoder(s, weights, kv_dtype=kv, max_seq=n + steps + 4)
    dec.prefill(prompt, is_last=True)
    ora = O.OracleDecoder(s, weights, kv_dtype=kv, max_seq=n + steps + 4)
    freq, factor = W.rope_frequencies(d, s.rope_theta)
    wd = torch.tensor(freq, dtype=torch.float64, device="cuda")
    pools = [[torch.full((B * width, s.n_kv, page, d), float("nan"), device="cuda").to(tdt(kv)) for _ in range(2)]
             for _ in range(s.layers)]
    table = rng.permutation(B * width).reshape(B, width)
    table_d, wide = ints(table), (s.n_q + 2 * s.n_kv) * d
    gains = [[torch.tensor(P.widen(w[g]).astype(np.float32), device="cuda") for g in ("g_q", "g_k")] for w in weights["layers"]]
    got = np.zeros((B, steps, s.vocab))
    W.gemv_device_errors()
    for i in range(steps):
        h = ora.E[rows[:, i]].copy()
        for l, w in enumerate(ora.layers):
            x = P.rmsnorm(h, w["g_in"], s.eps)
            qkv = torch.tensor(np.concatenate([x @ w[m].T for m in ("w_q", "w_k", "w_v")], 1).astype(np.float32), device="cuda")
            q_out = torch.empty((B, s.n_q * d), dtype=tdt(y), device="cuda")
            W.kv_append_paged(W.kv_append_args(
                rows=B, n_q=s.n_q, n_kv=s.n_kv, head_dim=d, xdtype=W.DEC_F32, ydtype=code(W, y), kvdtype=code(W, kv),
                q=qkv, k=qkv[:, s.n_q * d:], v=qkv[:, (s.n_q + s.n_kv) * d:], q_out=q_out, q_stride=wide, k_stride=wide,
                v_stride=wide, q_out_stride=s.n_q * d, g_q=gains[l][0], g_k=gains[l][1], positions=ints([n + i] * B),
                inv_freq=wd, eps=s.eps, rope_factor=factor, rot_dim=d, interleaved=0, k_pages=pools[l][0],
                v_pages=pools[l][1], page_table=table_d, seq=None, n_seq=B, num_pages=B * width, page_size=page,
                table_stride=width, base_pos=n))
            K, V, held = dec.kv(l)
            assert held == n
            out = torch.empty_like(q_out)
            a = W.attn_shared_args(
                batch=B, n_q=s.n_q, n_kv=s.n_kv, head_dim=d, qdtype=code(W, y), kvdtype=code(W, kv), q=q_out, out=out,
                q_stride=s.n_q * d, out_stride=s.n_q * d, prefix_k=K, prefix_v=V, prefix_len=n, prefix_stride=K.shape[1],
                k_pages=pools[l][0], v_pages=pools[l][1], page_table=table_d, seq_len=ints([i + 1] * B),
                num_pages=B * width, page_size=page, table_stride=width, scale=d ** -0.5)
            a.with_workspace(torch.empty(W.attn_shared_prefix_workspace(a), dtype=torch.uint8, device="cuda"))
            W.attn_shared_prefix(a)
            h = h + f64(out) @ w["w_o"].T
            x = P.rmsnorm(h, w["g_post"], s.eps)
            h = h + P.swiglu(x @ w["w_gate"].T, x @ w["w_up"].T) @ w["w_down"].T
        got[:, i] = P.rmsnorm(h, ora.g_final, s.eps) @ ora.E.T
    assert W.gemv_device_errors() == 0
    dec.close()
    i = np.arange(steps)
    for b in range(B):
        ref = O.OracleDecoder(s, weights, kv_dtype=kv, max_seq=n + steps + 4)
        ref.prefill(prompt)
        one = Decoder(s, weights, kv_dtype=kv, max_seq=n + steps + 4)
        one.prefill(prompt, is_last=True)
        logits = torch.empty(s.vocab, dtype=torch.float32, device="cuda")
        for j, t in enumerate(rows[b]):
            want = ref.step(int(t))
            one.step(int(t), logits=logits)
            close(got[b, j], want, tol, f"logits of branch {b}, step {j}")
            close(got[b, j], f64(logits), 2 * tol, f"the decoder's logits, branch {b}, step {j}")
        for l in range(s.layers):
            for pool, theirs, mine in zip(pools[l], ref.kv(l), one.kv(l)[:2]):
                rows_of = f64(pool)[table[b, i // page], :, i % page].transpose(1, 0, 2)
                close(rows_of, theirs[:, n:], tol, f"cache of branch {b}, layer {l}")
                close(rows_of, f64(mine)[:, n: n + steps], 2 * tol, f"the decoder's cache, branch {b}, layer {l}")
        one.close()


def test_operators_on_two_streams_at_once():
    """Calls with workspaces of their own that run beside each other give the bits that they give alone."""
    import torch

    W = lib()
    cases = []
    for k, (types, batch, n_q, n_kv, d, plen) in enumerate(((("bf16", "bf16"), 16, 16, 8, 128, 3000),
                                                            (("bf16", "bf16"), 40, 8, 2, 128, 1500),
                                                            (("f32", "f32"), 6, 8, 4, 64, 700))):
        a, t = attn_case(W, batch, n_q, n_kv, d, plen, [(7 * i + k) % 90 for i in range(batch)], 16, *types, seed=10 * k)
        logits, scores = rand((4 + k, 20000), "f32", 50 + k, 2.0), rand((4 + k,), "f32", 60 + k)
        outs = [torch.zeros(20, dtype=dt, device="cuda") for dt in (torch.float32, torch.int32, torch.int32)]
        b = W.beam_select_args(beams=4 + k, vocab=20000, n_out=20, logits=logits, logits_stride=20000, scores=scores,
                               out_scores=outs[0], out_parents=outs[1], out_tokens=outs[2])
        b.with_workspace(torch.empty(W.beam_select_workspace(b), dtype=torch.uint8, device="cuda"))
        cases.append((a, b, [t["out"], t["lse"], *outs]))
    want = []
    for a, b, outs in cases:
        W.attn_shared_prefix(a)
        W.beam_select(b)
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
        for x in outs:
            x.fill_(3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(30):
        for (a, b, _outs), st in zip(cases, streams):
            W.attn_shared_prefix(a, st)
            W.beam_select(b, st)
    torch.cuda.synchronize()
    assert W.gemv_device_errors() == 0
    for (_, _, outs), w in zip(cases, want):
        for x, y in zip(outs, w):
            assert torch.equal(x, y)


@pytest.mark.parametrize("types,d", [(("bf16", "bf16"), 128), (("bf16", "bf16"), 64), (("f32", "f32"), 128)], ids=str)
def test_a_captured_step_follows_its_lengths_and_tables(types, d):
    """A graph of append and attention is captured once; positions, lengths and tables change between its replays, as a
    decoding loop changes them, slots ending and starting again. Each replay gives an eager call's bits and the
    definition's values."""
    import torch

    W = lib()
    B, n_q, n_kv, plen, page, width = 5, 8, 4, 200, 8, 12
    full = [width * page] * B
    a, t = attn_case(W, B, n_q, n_kv, d, plen, full, page, *types, poison=False, width=width)
    s, ra, _, extra = rope_case(W, B, n_q, n_kv, d, d, 0, "f32", types[0], seed=30)
    v = rand((B, n_kv * d), "f32", 40)
    lens, pos, table = ints([-1] * B), ints([-1] * B), ints(t["table"])
    ra.update(q_out=t["q"], positions=pos)
    kv_args = W.kv_append_args(v=v, v_stride=n_kv * d, kvdtype=code(W, types[1]), k_pages=t["kp"], v_pages=t["vp"],
                               page_table=table, seq=None, n_seq=B, num_pages=t["kp"].shape[0], page_size=page,
                               table_stride=width, base_pos=plen, **ra)
    a.set("seq_len", lens).set("page_table", table)

    def step(stream=None):
        W.kv_append_paged(kv_args, stream)
        W.attn_shared_prefix(a, stream)

    side = torch.cuda.Stream()
    step(side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(side)
    rng = np.random.default_rng(8)
    for k in range(6):
        held = rng.integers(1, width * page + 1, B)
        held[k % B] = -1
        if k == 3:
            held[:] = -1  # every slot unused
        now = rng.permutation(t["table"].reshape(-1)).reshape(B, width).astype(np.int32)
        lens.copy_(ints(held)), pos.copy_(ints(np.where(held < 0, -1, plen + held - 1))), table.copy_(ints(now))
        t["table"] = now
        for x in (t["out"], t["lse"]):
            x.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert W.gemv_device_errors() == 0
        check_attn(t, B, n_q, n_kv, d, plen, held.tolist(), page, types[0])
        got = [x.clone() for x in (t["out"], t["lse"])]
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], t["out"]) and torch.equal(got[1], t["lse"])
