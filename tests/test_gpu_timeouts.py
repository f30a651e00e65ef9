"""The give-up path of the persistent engines' bounded waits, on the GPU.

Every wait of a persistent kernel on another CTA's results is bounded; when one
runs out the kernel records the cause in the device error word, waits for its
own copies in flight and returns, so the context stays usable. Here the limit is
set to 1 ns (dec_set_wait_limit), so any wait that is not already satisfied
gives up at once: the forward must end, the error bit must be set, dec_reset
must clear it, and after the default limit is restored the same context must
reproduce, bit for bit, what a fresh context computes.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

import workloads as Wl

from gpu_util import lib

pytestmark = pytest.mark.gpu

DEVERR_EXCHANGE_TIMEOUT = 0x10
DEVERR_BARRIER_TIMEOUT = 0x40
DEVERR_GEMM_TIMEOUT = 0x20


def _run(dec, prompt, n, vocab):
    import torch

    logits = torch.empty(vocab, dtype=torch.float32, device="cuda")
    dec.reset()
    tok = dec.prefill(prompt, is_last=True, logits=logits)
    out, rows = [tok], [logits.cpu().numpy().copy()]
    for _ in range(n):
        tok = dec.step(tok, logits=logits)
        out.append(tok)
        rows.append(logits.cpu().numpy().copy())
    return out, rows


@pytest.mark.parametrize("wd", ["f32", "q4"])
def test_persistent_wait_gives_up_and_context_recovers(wd):
    lib()
    from weight_streaming_gemv_token_gb300.decoder import Decoder

    if wd == "q4":
        shape, w, bit = Wl.Q4_SMALL, Wl.decoder_weights_q4(Wl.Q4_SMALL, seed=1), DEVERR_BARRIER_TIMEOUT
    else:
        shape, w, bit = Wl.TINY, Wl.decoder_weights(Wl.TINY, seed=1), DEVERR_EXCHANGE_TIMEOUT
    prompt = [int(t) for t in Wl.prompt_uniform(6, shape.vocab, seed=4)]
    ref = Decoder(shape, w, max_seq=32, engine="persistent")
    want_tok, want_logits = _run(ref, prompt, 4, shape.vocab)
    assert ref.device_errors() == 0
    ref.close()

    dec = Decoder(shape, w, max_seq=32, engine="persistent")
    dec.prefill(prompt[:-1], is_last=False)
    assert dec.device_errors() == 0
    dec.set_wait_limit(1)
    dec.step(prompt[-1])  # returns once the launch has given up; its token is undefined
    errs = dec.device_errors(clear=False)
    assert errs & bit, f"device errors {errs:#x}: the timeout bit {bit:#x} is not set"
    dec.set_wait_limit(0)
    dec.reset()
    assert dec.device_errors(clear=False) == 0, "dec_reset did not clear the device error word"
    got_tok, got_logits = _run(dec, prompt, 4, shape.vocab)
    assert got_tok == want_tok
    for j, (a, b) in enumerate(zip(got_logits, want_logits)):
        assert np.array_equal(a, b), f"logits of output {j} differ from a fresh context's"
    assert dec.device_errors() == 0
    dec.close()


_TREE = """
import sys, ctypes
sys.path.insert(0, sys.argv[1])
import numpy as np, torch
from weight_streaming_gemv_token_gb300 import build
build.LIB = sys.argv[2]
import weight_streaming_gemv_token_gb300 as W

def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")

def case(batch, rows, d, plen, ctx, page, width):
    n_q, n_kv = 16, 8
    starts = np.concatenate([[0], np.cumsum(rows)])
    total = int(starts[-1])
    bf = dict(dtype=torch.bfloat16, device="cuda")
    pk, pv, kp, vp = (torch.randn(s, **bf) for s in [(n_kv, max(plen, 1), d)] * 2 + [(64, n_kv, page, d)] * 2)
    q = torch.randn(total, n_q * d, **bf)
    a = W.attn_tree_args(
        batch=batch, rows=total, n_q=n_q, n_kv=n_kv, head_dim=d, qdtype=W.DEC_BF16, kvdtype=W.DEC_BF16, q=q, out=torch.empty_like(q),
        q_stride=n_q * d, out_stride=n_q * d, row_start=ints(starts), prefix_k=pk, prefix_v=pv, prefix_len=plen, prefix_stride=max(plen, 1),
        k_pages=kp, v_pages=vp, page_table=torch.arange(batch * width, dtype=torch.int32, device="cuda") % 64,
        seq_len=ints([ctx] * batch), num_pages=64, page_size=page, table_stride=width, scale=d ** -0.5)
    ws = torch.full((W.attn_tree_paged_workspace(a),), 255, dtype=torch.uint8, device="cuda")
    a.with_workspace(ws)
    a.ws = ws
    return a

few = np.zeros(4096, int)
few[np.arange(17) * 240] = 1
for kw in (dict(batch=4096, rows=few, d=128, plen=0, ctx=500, page=16, width=72), dict(batch=32, rows=[64] * 32, d=128, plen=0, ctx=4000, page=64, width=64),
           dict(batch=32, rows=[64] * 32, d=64, plen=3000, ctx=900, page=128, width=8), dict(batch=1, rows=[200], d=64, plen=0, ctx=3, page=8, width=30)):
    a = case(**kw)
    for _ in range(3):
        W.attn_tree_paged(a)
        torch.cuda.synchronize()
        errors = W.gemv_device_errors()
        # records of cut segments (32 bytes: number, pieces, ..) for 152 CTAs, in front of the line's length: the join's
        records = a.ws.cpu().numpy()[-256 - 32 * 152: -256 - 32 * (152 - 136)].view(np.int32).reshape(136, 8)
        print(errors, int((records[:, 2] < 0).sum()) if kw["batch"] == 4096 else 0)
x = torch.arange(1 << 20, device="cuda", dtype=torch.float64)
print(int(x.sum().item()) == (1 << 20) * ((1 << 20) - 1) // 2)
"""


def test_attention_of_drafted_trees_gives_up(tmp_path):
    """attn_tree_paged on the tensor cores, its waits' limit compiled as 1 ns and one try (in a library beside the package's):
    waits for the schedule, for keys and for products give up. The call ends, the error bit is set, the records that the join
    goes by are all there, and the process goes on. With the package's library the same calls run through."""
    lib()
    from weight_streaming_gemv_token_gb300 import build as bld

    nvcc, obj, so = bld._nvcc(), str(tmp_path / "tc.o"), str(tmp_path / "libwsg_short.so")
    src = os.path.join(bld.CSRC, "attn_tree_tc.cu")
    short = ["-DWSG_WAIT_LIMIT_NS=1ull", "-DWSG_WAIT_TRIES=1"]
    subprocess.run([nvcc, *bld.NVCC_FLAGS, *bld.ARCH, *short, "-c", src, "-o", obj], check=True)
    rest = [os.path.join(bld.BUILD, os.path.basename(s) + ".o") for s in bld.sources() if s != src]
    subprocess.run([nvcc, *bld.ARCH, "-shared", "-o", so, obj, *rest, "-lcudart"], check=True)
    root = os.path.dirname(bld.HERE)
    out = {}
    for path in (so, bld.LIB):
        r = subprocess.run([sys.executable, "-c", _TREE, root, path], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        out[path] = r.stdout.split("\n")
    for path, lines in out.items():
        assert lines[12] == "True"
        got = [[int(x) for x in l.split()] for l in lines[:12]]
        assert all(h == 0 for _, h in got), got
        if path == so:
            assert all(e & ~DEVERR_GEMM_TIMEOUT == 0 for e, _ in got) and all(e == DEVERR_GEMM_TIMEOUT for e, _ in got[:3]), got
        else:
            assert all(e == 0 for e, _ in got), got
