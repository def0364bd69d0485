"""The prompt side's first call of a process: captured into a graph, or made by several host threads at
once (each call sets its kernel's shared-memory limit and looks up the tensor map encoder the first time)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import paged_kv_decode_np_gb300 as npg
from prompt_helpers import chunk_inputs, chunk_reference, chunk_tolerance
rows = [(40, 300), (1, 700), (130, 130)]
dtype, d, bs = torch.{dtype}, {d}, {bs}
inp = chunk_inputs(dtype, d, 2, 4, bs, rows, seed=1)
n = inp["q"].shape[0]
slots = torch.cat([inp["block_tables"][r].long()[t // bs] * bs + t % bs for r, (m, c) in enumerate(rows)
                   for t in [torch.arange(c - m, c, device="cuda")]])
pos = torch.zeros(n, dtype=torch.int32, device="cuda")  # angle 0: k and v are put back as they were
table = npg.rope_table(8, d)
k, v = (inp[x].view(-1, 2, d)[slots].clone() for x in ("k_pool", "v_pool"))
def step(out, q, ws):
    npg.prefill_step(out, q, k, v, slots, inp["k_pool"], inp["v_pool"], inp["block_tables"], inp["context_lens"],
                     inp["query_starts"], d ** -0.5, ws, cos_sin=table, positions=pos, q_rotated=torch.empty_like(q))
def check(out):
    ref, bound = chunk_reference(inp, rows, d ** -0.5)
    assert ((out.double() - ref).abs() <= chunk_tolerance(ref, bound, dtype, d, 700)).all()
torch.cuda.synchronize()
"""

CAPTURED = """
out, ws, g = torch.zeros_like(inp["q"]), npg.prefill_workspace(d), torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step(out, inp["q"], ws)
assert (out == 0).all()
g.replay()
torch.cuda.synchronize()
check(out)
print("ok")
"""

THREADS = """
outs = [torch.zeros_like(inp["q"]) for _ in range(4)]
spaces = [npg.prefill_workspace(d) for _ in range(4)]
streams = [torch.cuda.Stream() for _ in range(4)]
torch.cuda.synchronize()
bad, gate = [], threading.Barrier(4)
def work(i):
    try:
        with torch.cuda.stream(streams[i]):
            gate.wait()
            for _ in range(20):
                npg.np_paged_prefill(outs[i], inp["q"], inp["k_pool"], inp["v_pool"], inp["block_tables"],
                                     inp["context_lens"], inp["query_starts"], d ** -0.5, spaces[i])
    except BaseException as e:
        bad.append(e)
ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[t.start() for t in ts]
[t.join() for t in ts]
torch.cuda.synchronize()
assert not bad, bad
for o in outs:
    check(o)
    assert torch.equal(o, outs[0])
print("ok")
"""


@pytest.mark.parametrize("body", [CAPTURED, THREADS], ids=["captured", "threads"])
@pytest.mark.parametrize("dtype,d,bs", [("bfloat16", 128, 16), ("bfloat16", 256, 5), ("bfloat16", 32, 16),
                                        ("float32", 128, 16), ("float32", 256, 16)])
def test_the_first_call_of_a_process(nplib, body, dtype, d, bs):
    src = HEAD.format(root=ROOT, tests=os.path.join(ROOT, "tests"), dtype=dtype, d=d, bs=bs) + body
    p = subprocess.run([sys.executable, "-c", src], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and p.stdout.strip().endswith("ok"), p.stdout + p.stderr
