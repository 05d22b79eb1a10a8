"""The first call that a process makes of an operator around the cache, made under stream capture: what a call sets up
once (kernel attributes, what the device holds at once, the status word) is set up without leaving the capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
import torch
import attention_attn_fwd_03_gb300 as attn
what, G, d = sys.argv[1], int(sys.argv[2]), int(sys.argv[3])
B, H_kv, page, pages, n = 2, 2, 16, 64, 400
g = torch.Generator(device="cuda").manual_seed(0)
r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
q, k, v, kc, vc = r(B, G * H_kv, d), r(B, H_kv, d), r(B, H_kv, d), r(pages, page, H_kv, d), r(pages, page, H_kv, d)
bt = torch.arange(2 * 32, dtype=torch.int32, device="cuda").view(2, 32)
lens, slots, pos, one = i32(n, 90), i32(3, 900), i32(7, 70000), i32(5)
f = attn.rope_inv_freq(d)[0].cuda()
sk = torch.randint(-127, 128, (pages, H_kv, 2 * d), dtype=torch.int8, device="cuda", generator=g)
amp = torch.rand((pages, H_kv), device="cuda", generator=g)
free = torch.arange(5, dtype=torch.int32, device="cuda")


def call():
    if what == "rope":
        return attn.rope(q, k, inv_freq=f, positions=pos)
    if what == "append":
        return [attn.paged_append(q, k, v, kc, vc, slots, positions=pos, inv_freq=f), kc, vc]
    if what == "plan":
        return [*attn.paged_plan(lens, bt, free, one, page, pages, 2), bt]
    if what == "sketch":
        return attn.page_sketch(kc, bt, lens, sk, amp, max_q_len=n)
    if what == "select":
        return attn.page_select(q, sk, amp, bt, lens, page, 4)
    return attn.paged_sparse_fwd(q, kc, vc, bt, lens, sk, amp, 4, return_tables=True)


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    got = call()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
want = call()
attn.device_status()
assert all(torch.equal(a, b) for a, b in zip(got, want)), what
"""


@pytest.mark.parametrize("what,G,d", [("rope", 4, 128), ("append", 4, 64), ("plan", 1, 64), ("sketch", 1, 128), ("select", 4, 64),
                                      ("sparse", 4, 128), ("sparse", 20, 64), ("sparse", 30, 128)])
def test_first_call_is_captured(what, G, d):
    r = subprocess.run([sys.executable, "-c", PROGRAM, what, str(G), str(d)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
