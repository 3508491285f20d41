"""Each operation on logits as the first call of a process: captured into a graph before anything ran eagerly, and from
several threads at once."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PRELUDE = r"""
import sys, threading
import torch
import neural_net_step_gb300 as nn
DEV = "cuda:0"
torch.cuda.init()
B, C, k, W = 24, 60000, 40, 4
def state(seed):
    torch.manual_seed(seed)
    f = lambda *s: torch.zeros(*s, device=DEV)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    z = (torch.randn(B, C, device=DEV) * 3).bfloat16()
    n = nn.mlp_op_beam_select_workspace_bytes(nn.BF16, B // W, W, C, W)
    return dict(z=z, v=f(B, k), i=i(B, k), lse=f(B), tail=f(B), dz=torch.zeros_like(z), loss=f(B),
                y=torch.randint(0, C, (B,), device=DEV).int(), s=-torch.rand(B // W, W, device=DEV), so=f(B // W, W), p=i(B // W, W),
                t=i(B // W, W), ws=torch.zeros(n, dtype=torch.uint8, device=DEV), st=torch.randn(3, B, 1000, device=DEV),
                sd=f(3, B, 1000))
def calls(t):
    p = {a: b.data_ptr() for a, b in t.items()}
    H, n = nn.BF16, t["ws"].numel()
    st = lambda: torch.cuda.current_stream().cuda_stream
    return dict(
        topk=lambda: nn.mlp_op_topk(H, B, C, k, p["z"], C, 1.5, p["v"], k, p["i"], k, p["lse"], p["tail"], st()),
        distill=lambda: nn.mlp_op_distill(H, B, C, k, p["z"], C, p["v"], k, p["i"], k, p["tail"], p["y"], None, 1.5, 0.5, 1.0,
                                          1.0, p["dz"], C, p["loss"], None, st()),
        select=lambda: nn.mlp_op_beam_select(H, B // W, W, C, W, p["z"], C, p["s"], None, -1, p["so"], p["p"], p["t"], None,
                                             p["ws"], n, st()),
        reorder=lambda: nn.mlp_op_beam_reorder(3, B // W, W, W, 4000, p["st"], 4000, 4000 * B, p["p"], W, p["sd"], 4000, 4000 * B,
                                               None, st()))
OUT = ("v", "i", "lse", "tail", "dz", "loss", "so", "p", "t", "sd")
"""

CAPTURE = PRELUDE + r"""
t = state(1)
c = calls(t)
first = sys.argv[1]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for name in [first] + [a for a in c if a != first]:
        c[name]()
for _ in range(3):   # (`first` reads what the replay before left)
    g.replay()
torch.cuda.synchronize()
got = {a: t[a].clone() for a in OUT}
for f in c.values():
    f()
torch.cuda.synchronize()
for a in OUT:
    assert torch.equal(got[a], t[a]), a
    assert torch.isfinite(t[a].float()).all() and t[a].float().abs().max() > 0, a
print("ok")
"""

THREADS = PRELUDE + r"""
ts = [state(j) for j in range(4)]
torch.cuda.synchronize()
errors = []
def work(t):
    try:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                for f in calls(t).values():
                    f()
        s.synchronize()
    except Exception as e:
        errors.append(e)
th = [threading.Thread(target=work, args=(t,)) for t in ts]
[x.start() for x in th]
[x.join() for x in th]
assert not errors, errors
for t in ts:
    got = {a: t[a].clone() for a in OUT}
    for f in calls(t).values():
        f()
    torch.cuda.synchronize()
    for a in OUT:
        assert torch.equal(got[a], t[a]), a
print("ok")
"""


def _run(program, *args):
    r = subprocess.run([sys.executable, "-c", program, *args], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@pytest.mark.parametrize("first", ["topk", "distill", "select", "reorder"])
def test_first_call_is_captured(first):
    _run(CAPTURE, first)


def test_first_calls_of_several_threads():
    _run(THREADS)
