"""Each operation of the block as the first call of a process: captured into
a graph before anything ran eagerly, and from two threads at once."""
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
M, D, F = 300, 1024, 520
def rand(*s):
    return torch.randn(*s, device=DEV).bfloat16()
def state(seed):
    torch.manual_seed(seed)
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device=DEV)
    f32, u8 = torch.float32, torch.uint8
    n = max(nn.mlp_op_layernorm_backward_workspace_bytes(nn.BF16, M, D), nn.mlp_op_wgrad8_workspace_bytes(nn.BF16, 2 * F, D, M))
    return dict(x=rand(M, D), dy=rand(M, D), w=rand(2 * F, D) * 0.03, wd=rand(D, F) * 0.03, n=z(M, D), mean=z(M, d=f32),
                rstd=z(M, d=f32), h=z(M, F), s=z(M, 2 * F, d=u8), e=z(M, 34, d=u8), nq=z(M, D, d=u8), ne=z(M, 32, d=u8),
                ds=z(M, 2 * F), h2=z(M, F), dx=z(M, D), dw=z(2 * F, D, d=f32), dg=z(D, d=f32), db=z(D, d=f32),
                ws=z(n, d=u8), back=z(M, D))
def calls(t):
    p = {k: v.data_ptr() for k, v in t.items()}
    n, B = t["ws"].numel(), nn.BF16
    st = lambda: torch.cuda.current_stream().cuda_stream
    return dict(
        layernorm=lambda: nn.mlp_op_layernorm(B, M, D, p["x"], D, None, None, 1e-5, p["n"], D, p["mean"], p["rstd"], st()),
        gated=lambda: nn.mlp_op_gated_linear(B, nn.ACT_SILU, M, F, D, p["n"], D, p["w"], D, None, p["h"], F, p["s"], 2 * F,
                                             p["e"], 34, None, st()),
        quant8=lambda: nn.mlp_op_quant8(B, M, D, p["n"], D, p["nq"], D, p["ne"], 32, st()),
        dequant8=lambda: nn.mlp_op_dequant8(B, M, D, p["nq"], D, p["ne"], 32, p["back"], D, st()),
        dgrad=lambda: nn.mlp_op_gated_dgrad(B, nn.ACT_SILU, M, D, F, p["dy"], D, p["wd"], F, p["s"], 2 * F, p["e"], 34,
                                            p["ds"], 2 * F, p["h2"], F, None, st()),
        wgrad8=lambda: nn.mlp_op_wgrad8(B, 2 * F, D, M, p["ds"], 2 * F, p["nq"], D, p["ne"], 32, p["dw"], D, None, p["ws"],
                                        n, None, st()),
        backward=lambda: nn.mlp_op_layernorm_backward(B, M, D, p["dy"], D, p["x"], D, None, p["mean"], p["rstd"], p["dx"], D,
                                                      p["dg"], p["db"], p["ws"], n, st()))
OUT = ("n", "mean", "rstd", "h", "s", "e", "nq", "ne", "back", "ds", "h2", "dw", "dx", "dg", "db")
"""

CAPTURE = PRELUDE + r"""
t = state(1)
c = calls(t)
first = sys.argv[1]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for name in [first] + [k for k in c if k != first]:
        c[name]()
for _ in range(3):   # (`first` reads what the replay before left)
    g.replay()
torch.cuda.synchronize()
got = {k: t[k].clone() for k in OUT}
for f in c.values():
    f()
torch.cuda.synchronize()
for k in OUT:
    assert torch.equal(got[k], t[k]), k
    assert torch.isfinite(t[k].float()).all() and t[k].float().abs().max() > 0, k
print("ok")
"""

THREADS = PRELUDE + r"""
ts = [state(i) for i in range(4)]
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
    got = {k: t[k].clone() for k in OUT}
    for f in calls(t).values():
        f()
    torch.cuda.synchronize()
    for k in OUT:
        assert torch.equal(got[k], t[k]), k
print("ok")
"""


def _run(program, *args):
    r = subprocess.run([sys.executable, "-c", program, *args], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@pytest.mark.parametrize("first", ["layernorm", "gated", "dgrad", "wgrad8", "backward"])
def test_first_call_is_captured(first):
    _run(CAPTURE, first)


def test_first_calls_of_several_threads():
    _run(THREADS)
