"""The operations on logits as a program runs them together: a distillation step behind two LM heads, and a beam search
with histories and states to the end, each against the fp64 oracle and captured."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import logits_oracle as lo
from tests.block_util import DEV, HALF, U32, assert_within, stream, sum_err

pytestmark = pytest.mark.gpu
H = nn.BF16


@pytest.mark.parametrize("captured", [False, True])
def test_distillation_step(captured):
    """teacher: linear -> top-k; student: linear -> distillation (in place) -> loss mean, dgrad, wgrad."""
    B, K, C, k, T = 264, 64, 2504, 16, 2.0
    rng = np.random.default_rng(1)
    bf = lambda *s, std=1.0: torch.from_numpy((rng.normal(size=s) * std).astype(np.float32)).bfloat16().to(DEV)
    f32 = lambda *s: torch.zeros(*s, device=DEV)
    xt, xs, wt, ws = bf(B, K), bf(B, K), bf(C, K, std=0.3), bf(C, K, std=0.3)
    xs.copy_(xt)
    y = torch.from_numpy(rng.integers(0, C, B).astype(np.int32)).to(DEV)
    w = torch.from_numpy((rng.uniform(size=B) < 0.9).astype(np.float32)).to(DEV)
    zt, z0 = torch.zeros(B, C, dtype=torch.bfloat16, device=DEV), torch.zeros(B, C, dtype=torch.bfloat16, device=DEV)
    z = torch.zeros_like(z0)
    tv, ti, tail = f32(B, k), torch.zeros(B, k, dtype=torch.int32, device=DEV), f32(B)
    rows, loss, dw, db = f32(B), f32(1), f32(C, K), f32(C)
    bias = f32(C)
    dx = torch.zeros(B, K, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    n = nn.mlp_op_wgrad_workspace_bytes(H, C, K, B)
    wsp = torch.zeros(max(n, 4), dtype=torch.uint8, device=DEV)
    p = lambda t: t.data_ptr()

    def step():
        nn.mlp_op_linear_act(H, nn.ACT_NONE, B, C, K, p(xt), K, p(wt), K, p(bias), p(zt), C, None, 0, p(err), stream())
        nn.mlp_op_topk(H, B, C, k, p(zt), C, T, p(tv), k, p(ti), k, None, p(tail), stream())
        nn.mlp_op_linear_act(H, nn.ACT_NONE, B, C, K, p(xs), K, p(ws), K, p(bias), p(z), C, None, 0, p(err), stream())
        z0.copy_(z)
        nn.mlp_op_distill(H, B, C, k, p(z), C, p(tv), k, p(ti), k, p(tail), p(y), p(w), T, 0.3, 0.7 * T * T, 1.0 / B, p(z), C,
                          p(rows), p(err), stream())
        nn.mlp_op_loss_mean(B, p(rows), p(loss), p(err), stream())
        nn.mlp_op_dgrad(H, nn.ACT_NONE, B, C, K, p(z), C, p(ws), K, None, 0, p(dx), K, p(err), stream())
        nn.mlp_op_wgrad(H, C, K, B, p(z), C, p(xs), K, p(dw), K, p(db), p(wsp), n, p(err), stream())

    step()
    torch.cuda.synchronize()
    if captured:
        want = [t.clone() for t in (tv, ti, tail, z, rows, loss, dx, dw, db)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for t in (tv, ti, tail, z, rows, loss, dx, dw, db):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (tv, ti, tail, z, rows, loss, dx, dw, db)):
            assert torch.equal(a, b)
        return
    d = lambda t: t.detach().double().cpu().numpy()
    assert err.item() == 0
    zt64 = d(zt)
    assert_within(zt64, d(xt) @ d(wt).T, HALF[H] * np.abs(zt64) + sum_err(np.abs(d(xt)) @ np.abs(d(wt)).T, K), "teacher's logits")
    v, i, _, tl = lo.topk(zt64, k, T)
    assert np.array_equal(d(tv), v) and np.array_equal(d(ti), i)
    assert_within(d(tail), tl, 1e-5 * np.ones(B), "tail")
    wl, wd, bad = lo.distill(d(z0), d(tv), d(ti).astype(int), d(tail), d(y).astype(int), d(w), T, float(np.float32(0.3)),
                             float(np.float32(0.7 * T * T)), 1.0 / B)
    assert not bad.any()
    assert_within(d(rows), wl, 1e-5 * np.abs(wl) + 1e-5, "loss rows")
    assert_within(d(z), wd, HALF[H] * np.abs(wd) + 2e-5 / B, "dz")
    assert abs(loss.item() - d(rows).mean()) < 1e-5 * abs(d(rows).mean())
    dz = d(z)
    assert_within(d(dx), dz @ d(ws), HALF[H] * np.abs(dz @ d(ws)) + 1.01 * sum_err(np.abs(dz) @ np.abs(d(ws)), C), "dx")
    assert_within(d(dw), dz.T @ d(xs), 1.01 * sum_err(np.abs(dz).T @ np.abs(d(xs)), B) + 8 * B / 16 * U32 * np.abs(dz).max(), "dw")
    assert_within(d(db), dz.sum(0), sum_err(np.abs(dz).sum(0), B), "db")


class ToyModel:
    """Logits from a table by the beam's last token and a running state: the state follows the beam, so that a wrong
    reordering changes every later step."""

    def __init__(self, rng, C, n):
        self.table = torch.from_numpy(rng.normal(size=(C, C)).astype(np.float32) * 2).to(DEV)
        self.mix = torch.from_numpy(rng.normal(size=(n, C)).astype(np.float32) * 0.3).to(DEV)
        self.embed = torch.from_numpy(rng.normal(size=(C, n)).astype(np.float32)).to(DEV)

    def step(self, tokens, states):
        new = 0.5 * states + self.embed[tokens.long()]
        return self.table[tokens.long()] + new @ self.mix, new


def test_beam_search_to_the_end():
    C, n, batch, W, steps, eos = 301, 24, 5, 4, 12, 7
    rng = np.random.default_rng(2)
    model = ToyModel(rng, C, n)
    start = torch.from_numpy(rng.integers(8, C, batch).astype(np.int32)).to(DEV)
    scores = torch.full((batch, W), -float("inf"), device=DEV)
    scores[:, 0] = 0
    done = torch.zeros(batch, W, dtype=torch.uint8, device=DEV)
    tokens = start[:, None].repeat(1, W).contiguous()
    states = torch.zeros(batch, W, n, device=DEV)
    history = torch.zeros(batch, W, steps, dtype=torch.int32, device=DEV)
    parents = torch.zeros(batch, W, dtype=torch.int32, device=DEV)
    nbytes = nn.mlp_op_beam_select_workspace_bytes(nn.F32, batch, W, C, W)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = lambda t: t.data_ptr()
    beams = None   # the oracle's: per batch entry a list of (score, tokens, ended)
    for t in range(steps):
        z, new = model.step(tokens.view(-1), states.view(batch * W, n))
        z = z.contiguous()
        states = new.view(batch, W, n).contiguous()
        zh = z.double().cpu().numpy().reshape(batch, W, C)
        # scores and done in place, states and histories in place
        nn.mlp_op_beam_select(nn.F32, batch, W, C, W, p(z), C, p(scores), p(done), eos, p(scores), p(parents), p(tokens),
                              p(done), p(ws), nbytes, stream())
        nn.mlp_op_beam_reorder(1, batch, W, W, 4 * n, p(states), 4 * n, 0, p(parents), W, p(states), 4 * n, 0, p(err), stream())
        nn.mlp_op_beam_reorder(1, batch, W, W, 4 * steps, p(history), 4 * steps, 0, p(parents), W, p(history), 4 * steps, 0,
                               p(err), stream())
        history[:, :, t] = tokens
        if beams is None:
            beams = [[(0.0 if w == 0 else -np.inf, [], False) for w in range(W)] for _ in range(batch)]
        for b in range(batch):
            sc = np.array([x[0] for x in beams[b]])
            dn = np.array([x[2] for x in beams[b]])
            wt, wp, wc, we = lo.beam_select(zh[b], sc, W, dn, eos)
            beams[b] = [(wt[j], beams[b][wp[j]][1] + [int(wc[j])], bool(we[j])) for j in range(W)]
            # the library's scores are rounded to fp32 every step; the choice is compared where it cannot matter
            assert parents[b].tolist() == wp.tolist() and tokens[b].tolist() == wc.tolist(), (t, b)
            assert done[b].tolist() == [int(x) for x in we]
    assert err.item() == 0
    got, s = history.cpu().numpy(), scores.cpu().numpy()
    for b in range(batch):
        for j in range(W):
            assert got[b, j].tolist() == beams[b][j][1]
            assert abs(s[b, j] - beams[b][j][0]) < 1e-4
    assert any(x[2] for e in beams for x in e) and len({tuple(r) for r in got[0].tolist()}) == W
