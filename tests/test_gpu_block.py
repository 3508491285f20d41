"""The feed-forward block as a program runs it: layer norm, gated projection
that keeps its pre-activations (in the dtype or in 8 bits), down projection;
and back: through the gate, the projections' gradients, the norm.  In fp32
end to end against the fp64 oracle and central differences; in bf16 stage by
stage, each against the oracle applied to what that stage read; captured."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests.block_util import DEV, HALF, TDT, U32, assert_within, stream, sum_err

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-5))


class Block:
    """Buffers and calls of one block: y = Wd (act(n Wg^T + bg) * (n Wu^T + bu)), n = layer norm of x."""

    def __init__(self, dtype, M, D, F, act, keep8, seed):
        td = TDT[dtype]
        self.dtype, self.M, self.D, self.F, self.act, self.keep8 = dtype, M, D, F, act, keep8
        rng = np.random.default_rng([seed, dtype, M, D, F])

        def put(shape, std, d=td):
            return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).to(d).to(DEV)

        f32, u8 = torch.float32, torch.uint8
        z = lambda *s, d=td: torch.empty(*s, dtype=d, device=DEV)   # noqa: E731
        self.x, self.dy = put((M, D), 2.0), put((M, D), 1e-2)
        self.gamma, self.beta = put((D,), 0.3, f32) + 1, put((D,), 0.3, f32)
        self.w, self.b = put((2 * F, D), 1 / np.sqrt(D)), put((2 * F,), 0.2, f32)
        self.wd, self.bd = put((D, F), 1 / np.sqrt(F)), torch.zeros(D, device=DEV)
        self.n, self.mean, self.rstd, self.h, self.y = z(M, D), z(M, d=f32), z(M, d=f32), z(M, F), z(M, D)
        self.nb, self.kb = -(-F // 32), -(-D // 32)
        self.s = z(M, 2 * F, d=u8) if keep8 else z(M, 2 * F)
        self.se = z(M, 2 * self.nb, d=u8) if keep8 else None
        self.nq, self.ne = z(M, D, d=u8), z(M, self.kb, d=u8)
        self.ds, self.h2, self.dn, self.dx = z(M, 2 * F), z(M, F), z(M, D), z(M, D)
        self.dw, self.db, self.dwd = z(2 * F, D, d=f32), z(2 * F, d=f32), z(D, F, d=f32)
        self.dgamma, self.dbeta = z(D, d=f32), z(D, d=f32)
        self.n_wd = nn.mlp_op_wgrad_workspace_bytes(dtype, D, F, M)
        self.n_w = (nn.mlp_op_wgrad8_workspace_bytes if keep8 else nn.mlp_op_wgrad_workspace_bytes)(dtype, 2 * F, D, M)
        self.n_ln = nn.mlp_op_layernorm_backward_workspace_bytes(dtype, M, D)
        self.ws = z(max(self.n_wd, self.n_w, self.n_ln, 16), d=u8)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def forward(self):
        M, D, F, dt, st = self.M, self.D, self.F, self.dtype, stream()
        p = lambda t: None if t is None else t.data_ptr()   # noqa: E731
        nn.mlp_op_layernorm(dt, M, D, p(self.x), D, p(self.gamma), p(self.beta), EPS, p(self.n), D, p(self.mean),
                            p(self.rstd), st)
        nn.mlp_op_gated_linear(dt, self.act, M, F, D, p(self.n), D, p(self.w), D, p(self.b), p(self.h), F, p(self.s),
                               2 * F, p(self.se), 2 * self.nb, p(self.err), st)
        if self.keep8:
            nn.mlp_op_quant8(dt, M, D, p(self.n), D, p(self.nq), D, p(self.ne), self.kb, st)
        nn.mlp_op_linear_act(dt, nn.ACT_NONE, M, D, F, p(self.h), F, p(self.wd), F, p(self.bd), p(self.y), D, None, 0,
                             p(self.err), st)

    def backward(self):
        M, D, F, dt, st = self.M, self.D, self.F, self.dtype, stream()
        p = lambda t: None if t is None else t.data_ptr()   # noqa: E731
        nn.mlp_op_gated_dgrad(dt, self.act, M, D, F, p(self.dy), D, p(self.wd), F, p(self.s), 2 * F, p(self.se),
                              2 * self.nb, p(self.ds), 2 * F, p(self.h2), F, p(self.err), st)
        nn.mlp_op_wgrad(dt, D, F, M, p(self.dy), D, p(self.h2), F, p(self.dwd), F, None, p(self.ws), self.n_wd,
                        p(self.err), st)
        nn.mlp_op_dgrad(dt, nn.ACT_NONE, M, 2 * F, D, p(self.ds), 2 * F, p(self.w), D, None, 0, p(self.dn), D,
                        p(self.err), st)
        if self.keep8:
            nn.mlp_op_wgrad8(dt, 2 * F, D, M, p(self.ds), 2 * F, p(self.nq), D, p(self.ne), self.kb, p(self.dw), D,
                             p(self.db), p(self.ws), self.n_w, p(self.err), st)
        else:
            nn.mlp_op_wgrad(dt, 2 * F, D, M, p(self.ds), 2 * F, p(self.n), D, p(self.dw), D, p(self.db), p(self.ws),
                            self.n_w, p(self.err), st)
        nn.mlp_op_layernorm_backward(dt, M, D, p(self.dn), D, p(self.x), D, p(self.gamma), p(self.mean), p(self.rstd),
                                     p(self.dx), D, p(self.dgamma), p(self.dbeta), p(self.ws), self.n_ln, st)

    OUT = ("n", "mean", "rstd", "h", "y", "s", "ds", "h2", "dn", "dx", "dw", "db", "dwd", "dgamma", "dbeta")


def _64(t):
    return t.double().cpu().numpy()


def _oracle(x, gamma, beta, w, b, wd, act):
    n, mean, rstd = bo.layer_norm(x, gamma, beta, EPS)
    h, s = bo.gated_linear(n, w, b, act)
    return n, mean, rstd, h, s, h @ wd.T


@pytest.mark.parametrize("act", [nn.ACT_SILU, nn.ACT_GELU_TANH])
def test_fp32_end_to_end(act):
    k = Block(nn.F32, 60, 48, 72, act, False, 1)
    k.forward()
    k.backward()
    assert k.err.item() == 0
    x, dy, gamma, beta, w, b, wd = (_64(t) for t in (k.x, k.dy, k.gamma, k.beta, k.w, k.b, k.wd))
    n, mean, rstd, h, s, y = _oracle(x, gamma, beta, w, b, wd, act)
    ds, _ = bo.gated_vjp(dy @ wd, s, act)
    dn = ds @ w
    dx, dg, dbt = bo.layer_norm_vjp(dn, x, mean, rstd, gamma)
    want = dict(n=n, h=h, s=s, y=y, ds=ds, dn=dn, dx=dx, dw=ds.T @ n, db=ds.sum(0), dwd=dy.T @ h, dgamma=dg, dbeta=dbt)
    for name, v in want.items():
        got = _64(getattr(k, name))
        # a chain of at most five sums of up to 144 terms, each 1e-6 of its absolute sum at most, whose results are
        # a tenth of that sum (random signs): 1e-5 of the largest value
        assert np.abs(got - v).max() <= 1e-5 * np.abs(v).max() + 1e-9, (name, np.abs(got - v).max(), np.abs(v).max())
    # the gradients are those of sum(y * dy): central differences in random directions
    rng = np.random.default_rng(5)
    args = dict(x=x, gamma=gamma, beta=beta, w=w, b=b, wd=wd)
    for name, grad in (("x", k.dx), ("gamma", k.dgamma), ("beta", k.dbeta), ("w", k.dw), ("b", k.db), ("wd", k.dwd)):
        d = rng.normal(size=args[name].shape)
        f = lambda e: (_oracle(**{**args, name: args[name] + e * d}, act=act)[5] * dy).sum()   # noqa: E731,B023
        diff = (f(1e-6) - f(-1e-6)) / 2e-6
        g = _64(grad)
        assert abs((g * d).sum() - diff) < 1e-5 * np.abs(g * d).sum() + 1e-7, name


@pytest.mark.parametrize("M,D,F,act,keep8", [
    (1, 64, 128, nn.ACT_SILU, False), (37, 72, 136, nn.ACT_GELU_TANH, True), (300, 264, 520, nn.ACT_SILU, True),
    (700, 512, 1000, nn.ACT_RELU, False), (260, 256, 264, nn.ACT_NONE, True)])
def test_bf16_stage_by_stage(M, D, F, act, keep8):
    k = Block(nn.BF16, M, D, F, act, keep8, 2)
    k.forward()
    k.backward()
    assert k.err.item() == 0
    half = HALF[nn.BF16]
    g = {name: _64(getattr(k, name)) for name in Block.OUT if name != "s"}
    x, dy, gamma, beta, w, b, wd = (_64(t) for t in (k.x, k.dy, k.gamma, k.beta, k.w, k.b, k.wd))

    def close(got, want, absum, n, what, rounded=True):
        t = sum_err(absum, n)
        assert_within(got, want, t + half * (np.abs(want) + t) * rounded + 2.0 ** -118, what)

    n, mean, rstd = bo.layer_norm(x, gamma, beta, EPS)
    close(g["n"], n, np.abs(n) + np.abs(gamma) * 8, D, "n")
    h, s = bo.gated_linear(g["n"], w, b, act)
    absum = np.abs(g["n"]) @ np.abs(w).T + np.abs(b)
    hs = (1.13 * absum[:, :F] + np.abs(bo.act(s[:, :F], act))) * (np.abs(s[:, F:]) + 1e-3 * absum[:, F:])
    hs += np.abs(bo.act(s[:, :F], act)) * absum[:, F:]
    close(g["h"], h, hs, D, "h")
    if keep8:
        q, e = k.s.cpu().numpy(), k.se.cpu().numpy()
        kept = np.concatenate([bo.q8_decode(q[:, :F], e[:, :k.nb]), bo.q8_decode(q[:, F:], e[:, k.nb:])], 1)
        top = np.abs(s).reshape(M, 2 * F).max()
        assert_within(kept, s, 2.0 ** -4 * (np.abs(s) + sum_err(absum, D)) + sum_err(absum, D) + 2.0 ** -17 * top, "s in 8 bits")
        nq, ne = bo.q8_encode(g["n"])
        assert np.array_equal(k.nq.cpu().numpy(), nq) and np.array_equal(k.ne.cpu().numpy(), ne)
        nk = bo.q8_decode(nq, ne)
    else:
        kept, nk = _64(k.s), g["n"]
        close(kept, s, absum, D, "s")
    close(g["y"], g["h"] @ wd.T, np.abs(g["h"]) @ np.abs(wd).T, F, "y")
    dh = dy @ wd
    ds, h2 = bo.gated_vjp(dh, kept, act)
    a, da = np.abs(bo.act(kept[:, :F], act)), np.abs(bo.act_grad(kept[:, :F], act))
    sc = np.concatenate([np.abs(kept[:, F:]) * (da + 0.01), a + 0.01], 1)
    close(g["ds"], ds, np.tile(np.abs(dy) @ np.abs(wd), (1, 2)) * sc, max(D, 256), "ds")
    close(g["h2"], h2, 32 * (a + 1e-3) * np.abs(kept[:, F:]), 1, "h2")
    close(g["dwd"], dy.T @ g["h2"], np.abs(dy).T @ np.abs(g["h2"]), M, "dwd", rounded=False)
    close(g["dn"], g["ds"] @ w, np.abs(g["ds"]) @ np.abs(w), 2 * F, "dn")
    close(g["dw"], g["ds"].T @ nk, np.abs(g["ds"]).T @ np.abs(nk), M, "dw", rounded=False)
    close(g["db"], g["ds"].sum(0), np.abs(g["ds"]).sum(0), M, "db", rounded=False)
    mu, r = g["mean"], g["rstd"]
    dx, dg, dbt = bo.layer_norm_vjp(g["dn"], x, mu, r, gamma)
    xh = np.abs((x - mu[:, None]) * r[:, None])
    dna = np.abs(g["dn"] * gamma)
    close(g["dx"], dx, r[:, None] * (dna + dna.mean(1, keepdims=True) + xh * (dna * xh).mean(1, keepdims=True)), D, "dx")
    close(g["dgamma"], dg, (np.abs(g["dn"]) * xh).sum(0), M, "dgamma", rounded=False)
    close(g["dbeta"], dbt, np.abs(g["dn"]).sum(0), M, "dbeta", rounded=False)


@pytest.mark.parametrize("dtype,M,keep8", [(nn.BF16, 1, False), (nn.BF16, 515, True), (nn.F32, 40, True)])
def test_block_captured(dtype, M, keep8):
    """Forward and backward as one graph, replayed on new inputs: what the
    eager calls give, bit for bit."""
    k = Block(dtype, M, 264, 520, nn.ACT_SILU, keep8, 3)
    rng = np.random.default_rng([4, M])
    k.forward()
    k.backward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k.forward()
        k.backward()
    for _ in range(2):
        k.x.copy_(torch.from_numpy(rng.normal(size=(M, 264)).astype(np.float32)))
        k.dy.copy_(torch.from_numpy(rng.normal(size=(M, 264)).astype(np.float32)))
        graph.replay()
        got = {name: getattr(k, name).clone() for name in Block.OUT}
        k.forward()
        k.backward()
        for name, t in got.items():
            assert torch.equal(t, getattr(k, name)), name
    assert k.err.item() == 0
