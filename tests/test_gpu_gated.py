"""The gated projection and its vector-Jacobian product against the fp64
oracle: types, activations, kept forms, ragged sizes, strides."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests.block_util import DEV, HALF, TDT, U32, Buf, assert_within, stream, sum_err

pytestmark = pytest.mark.gpu

NONE, RELU, GELU, SILU = nn.ACT_NONE, nn.ACT_RELU, nn.ACT_GELU_TANH, nn.ACT_SILU


# The relative bounds end where fp32's range does: e is clamped to 2^126 (so 1 / (1 + e) stops at 2^-126), the
# approximate exponential and reciprocal flush results below 2^-126 to zero, and bf16's steps are 2^-133 there.  With
# factors |g| <= 16, |u| <= 16 and |dh| <= 1 in these inputs each of the three moves a result by less than 2^-118.
TINY = 2.0 ** -118


def _gate_exponent(g, act):
    """|x| of the 2^x inside the activation: its rounding error grows with it."""
    if act == GELU:
        return np.minimum(np.abs(2.3022 * g * (1 + 0.044715 * g * g)), 130.0)
    return np.minimum(np.abs(1.4427 * g), 130.0) if act == SILU else np.zeros_like(g)


def _act_err(g, act):
    """Relative error of act(g) evaluated in fp32: 2^x from a rounded x (x ln2 steps), the approximate exponential
    and reciprocal (2 ulp each) and four multiplications."""
    return (12 + 4 * _gate_exponent(g, act)) * U32


def _check_kept8(q, e, s, ds, F):
    """Codes and scales of a checkpoint of s known to within ds: the scale is the smallest that holds some value in
    reach, and each value is within e4m3's rounding of one."""
    nb = -(-F // 32)
    for half in range(2):
        y = bo.q8_decode(q[:, half * F:(half + 1) * F], e[:, half * nb:(half + 1) * nb])
        v, d = s[:, half * F:(half + 1) * F], ds[:, half * F:(half + 1) * F]
        k = e[:, half * nb:(half + 1) * nb].astype(int) - 127
        pad = np.zeros((v.shape[0], nb * 32 - F))
        lo = np.concatenate([np.maximum(np.abs(v) - d, 0), pad], 1).reshape(v.shape[0], nb, 32).max(2)
        hi = np.concatenate([np.abs(v) + d, pad], 1).reshape(v.shape[0], nb, 32).max(2)
        assert np.all(lo <= 448.0 * 2.0 ** k) and np.all((hi > 448.0 * 2.0 ** (k - 1.0)) | (k == -120))
        kk = np.repeat(k, 32, axis=1)[:, :F].astype(float)
        assert_within(y, v, np.maximum(2.0 ** -4 * (np.abs(v) + d), 2.0 ** (kk - 10)) + d, "kept in 8 bits")


# M, F, K, pad of every leading dimension
BF16_SHAPES = [
    (1, 8, 8, 0), (1, 64, 64, 0), (1, 1000, 72, 8), (1, 4096, 1024, 0), (2, 136, 200, 0), (3, 264, 1000, 16),
    (7, 128, 64, 0), (8, 256, 512, 0), (9, 72, 128, 0), (16, 512, 256, 0), (17, 520, 264, 0), (31, 96, 1024, 0),
    (33, 1000, 200, 0), (64, 264, 264, 8), (65, 128, 8, 0), (100, 2056, 136, 0), (128, 136, 64, 0),
    (129, 256, 320, 0), (200, 120, 72, 0), (255, 384, 192, 24), (256, 128, 64, 0), (257, 264, 200, 0),
    (300, 1000, 1032, 0), (513, 640, 128, 0), (1000, 1096, 88, 0), (2048, 2560, 64, 0)]
F32_SHAPES = [(1, 1, 1, 0), (1, 100, 33, 0), (3, 7, 5, 2), (10, 64, 16, 0), (70, 65, 31, 1), (128, 64, 100, 0),
              (129, 130, 784, 0), (200, 333, 17, 3), (5, 1000, 257, 0)]
ACTS = [SILU, GELU, RELU, NONE]
SAVES = ["none", "full", "8bit"]
# every shape with one activation and kept form, rotating, and a small and a large one with all
FWD = [(nn.BF16, *s, ACTS[i % 4], i % 2 == 0, SAVES[i % 3]) for i, s in enumerate(BF16_SHAPES)]
FWD += [(nn.F32, *s, ACTS[(i + 1) % 4], i % 2 == 1, SAVES[(i + 1) % 3]) for i, s in enumerate(F32_SHAPES)]
FWD += [(nn.BF16, m, 264, 136, 0, a, True, sv) for m in (5, 40, 300) for a in ACTS for sv in SAVES]
FWD += [(nn.F32, 40, 100, 70, 0, a, True, sv) for a in ACTS for sv in SAVES]
BWD = [(nn.BF16, *s, ACTS[(i + 2) % 4], i % 2 == 0, SAVES[1 + i % 2]) for i, s in enumerate(BF16_SHAPES)]
BWD += [(nn.F32, *s, ACTS[i % 4], i % 2 == 1, SAVES[1 + i % 2]) for i, s in enumerate(F32_SHAPES)]
BWD += [(nn.BF16, m, 264, 136, 0, a, True, sv) for m in (5, 40, 300) for a in ACTS for sv in SAVES[1:]]
BWD += [(nn.F32, 40, 100, 70, 0, a, True, sv) for a in ACTS for sv in SAVES[1:]]
# fp32 tiles of every height (chosen by the number of tiles), reductions in one part and in several, in one chunk and in several
F32_HEIGHTS = [(5, 100, 2050), (300, 2000, 24), (383, 2047, 1030), (383, 4095, 20), (1000, 1000, 1040), (2500, 900, 24),
               (2500, 900, 1040), (4096, 1024, 16), (10000, 784, 20), (64, 512, 512), (200, 200, 200), (16, 256, 4000),
               (401, 1592, 1125), (1, 553, 1379)]
FWD += [(nn.F32, *s, 0, ACTS[i % 4], i % 2 == 0, SAVES[(i + 2) % 3]) for i, s in enumerate(F32_HEIGHTS)]
BWD += [(nn.F32, *s, 0, ACTS[(i + 1) % 4], i % 2 == 0, SAVES[1 + i % 2]) for i, s in enumerate(F32_HEIGHTS)]


def _rand(rng, shape, std, td):
    return torch.from_numpy((rng.normal(size=shape) * std).astype(np.float32)).to(td)


@pytest.mark.parametrize("dtype,M,F,K,pad,act,bias,save", FWD)
def test_forward(dtype, M, F, K, pad, act, bias, save):
    td = TDT[dtype]
    rng = np.random.default_rng([1, dtype, M, F, K, act])
    X = Buf(M, K, td, K + pad, 0, _rand(rng, (M, K), 1.0, td))
    W = Buf(2 * F, K, td, K + pad, 0, _rand(rng, (2 * F, K), 1.5 / np.sqrt(K), td))
    b = _rand(rng, (2 * F,), 0.3, torch.float32) if bias else None
    bd = b.to(DEV) if bias else None
    H = Buf(M, F, td, F + pad)
    nb = -(-F // 32)
    S = None if save == "none" else Buf(M, 2 * F, td if save == "full" else torch.uint8, 2 * F + pad)
    E = Buf(M, 2 * nb, torch.uint8, 2 * nb + pad) if save == "8bit" else None
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn.mlp_op_gated_linear(dtype, act, M, F, K, X.ptr, X.ld, W.ptr, W.ld, bd.data_ptr() if bias else None, H.ptr, H.ld,
                           S.ptr if S else None, S.ld if S else 0, E.ptr if E else None, E.ld if E else 0,
                           err.data_ptr(), stream())
    assert err.item() == 0
    x, w = X.np(), W.np()
    b64 = b.double().numpy() if bias else np.zeros(2 * F)
    h, s = bo.gated_linear(x, w, b64, act)
    ds = sum_err(np.abs(x) @ np.abs(w).T + np.abs(b64), K) + U32 * np.abs(s)
    g, u = s[:, :F], s[:, F:]
    a = bo.act(g, act)
    da = 1.13 * ds[:, :F] + np.abs(a) * _act_err(g, act)      # |act'| <= 1.13 for all four
    th = da * (np.abs(u) + ds[:, F:]) + np.abs(a) * ds[:, F:] + U32 * np.abs(h)
    assert_within(H.np(), h, th + HALF[dtype] * (np.abs(h) + th) + TINY, "h")
    if save == "full":
        assert_within(S.np(), s, ds + HALF[dtype] * (np.abs(s) + ds), "s")
    elif save == "8bit":
        _check_kept8(S.t.cpu().numpy(), E.t.cpu().numpy(), s, ds, F)
    for t in (H, S, E):
        if t is not None:
            t.check_canary()


@pytest.mark.parametrize("dtype,M,F,N,pad,act,want_h,save", BWD)
def test_backward(dtype, M, F, N, pad, act, want_h, save):
    td = TDT[dtype]
    rng = np.random.default_rng([2, dtype, M, F, N, act])
    dY = Buf(M, N, td, N + pad, 0, _rand(rng, (M, N), 1e-2, td))
    Wd = Buf(N, F, td, F + pad, 0, _rand(rng, (N, F), 1 / np.sqrt(F), td))
    pre = _rand(rng, (M, 2 * F), 2.0, td)
    nb, E = -(-F // 32), None
    if save == "full":
        S = Buf(M, 2 * F, td, 2 * F + pad, 0, pre)
        s = S.np()
    else:
        halves = [bo.q8_encode(pre[:, i * F:(i + 1) * F].double().numpy()) for i in range(2)]
        S = Buf(M, 2 * F, torch.uint8, 2 * F + pad, 0, torch.from_numpy(np.concatenate([halves[0][0], halves[1][0]], 1)))
        E = Buf(M, 2 * nb, torch.uint8, 2 * nb + pad, 0,
                torch.from_numpy(np.concatenate([halves[0][1], halves[1][1]], 1)))
        s = np.concatenate([bo.q8_decode(*halves[0]), bo.q8_decode(*halves[1])], 1)
    dS, H = Buf(M, 2 * F, td, 2 * F + pad), Buf(M, F, td, F + pad)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn.mlp_op_gated_dgrad(dtype, act, M, N, F, dY.ptr, dY.ld, Wd.ptr, Wd.ld, S.ptr, S.ld, E.ptr if E else None,
                          E.ld if E else 0, dS.ptr, dS.ld, H.ptr if want_h else None, H.ld if want_h else 0,
                          err.data_ptr(), stream())
    assert err.item() == 0
    dy, wd = dY.np(), Wd.np()
    dh = dy @ wd
    want, h = bo.gated_vjp(dh, s, act)
    tdh = sum_err(np.abs(dy) @ np.abs(wd), N)
    g, u = s[:, :F], s[:, F:]
    a, da = bo.act(g, act), bo.act_grad(g, act)
    ea = np.abs(a) * _act_err(g, act)
    # act' = s + (rest): the error of both terms, each at most 1.2 in size, relative to the larger
    eda = (24 + 8 * _gate_exponent(g, act)) * U32 * (np.abs(da) + np.minimum(np.abs(a), 1.2)) if act in (GELU, SILU) else 0.0
    tg = np.abs(u) * (tdh * (np.abs(da) + eda) + np.abs(dh) * eda) + 3 * U32 * np.abs(want[:, :F])
    tu = tdh * (np.abs(a) + ea) + np.abs(dh) * ea + 3 * U32 * np.abs(want[:, F:])
    t = np.concatenate([tg, tu], 1)
    assert_within(dS.np(), want, t + HALF[dtype] * (np.abs(want) + t) + TINY, "dS")
    if want_h:
        th = ea * np.abs(u) + 2 * U32 * np.abs(h)
        assert_within(H.np(), h, th + HALF[dtype] * (np.abs(h) + th) + TINY, "h")
    for b in (dS, H):
        b.check_canary()


def test_gradients_against_differences():
    """dS of the fp32 kernel against central differences of the fp64 formula."""
    M, N, F = 3, 20, 30
    rng = np.random.default_rng(4)
    dy, wd = rng.normal(size=(M, N)).astype(np.float32), rng.normal(size=(N, F)).astype(np.float32)
    s = rng.normal(size=(M, 2 * F)).astype(np.float32)
    for act in ACTS:
        dS = torch.empty(M, 2 * F, device=DEV)
        t = [torch.from_numpy(v).to(DEV) for v in (dy, wd, s)]
        nn.mlp_op_gated_dgrad(nn.F32, act, M, N, F, t[0].data_ptr(), N, t[1].data_ptr(), F, t[2].data_ptr(), 2 * F,
                              None, 0, dS.data_ptr(), 2 * F, None, 0, None, stream())
        dh = dy.astype(np.float64) @ wd.astype(np.float64)
        f = lambda z: (bo.act(z[:, :F], act) * z[:, F:] * dh).sum()   # noqa: E731
        d = rng.normal(size=s.shape)
        s64 = s.astype(np.float64)
        diff = (f(s64 + 1e-6 * d) - f(s64 - 1e-6 * d)) / 2e-6
        got = dS.double().cpu().numpy()
        assert abs((got * d).sum() - diff) < 256 * U32 * np.abs(got * d).sum() + 1e-7


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("act", ACTS)
def test_extreme_gates(M, act):
    """Gates far out in both tails stay finite, and a NaN or infinity in one
    token's row does not reach another's."""
    F, K = 128, 64
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = torch.linspace(-200, 200, M, device=DEV).bfloat16()
    x[M // 2, 5] = float("nan")
    w = torch.zeros(2 * F, K, dtype=torch.bfloat16, device=DEV)
    w[:F, 0], w[F:, 0] = 1.0, 0.5
    h, s = torch.empty(M, F, dtype=torch.bfloat16, device=DEV), torch.empty(M, 2 * F, dtype=torch.bfloat16, device=DEV)
    nn.mlp_op_gated_linear(nn.BF16, act, M, F, K, x.data_ptr(), K, w.data_ptr(), K, None, h.data_ptr(), F,
                           s.data_ptr(), 2 * F, None, 0, None, stream())
    rows = [m for m in range(M) if m != M // 2]
    g = x[rows, 0].double().cpu().numpy()[:, None]
    want = bo.act(g, act) * 0.5 * g
    assert np.abs(h[rows].double().cpu().numpy() - want).max() <= 2.0 ** -7 * np.abs(want).max()
    assert torch.isfinite(h[rows]).all() and torch.isnan(h[M // 2]).all()
    dy = torch.ones(M, 8, dtype=torch.bfloat16, device=DEV)
    wd = torch.ones(8, F, dtype=torch.bfloat16, device=DEV)
    ds = torch.empty_like(s)
    nn.mlp_op_gated_dgrad(nn.BF16, act, M, 8, F, dy.data_ptr(), 8, wd.data_ptr(), F, s.data_ptr(), 2 * F, None, 0,
                          ds.data_ptr(), 2 * F, h.data_ptr(), F, None, stream())
    assert torch.isfinite(ds[rows]).all() and torch.isfinite(h[rows]).all()
    want, _ = bo.gated_vjp(np.full((M - 1, F), 8.0), s[rows].double().cpu().numpy(), act)
    assert np.abs(ds[rows].double().cpu().numpy() - want).max() <= 2.0 ** -7 * np.abs(want).max()


@pytest.mark.parametrize("dtype,M", [(nn.F32, 50), (nn.BF16, 1), (nn.BF16, 20), (nn.BF16, 700)])
def test_captured_repeated_and_on_other_streams(dtype, M):
    """Forward and backward captured and replayed on new inputs, repeated, and
    on two streams at once: always the eager result, bit for bit."""
    F, K, td = 520, 264, TDT[dtype]
    rng = np.random.default_rng([8, dtype, M])

    def state():
        z = lambda *s, d=td: torch.empty(*s, dtype=d, device=DEV)   # noqa: E731
        return dict(x=z(M, K), w=_rand(rng, (2 * F, K), 0.06, td).to(DEV), h=z(M, F), s=z(M, 2 * F, d=torch.uint8),
                    e=z(M, 2 * 17, d=torch.uint8), dy=z(M, K), wd=_rand(rng, (K, F), 0.05, td).to(DEV), ds=z(M, 2 * F),
                    h2=z(M, F))

    def fill(s):
        s["x"].copy_(_rand(rng, (M, K), 1.0, td))
        s["dy"].copy_(_rand(rng, (M, K), 1.0, td))

    def call(s):
        p = {k: v.data_ptr() for k, v in s.items()}
        nn.mlp_op_gated_linear(dtype, SILU, M, F, K, p["x"], K, p["w"], K, None, p["h"], F, p["s"], 2 * F, p["e"], 34,
                               None, stream())
        nn.mlp_op_gated_dgrad(dtype, SILU, M, K, F, p["dy"], K, p["wd"], F, p["s"], 2 * F, p["e"], 34, p["ds"], 2 * F,
                              p["h2"], F, None, stream())

    outs = ("h", "s", "e", "ds", "h2")
    a, b = state(), state()
    fill(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a)
    for _ in range(2):
        fill(a)
        graph.replay()
        got = {k: a[k].clone() for k in outs}
        call(a)
        assert all(torch.equal(got[k], a[k]) for k in outs)
    fill(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            call(a)
        with torch.cuda.stream(s2):
            call(b)
    torch.cuda.synchronize()
    for s in (a, b):
        got = {k: s[k].clone() for k in outs}
        call(s)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], s[k]) for k in outs)
