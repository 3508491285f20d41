"""Workloads of the layer-norm, gated feed-forward and 8-bit checkpoint operations.

Each case is one call chain a training or serving program makes between two
residual additions: layer norm (forward, backward), the gated projection
H = act(X Wg^T + bg) * (X Wu^T + bu) (forward, backward), and activations kept
in 8 bits between the two (e4m3 codes with one power-of-two scale per row and
32 columns).  `run` computes a case from elementary torch operations, or, with
`own` set, through the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32          # columns that share one scale
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token's residual stream before a block: latency only
        {"name": "ln_fwd_token", "kind": "ln_fwd", "dtype": "bf16", "M": 1, "D": 1024},
        # a training batch of 64 Ki tokens at the LM block's width
        {"name": "ln_fwd_64k", "kind": "ln_fwd", "dtype": "bf16", "M": 65536, "D": 1024},
        # backward of a wide norm with the gradients of scale and shift
        {"name": "ln_bwd_16k_wide", "kind": "ln_bwd", "dtype": "bf16", "M": 16384, "D": 4096},
        # fp32 training with a width that is no power of two, few rows
        {"name": "ln_bwd_f32_odd", "kind": "ln_bwd", "dtype": "f32", "M": 777, "D": 1000},
        # decoding: one token through the gated projection, nothing kept for a backward pass
        {"name": "gated_fwd_token", "kind": "gated_fwd", "dtype": "bf16", "act": "silu", "M": 1, "F": 4096,
         "K": 1024, "bias": False, "save": "none"},
        # training forward at the LM block's sizes, pre-activations kept in bf16
        {"name": "gated_fwd_16k", "kind": "gated_fwd", "dtype": "bf16", "act": "gelu", "M": 16384, "F": 4096,
         "K": 1024, "bias": True, "save": "full"},
        # fp32 model with MNIST-shaped inputs and a ragged batch
        {"name": "gated_fwd_f32", "kind": "gated_fwd", "dtype": "f32", "act": "relu", "M": 1000, "F": 1000,
         "K": 784, "bias": True, "save": "full"},
        # training backward at the LM block's sizes
        {"name": "gated_bwd_16k", "kind": "gated_bwd", "dtype": "bf16", "act": "gelu", "M": 16384, "N": 1024,
         "F": 4096, "K": 1024, "save": "full"},
        # training forward that keeps its pre-activations in 8 bits
        {"name": "gated_fwd_8bit", "kind": "gated_fwd", "dtype": "bf16", "act": "silu", "M": 8192, "F": 4096,
         "K": 1024, "bias": False, "save": "8bit"},
        # backward from 8-bit pre-activations, ragged tokens and widths
        {"name": "gated_bwd_8bit_odd", "kind": "gated_bwd", "dtype": "bf16", "act": "silu", "M": 5003, "N": 1000,
         "F": 2728, "K": 1000, "save": "8bit"},
        # a layer's input kept in 8 bits and read back
        {"name": "ckpt_round_trip", "kind": "ckpt", "dtype": "bf16", "M": 16384, "K": 4096},
        # the gated weights' gradient from an 8-bit checkpoint of the block's input
        {"name": "wgrad_8bit", "kind": "wgrad", "dtype": "bf16", "N": 8192, "K": 1024, "B": 8192},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(v, m):
    return max(m, v // m * m)


def draw(rng):
    kind = rng.choice(["ln_fwd", "ln_bwd", "gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd", "ckpt", "wgrad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("ln_fwd", "ln_bwd"):
        D = _logint(rng, 16, 8192)
        if rng.random() < 0.5:
            D = _mult(D, 8)
        return {"kind": kind, "dtype": dtype, "M": min(_logint(rng, 1, 65536), (1 << 26) // D), "D": D}
    if kind == "ckpt":
        K = _logint(rng, 16, 8192)
        return {"kind": kind, "dtype": dtype, "M": min(_logint(rng, 1, 65536), (1 << 26) // K), "K": K}
    # the products: bf16 widths are multiples of 8 (16-byte rows), fp32 ones any
    step = 8 if dtype == "bf16" else 1
    F = _mult(_logint(rng, 64, 6144), step)
    K = _mult(_logint(rng, 64, 4096), step)
    # fp32 products are at most a hundredth of the largest bf16 ones
    most = (1 << 36) if dtype == "bf16" else (1 << 30)
    if kind == "wgrad":
        N = _mult(_logint(rng, 64, 8192), step)
        return {"kind": kind, "dtype": dtype, "N": N, "K": K, "B": max(1, min(_logint(rng, 1, 8192), most // (N * K)))}
    act = rng.choice(["none", "relu", "gelu", "silu"])
    if kind == "gated_fwd":
        return {"kind": kind, "dtype": dtype, "act": act, "M": max(1, min(_logint(rng, 1, 16384), most // (F * K))),
                "F": F, "K": K, "bias": rng.random() < 0.5, "save": rng.choice(["none", "full", "8bit"])}
    N = _mult(_logint(rng, 64, 4096), step)
    return {"kind": kind, "dtype": dtype, "act": act, "M": max(1, min(_logint(rng, 1, 16384), most // (F * (N + K)))),
            "N": N, "F": F, "K": K, "save": rng.choice(["full", "8bit"])}


# ---- inputs ------------------------------------------------------------------
def _normal(gen, shape, std, td=torch.float32):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(td)


def _codes(x):
    """Codes and scale exponents (k + 127) of x, as a program finds them in a stored checkpoint."""
    rows, cols = x.shape
    pad = -cols % BLOCK
    b = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, BLOCK)
    m, e = torch.frexp(b.abs().amax(2))
    k = (e - 9 + (m > 0.875).int()).clamp_min(-120)
    k = torch.where(m == 0, torch.full_like(k, -120), k)
    q = torch.ldexp(b, -k[..., None]).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return q.view(torch.uint8).contiguous(), (k + 127).to(torch.uint8)


def _stream_rows(gen, M, D, td):
    # a residual stream: rows of different scale and offset, a few columns that stand out
    x = torch.randn((M, D), generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn((M, 1), generator=gen, device=DEV))
    x += 0.3 * torch.randn((M, 1), generator=gen, device=DEV)
    x *= torch.exp(0.7 * torch.randn((D,), generator=gen, device=DEV))
    return x.to(td)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind, td = case["kind"], TD[case["dtype"]]
    s = dict(case)
    s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if kind in ("ln_fwd", "ln_bwd"):
        M, D = case["M"], case["D"]
        s["eps"] = 1e-5
        s["x"] = _stream_rows(gen, M, D, td)
        s["gamma"] = 1.0 + _normal(gen, (D,), 0.2)
        s["beta"] = _normal(gen, (D,), 0.2)
        s["y"] = torch.empty((M, D), dtype=td, device=DEV)
        s["mean"] = torch.empty(M, dtype=torch.float32, device=DEV)
        s["rstd"] = torch.empty(M, dtype=torch.float32, device=DEV)
        if kind == "ln_bwd":
            s["dy"] = _normal(gen, (M, D), 1e-2, td)
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + s["eps"]).rsqrt().float()
            s["dx"] = torch.empty_like(s["x"])
            s["dgamma"] = torch.empty(D, dtype=torch.float32, device=DEV)
            s["dbeta"] = torch.empty(D, dtype=torch.float32, device=DEV)
    elif kind == "gated_fwd":
        M, F, K = case["M"], case["F"], case["K"]
        s["x"] = _normal(gen, (M, K), 1.0, td)
        s["w"] = _normal(gen, (2 * F, K), 1.0 / math.sqrt(K), td)
        s["b"] = _normal(gen, (2 * F,), 0.1) if case["bias"] else None
        s["h"] = torch.empty((M, F), dtype=td, device=DEV)
        if case["save"] == "full":
            s["s"] = torch.empty((M, 2 * F), dtype=td, device=DEV)
        elif case["save"] == "8bit":
            s["q"] = torch.empty((M, 2 * F), dtype=torch.uint8, device=DEV)
            s["e"] = torch.empty((M, 2 * (-(-F // BLOCK))), dtype=torch.uint8, device=DEV)
            s["s"] = torch.empty((M, 2 * F), dtype=td, device=DEV)
    elif kind == "gated_bwd":
        M, N, F, K = case["M"], case["N"], case["F"], case["K"]
        s["dy"] = _normal(gen, (M, N), 1e-3, td)
        s["wd"] = _normal(gen, (N, F), 1.0 / math.sqrt(F), td)
        s["w"] = _normal(gen, (2 * F, K), 1.0 / math.sqrt(K), td)
        pre = _normal(gen, (M, 2 * F), 1.0, td)
        if case["save"] == "full":
            s["s"] = pre
        else:
            (qg, eg), (qu, eu) = _codes(pre[:, :F]), _codes(pre[:, F:])
            s["q"], s["e"] = torch.cat([qg, qu], 1), torch.cat([eg, eu], 1)
        s["ds"] = torch.empty((M, 2 * F), dtype=td, device=DEV)
        s["h"] = torch.empty((M, F), dtype=td, device=DEV)
        s["dx"] = torch.empty((M, K), dtype=td, device=DEV)
    elif kind == "ckpt":
        M, K = case["M"], case["K"]
        s["x"] = _stream_rows(gen, M, K, td)
        s["q"] = torch.empty((M, K), dtype=torch.uint8, device=DEV)
        s["e"] = torch.empty((M, -(-K // BLOCK)), dtype=torch.uint8, device=DEV)
        s["y"] = torch.empty_like(s["x"])
    else:
        N, K, B = case["N"], case["K"], case["B"]
        s["dy"] = _normal(gen, (B, N), 1e-3, td)
        s["q"], s["e"] = _codes(_normal(gen, (B, K), 1.0, td))
        s["dw"] = torch.empty((N, K), dtype=torch.float32, device=DEV)
        s["db"] = torch.empty(N, dtype=torch.float32, device=DEV)
    return s


# ---- the plain form ----------------------------------------------------------
def _values(q, e):
    """The values that codes q and scale exponents e stand for, in fp32."""
    k = (e.int() - 127).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return torch.ldexp(q.view(torch.float8_e4m3fn).float(), k)


def _act(g, act):
    if act == "relu":
        return g.clamp_min(0)
    if act == "gelu":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return g


def _act_grad(g, act):
    if act == "relu":
        return (g > 0).to(g.dtype)
    if act == "gelu":
        t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return p * (1 + g * (1 - p))
    return torch.ones_like(g)


def _stored(s):
    """The saved pre-activations [M, 2F] in fp32."""
    if s["save"] == "full":
        return s["s"].float()
    F, ne = s["F"], s["e"].shape[1] // 2
    return torch.cat([_values(s["q"][:, :F].contiguous(), s["e"][:, :ne]),
                      _values(s["q"][:, F:].contiguous(), s["e"][:, ne:])], 1)


def _plain(s):
    kind, td = s["kind"], TD[s["dtype"]]
    if kind == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + s["eps"])
        return {"y": (d * rstd * s["gamma"] + s["beta"]).to(td), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if kind == "ln_bwd":
        dy = s["dy"].float()
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        gy = dy * s["gamma"]
        dx = s["rstd"][:, None] * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
        return {"dx": dx.to(td), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
    if kind == "gated_fwd":
        F = s["F"]
        pre = s["x"].float() @ s["w"].float().T
        if s["b"] is not None:
            pre = pre + s["b"]
        out = {"h": (_act(pre[:, :F], s["act"]) * pre[:, F:]).to(td)}
        if s["save"] == "full":
            out["s"] = pre.to(td)
        elif s["save"] == "8bit":
            out["s"] = torch.cat([_values(*_codes(pre[:, :F])), _values(*_codes(pre[:, F:]))], 1).to(td)
        return out
    if kind == "gated_bwd":
        F = s["F"]
        pre = _stored(s)
        g, u = pre[:, :F], pre[:, F:]
        dh = s["dy"].float() @ s["wd"].float()
        a = _act(g, s["act"])
        ds = torch.cat([dh * u * _act_grad(g, s["act"]), dh * a], 1)
        return {"ds": ds.to(td), "h": (a * u).to(td), "dx": (ds @ s["w"].float()).to(td)}
    if kind == "ckpt":
        return {"y": _values(*_codes(s["x"])).to(td)}
    dy = s["dy"].float()
    return {"dw": dy.T @ _values(s["q"], s["e"]), "db": dy.sum(0)}


# ---- the library's calls -------------------------------------------------------
def _own(s):
    import neural_net_step_gb300 as nn
    kind = s["kind"]
    st = torch.cuda.current_stream().cuda_stream
    dt = nn.BF16 if s["dtype"] == "bf16" else nn.F32
    err = s["err"].data_ptr()
    if kind == "ln_fwd":
        M, D = s["M"], s["D"]
        nn.mlp_op_layernorm(dt, M, D, s["x"].data_ptr(), D, s["gamma"].data_ptr(), s["beta"].data_ptr(), s["eps"],
                            s["y"].data_ptr(), D, s["mean"].data_ptr(), s["rstd"].data_ptr(), st)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if kind == "ln_bwd":
        M, D = s["M"], s["D"]
        n = nn.mlp_op_layernorm_backward_workspace_bytes(dt, M, D)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        nn.mlp_op_layernorm_backward(dt, M, D, s["dy"].data_ptr(), D, s["x"].data_ptr(), D, s["gamma"].data_ptr(),
                                     s["mean"].data_ptr(), s["rstd"].data_ptr(), s["dx"].data_ptr(), D,
                                     s["dgamma"].data_ptr(), s["dbeta"].data_ptr(), ws.data_ptr(), n, st)
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if kind == "ckpt":
        M, K, ne = s["M"], s["K"], s["e"].shape[1]
        nn.mlp_op_quant8(dt, M, K, s["x"].data_ptr(), K, s["q"].data_ptr(), K, s["e"].data_ptr(), ne, st)
        nn.mlp_op_dequant8(dt, M, K, s["q"].data_ptr(), K, s["e"].data_ptr(), ne, s["y"].data_ptr(), K, st)
        return {"y": s["y"]}
    if kind == "wgrad":
        N, K, B, ne = s["N"], s["K"], s["B"], s["e"].shape[1]
        n = nn.mlp_op_wgrad8_workspace_bytes(dt, N, K, B)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        nn.mlp_op_wgrad8(dt, N, K, B, s["dy"].data_ptr(), N, s["q"].data_ptr(), K, s["e"].data_ptr(), ne,
                         s["dw"].data_ptr(), K, s["db"].data_ptr(), ws.data_ptr(), n, err, st)
        return {"dw": s["dw"], "db": s["db"]}
    act = {"none": nn.ACT_NONE, "relu": nn.ACT_RELU, "gelu": nn.ACT_GELU_TANH, "silu": nn.ACT_SILU}[s["act"]]
    M, F, K = s["M"], s["F"], s["K"]
    q8 = s["save"] == "8bit"
    ne = s["e"].shape[1] // 2 if q8 else 0
    kept = s["q"] if q8 else s.get("s")
    kp, ep = kept.data_ptr() if kept is not None else None, s["e"].data_ptr() if q8 else None
    if kind == "gated_fwd":
        b = s["b"].data_ptr() if s["b"] is not None else None
        nn.mlp_op_gated_linear(dt, act, M, F, K, s["x"].data_ptr(), K, s["w"].data_ptr(), K, b, s["h"].data_ptr(), F,
                               kp, 2 * F, ep, 2 * ne, err, st)
        out = {"h": s["h"]}
        if q8:   # the two halves of the checkpoint, read back as the values they stand for
            es, v = s["s"].element_size(), s["s"].data_ptr()
            nn.mlp_op_dequant8(dt, M, F, kp, 2 * F, ep, 2 * ne, v, 2 * F, st)
            nn.mlp_op_dequant8(dt, M, F, kp + F, 2 * F, ep + ne, 2 * ne, v + F * es, 2 * F, st)
        if kept is not None:
            out["s"] = s["s"]
        return out
    N = s["N"]
    nn.mlp_op_gated_dgrad(dt, act, M, N, F, s["dy"].data_ptr(), N, s["wd"].data_ptr(), F, kp, 2 * F, ep, 2 * ne,
                          s["ds"].data_ptr(), 2 * F, s["h"].data_ptr(), F, err, st)
    nn.mlp_op_dgrad(dt, nn.ACT_NONE, M, 2 * F, K, s["ds"].data_ptr(), 2 * F, s["w"].data_ptr(), K, None, 0,
                    s["dx"].data_ptr(), K, err, st)
    return {"ds": s["ds"], "h": s["h"], "dx": s["dx"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- work ----------------------------------------------------------------------
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if kind == "ln_fwd":
        M, D = case["M"], case["D"]
        return {"bytes": 2 * es * M * D + 8 * D + 8 * M, "flops": 8 * M * D}
    if kind == "ln_bwd":
        M, D = case["M"], case["D"]
        return {"bytes": 3 * es * M * D + 12 * D + 8 * M, "flops": 14 * M * D}
    if kind == "ckpt":
        M, K = case["M"], case["K"]
        return {"bytes": 2 * (es * M * K + M * K + M * -(-K // BLOCK)), "flops": 4 * M * K}
    if kind == "wgrad":
        N, K, B = case["N"], case["K"], case["B"]
        return {"bytes": es * B * N + B * K + B * -(-K // BLOCK) + 4 * N * K + 4 * N, "flops": 2 * N * K * B}
    M, F, K = case["M"], case["F"], case["K"]
    s8 = 2 * M * F + 2 * M * -(-F // BLOCK)
    if kind == "gated_fwd":
        # the 8-bit case also reads its checkpoint back as values
        kept = {"none": 0, "full": 2 * es * M * F, "8bit": 2 * s8 + 2 * es * M * F}[case["save"]]
        return {"bytes": es * (M * K + 2 * F * K + M * F) + (8 * F if case["bias"] else 0) + kept,
                "flops": 4 * M * F * K}
    N = case["N"]
    kept = 2 * es * M * F if case["save"] == "full" else s8
    # dS is written by one operator and read by the next
    return {"bytes": es * (M * N + N * F + 2 * F * K + 4 * M * F + M * F + M * K) + kept,
            "flops": 2 * M * N * F + 4 * M * F * K}


# ---- the definition in 64 bits ---------------------------------------------------
def _round_e4m3(v):
    """v (64 bits, |v| <= 448) to the nearest multiple of its step, ties to even: 3 bits after the leading one, and
    multiples of 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(-6, 8).double() - 3)
    return torch.round(v / step) * step


def _kept8(v):
    """What an 8-bit checkpoint of v (64 bits) stands for: per row and 32 columns the smallest scale 2^k, k >= -120,
    with every |v| <= 448 * 2^k."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], BLOCK):
        b = v[:, c:c + BLOCK]
        top = b.abs().amax(1, keepdim=True)
        k = torch.ceil(torch.log2(top / 448)).clamp(-120, 120)
        k = torch.where(top > 448 * torch.exp2(k), k + 1, k)
        k = torch.where((top <= 448 * torch.exp2(k - 1)) & (k > -120), k - 1, k)
        out[:, c:c + BLOCK] = _round_e4m3(b / torch.exp2(k)) * torch.exp2(k)
    return out


def _sigmoid64(t):
    return torch.where(t >= 0, 1 / (1 + torch.exp(-t.abs())), torch.exp(-t.abs()) / (1 + torch.exp(-t.abs())))


def _gate64(g, act):
    """act(g) and act'(g) in 64 bits."""
    if act == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g)), torch.where(g > 0, torch.ones_like(g), torch.zeros_like(g))
    if act == "none":
        return g, torch.ones_like(g)
    # x s(c(x)): the tanh form of GELU has 1 + tanh(a) = 2 s(2a)
    if act == "gelu":
        r = math.sqrt(8 / math.pi)
        c, dc = r * (g + 0.044715 * g * g * g), r * (1 + 0.134145 * g * g)
    else:
        c, dc = g, torch.ones_like(g)
    p = _sigmoid64(c)
    return g * p, p + g * p * _sigmoid64(-c) * dc


def _read64(q, e):
    """Codes (sign, 4 exponent bits, 3 bits of fraction) times their scale, in 64 bits."""
    v = q.to(torch.int64)
    sign = 1.0 - 2.0 * (v >> 7).double()
    ex, fr = (v >> 3) & 15, (v & 7).double()
    mag = torch.where(ex == 0, fr / 512, (1 + fr / 8) * torch.exp2(ex.double() - 7))
    at = torch.arange(q.shape[1], device=q.device) // BLOCK
    return sign * mag * torch.exp2(e.double() - 127)[:, at]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "ln_fwd":
        x = s["x"].double()
        mu = x.sum(1) / x.shape[1]
        var = ((x - mu[:, None]) ** 2).sum(1) / x.shape[1]
        r = (var + s["eps"]) ** -0.5
        y = s["gamma"].double() * (x - mu[:, None]) * r[:, None] + s["beta"].double()
        return {"y": y, "mean": mu, "rstd": r}
    if kind == "ln_bwd":
        x, dy = s["x"].double(), s["dy"].double()
        r = s["rstd"].double()[:, None]
        xh = r * (x - s["mean"].double()[:, None])
        w = s["gamma"].double() * dy
        D = x.shape[1]
        dx = r * (w - (w.sum(1, keepdim=True) + xh * (w * xh).sum(1, keepdim=True)) / D)
        return {"dx": dx, "dgamma": torch.einsum("ij,ij->j", dy, xh), "dbeta": torch.einsum("ij->j", dy)}
    if kind == "ckpt":
        return {"y": _kept8(s["x"].double())}
    if kind == "wgrad":
        dy = s["dy"].double()
        return {"dw": torch.einsum("bn,bk->nk", dy, _read64(s["q"], s["e"])), "db": torch.einsum("bn->n", dy)}
    F = case["F"]
    if kind == "gated_fwd":
        x, w = s["x"].double(), s["w"].double()
        g, u = x @ w[:F].T, x @ w[F:].T
        if s["b"] is not None:
            g, u = g + s["b"][:F].double(), u + s["b"][F:].double()
        out = {"h": _gate64(g, case["act"])[0] * u}
        if case["save"] == "full":
            out["s"] = torch.cat([g, u], 1)
        elif case["save"] == "8bit":
            out["s"] = torch.cat([_kept8(g), _kept8(u)], 1)
        return out
    if case["save"] == "full":
        g, u = s["s"][:, :F].double(), s["s"][:, F:].double()
    else:
        ne = s["e"].shape[1] // 2
        g, u = _read64(s["q"][:, :F], s["e"][:, :ne]), _read64(s["q"][:, F:], s["e"][:, ne:])
    dh = s["dy"].double() @ s["wd"].double()
    a, da = _gate64(g, case["act"])
    dg, du = dh * da * u, dh * a
    w = s["w"].double()
    return {"ds": torch.cat([dg, du], 1), "h": a * u, "dx": dg @ w[:F] + du @ w[F:]}
