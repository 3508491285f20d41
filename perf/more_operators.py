"""Workloads of the operations on an LM head's logits: top-k with its log-sums,
distillation from a teacher's top logits, beam search's selection and the
reordering of its states.

Each case is one call that a training or serving program makes behind the
output layer.  `run` computes it from elementary torch operations, or, with
`own` set, through the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


def listed():
    return [
        # serving: the candidates of one token for a sampler; latency only
        {"name": "topk_token", "kind": "topk", "dtype": "bf16", "B": 1, "C": 32000, "k": 50, "T": 1.0},
        # a teacher's batch of 16 Ki tokens, its top logits kept for a student
        {"name": "topk_teacher_16k", "kind": "topk", "dtype": "bf16", "B": 16384, "C": 32000, "k": 64, "T": 2.0},
        # fp32 logits of a vocabulary that is no multiple of anything, a ragged batch
        {"name": "topk_f32_odd", "kind": "topk", "dtype": "f32", "B": 777, "C": 50001, "k": 100, "T": 1.0},
        # a serving batch over the widest vocabulary, the most candidates
        {"name": "topk_wide", "kind": "topk", "dtype": "bf16", "B": 48, "C": 262144, "k": 256, "T": 0.7},
        # a student's training batch at the LM block's sizes, soft targets alone, the teacher's tail as one class
        {"name": "distill_16k", "kind": "distill", "dtype": "bf16", "B": 16384, "C": 32000, "k": 64, "T": 2.0,
         "tail": True, "labels": False, "ragged": False},
        # soft and hard targets together, padded rows of weight zero, teacher rows of differing lengths
        {"name": "distill_labels_8k", "kind": "distill", "dtype": "bf16", "B": 8192, "C": 32000, "k": 32, "T": 2.0,
         "tail": True, "labels": True, "ragged": True},
        # fp32 training over an odd vocabulary, the teacher's top renormalised
        {"name": "distill_f32_odd", "kind": "distill", "dtype": "f32", "B": 1000, "C": 10007, "k": 20, "T": 1.0,
         "tail": False, "labels": True, "ragged": False},
        # one request's decoding step with four beams
        {"name": "select_one", "kind": "select", "dtype": "bf16", "batch": 1, "W": 4, "C": 32000, "m": 4,
         "first": False},
        # a serving batch of 64 requests with eight beams, twice as many candidates as beams
        {"name": "select_64", "kind": "select", "dtype": "bf16", "batch": 64, "W": 8, "C": 32000, "m": 16,
         "first": False},
        # fp32 logits, odd vocabulary and beam count
        {"name": "select_f32_odd", "kind": "select", "dtype": "f32", "batch": 7, "W": 5, "C": 50001, "m": 10,
         "first": False},
        # recurrent states of one request, two layers
        {"name": "reorder_one", "kind": "reorder", "dtype": "bf16", "planes": 2, "batch": 1, "W": 4, "n": 1024},
        # keys and values of twelve layers, sixteen requests with four beams, 256 tokens of 1024
        {"name": "reorder_cache", "kind": "reorder", "dtype": "bf16", "planes": 24, "batch": 16, "W": 4,
         "n": 256 * 1024},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["topk", "topk", "distill", "distill", "select", "select", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    half = 1 if dtype == "bf16" else 2
    C = _logint(rng, 1000, 262144)
    if rng.random() < 0.5:
        C = C // 8 * 8
    if kind == "topk":
        return {"kind": kind, "dtype": dtype, "B": max(1, min(_logint(rng, 1, 16384), 524288000 // half // C)), "C": C,
                "k": _logint(rng, 1, 256), "T": rng.choice([0.7, 1.0, 2.0])}
    if kind == "distill":
        return {"kind": kind, "dtype": dtype, "B": max(1, min(_logint(rng, 1, 16384), 524288000 // half // C)), "C": C,
                "k": _logint(rng, 1, 256), "T": rng.choice([1.0, 2.0, 4.0]), "tail": rng.random() < 0.7,
                "labels": rng.random() < 0.5, "ragged": rng.random() < 0.5}
    if kind == "select":
        W = rng.randint(1, 16)
        return {"kind": kind, "dtype": dtype, "batch": max(1, min(_logint(rng, 1, 64), 16384000 // half // (W * C))),
                "W": W, "C": C, "m": W * rng.choice([1, 2]), "first": rng.random() < 0.2}
    W, planes, batch = rng.randint(2, 16), _logint(rng, 1, 48), _logint(rng, 1, 64)
    n = min(_logint(rng, 8, 262144), 402653184 // half // (W * planes * batch))
    return {"kind": kind, "dtype": dtype, "planes": planes, "batch": batch, "W": W,
            "n": n // 8 * 8 if rng.random() < 0.7 and n >= 8 else n}


# ---- inputs ------------------------------------------------------------------
def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEV)


def _logits(gen, rows, C, td):
    # tokens differ in frequency, a row favours a few of them; the vocabulary's last columns are padding
    z = torch.randn((rows, C), generator=gen, device=DEV)
    z *= 2.0
    z += 1.5 * torch.randn((C,), generator=gen, device=DEV)
    at = torch.randint(0, C, (rows, 4), generator=gen, device=DEV)
    z.scatter_add_(1, at, 10.0 * _rand(gen, rows, 4))
    z[:, C - C // 500:] = -INF
    return z.to(td)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind, td = case["kind"], TD[case["dtype"]]
    s = dict(case)
    i32, f32 = dict(dtype=torch.int32, device=DEV), dict(dtype=torch.float32, device=DEV)
    s["err"] = torch.zeros(1, **i32)
    if kind == "topk":
        B, C, k = case["B"], case["C"], case["k"]
        s["z"] = _logits(gen, B, C, td)
        s["values"], s["indices"] = torch.empty((B, k), **f32), torch.empty((B, k), **i32)
        s["lse"], s["tail_out"] = torch.empty(B, **f32), torch.empty(B, **f32)
    elif kind == "distill":
        B, C, k, T = case["B"], case["C"], case["k"], case["T"]
        s["z"] = _logits(gen, B, C, td)
        # a teacher that agrees with the student in part
        t = torch.randn((B, C), generator=gen, device=DEV)
        t += s["z"]
        tv, ti = torch.topk(t, k, dim=1)
        if case["tail"]:
            t.scatter_(1, ti, -INF)
            t /= T
            s["t_tail"] = torch.logsumexp(t, 1)
        else:
            s["t_tail"] = None
        del t
        ti = ti.to(torch.int32)
        if case["ragged"]:   # rows with fewer kept logits end in unused entries
            used = 1 + (_rand(gen, B) * k).long().clamp_max(k - 1)
            off = torch.arange(k, device=DEV)[None] >= used[:, None]
            ti[off], tv[off] = -1, 0.0
        s["tv"], s["ti"] = tv, ti
        s["labels"] = None
        if case["labels"]:
            rnd = torch.randint(0, C - C // 500, (B,), generator=gen, device=DEV).int()
            s["labels"] = torch.where(_rand(gen, B) < 0.7, ti[:, 0], rnd)
        s["w"] = None
        if case["ragged"]:   # sequences of 64 tokens whose ends are padding
            s["w"] = ((torch.arange(B, device=DEV) % 64) < 56 + (seed & 7)).float() * (0.5 + _rand(gen, B))
            if s["labels"] is not None:
                s["labels"] = torch.where(s["w"] > 0, s["labels"], torch.full_like(s["labels"], -100))
        s["a"], s["b"] = (0.5, 0.5 * T * T) if case["labels"] else (0.0, T * T)
        s["g"] = 1.0 / B
        s["dz"], s["loss"] = torch.empty_like(s["z"]), torch.empty(B, **f32)
    elif kind == "select":
        batch, W, C, m = case["batch"], case["W"], case["C"], case["m"]
        s["z"] = _logits(gen, batch * W, C, td)
        s["eos"] = 2
        if case["first"]:   # a search starts with one live beam
            s["scores"] = torch.full((batch, W), -INF, device=DEV)
            s["scores"][:, 0] = 0
            s["done"] = torch.zeros((batch, W), dtype=torch.uint8, device=DEV)
        else:
            s["scores"] = torch.sort(-30 - 3 * _rand(gen, batch, W), dim=1, descending=True)[0]
            s["done"] = (_rand(gen, batch, W) < 0.15).to(torch.uint8)
        s["scores_out"] = torch.empty((batch, m), **f32)
        s["parents"], s["tokens"] = torch.empty((batch, m), **i32), torch.empty((batch, m), **i32)
        s["done_out"] = torch.empty((batch, m), dtype=torch.uint8, device=DEV)
    else:
        planes, batch, W, n = case["planes"], case["batch"], case["W"], case["n"]
        s["src"] = torch.randn((planes, batch, W, n), generator=gen, device=DEV, dtype=td)
        s["dst"] = torch.empty_like(s["src"])
        # most children come from the better beams
        s["parents"] = (_rand(gen, batch, W) ** 2 * W).int().clamp_max(W - 1)
    return s


# ---- the plain form ----------------------------------------------------------
def _lse(x):
    """log sum exp over the rows of x (-inf where a row has nothing)."""
    m = x.amax(1, keepdim=True).clamp_min(torch.finfo(x.dtype).min)
    return m[:, 0] + torch.log(torch.exp(x - m).sum(1))


def _plain(s):
    kind = s["kind"]
    if kind == "topk":
        k, z = s["k"], s["z"].float()
        v, i = torch.sort(z, dim=1, descending=True, stable=True)
        rest = v[:, k:] / s["T"]
        tail = _lse(rest) if rest.shape[1] else torch.full_like(v[:, 0], -INF)
        return {"values": v[:, :k].contiguous(), "indices": i[:, :k].int(), "lse": _lse(z / s["T"]), "tail": tail}
    if kind == "distill":
        # a divergence is a small difference of large logarithms: those in 64 bits, the gradient's classes in 32
        T, z, k = s["T"], s["z"].float(), s["k"]
        used = s["ti"] >= 0
        at = torch.where(used, s["ti"], torch.zeros_like(s["ti"])).long()
        t = torch.where(used, s["tv"].double() / T, -INF)
        if s["t_tail"] is not None:
            t = torch.cat([t, s["t_tail"].double()[:, None]], 1)
        logp = t - _lse(t)[:, None]
        p = torch.exp(logp)
        pk = p[:, :k]
        lse = _lse(z.double() / T)
        q = torch.exp(z / T - lse.float()[:, None])
        top = torch.zeros_like(z)
        top.scatter_add_(1, at, used.float())
        logq = torch.gather(z, 1, at).double() / T - lse[:, None]
        kd = torch.where(pk > 0, pk * (logp[:, :k] - logq), 0.0).sum(1)
        d = q
        if s["t_tail"] is not None:
            pr = p[:, -1]
            logr = _lse(torch.where(top > 0, -INF, z).double() / T) - lse
            kd = kd + torch.where(pr > 0, pr * (logp[:, -1] - logr), 0.0)
            rest = (1 - pr / torch.exp(logr)).float()
            d = torch.where(top > 0, q, q * rest[:, None])
        d.scatter_add_(1, at, -pk.float())
        d *= s["b"] / T
        loss = s["b"] * kd
        if s["labels"] is not None:
            y = s["labels"].long().clamp_min(0)[:, None]
            l1 = _lse(z)
            loss = loss + s["a"] * (l1.double() - torch.gather(z, 1, y)[:, 0])
            d += s["a"] * torch.exp(z - l1[:, None])
            d.scatter_add_(1, y, torch.full_like(d[:, :1], -s["a"]))
        if s["w"] is not None:
            loss, d = loss * s["w"], d * s["w"][:, None]
        return {"loss": loss.float(), "dz": (d * s["g"]).to(TD[s["dtype"]])}
    if kind == "select":
        # totals of different beams can lie next to each other: 64 bits
        batch, W, C, m = s["batch"], s["W"], s["C"], s["m"]
        z = s["z"].double()
        logp = (z - _lse(z)[:, None]).view(batch, W, C)
        only = torch.full((C,), -INF, dtype=torch.float64, device=DEV)
        only[s["eos"]] = 0
        logp = torch.where(s["done"][:, :, None] > 0, only, logp)
        total = (s["scores"].double()[:, :, None] + logp).view(batch, W * C)
        v, i = torch.sort(total, dim=1, descending=True, stable=True)
        v, i = v[:, :m], i[:, :m]
        parents, tokens = i // C, i % C
        done = (torch.gather(s["done"], 1, parents) > 0) | (tokens == s["eos"])
        return {"scores": v.float(), "parents": parents.int(), "tokens": tokens.int(), "done": done.to(torch.uint8)}
    b = torch.arange(s["batch"], device=DEV)[:, None]
    return {"dst": s["src"][:, b, s["parents"].long()]}


# ---- the library's calls -------------------------------------------------------
def _own(s):
    import neural_net_step_gb300 as nn
    kind = s["kind"]
    st = torch.cuda.current_stream().cuda_stream
    dt = nn.BF16 if s["dtype"] == "bf16" else nn.F32
    if kind == "topk":
        B, C, k = s["B"], s["C"], s["k"]
        nn.mlp_op_topk(dt, B, C, k, s["z"].data_ptr(), C, s["T"], s["values"].data_ptr(), k, s["indices"].data_ptr(), k,
                       s["lse"].data_ptr(), s["tail_out"].data_ptr(), st)
        return {"values": s["values"], "indices": s["indices"], "lse": s["lse"], "tail": s["tail_out"]}
    if kind == "distill":
        B, C, k = s["B"], s["C"], s["k"]
        ptr = {n: s[n].data_ptr() if s[n] is not None else None for n in ("t_tail", "labels", "w")}
        nn.mlp_op_distill(dt, B, C, k, s["z"].data_ptr(), C, s["tv"].data_ptr(), k, s["ti"].data_ptr(), k,
                          ptr["t_tail"], ptr["labels"], ptr["w"], s["T"], s["a"], s["b"], s["g"], s["dz"].data_ptr(), C,
                          s["loss"].data_ptr(), s["err"].data_ptr(), st)
        return {"loss": s["loss"], "dz": s["dz"]}
    if kind == "select":
        batch, W, C, m = s["batch"], s["W"], s["C"], s["m"]
        n = nn.mlp_op_beam_select_workspace_bytes(dt, batch, W, C, m)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        nn.mlp_op_beam_select(dt, batch, W, C, m, s["z"].data_ptr(), C, s["scores"].data_ptr(), s["done"].data_ptr(),
                              s["eos"], s["scores_out"].data_ptr(), s["parents"].data_ptr(), s["tokens"].data_ptr(),
                              s["done_out"].data_ptr(), ws.data_ptr(), n, st)
        return {"scores": s["scores_out"], "parents": s["parents"], "tokens": s["tokens"], "done": s["done_out"]}
    planes, batch, W = s["planes"], s["batch"], s["W"]
    row = s["n"] * s["src"].element_size()
    nn.mlp_op_beam_reorder(planes, batch, W, W, row, s["src"].data_ptr(), row, batch * W * row, s["parents"].data_ptr(),
                           W, s["dst"].data_ptr(), row, batch * W * row, s["err"].data_ptr(), st)
    return {"dst": s["dst"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- work ----------------------------------------------------------------------
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if kind == "topk":
        B, C, k = case["B"], case["C"], case["k"]
        return {"bytes": es * B * C + B * (8 * k + 8), "flops": 4 * B * C}
    if kind == "distill":
        B, C, k = case["B"], case["C"], case["k"]
        row = 8 * k + 4 + (4 if case["tail"] else 0) + (4 if case["labels"] else 0) + (4 if case["ragged"] else 0)
        return {"bytes": 2 * es * B * C + B * row, "flops": (12 if case["labels"] and case["T"] != 1 else 8) * B * C}
    if kind == "select":
        batch, W, C, m = case["batch"], case["W"], case["C"], case["m"]
        return {"bytes": es * batch * W * C + 5 * batch * W + 13 * batch * m, "flops": 4 * batch * W * C}
    planes, batch, W, n = case["planes"], case["batch"], case["W"], case["n"]
    return {"bytes": 2 * es * planes * batch * W * n + 4 * batch * W, "flops": 0}


# ---- the definition in 64 bits ---------------------------------------------------
def _largest(x, k):
    """The k largest of each row of x (64 bits, used up), one after another; the lowest index among equals."""
    vals, at = [], []
    place = torch.arange(x.shape[1], device=x.device)
    gone = torch.zeros(x.shape, dtype=torch.bool, device=x.device)
    for _ in range(k):
        left = torch.where(gone, torch.full_like(x, -INF), x)
        v = left.max(1, keepdim=True).values
        i = torch.where((left == v) & ~gone, place, x.shape[1]).min(1, keepdim=True).values
        gone.scatter_(1, i, True)
        vals.append(v)
        at.append(i)
    return torch.cat(vals, 1), torch.cat(at, 1), gone


def _exact_topk(z, k, T):
    v, i, gone = _largest(z, k)
    lse = torch.logsumexp(z / T, 1)
    tail = torch.logsumexp(torch.where(gone, torch.full_like(z, -INF), z / T), 1)
    return v, i, lse, tail


def _exact_distill(s, r):
    """Rows r of the loss and its gradient, class by class: the teacher's distribution written over the whole
    vocabulary, the tail's share handed out in the student's own proportions."""
    T, z = s["T"], s["z"][r].double()
    rows = torch.arange(z.shape[0], device=DEV)
    t = torch.full_like(z, -INF)
    for j in range(s["k"]):
        i = s["ti"][r, j].long()
        ok = i >= 0
        t[rows[ok], i[ok]] = s["tv"][r, j].double()[ok] / T
    kept = t > -INF
    q = torch.softmax(z / T, 1)
    norm = torch.logsumexp(t, 1)
    p = torch.zeros_like(z)
    kd = torch.zeros_like(norm)
    if s["t_tail"] is not None:
        tail = s["t_tail"][r].double()
        norm = torch.logaddexp(norm, tail)
        pr = torch.exp(tail - norm)[:, None]
        rest = torch.where(kept, torch.full_like(z, -INF), z / T)
        share = torch.softmax(rest, 1)
        p = torch.where(kept, p, pr * share)
        kd = (pr * (torch.log(pr) - (torch.logsumexp(rest, 1) - torch.logsumexp(z / T, 1))[:, None]))[:, 0]
    pt = torch.exp(t - norm[:, None])
    p = torch.where(kept, pt, p)
    kd = kd + torch.where(kept, pt * (t - norm[:, None] - torch.log_softmax(z / T, 1)), torch.zeros_like(z)).sum(1)
    d = s["b"] / T * (q - p)
    loss = s["b"] * kd
    if s["labels"] is not None:
        y = s["labels"][r].long()
        y = torch.where(y < 0, torch.zeros_like(y), y)
        logs = torch.log_softmax(z, 1)
        hot = torch.zeros_like(z)
        hot[rows, y] = 1.0
        loss = loss - s["a"] * logs[rows, y]
        d = d + s["a"] * (torch.exp(logs) - hot)
    w = torch.ones_like(loss) if s["w"] is None else s["w"][r].double()
    return loss * w, d * (w * s["g"])[:, None]


def exact(case, seed):
    kind = case["kind"]
    s = prepare(case, seed)
    if kind == "topk":
        rows = max(1, (1 << 27) // case["C"])
        parts = [_exact_topk(z.double(), case["k"], case["T"]) for z in s["z"].split(rows)]
        v, i, lse, tail = (torch.cat(p) for p in zip(*parts))
        return {"values": v, "indices": i.int(), "lse": lse, "tail": tail}
    if kind == "distill":
        rows = max(1, (1 << 27) // case["C"])
        loss = torch.empty(case["B"], dtype=torch.float64, device=DEV)
        dz = torch.empty(case["B"], case["C"], dtype=torch.float64, device=DEV)
        for a in range(0, case["B"], rows):
            r = slice(a, min(case["B"], a + rows))
            loss[r], dz[r] = _exact_distill(s, r)
        return {"loss": loss, "dz": dz}
    if kind == "select":
        batch, W, C, m = case["batch"], case["W"], case["C"], case["m"]
        out = {"scores": [], "parents": [], "tokens": [], "done": []}
        for b in range(batch):
            lp = torch.log_softmax(s["z"][b * W:(b + 1) * W].double(), 1)
            for w in range(W):
                if s["done"][b, w]:
                    lp[w].fill_(-INF)
                    lp[w, s["eos"]] = 0
            v, i, _ = _largest((lp + s["scores"][b].double()[:, None]).reshape(1, W * C), m)
            p, t = torch.div(i[0], C, rounding_mode="floor"), i[0].remainder(C)
            out["scores"].append(v[0])
            out["parents"].append(p.int())
            out["tokens"].append(t.int())
            out["done"].append((s["done"][b][p].bool() | (t == s["eos"])).to(torch.uint8))
        return {n: torch.stack(x) for n, x in out.items()}
    dst = torch.empty_like(s["src"], dtype=torch.float64)
    for b in range(case["batch"]):
        for w in range(case["W"]):
            dst[:, b, w] = s["src"][:, b, int(s["parents"][b, w])].double()
    return {"dst": dst}
