"""Helpers of the logits operations' GPU tests: calls on Buf matrices, and error bounds."""
import numpy as np
import torch

import neural_net_step_gb300 as nn
from tests.block_util import DEV, TDT, U32, Buf, stream


class IntBuf(Buf):
    """A Buf of int32."""

    def __init__(self, rows, cols, ld=None, off=0):
        self.rows, self.cols, self.ld, self.off = rows, cols, ld or cols, off
        self.flat = torch.full((off + rows * self.ld + 64,), -777, dtype=torch.int32, device=DEV)
        self.before = self.flat.clone()
        self.t = torch.as_strided(self.flat, (rows, cols), (self.ld, 1), off)


EX2 = 2.0 ** -22   # the hardware's base-2 exponential, relative
# an fp32 sum of the row: a thread's at most 224 terms one after another, then trees (8x the rms growth of 224, and 16)
SUM = (8.0 * np.sqrt(224.0) + 16.0) * U32


def logits(rng, B, C, td, scale=2.0):
    z = rng.normal(size=(B, C)) * scale + rng.normal(size=(1, C))
    return torch.from_numpy(z.astype(np.float32)).to(td)


def term_err(d):
    """Relative error of exp(d) formed as ex2(d c): c, the product and the difference are rounded, then ex2."""
    return EX2 + 4 * U32 * np.abs(d)


def lse_tol(x, chosen):
    """Error of log sum exp over the columns `chosen` of x [B, C] (in units of 1 / T), relative terms weighted by their share."""
    out = np.zeros(len(x))
    for i in range(len(x)):
        v = x[i][chosen[i] & (x[i] > -np.inf)]
        if len(v):
            p = np.exp(v - v.max())
            p /= p.sum()
            # terms are relative to the largest column taken or left: no further than the row's largest
            d = np.abs(v - x[i].max()) + abs(v.max() - x[i].max())
            # (terms so small that fp32 drops them: at most 2^-126 of the largest each)
            out[i] = (p * term_err(d)).sum() + SUM + 2 * U32 * (np.abs(v).max() + np.log(len(v)) + np.abs(x[i]).max()) + 4 * U32
    return out


def run_topk(dtype, z, k, T=1.0, lse=True, tail=True, pad=0, off=0):
    B, C = z.shape
    Z = Buf(B, C, TDT[dtype], C + pad, off, z)
    V, I = Buf(B, k, torch.float32, k + 3, 1), IntBuf(B, k, k + 1, 3)
    L, R = Buf(1, B, torch.float32), Buf(1, B, torch.float32)
    nn.mlp_op_topk(dtype, B, C, k, Z.ptr, Z.ld, T, V.ptr, V.ld, I.ptr, I.ld, L.ptr if lse else None,
                   R.ptr if tail else None, stream())
    torch.cuda.synchronize()
    for b in (Z, V, I, L, R):
        b.check_canary()
    return V.np(), I.np().astype(np.int64), L.np()[0], R.np()[0], Z.np()


def run_distill(dtype, z, tv, ti, tail=None, labels=None, w=None, T=1.0, a=0.0, b=1.0, g=1.0, pad=0, off=0, dpad=0,
                doff=0, in_place=False, grad=True):
    """(loss, dz, error bits, z as stored)"""
    B, C = z.shape
    k = ti.shape[1]
    td = TDT[dtype]
    f = lambda x, t: None if x is None else torch.as_tensor(np.asarray(x)).to(t).to(DEV).contiguous()
    Z = Buf(B, C, td, C + pad, off, z)
    stored = Z.np()
    D = Z if in_place else Buf(B, C, td, C + dpad, doff)
    tv_, ti_ = f(tv, torch.float32), f(ti, torch.int32)
    tail_, y_, w_ = f(tail, torch.float32), f(labels, torch.int32), f(w, torch.float32)
    L = Buf(1, B, torch.float32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = lambda t: None if t is None else t.data_ptr()
    nn.mlp_op_distill(dtype, B, C, k, Z.ptr, Z.ld, tv_.data_ptr(), k, ti_.data_ptr(), k, p(tail_), p(y_), p(w_), T, a, b, g,
                      D.ptr if grad else None, D.ld, L.ptr, err.data_ptr(), stream())
    torch.cuda.synchronize()
    for x in (Z, D, L):
        x.check_canary()
    return L.np()[0], D.np(), int(err.item()), stored


def teacher(rng, z, k, T, noise=1.0):
    """A teacher near the student z: (values, columns, tail) in fp32 / int."""
    from oracle import logits_oracle as lo
    t = (z + noise * rng.normal(size=z.shape)).astype(np.float32).astype(np.float64)
    v, i, _, tail = lo.topk(t, k, T)
    return v.astype(np.float32), i, tail.astype(np.float32)


def distill_tol(z, tv, ti, tail, labels, w, T, a, b, g, loss, dz, half):
    """Bounds of loss and gradient from the kernel's roundings.

    A class's share is exp((z - m) / T) / S: its exponent's error (term_err) and its sum's (SUM and the terms').
    The gradient's terms carry those of q and p and two roundings; the loss carries p_j times the error of log(p_j /
    q_j), whose parts are rounded at their own size."""
    B, C = z.shape
    tl, td = np.zeros(B), np.zeros((B, C))
    for i in range(B):
        ww = 1.0 if w is None else float(w[i])
        if ww == 0.0:
            continue
        fin = z[i] > -np.inf
        m = z[i][fin].max()
        d = np.where(fin, np.abs(z[i] - m), 0.0) / T
        q = np.where(fin, np.exp(-d), 0.0)
        q /= q.sum()
        S = SUM + (q * term_err(d)).sum()
        e = 2 * term_err(d) + 2 * S + 8 * U32
        use = ti[i] >= 0
        cols, tj = ti[i][use], tv[i][use].astype(np.float64) / T
        tj = np.append(tj, -np.inf if tail is None else float(tail[i]))
        grad = np.zeros(C)
        if tj.max() > -np.inf:
            lt = tj.max() + np.log(np.exp(tj - tj.max()).sum())
            p = np.exp(tj - lt)
            dt = np.where(p > 0, np.abs(tj - tj.max()), 0.0)
            ep = 2 * term_err(dt) + 2 * ((p * term_err(dt)).sum() + SUM) + 8 * U32
            others = np.ones(C, bool)
            others[cols] = False
            R = q[others].sum()
            grad = q * e
            grad[cols] += p[:-1] * ep[:-1]
            if p[-1] > 0 and R > 0:
                grad[others] += (q * (e + ep[-1] + S))[others] * p[-1] / R
            lr = np.zeros(len(p))
            ok = p[:-1] > 0
            size = (np.abs(tv[i][use]) + np.abs(z[i][cols]) + np.abs(m) + np.abs(tv[i][use]).max(initial=0)) / T
            with np.errstate(invalid="ignore", divide="ignore"):
                lr[:-1][ok] = (4 * U32 * size + 2 * S + ep[:-1] + np.abs(np.log(p[:-1] / q[cols])) * (ep[:-1] + 4 * U32))[ok]
                if p[-1] > 0:
                    lr[-1] = ep[-1] + 2 * e.min() + 2 * S + 4 * U32 * (np.abs(np.log(p[-1] / R)) + 1) + 2 * term_err(d[others].min())
            tl[i] += abs(b) * ((p * lr).sum() + 4 * U32 * abs(loss[i]))
        td[i] += abs(b) / T * grad
        if labels is not None and a != 0.0:
            d1 = d * T
            s1 = np.where(fin, np.exp(-d1), 0.0)
            s1 /= s1.sum()
            S1 = SUM + (s1 * term_err(d1)).sum()
            td[i] += abs(a) * s1 * (2 * term_err(d1) + 2 * S1 + 8 * U32)
            td[i][labels[i]] += abs(a) * 4 * U32
            tl[i] += abs(a) * (2 * S1 + 4 * U32 * (abs(m) + abs(z[i][labels[i]]) + np.log(C) + 1))
        tl[i] = ww * tl[i] + 4 * U32 * abs(loss[i])
        td[i] = td[i] * abs(ww * g) + 4 * U32 * np.abs(dz[i])
    return tl, td + half * (np.abs(dz) + td) + 1e-40 + (half > U32) * 2.0 ** -134   # (bf16's smallest step)
