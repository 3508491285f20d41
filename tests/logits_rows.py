"""Rows that an ordinary logits row is not, and the calls whose rows they fill: for every instance of the top-k, distillation
and selection kernels a size that runs it over many rounds of its threads, or over the blocks of a cluster.

The kernels' launches are chosen by rules on sizes; test_logits_cuts_cpu.py holds each call below to the instance that it is
listed for, so that a later rule cannot take a test away from what it is here to run."""
import numpy as np
import torch

import neural_net_step_gb300 as nn
from tests.block_util import TDT, U32
from tests.logits_util import term_err, SUM

F, H = nn.F32, nn.BF16
ALONE, SLICES, BEAMS = 0, 1, 2

# dtype, rows, columns, k: mode, threads, blocks a row, rounds of 16-byte units a thread
TOPK = [
    (H, 2440, 8000, 24, ALONE, 32, 1, 31), (F, 2440, 4001, 20, ALONE, 32, 1, 31),
    (H, 1300, 32003, 40, ALONE, 64, 1, 62), (F, 1300, 16001, 48, ALONE, 64, 1, 62),
    (H, 640, 32000, 64, ALONE, 128, 1, 31), (F, 640, 31999, 90, ALONE, 128, 1, 62),
    (H, 320, 60001, 180, ALONE, 256, 1, 29), (F, 320, 40000, 100, ALONE, 256, 1, 39),
    (H, 700, 1500, 192, ALONE, 256, 1, 0), (F, 2440, 4096, 96, ALONE, 128, 1, 8),
    (H, 100, 65000, 200, ALONE, 512, 1, 15), (F, 100, 65000, 250, ALONE, 512, 1, 31),
    (H, 1300, 70001, 33, ALONE, 256, 1, 34), (H, 700, 70001, 33, ALONE, 128, 1, 68), (H, 100, 70001, 33, ALONE, 512, 1, 17),
    (F, 54, 33001, 33, SLICES, 512, 2, 8), (F, 36, 70001, 256, SLICES, 512, 4, 8), (F, 18, 140001, 33, SLICES, 512, 8, 8),
    (F, 18, 384000, 1, SLICES, 512, 8, 23),
    (H, 54, 70001, 33, SLICES, 512, 2, 8), (H, 36, 140001, 256, SLICES, 512, 4, 8), (H, 18, 270001, 33, SLICES, 512, 8, 8),
    (H, 54, 200001, 33, SLICES, 512, 2, 24), (H, 54, 384000, 256, SLICES, 512, 2, 46)]

# dtype, batch, beams, columns, m: mode, threads, blocks in a cluster, rounds
SELECT = [
    (H, 310, 8, 8000, 8, BEAMS, 32, 8, 31), (F, 620, 4, 4001, 8, BEAMS, 32, 4, 31),
    (H, 170, 8, 32003, 40, BEAMS, 64, 8, 62), (F, 660, 2, 16001, 30, BEAMS, 64, 2, 62),
    (H, 110, 6, 32000, 64, BEAMS, 128, 8, 31), (F, 215, 3, 31999, 50, BEAMS, 128, 4, 62),
    (H, 80, 5, 32000, 10, BEAMS, 256, 8, 15), (F, 8, 4, 60001, 10, BEAMS, 512, 4, 29), (H, 8, 4, 120001, 9, BEAMS, 512, 4, 29),
    (F, 3, 12, 70001, 20, SLICES, 512, 4, 8), (H, 3, 12, 140001, 20, SLICES, 512, 4, 8), (H, 2, 9, 270001, 64, SLICES, 512, 8, 8),
    (H, 2, 32, 70001, 64, SLICES, 512, 2, 8), (F, 2, 5, 90001, 7, SLICES, 512, 4, 10), (H, 1, 2, 200001, 4, SLICES, 512, 4, 12)]

# dtype, rows, columns, k: blocks a row, threads, rounds
DISTILL = [
    (H, 1300, 4096, 32, 1, 32, 16), (F, 1300, 2041, 30, 1, 32, 15), (H, 700, 16384, 64, 1, 64, 32), (F, 700, 8100, 50, 1, 64, 31),
    (H, 310, 24576, 128, 1, 128, 24), (F, 310, 12288, 100, 1, 128, 24), (H, 310, 32000, 64, 1, 256, 15), (F, 160, 16384, 200, 1, 256, 16),
    (H, 160, 60001, 33, 2, 256, 14), (F, 160, 30001, 256, 2, 256, 14), (H, 80, 120001, 20, 4, 256, 14), (F, 40, 120001, 20, 8, 256, 14),
    (H, 20, 384000, 40, 8, 256, 23), (F, 20, 300001, 40, 8, 512, 18)]

KINDS = ["ordinary", "constant", "two_values", "rising", "falling", "few_left", "lowest", "one_left", "all_masked",
         "one_thread", "zeros", "stands_out", "front_masked", "back_masked", "one_part", "lowest_but_one_part", "front_nan",
         "back_nan", "one_part_not_nan", "all_nan", "one_nan", "one_inf", "two_inf_and_masks"]


def row(kind, rng, C, dtype, k):
    """One row [C] of the kind, in the type's values.  Halves and eighths are whole slices of a row that a cluster shares."""
    low = torch.finfo(TDT[dtype]).min
    z = torch.from_numpy((rng.normal(size=C) * 2.0 + rng.normal(size=C)).astype(np.float32))
    some = lambda n: torch.from_numpy(rng.permutation(C)[:n])
    part = slice(C // 8, C // 4)
    if kind == "constant":
        z[:] = -3.25
    elif kind == "two_values":
        z = torch.from_numpy((rng.uniform(size=C) < 0.5).astype(np.float32))
    elif kind == "rising":
        z = torch.linspace(-30, 30, C)
    elif kind == "falling":
        z = torch.linspace(30, -30, C)
    elif kind == "few_left":
        z[some(C - 10)] = -np.inf
    elif kind == "lowest":
        z[some(C - 10)] = low
    elif kind == "one_left":
        z[1:] = -np.inf
    elif kind == "all_masked":
        z[:] = -np.inf
    elif kind == "one_thread":   # the largest are all in a few threads' elements
        z[(torch.arange(C) // (16 // TDT[dtype].itemsize)) % 128 == 5] += 40
    elif kind == "zeros":
        z = torch.where(torch.from_numpy(rng.uniform(size=C) < 0.5), torch.tensor(0.0), torch.tensor(-0.0))
    elif kind == "stands_out":
        z[some(k)] += 200.0
    elif kind == "front_masked":
        z[:C // 2] = -np.inf
    elif kind == "back_masked":
        z[C // 2:] = -np.inf
    elif kind == "one_part":
        z[:part.start], z[part.stop:] = -np.inf, -np.inf
    elif kind == "lowest_but_one_part":
        z[:part.start], z[part.stop:] = low, low
    elif kind == "front_nan":
        z[:C // 2] = np.nan
    elif kind == "back_nan":
        z[C // 2:] = np.nan
    elif kind == "one_part_not_nan":
        z[:part.start], z[part.stop:] = np.nan, np.nan
    elif kind == "all_nan":
        z[:] = np.nan
    elif kind == "one_nan":
        z[some(1)] = np.nan
    elif kind == "one_inf":
        z[some(1)] = np.inf
    elif kind == "two_inf_and_masks":
        z[some(C // 2)] = -np.inf
        z[some(2)] = np.inf
    return z.to(TDT[dtype])


def sum_tol(n):
    """An fp32 sum of the row whose threads add n terms one after another (8x the rms growth), over what SUM has."""
    return max(0.0, (8.0 * np.sqrt(n) + 16.0) * U32 - SUM)


def log_sum_tol(v, most, n):
    """Error of log sum exp over v (in units of 1 / T), formed relative to values no further from the row's largest `most`
    than v's own: each term's share times its error, the sum's, and the roundings of largest, logarithm and result."""
    v = v[v > -np.inf]
    p = np.exp(v - v.max())
    p /= p.sum()
    there = p > 0
    d = np.abs(v[there] - most) + abs(v.max() - most)
    if not np.isfinite(most) or d.max() > 1e30:   # (relative to its own largest: nothing else is near)
        d = np.abs(v[there] - v.max())
    return (p[there] * term_err(d)).sum() + SUM + sum_tol(n) + 2 * U32 * (abs(v.max()) + np.log(len(v)) + (
        abs(most) if np.isfinite(most) and abs(most) < 1e30 else 0.0)) + 4 * U32
