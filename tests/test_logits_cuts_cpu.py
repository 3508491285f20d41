"""The sizes that tests/logits_rows.py lists for an instance of a kernel run that instance: the launch rules themselves, compiled
here behind stand-ins for the kernels (nvcc, no GPU)."""
import os
import subprocess

import pytest

from neural_net_step_gb300 import build
from tests import logits_rows as lr

PROGRAM = r"""
#include <cstdlib>
#include <initializer_list>
#include "topk.cu"
#include "distill.cu"
static int last_mode;
namespace mlpk {
namespace tk {
const void* topk_func_f32(int mode, int) { last_mode = mode; return &last_mode; }
const void* topk_func_bf16(int mode, int) { last_mode = mode; return &last_mode; }
const void* topk_func_bf16_wide(int mode, int) { last_mode = mode; return &last_mode; }
}
namespace ds {
const void* distill_func_f32(bool, int, int) { return &last_mode; }
const void* distill_func_bf16(bool, int, int) { return &last_mode; }
}
}
using namespace mlpk;
int main(int argc, char** argv) {
  char err[512];
  for (int i = 1; i < argc; i += 6) {
    const char op = argv[i][0];
    long long a[5];
    for (int j = 0; j < 5; ++j) a[j] = atoll(argv[i + 1 + j]);
    LaunchRec r;
    int per;
    if (op == 'd') {
      DistillOp o;
      o.dtype = (int)a[0]; o.B = a[1]; o.C = a[3]; o.k = a[4]; o.ldz = o.C; o.ldtv = o.ldti = o.k;
      if (distill_plan(o, &r, err, sizeof(err)) < 0) return 1;
      ds::DistillParams p;
      memcpy(&p, r.args, sizeof(p));
      per = p.per;
      last_mode = -1;
    } else {
      if (op == 't') {
        TopkOp o;
        o.dtype = (int)a[0]; o.B = a[1]; o.C = a[3]; o.k = a[4]; o.ldz = o.C; o.ldv = o.ldi = o.k;
        if (topk_plan(o, &r, err, sizeof(err)) < 0) return 1;
      } else {
        BeamSelectOp o;
        o.dtype = (int)a[0]; o.batch = a[1]; o.beams = a[2]; o.C = a[3]; o.m = a[4]; o.ldz = o.C;
        beam_rows_plan(o, (int)std::min(o.m, o.C), nullptr, nullptr, &r);
      }
      tk::TopkParams p;
      memcpy(&p, r.args, sizeof(p));
      per = p.per;
    }
    const long long units = (long long)per * (a[0] == DT_F32 ? 4 : 2) / 16;
    printf("%d %u %u %lld\n", last_mode, r.block.x, r.grid.z, units / r.block.x);
  }
  return 0;
}
"""


def _plans(tmp, calls):
    src, exe = os.path.join(tmp, "plans.cu"), os.path.join(tmp, "plans")
    with open(src, "w") as f:
        f.write(PROGRAM)
    r = subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-O0", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"),
                        src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe, *(str(x) for c in calls for x in c)], capture_output=True, text=True, check=True).stdout
    return [tuple(int(x) for x in line.split()) for line in out.splitlines()]


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    calls = [("t", d, B, 0, C, k) for d, B, C, k, *_ in lr.TOPK]
    calls += [("s", d, b, W, C, m) for d, b, W, C, m, *_ in lr.SELECT]
    calls += [("d", d, B, 0, C, k) for d, B, C, k, *_ in lr.DISTILL]
    out = _plans(str(tmp_path_factory.mktemp("plans")), calls)
    assert len(out) == len(calls)
    n, m = len(lr.TOPK), len(lr.TOPK) + len(lr.SELECT)
    return out[:n], out[n:m], out[m:]


def test_topk(plans):
    for case, (mode, threads, blocks, rounds) in zip(lr.TOPK, plans[0]):
        assert (mode, threads, blocks) == case[4:7] and rounds >= case[7], (case, mode, threads, blocks, rounds)


def test_select(plans):
    for case, (mode, threads, blocks, rounds) in zip(lr.SELECT, plans[1]):
        assert (mode, threads, blocks) == case[5:8] and rounds >= case[8], (case, mode, threads, blocks, rounds)


def test_distill(plans):
    for case, (_, threads, blocks, rounds) in zip(lr.DISTILL, plans[2]):
        assert (blocks, threads) == case[4:6] and rounds >= case[6], (case, blocks, threads, rounds)


def test_every_instance_is_listed():
    """Each mode and block size there is, in both types; rows shared by 2, 4 and 8 blocks, with 32- and 64-bit candidates."""
    for d in (lr.F, lr.H):
        assert {(c[4], c[5]) for c in lr.TOPK if c[0] == d} >= {(lr.ALONE, t) for t in (32, 64, 128, 256, 512)} | {(lr.SLICES, 512)}
        assert {c[6] for c in lr.TOPK if c[0] == d} == {1, 2, 4, 8}
        assert {c[4:6] for c in lr.DISTILL if c[0] == d and c[4] == 1} == {(1, t) for t in (32, 64, 128, 256)}
        assert {c[4] for c in lr.DISTILL if c[0] == d} >= {1, 2, 8}
    assert {c[6] for c in lr.SELECT} >= {32, 64, 128, 256, 512} and {c[5] for c in lr.SELECT} == {lr.SLICES, lr.BEAMS}
    wide = [c for c in lr.TOPK if c[0] == lr.H and -(-c[2] // c[6]) > 65535]
    assert {c[5] for c in wide} == {128, 256, 512} and {c[4] for c in wide} == {lr.ALONE, lr.SLICES}
