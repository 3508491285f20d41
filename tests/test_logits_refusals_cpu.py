"""Refusals of the operations on logits: every bad argument is turned down before anything is enqueued (no GPU needed)."""
import pytest

import neural_net_step_gb300 as nn

P = 1 << 20   # a well-aligned stand-in for a device address (never read)
BIG = nn.TOPK_MAX_COLUMNS


@pytest.fixture(scope="module", autouse=True)
def lib():
    from neural_net_step_gb300 import build
    build.build()
    return nn.lib()


def _refused(f, good, **bad):
    args = dict(good)
    args.update(bad)
    assert set(args) == set(good)
    with pytest.raises(nn.MlpError) as e:
        f(*args.values())
    assert e.value.status in (1, 2, 3), e.value   # argument, shape or dtype; not a CUDA error


TOPK = dict(dtype=nn.BF16, B=4, C=64, k=8, z=P, ldz=64, temperature=1.0, values=P, ldv=8, indices=P, ldi=8, lse=P, tail=P,
            stream=None)
DIST = dict(dtype=nn.BF16, B=4, C=64, k=8, z=P, ldz=64, t_values=P, ldtv=8, t_indices=P, ldti=8, t_tail=P, labels=P,
            row_weights=P, temperature=1.0, ce_weight=0.5, kd_weight=0.5, grad_scale=1.0, dz=2 * P, lddz=64, loss_rows=P,
            err=P, stream=None)
SEL = dict(dtype=nn.BF16, batch=2, beams=4, C=64, m=8, z=P, ldz=64, scores=P, done=P, eos=2, scores_out=P, parents=P,
           tokens=P, done_out=P, ws=P, ws_bytes=1 << 20, stream=None)
REO = dict(planes=2, batch=3, beams_in=4, beams_out=4, row_bytes=64, src=P, src_pitch=64, src_plane=768, parents=P, ldp=4,
           dst=2 * P, dst_pitch=64, dst_plane=768, err=P, stream=None)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [
    dict(dtype=nn.F32X3), dict(dtype=-1), dict(B=0), dict(B=-1), dict(B=1 << 31), dict(C=0), dict(C=7), dict(k=0), dict(k=-1),
    dict(k=65), dict(C=512, ldz=512, k=257, ldv=512, ldi=512), dict(C=BIG + 1, ldz=1 << 20), dict(ldz=63), dict(ldv=7),
    dict(ldi=7), dict(z=None), dict(values=None), dict(indices=None), dict(z=P + 1), dict(values=P + 2),
    dict(indices=P + 2), dict(lse=P + 1), dict(tail=P + 2), dict(temperature=0.0), dict(temperature=-1.0),
    dict(temperature=NAN), dict(temperature=INF), dict(temperature=1e-7), dict(temperature=1e7)])
def test_topk_refuses(bad):
    _refused(nn.mlp_op_topk, TOPK, **bad)


@pytest.mark.parametrize("bad", [
    dict(dtype=nn.F32X3), dict(B=0), dict(B=1 << 31), dict(C=0), dict(C=7), dict(k=0), dict(k=65),
    dict(C=512, ldz=512, lddz=512, k=257, ldtv=512, ldti=512), dict(C=BIG + 1, ldz=1 << 20, lddz=1 << 20), dict(ldz=63),
    dict(lddz=63), dict(ldtv=7), dict(ldti=7), dict(z=None), dict(t_values=None), dict(t_indices=None),
    dict(loss_rows=None), dict(labels=None), dict(temperature=0.0), dict(temperature=NAN), dict(temperature=INF),
    dict(ce_weight=NAN), dict(kd_weight=INF), dict(grad_scale=NAN), dict(z=P + 1), dict(dz=P + 1), dict(t_values=P + 1),
    dict(t_indices=P + 2), dict(t_tail=P + 2), dict(labels=P + 2), dict(row_weights=P + 1), dict(loss_rows=P + 2),
    dict(err=P + 2), dict(dz=P, ldz=72)])
def test_distill_refuses(bad):
    _refused(nn.mlp_op_distill, DIST, **bad)


@pytest.mark.parametrize("bad", [
    dict(dtype=nn.F32X3), dict(batch=0), dict(batch=1 << 30), dict(beams=0), dict(beams=33), dict(C=0), dict(m=0),
    dict(m=65), dict(C=1, m=5, eos=0), dict(C=BIG + 1, ldz=1 << 20), dict(ldz=63), dict(z=None), dict(scores=None),
    dict(scores_out=None), dict(parents=None), dict(tokens=None), dict(eos=-1), dict(eos=64), dict(ws=None),
    dict(ws_bytes=2 * 4 * (8 * 8 + 8) - 1), dict(ws=P + 4), dict(z=P + 1), dict(scores=P + 2), dict(scores_out=P + 1),
    dict(parents=P + 2), dict(tokens=P + 2)])
def test_beam_select_refuses(bad):
    _refused(nn.mlp_op_beam_select, SEL, **bad)


def test_beam_select_workspace():
    f = nn.mlp_op_beam_select_workspace_bytes
    assert f(nn.BF16, 2, 4, 64, 8) == f(nn.F32, 2, 4, 64, 8) == 2 * 4 * (8 * 8 + 8)
    assert f(nn.F32, 1, 2, 3, 6) == 2 * (8 * 3 + 8)   # (no beam has more than its tokens)
    for bad in [(9, 2, 4, 64, 8), (1, 0, 4, 64, 8), (1, 2, 33, 64, 8), (1, 2, 4, 0, 8), (1, 2, 4, 64, 65), (1, 1, 2, 2, 5),
                (1, 1 << 62, 4, 64, 8), (1, 2, 4, BIG + 1, 8)]:
        assert f(*bad) == 0


@pytest.mark.parametrize("bad", [
    dict(planes=0), dict(batch=0), dict(beams_in=0), dict(beams_out=0), dict(beams_in=33), dict(beams_out=33, ldp=33),
    dict(row_bytes=0), dict(row_bytes=65), dict(src=None), dict(dst=None), dict(parents=None), dict(ldp=3),
    dict(src_pitch=63), dict(dst_pitch=63), dict(parents=P + 2), dict(err=P + 1), dict(planes=1 << 31),
    dict(planes=1 << 40, batch=1 << 30), dict(row_bytes=1 << 60, src_pitch=1 << 60, dst_pitch=1 << 60),
    dict(dst=P, dst_pitch=80), dict(dst=P, dst_plane=1024), dict(dst=P, beams_out=3)])
def test_beam_reorder_refuses(bad):
    _refused(nn.mlp_op_beam_reorder, REO, **bad)


def test_every_kernel_in_a_header_takes_one_parameter_block():
    """Launches pass one argument pointer, so every __global__ function takes exactly one `const __grid_constant__` struct
    (test_capi_cpu looks at the .cu files)."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.abspath(nn.__file__)), "csrc")
    n = 0
    for f in sorted(os.listdir(csrc)):
        if f.endswith(".cuh"):
            txt = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, f)).read())
            for m in re.finditer(r"__global__", txt):
                seg = txt[m.end():txt.index("{", m.end())]
                assert re.fullmatch(r"const __grid_constant__ \w+ \w+", seg[seg.rindex("(") + 1:seg.rindex(")")].strip()), f
                n += 1
    assert n >= 2
