"""Refusals of the feed-forward block's operations: every bad argument is
turned down before anything is enqueued (no GPU needed), and workspace sizes."""
import pytest

import neural_net_step_gb300 as nn

P = 1 << 20   # a well-aligned stand-in for a device address (never read)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from neural_net_step_gb300 import build
    build.build()
    return nn.lib()


def _refused(f, good, **bad):
    args = dict(good)
    args.update(bad)
    with pytest.raises(nn.MlpError) as e:
        f(*args.values())
    assert e.value.status in (1, 2, 3), e.value   # argument, shape or dtype; not a CUDA error
    return e.value.status


LN = dict(dtype=nn.BF16, M=4, D=64, X=P, ldx=64, gamma=P, beta=P, eps=1e-5, Y=P, ldy=64, mean=P, rstd=P, stream=None)
LNB = dict(dtype=nn.BF16, M=4, D=64, dY=P, lddy=64, X=P, ldx=64, gamma=P, mean=P, rstd=P, dX=P, lddx=64, dgamma=P,
           dbeta=P, ws=P, ws_bytes=1 << 30, stream=None)
Q8 = dict(dtype=nn.BF16, rows=4, cols=64, X=P, ldx=64, Q=P, ldq=64, E=P, lde=2, stream=None)
D8 = dict(dtype=nn.BF16, rows=4, cols=64, Q=P, ldq=64, E=P, lde=2, Y=P, ldy=64, stream=None)
W8 = dict(dtype=nn.BF16, N=64, K=64, B=16, dY=P, ldy=64, Q=P, ldq=64, E=P, lde=2, dW=P, lddw=64, db=P, ws=P,
          ws_bytes=1 << 30, err=None, stream=None)


@pytest.mark.parametrize("bad", [
    dict(dtype=nn.F32X3), dict(dtype=9), dict(X=None), dict(Y=None), dict(M=0), dict(M=-1), dict(D=0), dict(D=1 << 30),
    dict(M=1 << 40), dict(ldx=63), dict(ldy=63), dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf"))])
def test_layernorm_refuses(bad):
    _refused(nn.mlp_op_layernorm, LN, **bad)


@pytest.mark.parametrize("bad", [
    dict(dtype=nn.F32X3), dict(dY=None), dict(X=None), dict(mean=None), dict(rstd=None), dict(dX=None), dict(M=0),
    dict(D=0), dict(D=1 << 30), dict(lddy=63), dict(ldx=63), dict(lddx=63), dict(ws=None), dict(ws_bytes=0),
    dict(ws_bytes=4 * 2 * 64 - 1), dict(ws=P + 2)])
def test_layernorm_backward_refuses(bad):
    _refused(nn.mlp_op_layernorm_backward, LNB, **bad)


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(X=None), dict(Q=None), dict(E=None), dict(rows=0), dict(cols=0),
                                 dict(cols=1 << 40), dict(ldx=63), dict(ldq=63), dict(lde=1), dict(rows=-3)])
def test_quant8_refuses(bad):
    _refused(nn.mlp_op_quant8, Q8, **bad)


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(Y=None), dict(Q=None), dict(E=None), dict(rows=0), dict(cols=0),
                                 dict(ldy=63), dict(ldq=63), dict(lde=1)])
def test_dequant8_refuses(bad):
    _refused(nn.mlp_op_dequant8, D8, **bad)


@pytest.mark.parametrize("bad", [
    dict(dtype=nn.F32X3), dict(dY=None), dict(Q=None), dict(E=None), dict(dW=None), dict(ws=None), dict(N=0),
    dict(K=0), dict(B=0), dict(B=1 << 40), dict(ldy=63), dict(ldy=65), dict(dY=P + 2), dict(ldq=63), dict(lde=1),
    dict(lddw=63), dict(K=33, lddw=36), dict(lddw=66), dict(dW=P + 8), dict(ws_bytes=64 * 16 * 2 - 1), dict(ws=P + 8)])
def test_wgrad8_refuses(bad):
    _refused(nn.mlp_op_wgrad8, W8, **bad)


def test_workspace_sizes():
    for dt in (nn.F32, nn.BF16):
        n = nn.mlp_op_layernorm_backward_workspace_bytes(dt, 65536, 1024)
        assert n % (2 * 1024 * 4) == 0 and 1 <= n // (2 * 1024 * 4) <= 1216
        assert nn.mlp_op_layernorm_backward_workspace_bytes(dt, 1, 8) == 2 * 8 * 4
        # the values, 256-byte rounded, then the weight gradient's own
        assert nn.mlp_op_wgrad8_workspace_bytes(dt, 64, 100, 10) >= 10 * 104 * (4 if dt == nn.F32 else 2)
    for bad in ((2, 4, 4), (nn.BF16, 0, 4), (nn.BF16, 4, 0)):
        assert nn.mlp_op_layernorm_backward_workspace_bytes(*bad) == 0
        assert nn.mlp_op_wgrad8_workspace_bytes(*bad, 4) == 0
    assert nn.mlp_op_wgrad8_workspace_bytes(nn.BF16, 1 << 30, 1 << 30, 1 << 30) == 0


GF = dict(dtype=nn.BF16, act=nn.ACT_SILU, M=4, F=64, K=32, X=P, ldx=32, W=P, ldw=32, b=P, H=P, ldh=64, S=P, lds=128,
          SE=None, ldse=4, err=None, stream=None)
GB = dict(dtype=nn.BF16, act=nn.ACT_SILU, M=4, N=32, F=64, dY=P, lddy=32, Wd=P, ldw=64, S=P, lds=128, SE=None, ldse=4,
          dS=P, ldds=128, H=P, ldh=64, err=None, stream=None)


@pytest.mark.parametrize("bad", [
    dict(dtype=nn.F32X3), dict(act=4), dict(act=-1), dict(X=None), dict(W=None), dict(H=None), dict(S=None, SE=P),
    dict(M=0), dict(F=0), dict(K=0), dict(M=1 << 33), dict(M=(1 << 31) - 1), dict(F=1 << 31), dict(K=1 << 33), dict(ldx=24), dict(ldw=24),
    dict(ldh=56), dict(lds=120), dict(SE=P, ldse=3), dict(F=60), dict(K=28), dict(X=P + 2), dict(W=P + 8),
    dict(H=P + 4), dict(S=P + 8), dict(SE=P, S=P + 4), dict(ldx=33), dict(ldw=36), dict(ldh=68), dict(lds=132),
    dict(SE=P, lds=132)])
def test_gated_linear_refuses(bad):
    _refused(nn.mlp_op_gated_linear, GF, **bad)


@pytest.mark.parametrize("bad", [
    dict(dtype=nn.F32X3), dict(act=4), dict(dY=None), dict(Wd=None), dict(S=None), dict(dS=None), dict(M=0), dict(N=0),
    dict(F=0), dict(M=1 << 33), dict(F=1 << 31), dict(lddy=24), dict(ldw=56), dict(lds=120), dict(ldds=120),
    dict(ldh=56), dict(SE=P, ldse=3), dict(F=60), dict(N=28), dict(dY=P + 2), dict(Wd=P + 8), dict(dS=P + 4),
    dict(H=P + 8), dict(S=P + 2), dict(SE=P, S=P + 4), dict(ldds=132), dict(lddy=36)])
def test_gated_dgrad_refuses(bad):
    _refused(nn.mlp_op_gated_dgrad, GB, **bad)


def test_silu_belongs_to_the_gated_operations():
    with pytest.raises(nn.MlpError):
        nn.mlp_op_linear_act(nn.BF16, nn.ACT_SILU, 4, 64, 64, P, 64, P, 64, P, P, 64, None, 0, None, None)
    with pytest.raises(nn.MlpError):
        nn.mlp_arena_bytes([8, 8, 4], None, nn.ACT_SILU, nn.F32, 4)


@pytest.mark.parametrize("f,good,names", [
    (nn.mlp_op_layernorm, LN, "X Y gamma beta mean rstd"), (nn.mlp_op_layernorm_backward, LNB, "dY X dX gamma mean rstd dgamma dbeta"),
    (nn.mlp_op_quant8, Q8, "X"), (nn.mlp_op_dequant8, D8, "Y"), (nn.mlp_op_wgrad8, W8, "dY dW db"),
    (nn.mlp_op_gated_linear, GF, "X W b H S"), (nn.mlp_op_gated_dgrad, GB, "dY Wd S dS H")])
@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
def test_addresses_between_elements_are_refused(f, good, names, dtype):
    """An address that is no multiple of an element's size."""
    for name in names.split():
        _refused(f, dict(good, dtype=dtype), **{name: P + 1})
        _refused(f, dict(good, dtype=nn.F32), **{name: P + 2})
