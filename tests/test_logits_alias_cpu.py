"""A beam selection of another number of pairs than beams is refused where its results would lie over the scores or flags
that it reads: entry b's m results would overwrite what other entries' blocks are still reading (no GPU needed)."""
import pytest

import neural_net_step_gb300 as nn
from tests.test_logits_refusals_cpu import P, SEL, _refused, lib  # noqa: F401

APART = dict(SEL, z=64 * P, scores=P, done=2 * P, scores_out=3 * P, parents=4 * P, tokens=5 * P, done_out=6 * P, ws=7 * P)


@pytest.mark.parametrize("m", [1, 3, 5, 8])
@pytest.mark.parametrize("alias", [dict(scores_out=P), dict(done_out=2 * P), dict(scores_out=P, done_out=2 * P)])
def test_results_over_the_inputs_need_as_many_pairs_as_beams(m, alias):
    _refused(nn.mlp_op_beam_select, APART, m=m, **alias)


def test_no_flags_are_no_alias():
    """done and done_out both null, and m other than beams: not an alias (the workspace is refused instead)."""
    with pytest.raises(nn.MlpError) as e:
        nn.mlp_op_beam_select(*dict(APART, done=None, done_out=None, ws_bytes=0).values())
    assert "workspace" in str(e.value)


def test_as_many_pairs_as_beams_may_lie_over_the_inputs():
    with pytest.raises(nn.MlpError) as e:
        nn.mlp_op_beam_select(*dict(APART, m=4, scores_out=P, done_out=2 * P, ws_bytes=0).values())
    assert "workspace" in str(e.value)
