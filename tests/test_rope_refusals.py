"""What a refused call, and a side without heads, may not touch (CPU)."""
import pytest
import torch

from test_rope_args import FAKE, FAR, call


@pytest.mark.parametrize("kw,status", [
    (dict(qo=FAKE + 256), 1),   # dq inside q, a row on
    (dict(q=None), 1), (dict(dqo=3 * FAKE + 1), 2), (dict(ws=None), 1), (dict(ws_bytes=16), 1), (dict(qos=(1024, 0, 128)), 1),
])
def test_checks_come_before_any_write(kw, status):
    """K has no heads, so that its weight's gradient is zeros: they are not written by a call that is refused (without a GPU the
    write itself is what would fail)."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    assert call("qk_norm_rope_bwd", Hk=0, k=None, ko=None, dko=None, dkw=FAR, **kw) == status


@pytest.mark.parametrize("name", ["qk_norm_rope_fwd", "qk_norm_rope_bwd"])
def test_the_weight_of_a_side_without_heads_is_not_looked_at(name):
    """Its address may be anything (both kernels read the weights that they are given)."""
    if torch.cuda.is_available():
        pytest.skip("would run")
    assert call(name, Hk=0, k=None, ko=None, dko=None, dkw=None, kw=FAKE + 1) in (3, 4)
    assert call(name, Hq=0, q=None, qo=None, dqo=None, dqw=None, qw=FAKE + 1) in (3, 4)
    assert call(name, Hk=0, k=None, ko=None, dko=None, dkw=None, qw=FAKE + 1) == 2
