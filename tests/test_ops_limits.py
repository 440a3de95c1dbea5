"""The ends of what the operators around the MoE layer accept, without a GPU."""
import pytest
from test_ops_args import Q, _lp  # noqa: F401


@pytest.mark.parametrize("temp", [1e-45, 2e-39, 9e-37, 1.1e36, 5e37, 3e38])
def test_logprob_refuses_far_temperatures(Q, temp):  # noqa: F811
    assert _lp(Q, Q.make_logprob_cfg(1000, temperature=temp), m=0) == Q.MOE_ERR_ARG


@pytest.mark.parametrize("temp", [1e-36, 1e-3, 1.0, 1e36])
def test_logprob_accepts_temperatures(Q, temp):  # noqa: F811
    assert _lp(Q, Q.make_logprob_cfg(1000, temperature=temp), m=0) == Q.MOE_OK


def test_logprob_vocabulary_limit(Q):  # noqa: F811
    assert _lp(Q, Q.make_logprob_cfg(1 << 28), m=0) == Q.MOE_OK
    assert _lp(Q, Q.make_logprob_cfg((1 << 28) + 1), m=0) == Q.MOE_ERR_ARG
