"""The example of a hybrid stack: all operators together against a dense fp32 computation without a cache.

Bound.  Every bf16 rounding is off by at most 2^-8 of its value, about 2^-9.5 of it in the mean square.  The served path
rounds some eight times per layer (norm, projection, rotation, weights, sums, output projection, residual) and a few times
more at the ends, 30 in all; independent roundings of that size add up to sqrt(30) 2^-9.5 < 0.008 of a signal, and the
layers pass an error on with a gain of about one each.  0.03 leaves room for that gain."""
import pytest

pytestmark = pytest.mark.gpu


def test_hybrid_stack_matches_dense_computation():
    import __graft_entry__
    __graft_entry__.build()
    from examples import hybrid
    assert hybrid.main(quiet=True) < 0.03
