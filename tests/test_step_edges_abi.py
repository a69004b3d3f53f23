"""CPU-only checks of the limits of the calls that end a training step.  No compute call is made."""
from test_step_abi import P, grads, pkg  # noqa: F401


def test_gradients_of_more_bytes_than_are_counted(pkg):  # noqa: F811
    """A launch counts pieces of 32 KB in 32 bits.  The same tensor may stand in the norm's list
    many times, so that their sum passes any memory's size: 1024 times 64 GB are 2^31 pieces."""
    many = dict(data=[P] * 1024, types=[2] * 1024, counts=[1 << 34] * 1024)
    assert grads(pkg, **many) == -2
    assert grads(pkg, **many, outs=[P] * 1024, out_types=[2] * 1024) == -2
    for types, count in ((0, 1 << 42), (2, 1 << 41)):        # 2^43 bytes each: five are too many
        assert grads(pkg, data=[P] * 5, types=[types] * 5, counts=[count] * 5) == -2
        # four are within the limit: the next check answers (no GPU here, or no norm to write)
        assert grads(pkg, data=[P] * 4, types=[types] * 4, counts=[count] * 4, norm=None) == -1
