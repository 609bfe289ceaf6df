"""CPU tests of the block operators' C ABI at its edges: what empty sequences
and the largest sizes still need, before any HIP call."""
from selective_state_space_56_amd import binding as bd
from test_block_abi import INVALID, conv, err, lib  # noqa: F401


def test_conv_bwd_of_no_tokens_needs_its_weight(lib):  # noqa: F811
    """A sequence of no tokens still has its state's gradient, and its kernel
    reads the taps: refused without them, as the forward is."""
    for state in (dict(), dict(dstate_out=None), dict(state_in=None, dstate_in=None)):
        d = bd.ConvDesc(2, 0, 16, 4, 1, 0)
        assert conv(lib, d, weight=None, xin=None, dout=None, dxin=None, **state) == INVALID
        assert "weight is NULL" in err(lib)
    # no rows: nothing is read
    d = bd.ConvDesc(0, 0, 0, 4, 1, 0)
    assert conv(lib, d, weight=None, dweight=None) == 0
