"""Arrays of the verification step's calls that claim more memory than lies behind their address: what they span
still counts as overlapping.  Host checks alone, on addresses that are never dereferenced."""
import ctypes

import pytest

FAKE = 1 << 20


@pytest.fixture(scope="module")
def ia():
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    ia.lib()
    return ia


@pytest.mark.parametrize("n_tok", [2, 1 << 20, (1 << 31) - 1])
def test_rollback_rows_that_reach_the_end_of_the_addresses(ia, n_tok):
    """Rows of x 2^33 bytes apart: from its first to its last, 2^31 - 1 of them end just below 2^64 bytes on,
    past the largest address.  A state_after between them lies in that span."""
    def params(after):
        p = ia.ConvRollbackParams()
        p.struct_size = ctypes.sizeof(p)
        p.B, p.N_tok, p.num_state_slots, p.n_states = 1, n_tok, 1, 1
        p.cu_seqlens_q, p.state_slot, p.n_keep = (FAKE + 64 * i for i in range(3))
        c = p.states[0]
        c.C, c.x_stride = 8, 1 << 32
        c.x, c.state_before, c.state_after = 1 << 44, FAKE + 4096, after
        return p
    inside = (1 << 44) + (1 << 33) - 48        # ends where the second row starts
    none = dict(stream=0, raise_on_error=False)
    assert ia.inkattn_conv_rollback(params(inside), **none) == ia.INKATTN_ERR_INVALID_ARG
    assert ia.inkattn_conv_rollback(params((1 << 44) - 48), **none) != ia.INKATTN_OK      # (not on a device)
