"""A workspace tensor whose elements share memory is refused: it claims more bytes than it has, and
the kernels would write behind them."""
import pytest
import torch


@pytest.fixture(scope="module")
def ia():
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    ia.lib()
    return ia


@pytest.mark.parametrize("make", [lambda: torch.zeros(1, dtype=torch.uint8).expand(1 << 22),
                                  lambda: torch.zeros(16, 1).expand(16, 64),
                                  lambda: torch.zeros(1 << 12).as_strided((64, 64), (1, 1))])
def test_workspaces_share_no_elements(ia, make):
    ws = make()
    calls = [lambda: ia.inkattn_route(ia.RouteParams(), ws, stream=0, raise_on_error=False),
             lambda: ia.inkattn_prefill_e4m3(ia.AttnParams(), ws, stream=0, raise_on_error=False),
             lambda: ia.inkattn_decode(ia.AttnParams(), 2, ws, stream=0, raise_on_error=False),
             lambda: ia.inkattn_combine(ia.AttnParams(), 2, ws, stream=0, raise_on_error=False)]
    for call in calls:
        with pytest.raises(ValueError, match="share memory"):
            call()


def test_other_workspaces_pass(ia):
    """Others, an empty one and none reach the library, which refuses the empty params."""
    for ws in (torch.zeros(64, dtype=torch.uint8), torch.zeros(1 << 12)[::2], torch.zeros(64, 32).t(), torch.zeros(0), None):
        assert ia.inkattn_route(ia.RouteParams(), ws, stream=0, raise_on_error=False) == ia.INKATTN_ERR_INVALID_ARG
