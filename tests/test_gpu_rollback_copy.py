"""inkattn_conv_rollback into another array: what is written is written whatever n_keep is, and nothing else."""
import pytest
import torch

pytestmark = pytest.mark.gpu

I32, BF16 = torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def ia():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    return ia


@pytest.mark.parametrize("lens, keep", [([1], [0]), ([0], [0]), ([9, 9, 9, 9], [0, 1, 2, 9]), ([0, 3, 0, 2], [0, 0, 0, 2]),
                                        ([3] * 40, [0] * 40)])
@pytest.mark.parametrize("widths", [(8,), (1016, 2056, 24)])
def test_states_are_copied_also_where_nothing_is_kept(ia, widths, lens, keep):
    """The array written starts as another value than the state before: slots of the sequences get their state,
    also those that keep no row, and the other slots stay."""
    g = torch.Generator(device="cuda").manual_seed(len(lens))
    N, B, slots = sum(lens), len(lens), len(lens) + 2
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    slot = torch.randperm(slots, generator=torch.Generator().manual_seed(3))[:B].tolist()
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(BF16)     # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=I32, device="cuda")                        # noqa: E731
    x, before = [rand(N, w) for w in widths], [rand(slots, 3, w) for w in widths]
    after = [torch.full_like(s, 7.0) for s in before]
    want = [s.clone() for s in after]
    for rows, old, new in zip(x, before, want):
        for b in range(B):
            new[slot[b]] = torch.cat([old[slot[b]], rows[cu[b]:cu[b] + keep[b]]])[-3:]
    kept = [s.clone() for s in before]
    status = ints([0])
    ia.inkattn_conv_rollback(ia.conv_rollback_params(x=x, state_before=before, state_after=after, n_keep=ints(keep),
                                                     cu_seqlens_q=ints(cu), state_slot=ints(slot), dev_status=status))
    torch.cuda.synchronize()
    assert int(status) == 0
    assert all(torch.equal(a, b) for a, b in zip(after, want))
    assert all(torch.equal(a, b) for a, b in zip(before, kept))
