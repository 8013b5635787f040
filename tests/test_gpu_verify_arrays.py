"""Arrays of a verification step's calls that are not in memory of the current device: refused on the host,
whichever array it is, before anything is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, I32, BF16 = torch.float32, torch.int32, torch.bfloat16
N, B, V, C, SLOTS = 5, 2, 40, 16, 3


@pytest.fixture(scope="module")
def ia():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    import relative_bias_hybrid_gb300.inkattn as ia
    return ia


def _ints(*v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _probs(ia):
    t = dict(logits=torch.randn((N, V), device="cuda"), probs=torch.full((N, V), 7.0, device="cuda"),
             temperature=torch.ones(N, device="cuda"))
    return ia.inkattn_token_probs, ia.token_probs_params(**t), t, ("probs",)


def _verify(ia):
    t = dict(target_p=torch.rand((N, V), device="cuda"), draft_p=torch.rand((N, V), device="cuda"),
             token_ids=torch.zeros(N, dtype=I32, device="cuda"), cu_seqlens_q=_ints(0, 3, 5),
             u_accept=torch.rand(N, device="cuda"), u_sample=torch.rand(B, device="cuda"), n_new=_ints(7, 7),
             out_tokens=_ints(7, 7, 7, 7, 7))
    return ia.inkattn_verify_drafts, ia.verify_drafts_params(**t), t, ("n_new", "out_tokens")


def _rollback(ia, states=2):
    rand = lambda *shape: torch.randn(shape, device="cuda").to(BF16)     # noqa: E731
    t = dict(x=[rand(N, C) for _ in range(states)], state_before=[rand(SLOTS, 3, C) for _ in range(states)],
             state_after=[torch.full((SLOTS, 3, C), 7.0, dtype=BF16, device="cuda") for _ in range(states)],
             n_keep=_ints(1, 2), cu_seqlens_q=_ints(0, 3, 5), state_slot=_ints(2, 0))
    return ia.inkattn_conv_rollback, ia.conv_rollback_params(**t), t, ("state_after",)


def _refused(ia, made, holder, field, like):
    call, p, t, outputs = made
    before = [x.clone() for o in outputs for x in (t[o] if isinstance(t[o], list) else [t[o]])]
    good = getattr(holder, field)
    for host in (like.cpu(), like.cpu().pin_memory()):
        setattr(holder, field, host.data_ptr())
        assert call(p, raise_on_error=False) == ia.INKATTN_ERR_INVALID_ARG, field
    setattr(holder, field, good)
    torch.cuda.synchronize()
    after = [x for o in outputs for x in (t[o] if isinstance(t[o], list) else [t[o]])]
    assert all(torch.equal(a, b) for a, b in zip(before, after)), field
    assert call(p, raise_on_error=False) == ia.INKATTN_OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("make, fields", [
    (_probs, ("logits", "probs", "temperature")),
    (_verify, ("target_p", "draft_p", "token_ids", "cu_seqlens_q", "u_accept", "u_sample", "n_new", "out_tokens")),
    (_rollback, ("n_keep", "cu_seqlens_q", "state_slot"))])
def test_arrays_in_host_memory_are_refused(ia, make, fields):
    for field in fields:
        made = make(ia)
        _refused(ia, made, made[1], field, made[2][field])


@pytest.mark.parametrize("state", [0, 1, 7])
def test_conv_states_in_host_memory_are_refused(ia, state):
    for field in ("x", "state_before", "state_after"):
        made = _rollback(ia, 8)
        _refused(ia, made, made[1].states[state], field, made[2][field][state])


def test_arrays_without_rows_may_be_null(ia):
    """A step without rows: the arrays of rows are not looked at."""
    call, p, t, _ = _verify(ia)
    p.N_tok = 0
    for f in ("target_p", "draft_p", "token_ids", "u_accept", "out_tokens"):
        setattr(p, f, None)
    t["cu_seqlens_q"].zero_()
    assert call(p, raise_on_error=False) == ia.INKATTN_OK
    torch.cuda.synchronize()
    assert t["n_new"].tolist() == [0, 0]
    call, p, t, _ = _rollback(ia)
    p.N_tok = 0
    for s in range(2):
        p.states[s].x = None
    t["cu_seqlens_q"].zero_(), t["n_keep"].zero_()
    assert call(p, raise_on_error=False) == ia.INKATTN_OK
    torch.cuda.synchronize()
    for before, after in zip(t["state_before"], t["state_after"]):
        assert torch.equal(after[[2, 0]], before[[2, 0]]) and bool((after[1] == 7).all())
