"""The decode over a cache of codes holds q as fp16: a q beyond that range is flagged (its row's result is not
defined), the largest inside is not; the prefill over the same cache holds q as bf16 and takes any."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    from relative_bias_hybrid_gb300 import inputs as gen
    import relative_bias_hybrid_gb300.inkattn as ia
    from relative_bias_hybrid_gb300.step import AttentionStep
    return gen, ia, AttentionStep


@pytest.mark.parametrize("kv", ["e4m3", "i4"])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("value, flagged", [(65280.0, False), (-65280.0, False), (65536.0, True), (-3e38, True)])
def test_q_beyond_fp16_is_flagged(env, kv, splits, value, flagged):
    gen, ia, AttentionStep = env
    w = gen.custom("q-range", Hq=16, Hkv=2, q_lens=[3, 0, 5], prefix_lens=[300, 4, 70], rel_extent=32)
    for token, head, dim in ((0, 0, 0), (7, 15, 127), (2, 9, 64)):
        x = gen.make_inputs(w, seed=1, device="cuda", kv_dtype=kv)
        step = AttentionStep(w, x, mode="decode", num_splits=splits, out_dtype=torch.float32)
        step.run_prologue()
        step.run_attention()
        plain = step.out.clone()
        assert step.device_status() == 0
        step.q_out[token, head, dim] = value
        step.run_attention()
        assert step.device_status() == (ia.INKATTN_ERR_DEVICE_BOUNDS if flagged else 0)
        if not flagged:
            assert bool(torch.isfinite(step.out).all())
        # the other rows stay as they were
        other = torch.ones(plain.shape[:2], dtype=torch.bool, device="cuda")
        other[token, head] = False
        assert torch.equal(step.out[other], plain[other])


@pytest.mark.parametrize("kv", ["e4m3", "i4"])
def test_the_prefill_takes_any_q(env, kv):
    gen, ia, AttentionStep = env
    w = gen.custom("q-prefill", Hq=8, Hkv=1, q_lens=[5], prefix_lens=[70], rel_extent=0)
    x = gen.make_inputs(w, seed=1, device="cuda", kv_dtype=kv)
    step = AttentionStep(w, x, mode="prefill", out_dtype=torch.float32)
    step.run_prologue()
    step.q_out[3, 2, 5] = 1e6
    step.run_attention()
    assert step.device_status() == 0 and bool(torch.isfinite(step.out).all())
