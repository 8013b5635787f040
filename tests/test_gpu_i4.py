"""GPU parity of the 4-bit KV cache: the rows that the prologue and the qkvr projections write, and the
decode and the prefill over such a cache.

Bars: codes and scale bytes are bit-exact against the oracle's quantisation of the very bf16 rows that
the bf16 run writes.  n * s is exact in the decode's fp16 and the prefill's bf16 operands, so both are held to
the bf16 path's bar against the oracle on the dequantised cache: max-abs <= 1e-2, mean-abs <=
1e-3, |dLSE| <= 2e-3."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAX_ABS, MEAN_ABS, LSE_ABS = 1e-2, 1e-3, 2e-3


@pytest.fixture(scope="module")
def env(oracle_mod):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    from relative_bias_hybrid_gb300 import inputs as gen
    import relative_bias_hybrid_gb300.inkattn as ia
    from relative_bias_hybrid_gb300.step import AttentionStep
    return gen, AttentionStep, oracle_mod, ia


def _dequant_bits(oracle, gen, codes, scales):
    vals = oracle.dequantize_i4(codes, scales)
    t = torch.from_numpy(vals).to(torch.bfloat16)
    assert np.array_equal(t.double().numpy(), vals)
    return gen.bits(t)


def _check(env, w, x, step, lse_tol=LSE_ABS, rows=None):
    gen, _, oracle, _ = env
    assert step.device_status() == 0
    kc = _dequant_bits(oracle, gen, x["k_cache"].cpu().numpy(), x["k_scale"].cpu().numpy())
    vc = _dequant_bits(oracle, gen, x["v_cache"].cpu().numpy(), x["v_scale"].cpu().numpy())
    xs = {k: x[k].cpu() for k in ("cu_seqlens_q", "seqlen_k", "r", "P", "block_table")}
    o_ref, lse_ref = oracle.attention_for_inputs(xs, w, gen.bits(step.q_out), kc, vc, rows=rows)
    out, lse = step.out.float().cpu().numpy(), step.lse.cpu().numpy()
    if rows is not None:
        out, lse = out[rows], lse[rows]
    err = np.abs(out - o_ref)
    assert np.isfinite(out).all(), w.name
    assert err.max() <= MAX_ABS and err.mean() <= MEAN_ABS, (w.name, err.max(), err.mean())
    assert (np.abs(lse - lse_ref) <= lse_tol).all(), (w.name, np.abs(lse - lse_ref).max())


def _run(env, w, seed, mode="decode", splits=0, x=None):
    gen, AttentionStep, _, _ = env
    x = gen.make_inputs(w, seed=seed, device="cuda", kv_dtype="i4") if x is None else x
    step = AttentionStep(w, x, mode=mode, num_splits=splits, out_dtype=torch.float32)
    step.run()
    torch.cuda.synchronize()
    return x, step


def _same_rows(oracle, gen, w, xb, x4, before):
    """The mapped slots hold the quantised rows of the bf16 cache, the others what they held."""
    slots = x4["slot_mapping"].cpu().numpy().astype(np.int64)
    blk, off = slots // 64, slots % 64
    keep = np.ones(x4["k_cache"].shape[0] * 64, bool)
    keep[slots] = False
    for name in ("k", "v"):
        codes, scales = oracle.quantize_rows_i4(gen.bits(xb[f"{name}_cache"])[blk, :, off, :])
        for part, want in ((f"{name}_cache", codes), (f"{name}_scale", scales)):
            got = x4[part].cpu().numpy()
            assert np.array_equal(got[blk, :, off], want), part
            g = got.transpose(0, 2, 1, 3).reshape(keep.size, w.Hkv, -1)
            b = before[part].cpu().numpy().transpose(0, 2, 1, 3).reshape(keep.size, w.Hkv, -1)
            assert np.array_equal(g[keep], b[keep]), part


def test_prologue_writes_quantised_rows(env):
    gen, AttentionStep, oracle, _ = env
    w = gen.custom("pro4", Hq=16, Hkv=2, q_lens=[9, 40, 0, 3, 1], prefix_lens=[100, 0, 5, 1, 70], rel_extent=64)
    xb = gen.make_inputs(w, seed=3, device="cuda")
    x4 = gen.make_inputs(w, seed=3, device="cuda", kv_dtype="i4")
    # rows of all sizes: small ones (subnormal scales), zeros, and ones beyond the largest scale
    for x in (xb, x4):
        for i, f in enumerate((1e-7, 2.0 ** -14, 1e-3, 0.0, 300.0, 1e4, 1e6)):
            x["v"][9 + i] *= f
    before = {k: x4[k].clone() for k in ("k_cache", "v_cache", "k_scale", "v_scale")}
    sb, s4 = AttentionStep(w, xb, mode="prefill"), AttentionStep(w, x4, mode="decode", num_splits=1)
    sb.run_prologue()
    s4.run_prologue()
    torch.cuda.synchronize()
    assert sb.device_status() == 0 and s4.device_status() == 0
    assert torch.equal(sb.q_out, s4.q_out)
    assert torch.equal(xb["conv_state_k"], x4["conv_state_k"]) and torch.equal(xb["conv_state_v"], x4["conv_state_v"])
    _same_rows(oracle, gen, w, xb, x4, before)


def test_prologue_stores_a_nan_as_zero(env):
    """NaN and infinite inputs (whose conv is a NaN, in the bf16 cache too) leave the other values of their group as
    they are."""
    gen, AttentionStep, oracle, _ = env
    w = gen.custom("pro4-nan", Hq=8, Hkv=1, q_lens=[4], prefix_lens=[0], rel_extent=16)
    xb = gen.make_inputs(w, seed=4, device="cuda")
    x = gen.make_inputs(w, seed=4, device="cuda", kv_dtype="i4")
    before = {k: x[k].clone() for k in ("k_cache", "v_cache", "k_scale", "v_scale")}
    for y in (x, xb):
        y["conv_w_v"][:] = 0.0
        y["conv_w_v"][:, 3] = 1.0
        y["v"][:, 5] = float("nan")
        y["v"][1:, 40] = float("inf")
        AttentionStep(w, y, mode="decode", num_splits=1).run_prologue()
    torch.cuda.synchronize()
    _same_rows(oracle, gen, w, xb, x, before)
    slots = x["slot_mapping"].cpu().numpy()
    got = oracle.dequantize_i4(x["v_cache"].cpu().numpy()[slots // 64, 0, slots % 64],
                               x["v_scale"].cpu().numpy()[slots // 64, 0, slots % 64])
    assert (got[:, 5] == 0).all() and np.isfinite(got).all() and (got != 0).mean() > 0.8


def test_prologue_ties_at_every_scale(env):
    """Every scale in a group that reaches 7 s, with each tie (n + 1/2) s and the bf16 values on both sides of it; and
    groups whose largest value is the bf16 value above 7 s."""
    gen, AttentionStep, oracle, _ = env
    groups = []
    for s in oracle.i4_scales()[1:]:
        ties = torch.tensor([(n + 0.5) * s for n in range(7)], dtype=torch.float64).to(torch.bfloat16)
        near = torch.cat([ties, (ties.view(torch.int16) + 1).view(torch.bfloat16), (ties.view(torch.int16) - 1).view(torch.bfloat16)])
        near = torch.cat([near[:14], -near[14:], -ties])             # 28 values
        top = torch.tensor([7 * s], dtype=torch.float64).to(torch.bfloat16)
        above = (top.view(torch.int16) + 1).view(torch.bfloat16)
        for most in (top, above):
            groups.append(torch.cat([near, most, -most, torch.zeros(2, dtype=torch.bfloat16)]))
    groups = torch.stack(groups)
    rows = groups.reshape(-1, 128)
    w = gen.custom("ties4", Hq=8, Hkv=1, q_lens=[rows.shape[0]], prefix_lens=[0], rel_extent=16)
    x = gen.make_inputs(w, seed=4, device="cuda", kv_dtype="i4")
    x["conv_w_v"][:] = 0.0
    x["conv_w_v"][:, 3] = 1.0
    x["v"].copy_(rows)
    AttentionStep(w, x, mode="prefill").run_prologue()
    torch.cuda.synchronize()
    slots = x["slot_mapping"].cpu().numpy()
    codes, scales = oracle.quantize_rows_i4(gen.bits(rows))
    assert np.array_equal(x["v_scale"].cpu().numpy()[slots // 64, 0, slots % 64], scales)
    assert np.array_equal(x["v_cache"].cpu().numpy()[slots // 64, 0, slots % 64], codes)


def test_qkvr_writes_the_prologues_rows(env):
    """The fused projections on integer-grid inputs (exact sums): cache rows, scales, queries and states as
    the bf16 run's, quantised."""
    from relative_bias_hybrid_gb300.step import QkvrStep
    gen, _, oracle, _ = env
    w = gen.custom("qkvr4", Hq=16, Hkv=2, q_lens=[130, 9, 2], prefix_lens=[0, 40, 1], rel_extent=16)
    xb = gen.make_qkvr_inputs(w, 256, seed=0, device="cuda", grid=True)
    x4 = gen.make_qkvr_inputs(w, 256, seed=0, device="cuda", grid=True, kv_dtype="i4")
    before = {k: x4[k].clone() for k in ("k_cache", "v_cache", "k_scale", "v_scale")}
    sb, s4 = QkvrStep(w, xb), QkvrStep(w, x4)
    sb.run()
    s4.run()
    torch.cuda.synchronize()
    assert sb.device_status() == 0 and s4.device_status() == 0
    assert torch.equal(sb.q_out, s4.q_out) and torch.equal(sb.r_out, s4.r_out)
    assert torch.equal(sb.state_k, s4.state_k) and torch.equal(sb.state_v, s4.state_v)
    _same_rows(oracle, gen, w, xb, x4, before)


@pytest.mark.parametrize("splits", [1, 0, 2, 3])
def test_decode_small(env, splits):
    w = env[0].custom("dec4", Hq=16, Hkv=2, q_lens=[9, 9, 4, 1, 0], prefix_lens=[700, 40, 1500, 3000, 200],
                      rel_extent=200, log_scale_base=256.0)
    _check(env, w, *_run(env, w, seed=4, splits=splits))


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 191, 257])
def test_decode_lengths_around_a_page(env, T):
    """One query row and two over caches that end anywhere in a page or a tile, without a bias."""
    n = min(T, 2)
    w = env[0].custom("dec4-T", Hq=6, Hkv=2, q_lens=[1, n], prefix_lens=[T - 1, T - n])
    _check(env, w, *_run(env, w, seed=T, splits=1))


def test_decode_at_the_row_limit_with_window(env):
    w = env[0].custom("dec4-rows", Hq=32, Hkv=2, q_lens=[8, 8], prefix_lens=[1000, 2989], rel_extent=300,
                      window=1024)
    _check(env, w, *_run(env, w, seed=8, splits=3))


def test_decode_scales_of_every_size(env):
    """Scales from subnormal ones to the largest in the same cache, K and V."""
    gen = env[0]
    w = gen.custom("dec4-scales", Hq=8, Hkv=2, q_lens=[3], prefix_lens=[600], rel_extent=32)
    x = gen.make_inputs(w, seed=6, device="cuda", kv_dtype="i4")
    g = torch.Generator(device="cuda").manual_seed(1)
    shape = x["k_scale"].shape
    x["k_scale"].copy_(torch.randint(0, 0x71, shape, generator=g, device="cuda"))     # up to 0.5625
    x["v_scale"].copy_(torch.randint(0, 0x71, shape, generator=g, device="cuda"))
    _check(env, w, *_run(env, w, seed=6, splits=1, x=x))
    # the largest scales: outputs of up to 6272, held to the same bar relative to them
    x["v_scale"].fill_(0xC6)
    x["v_cache"].fill_(0xFF)
    _, step = _run(env, w, seed=6, splits=1, x=x)
    assert step.device_status() == 0
    # (the step's own three rows are the prologue's, so below the largest)
    assert step.out.max() <= 6272 * (1 + 1e-2) and step.out.min() > 5000


def test_decode_strong_bias_mtp_shape(env):
    gen = env[0]
    from test_gpu_attention import _decode_table_lse_bound
    w = gen.custom("dec4-strong", Hq=64, Hkv=8, q_lens=[9, 9, 9], prefix_lens=[32759] * 3, rel_extent=1024,
                   log_scale_base=8192.0, p_std=0.5)
    x0 = gen.make_inputs(w, seed=19, device="cuda", kv_dtype="i4")
    xc = {k: x0[k].cpu() for k in ("r", "P", "cu_seqlens_q")}
    _check(env, w, *_run(env, w, seed=19), lse_tol=LSE_ABS + _decode_table_lse_bound(w, xc))


def test_decode_full_size_sampled(env):
    """The MTP-verify workload (32 x 9 queries, 32768 keys each): three sequences against the oracle."""
    gen, _, oracle, _ = env
    w = gen.workload("decode")
    x, step = _run(env, w, seed=2)
    assert step.device_status() == 0
    seqs = [0, 17, 31]
    bt = x["block_table"].cpu().numpy()
    idx = torch.as_tensor(np.concatenate([bt[b] for b in seqs]).astype(np.int64), device="cuda")
    kc = _dequant_bits(oracle, gen, x["k_cache"][idx].cpu().numpy(), x["k_scale"][idx].cpu().numpy())
    vc = _dequant_bits(oracle, gen, x["v_cache"][idx].cpu().numpy(), x["v_scale"][idx].cpu().numpy())
    rows = np.concatenate([np.arange(b * 9, b * 9 + 9) for b in seqs])
    ridx = torch.as_tensor(rows.astype(np.int64), device="cuda")
    sub = gen.custom("dec4-3", Hq=64, Hkv=8, q_lens=[9] * 3, prefix_lens=[32759] * 3, rel_extent=1024,
                     log_scale_base=8192.0)
    xs = {"cu_seqlens_q": torch.tensor([0, 9, 18, 27], dtype=torch.int32),
          "seqlen_k": torch.tensor([32768] * 3, dtype=torch.int32), "r": x["r"][ridx].cpu(), "P": x["P"].cpu(),
          "block_table": torch.arange(3 * 512, dtype=torch.int32).reshape(3, 512)}
    o_ref, lse_ref = oracle.attention_for_inputs(xs, sub, gen.bits(step.q_out)[rows], kc, vc)
    err = np.abs(step.out[ridx].cpu().numpy() - o_ref)
    assert err.max() <= MAX_ABS and err.mean() <= MEAN_ABS
    assert (np.abs(step.lse[ridx].cpu().numpy() - lse_ref) <= LSE_ABS).all()


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_bad_scale_is_flagged_and_read_as_zeros(env, mode):
    gen, _, _, ia = env
    w = gen.custom("bad4", Hq=8, Hkv=2, q_lens=[9], prefix_lens=[500], rel_extent=64)
    x = gen.make_inputs(w, seed=5, device="cuda", kv_dtype="i4")
    blk = int(x["block_table"][0, 2].item())
    x["v_scale"][blk, 1, 7, 2] = 0xC7
    x, step = _run(env, w, seed=5, mode=mode, splits=1, x=x)
    assert step.device_status() == ia.INKATTN_ERR_DEVICE_BOUNDS
    step.status.zero_()
    _check(env, w, x, step)                            # (the oracle reads the group as zeros too)


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_rows_behind_the_last_key_are_ignored(env, mode):
    """Bad scales and the code no value has in every row past a sequence's end inside its last page."""
    gen = env[0]
    w = gen.custom("end4", Hq=16, Hkv=2, q_lens=[9, 4], prefix_lens=[291, 1000], rel_extent=100)
    x = gen.make_inputs(w, seed=7, device="cuda", kv_dtype="i4")
    bt = x["block_table"].cpu().numpy()
    for b, T in enumerate(w.seqlen_k):
        last = int(bt[b, (T - 1) // 64])
        for name in ("k", "v"):
            x[f"{name}_cache"][last, :, T % 64:] = 0
            x[f"{name}_scale"][last, :, T % 64:] = 0xFF
    _check(env, w, *_run(env, w, seed=7, mode=mode, splits=1, x=x))


def test_block_ids_out_of_range_are_flagged(env):
    gen, _, _, ia = env
    w = gen.custom("blk4", Hq=8, Hkv=2, q_lens=[2], prefix_lens=[400], rel_extent=0)
    x = gen.make_inputs(w, seed=8, device="cuda", kv_dtype="i4")
    x["block_table"][0, 1] = x["k_cache"].shape[0]
    x["block_table"][0, 3] = -5
    for mode in ("decode", "prefill"):
        _, step = _run(env, w, seed=8, mode=mode, splits=1, x=x)
        assert step.device_status() == ia.INKATTN_ERR_DEVICE_BOUNDS
        assert torch.isfinite(step.out).all()


def test_decode_noalloc_and_graph_replay_are_bit_identical(env):
    gen, _, _, ia = env
    w = gen.custom("na4", Hq=16, Hkv=2, q_lens=[9, 9], prefix_lens=[2000, 700], rel_extent=128)
    x, step = _run(env, w, seed=9, splits=3)
    ref = step.out.clone()
    step.out.zero_()
    ia.inkattn_decode_noalloc(step.attn, 3)
    torch.cuda.synchronize()
    assert step.device_status() == 0 and torch.equal(step.out, ref)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        step.run_attention(s)
    step.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, ref)


def test_prefill_copy_is_the_dequantised_cache(env):
    gen, _, oracle, _ = env
    w = gen.custom("copy4", Hq=8, Hkv=2, q_lens=[70, 5], prefix_lens=[100, 250], rel_extent=64)
    x, step = _run(env, w, seed=12, mode="prefill")
    assert step.device_status() == 0
    mb = x["block_table"].shape[1]
    per = w.B * mb * w.Hkv * 64 * 128 * 2
    pad = (per + 255) // 256 * 256
    ws = step.workspace
    copies = {"k": gen.bits(ws[:per].view(torch.bfloat16)).reshape(w.B * mb, w.Hkv, 64, 128),
              "v": gen.bits(ws[pad:pad + per].view(torch.bfloat16)).reshape(w.B * mb, w.Hkv, 64, 128)}
    bt = x["block_table"].cpu().numpy()
    for b, T in enumerate(w.seqlen_k):
        for j in range((T + 63) // 64):
            rows = min(64, T - 64 * j)
            for name, got in copies.items():
                phys = int(bt[b, j])
                want = _dequant_bits(oracle, gen, x[f"{name}_cache"][phys].cpu().numpy(),
                                     x[f"{name}_scale"][phys].cpu().numpy())
                assert np.array_equal(got[b * mb + j][:, :rows] & 0x7FFF, want[:, :rows] & 0x7FFF)
                assert not got[b * mb + j][:, rows:].any()


@pytest.mark.parametrize("case", ["window_strong_bias", "full_lambda", "no_bias"])
def test_prefill_small(env, case):
    gen = env[0]
    w = {"window_strong_bias": gen.custom(case, Hq=8, Hkv=2, q_lens=[700, 130, 3], prefix_lens=[0, 200, 61],
                                          window=400, rel_extent=600, p_std=0.5),
         "full_lambda": gen.custom(case, Hq=16, Hkv=2, q_lens=[300, 260], prefix_lens=[900, 0], rel_extent=256,
                                   log_scale_base=256.0),
         "no_bias": gen.custom(case, Hq=12, Hkv=4, q_lens=[1, 333], prefix_lens=[77, 0])}[case]
    _check(env, w, *_run(env, w, seed=11, mode="prefill"))


CHILD = r"""
import json, sys
sys.path.insert(0, sys.argv[1])
import torch
from relative_bias_hybrid_gb300 import inputs as gen
from relative_bias_hybrid_gb300.step import AttentionStep
w = gen.custom("t4", Hq=16, Hkv=2, q_lens=[9, 4], prefix_lens=[2000, 700], rel_extent=200)
x = gen.make_inputs(w, seed=3, device="cuda", kv_dtype="i4")
st = AttentionStep(w, x, mode="decode", num_splits=1)
st.run_prologue()
torch.cuda.synchronize()
st.run_attention()
torch.cuda.synchronize()
print("RESULT " + json.dumps({"status": st.device_status(),
                              "usable": torch.arange(1000, device="cuda").sum().item() == 499500}))
"""


def test_decode_winds_down_when_a_wait_runs_out(env):
    """The softmax withholds its first arrival, so the MMA warp's bounded wait runs out: the kernel
    reports it, drains its copies and leaves."""
    e = dict(os.environ, INKATTN_TEST_WITHHOLD_ARRIVAL="1", INKATTN_TEST_WAIT_LIMIT_US="2000")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=e, capture_output=True, text=True, timeout=300)
    line = [ln for ln in r.stdout.splitlines() if ln.startswith("RESULT ")]
    assert r.returncode == 0 and line, r.stderr[-2000:]
    got = json.loads(line[0][7:])
    assert got == {"status": env[3].INKATTN_ERR_DEVICE_TIMEOUT, "usable": True}


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_blocks_past_32_bits_of_a_long_cache(env, mode):
    """The same sequences at the end of a cache whose codes lie past 4 GiB: the same rows and results, bit for bit."""
    gen, AttentionStep, _, _ = env
    w = gen.custom("far4", Hq=16, Hkv=8, q_lens=[9, 3], prefix_lens=[300, 70], rel_extent=64)
    x, step = _run(env, w, seed=15, mode=mode)
    assert step.device_status() == 0
    small, far = x["k_cache"].shape[0], 2 ** 32 // (8 * 64 * 64) + 5
    y = gen.make_inputs(w, seed=15, device="cuda", kv_dtype="i4")
    for c in ("k_cache", "v_cache", "k_scale", "v_scale"):
        # only the last blocks are ever read or written
        big = torch.empty((far + small, *y[c].shape[1:]), dtype=torch.uint8, device="cuda")
        big[far:] = y[c]
        y[c] = big
    y["block_table"] = torch.where(y["block_table"] < 0, y["block_table"], y["block_table"] + far)
    y["slot_mapping"] = y["slot_mapping"] + far * 64
    _, again = _run(env, w, seed=15, mode=mode, x=y)
    assert again.device_status() == 0
    for c in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(y[c][far:], x[c]), c
    assert torch.equal(again.out, step.out) and torch.equal(again.lse, step.lse)
