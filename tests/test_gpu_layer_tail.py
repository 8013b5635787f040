"""The products of the layer's second half used together and in the ways a program uses them:
the whole rest of the layer against 64-bit forms stage by stage, CUDA graphs, streams, large
arrays, the command line, and the failure path of the bounded waits."""
import json
import os
import subprocess
import sys
import threading

import pytest
import torch

from test_gpu_layer_products import _check, _check_route

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    from relative_bias_hybrid_gb300 import inputs as gen
    import relative_bias_hybrid_gb300.inkattn as ia
    from relative_bias_hybrid_gb300.step import LayerTailStep
    return gen, ia, LayerTailStep


def _tail(env, q_lens, seed=0, Hq=4, **kw):
    gen, _, LayerTailStep = env
    w = gen.custom("tail", Hq=Hq, Hkv=1, q_lens=q_lens, prefix_lens=[5] * len(q_lens))
    x = gen.make_layer_tail_inputs(w, seed=seed, device="cuda", **kw)
    attn = torch.randn((w.N_tok, Hq, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(BF16)
    return LayerTailStep(w, x, attn, top_k=3), x, attn


def _near_product(got, x, w, act="none"):
    """Within the rounding of got's type and of K fp32 additions, each off by at most a step of the
    sum of magnitudes."""
    x, w = x.cpu().double(), w.cpu().double()
    _check(got, x @ w.t(), act, sum_slack=x.shape[1] * 2.0 ** -23 * (x.abs() @ w.abs().t()))


@pytest.mark.parametrize("q_lens", [[1], [9, 3, 1], [150, 40, 300]])
def test_tail_stage_by_stage(env, q_lens):
    step, x, attn = _tail(env, q_lens, seed=len(q_lens), experts=12, n_shared=2, ff=136)
    resid = x["attn"]["residual"].clone()
    step.run()
    torch.cuda.synchronize()
    assert step.device_status() == 0
    assert torch.equal(x["attn"]["residual"], resid)
    N, r = attn.shape[0], step.route
    _near_product(step.proj, attn.view(N, -1), x["w_o"])
    _near_product(step.logits, step.normed, x["w_router"])
    _check_route({k: v.cpu() for k, v in r.items()}, step.logits.cpu(), 2, 3, "sigmoid")
    offs = r["expert_offsets"].tolist()
    for e in range(12):
        rows = slice(offs[e], offs[e + 1])
        _near_product(step.inner[rows], step.normed[r["row_token"][rows].long()], x["w_up"][e], "swiglu")
        _near_product(step.rows[rows], step.inner[rows], x["w_down"][e])
    # (the inner rows that are still there are the last shared expert's)
    _near_product(step.shared_inner, step.normed, x["w_shared_up"][1], "swiglu")
    _near_product(step.shared_rows[1], step.shared_inner, x["w_shared_down"][1])
    w = r["weights"].double()
    terms = torch.cat([step.rows[r["token_rows"].long()].double() * w[:, :3, None],
                       step.shared_rows.double().transpose(0, 1) * w[:, 3:, None]], 1)
    want, slack = terms.sum(1), 5 * 2.0 ** -24 * terms.abs().sum(1)        # one rounding a term
    assert bool(((step.mlp.double() - want).abs() <= slack + 2.0 ** -8 * (want.abs() + slack)).all())
    assert bool(torch.isfinite(step.out.float()).all()) and float(step.out.float().abs().max()) > 0


def test_tail_replays_from_a_cuda_graph_with_other_tokens(env):
    """One captured graph serves other hidden states, and so another split of the rows among the
    experts: a replay writes what the direct calls write, bit for bit."""
    step, x, attn = _tail(env, [60, 9], seed=3, experts=10, n_shared=1, ff=264)
    states = [x["attn"]["conv_state"], x["mlp"]["conv_state"]]
    saved = [t.clone() for t in states]

    def reset(seed):
        attn.copy_(torch.randn(attn.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        for t, s in zip(states, saved):
            t.copy_(s)

    step.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    seen = []
    for seed in (11, 12):
        outs = []
        for direct in (True, False):
            reset(seed)
            for t in (step.out, step.h, step.rows, step.route["row_token"]):
                t.zero_()
            step.run() if direct else graph.replay()
            torch.cuda.synchronize()
            outs.append([t.clone() for t in (step.out, step.h, step.rows, step.route["row_token"],
                                             step.route["expert_offsets"], *states)])
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        seen.append(outs[0])
    assert not torch.equal(seen[0][4], seen[1][4])          # another split of the rows
    assert step.device_status() == 0


def test_two_streams_and_two_threads(env):
    """Two steps of their own buffers at once, each from its own host thread and stream."""
    steps = [_tail(env, [200, 31], seed=s, experts=16, n_shared=2, ff=128)[0] for s in (5, 6)]
    alone = []
    for st in steps:
        saved = [st.x[p]["conv_state"].clone() for p in ("attn", "mlp")]
        st.run()
        torch.cuda.synchronize()
        alone.append(st.out.clone())
        for p, t in zip(("attn", "mlp"), saved):
            st.x[p]["conv_state"].copy_(t)
        st.out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    threads = [threading.Thread(target=st.run, args=(s,)) for st, s in zip(steps, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for st, want in zip(steps, alone):
        assert st.device_status() == 0 and torch.equal(st.out, want)


def test_calls_wait_for_the_work_before_them(env):
    """A product reads what the calls just before it on the stream wrote, over and over."""
    _, ia, _ = env
    T, K = 64, 512
    g = torch.Generator().manual_seed(1)
    eye = torch.eye(K, dtype=BF16, device="cuda")
    a = (torch.randint(-8, 9, (T, K), generator=g) / 8).to(BF16).cuda()
    b, first = torch.empty_like(a), a.clone()
    p = [ia.linear_params(x=a, w=eye, out=b), ia.linear_params(x=b, w=eye, out=a, residual=b)]
    for i in range(6):                                      # a <- 2 a, exactly, each round
        ia.inkattn_linear(p[0])
        ia.inkattn_linear(p[1])
    torch.cuda.synchronize()
    assert torch.equal(a.float(), first.float() * 64)


def test_host_memory_is_refused(env):
    """Tensors in host memory, pinned or not: refused by the library, nothing launched."""
    _, ia, _ = env
    x, w, out = (torch.zeros(s, dtype=BF16) for s in ((4, 16), (8, 16), (4, 8)))
    i32 = torch.int32
    for pin in (False, True):
        a, b, c = (t.pin_memory() if pin else t for t in (x, w, out))
        calls = [
            (ia.inkattn_linear, ia.linear_params(x=a, w=b, out=c)),
            (ia.inkattn_grouped_linear, ia.grouped_linear_params(
                x=a, w=b[None], out=c, expert_offsets=torch.zeros(2, dtype=i32))),
            (ia.inkattn_expert_combine, ia.expert_combine_params(
                y=a, weights=torch.zeros(4, 1), token_rows=torch.zeros(4, 1, dtype=i32), out=torch.zeros_like(a))),
            (ia.inkattn_route, ia.route_params(
                logits=torch.zeros(4, 8), topk_ids=torch.zeros(4, 1, dtype=i32), weights=torch.zeros(4, 1),
                expert_offsets=torch.zeros(9, dtype=i32), row_token=torch.zeros(4, dtype=i32),
                token_rows=torch.zeros(4, 1, dtype=i32)))]
        for call, p in calls:
            assert call(p, raise_on_error=False) == ia.INKATTN_ERR_INVALID_ARG, call.__name__


def test_arrays_past_32_bits(env):
    """Outputs, weights and inputs of more than 2^31 elements: rows at the far end."""
    _, ia, _ = env
    g = torch.Generator("cuda").manual_seed(2)

    def grid(shape, unit):
        return (torch.randint(-8, 9, shape, generator=g, device="cuda", dtype=torch.int8).to(BF16) * unit)

    # 66000 x 33000 outputs
    x, w = grid((66000, 16), 1 / 8), grid((33000, 16), 1 / 64)
    out = torch.empty((66000, 33000), dtype=BF16, device="cuda")
    ia.inkattn_linear(ia.linear_params(x=x, w=w, out=out))
    for rows in (slice(0, 3), slice(40000, 40003), slice(65997, 66000)):
        assert torch.equal(out[rows], (x[rows].double() @ w.double().t()).to(F32).to(BF16))
    del out, x, w
    # 70 experts of 8192 x 4096 weights, and 600000 rows of x that the last row indices name
    E, F, K, N = 70, 8192, 4096, 600000
    w, x = grid((E, F, K), 1 / 64), grid((N, K), 1 / 8)
    tok = torch.tensor([N - 1, 5, N - 2, 0, N - 7], dtype=I32, device="cuda")
    offs = torch.tensor([0] * (E - 1) + [2, 5], dtype=I32, device="cuda")
    out = torch.empty((5, F), dtype=F32, device="cuda")
    ia.inkattn_grouped_linear(ia.grouped_linear_params(x=x, w=w, expert_offsets=offs, row_token=tok, out=out))
    for i in range(5):
        e = E - 2 if i < 2 else E - 1
        assert torch.equal(out[i], (w[e].double() @ x[int(tok[i])].double()).to(F32))


def test_expert_combine_past_32_bits(env):
    _, ia, _ = env
    M, F = 140000, 16384
    y = torch.zeros((M, F), dtype=BF16, device="cuda")
    y[M - 1], y[M - 2] = 2.0, 3.0
    rows = torch.tensor([[M - 1, M - 2]], dtype=I32, device="cuda")
    w = torch.tensor([[0.5, 2.0]], device="cuda")
    out = torch.empty((1, F), dtype=BF16, device="cuda")
    ia.inkattn_expert_combine(ia.expert_combine_params(y=y, weights=w, token_rows=rows, out=out))
    assert bool((out == 7).all())


def test_command_line(env):
    r = subprocess.run([sys.executable, "-m", "relative_bias_hybrid_gb300.run", "tiny", "--iters", "2", "--layer-tail",
                        "--experts", "8", "--expert-width", "256"], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "rest of the layer" in r.stdout and "device status 0" in r.stdout


CHILD = r"""
import json, sys, time
sys.path.insert(0, sys.argv[1])
import torch
import relative_bias_hybrid_gb300.inkattn as ia
BF = torch.bfloat16
res = {}
def go(name, make, call):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = make(status)
    torch.cuda.synchronize()
    t0 = time.time()
    call(p)
    torch.cuda.synchronize()
    res[name] = {"status": int(status), "seconds": time.time() - t0}
# enough items that every pair takes at least three: the first accumulator is wanted again
x, w = torch.zeros((20000, 64), dtype=BF, device="cuda"), torch.zeros((4096, 64), dtype=BF, device="cuda")
out = torch.empty((20000, 4096), dtype=BF, device="cuda")
go("linear", lambda s: ia.linear_params(x=x, w=w, out=out, dev_status=s), ia.inkattn_linear)
we = w.view(4, 1024, 64)
offs = torch.tensor([0, 5000, 10000, 10000, 20000], dtype=torch.int32, device="cuda")
tok = torch.arange(20000, dtype=torch.int32, device="cuda").flip(0)
half = out.view(-1)[:20000 * 512].view(20000, 512)
go("gathered", lambda s: ia.grouped_linear_params(x=x, w=we, expert_offsets=offs, row_token=tok, out=half,
                                                  act="swiglu", dev_status=s), ia.inkattn_grouped_linear)
res["context_usable"] = torch.arange(1000, device="cuda", dtype=torch.float32).sum().item() == 499500.0
print("RESULT " + json.dumps(res))
"""


@pytest.mark.parametrize("withhold", [False, True])
def test_withheld_release_times_out_cleanly(env, withhold):
    """With one release of an accumulator withheld and a wait limit of 2 ms, the products report
    INKATTN_ERR_DEVICE_TIMEOUT and return; without the setting the same calls succeed."""
    e = {k: v for k, v in os.environ.items() if not k.startswith("INKATTN_TEST_")}
    if withhold:
        e.update(INKATTN_TEST_WITHHOLD_ARRIVAL="1", INKATTN_TEST_WAIT_LIMIT_US="2000")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=e, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    res = json.loads([l for l in r.stdout.splitlines() if l.startswith("RESULT ")][-1][len("RESULT "):])
    assert res.pop("context_usable") is True
    for name, v in res.items():
        assert v["status"] == (4 if withhold else 0) and v["seconds"] < 10.0, (name, v)
