"""The bench and the workload runner make their inputs on one stream and run on another: the first pass waits for
them.  Inputs here become right only a while after they were asked for; before that their sequence offsets are out
of range, which the kernels flag and both programs report.  Twice each: loading a kernel for the first time waits
for the device anyway."""
import argparse

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def late(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import build
    build.build()
    from relative_bias_hybrid_gb300 import inputs as gen
    asked = []

    def slowly(make):
        def wrapped(*args, **kwargs):
            x = make(*args, **kwargs)
            cu = x["cu_seqlens_q"]
            if cu.is_cuda:
                right = cu.clone()
                cu.fill_(-1)
                torch.cuda.synchronize()
                torch.cuda._sleep(100_000_000)               # some 50 ms
                cu.copy_(right)
                asked.append(make.__name__)
            return x
        return wrapped

    def small(name, seed=0):
        q, cached = ([9, 4] * 16, [300, 40] * 16) if name == "decode" else ([200, 70], [300, 40])
        return gen.custom(name, Hq=16, Hkv=2, q_lens=q, prefix_lens=cached, rel_extent=32)

    for name in ("make_inputs", "make_output_conv_inputs", "make_qkvr_inputs"):
        monkeypatch.setattr(gen, name, slowly(getattr(gen, name)))
    monkeypatch.setattr(gen, "workload", small)
    return asked


@pytest.mark.parametrize("name", ["decode", "decode_e4m3", "full", "full_e4m3"])
def test_the_bench_waits_for_its_inputs(late, name):
    import bench
    dev = torch.device("cuda", 0)
    flush = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    for _ in range(2):
        _, launches, _ = bench.measure(name, argparse.Namespace(steps=2, warmup=3, gpus=1), bench.load_peaks(), dev,
                                       torch.cuda.Stream(device=dev), flush)
        assert launches > 0
    assert "make_inputs" in late
    if name == "full":
        assert {"make_output_conv_inputs", "make_qkvr_inputs"} <= set(late)


@pytest.mark.parametrize("args", [["decode", "--kv", "i4"], ["full", "--output-conv", "--qkvr"], ["decode", "--verify", "1003"]])
def test_the_runner_waits_for_its_inputs(late, monkeypatch, args):
    """One pass: had it run ahead, it would have skipped every sequence (and its status been zeroed behind it)."""
    from relative_bias_hybrid_gb300 import run
    made = []

    class Step(run.AttentionStep):
        def __init__(self, *a, **k):
            super().__init__(*a, **k)
            self.q_out.fill_(7.0)
            made.append(self)

    monkeypatch.setattr(run, "AttentionStep", Step)
    for _ in range(2):
        run.main([*args, "--iters", "1"])
        torch.cuda.synchronize()
        got = made[-1].q_out.clone()
        made[-1].q_out.zero_()
        made[-1].run_prologue()
        torch.cuda.synchronize()
        assert torch.equal(got, made[-1].q_out)
    assert "make_inputs" in late
