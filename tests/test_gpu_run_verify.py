"""`run --verify`: every pass rolls back from the conv states that this pass started from."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "i4"])
def test_every_pass_rolls_back_from_its_own_states(monkeypatch, kv):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from relative_bias_hybrid_gb300 import run
    started, checked = [], []

    class Step(run.AttentionStep):
        def run_prologue(self, stream=None):
            started.append([self.x[f"conv_state_{n}"].clone() for n in ("k", "v")])
            super().run_prologue(stream)

    class End(run.VerifyStep):
        def __init__(self, w, inputs, logits, convs=()):
            super().__init__(w, inputs, logits, convs)
            self.convs = convs

        def run(self, stream=None):
            super().run(stream)
            torch.cuda.synchronize()
            cu, keep = self.x["cu_seqlens_q"].tolist(), self.n_new.tolist()
            slots = self.x["state_slot"].tolist()
            for (x, _, after), before in zip(self.convs, started[-1]):
                for b, n in enumerate(keep):
                    want = torch.cat([before[slots[b]], x[cu[b]:cu[b] + n]])[-3:]
                    checked.append((n, torch.equal(after[slots[b]], want)))

    monkeypatch.setattr(run, "AttentionStep", Step)
    monkeypatch.setattr(run, "VerifyStep", End)
    run.main(["decode", "--seqs", "3", "--iters", "3", "--verify", "1003", "--kv", kv])
    assert len(started) == 3 and len(checked) == 3 * 2 * 3
    # (rows of the state before stay where fewer than three are kept)
    assert any(n < 3 for n, _ in checked)
    assert all(same for _, same in checked)
