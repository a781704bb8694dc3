"""The balance loss of the training step (Layer.set_balance) between steps: what a later call may count on."""
import numpy as np
import pytest
import torch

import datagen
import latent_routing_quantile_b200 as lq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latent_routing_quantile_b200 import build
    build.build()
    yield


class Step:
    """A small layer with its inputs."""

    def __init__(self, T=256, E=64, k=4, seed=95):
        self.shape = s = datagen.LayerShape("bal_step", T, 256, 128, E, k, 128, 0, "bf16", seed=seed, offset_var=0.5)
        self.w = datagen.layer_weights(s)
        self.w_dev = {n: t.cuda() for n, t in self.w.items()}
        self.x, self.dy = datagen.tokens(s).cuda(), datagen.output_grad(s, seed=seed + 100).cuda()
        self.layer = lq.Layer(s.d, s.l, E, k, s.h, s.hs, lq.BF16, T, self.w_dev, rms_eps=s.rms_eps)

    def run(self, **kw):
        return self.layer.forward_backward(self.x, self.dy, self.w_dev, **kw)[1]


def bounds(*cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


@pytest.fixture
def step():
    s = Step()
    yield s
    s.layer.close()


def test_set_balance_returns_once_no_step_reads_the_old_bounds(step):
    """The binding drops the old bounds when it returns: a step on another stream has to be done with them,
    whatever changed (bounds, weight, off)."""
    side, gate = torch.cuda.Stream(), torch.cuda.Event()
    step.layer.set_balance(1.0, bounds(0, 100, 256))
    torch.cuda.synchronize()
    for change in ((1.0, bounds(0, 50, 256)), (2.0, bounds(0, 256)), (0.0, None)):
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)  # some 25 ms before the step begins
        step.run(stream=side)
        gate.record(side)
        step.layer.set_balance(*change)
        assert gate.query()
    assert step.layer.status() == 0


def test_more_sequences_than_a_step_takes_are_refused_at_once(step):
    """Not by the steps, after their forward; the settings before stay."""
    step.layer.set_balance(1.0)
    cu = torch.zeros((1 << 24) + 2, dtype=torch.int32, device="cuda")
    with pytest.raises(lq.LmoeError, match="unsupported"):
        step.layer.set_balance(1.0, cu)
    step.run()
    assert step.layer.balance()[1].shape == (1, 64) and float(step.layer.balance()[0]) > 0


def test_no_results_of_steps_before_the_settings(step):
    """Fewer sequences fit the buffers of more: what balance() gives before the next step is not the old step's
    counts in another shape."""
    step.layer.set_balance(1.0, bounds(0, 50, 100, 150, 200, 256))
    step.run()
    loss, counts = step.layer.balance()
    assert float(loss) > 0 and counts.sum(1).tolist() == [200, 200, 200, 200, 224]
    for change in ((1.0, bounds(0, 100, 256)), (2.0, bounds(0, 100, 256)), (1.0, None)):
        step.layer.set_balance(*change)
        loss, counts = step.layer.balance()
        assert not loss.any() and not counts.any()
        step.run()
        loss, counts = step.layer.balance()
        assert float(loss) > 0 and int(counts.sum()) == 4 * 256
