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


def test_total_of_all_ranks_scales_the_steps_loss_and_gradient(step):
    """S' of the whole group in the place of the step's own 2: loss and gradient 2 / 5 of what they were, in
    steps that replay one graph, until it is taken back."""
    g0 = {n: t.clone() for n, t in step.run().items()}
    step.layer.set_balance(2e4, bounds(0, 100, 100, 256))
    grads = step.run()
    for _ in range(3):  # eager, captured, replayed
        step.run(grads=grads)
    own, (loss, counts) = {n: t.clone() for n, t in grads.items()}, step.layer.balance()
    for total, share in ((5, 0.4), (1000, 0.002), (None, 1.0), (2, 1.0), (0, 1.0)):
        step.layer.set_balance_total(None if total is None else torch.tensor([total], dtype=torch.int32, device="cuda"))
        step.run(grads=grads)
        got, cnt = step.layer.balance()
        assert torch.equal(cnt, counts)
        assert abs(float(got) - share * float(loss)) <= 8 * 2.0 ** -24 * float(loss)
        for n in ("w_router", "router_bias", "w_down"):
            # bf16 operands: 2^-8 of the larger of the two gradients' sizes a rounding, two on the way
            size = float(own[n].abs().max())
            want = g0[n] + share * (own[n] - g0[n])
            assert float((grads[n] - want).abs().max()) <= 4 * 2.0 ** -8 * size, (n, total)
        assert float((own["router_bias"] - g0["router_bias"]).abs().max()) > 0.2 * float(g0["router_bias"].abs().max())
    step.layer.set_balance_total(torch.tensor([9], dtype=torch.int32, device="cuda"))
    step.layer.set_balance(2e4, bounds(0, 100, 100, 256))  # its own again
    step.run(grads=grads)
    assert abs(float(step.layer.balance()[0]) - float(loss)) <= 8 * 2.0 ** -24 * float(loss)
    step.layer.set_balance(0.0)
    with pytest.raises(lq.LmoeError, match="invalid"):
        step.layer.set_balance_total(None)


def test_data_parallel_step_of_one_rank_on_a_named_stream(step):
    """dp_train_step with a balance loss in a group of one: the step's own gradients and loss."""
    import datetime
    import socket
    import torch.distributed as dist
    step.layer.set_balance(2e4, bounds(0, 100, 100, 256))
    ref = step.run()
    loss = float(step.layer.balance()[0])
    torch.cuda.synchronize()
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    dist.init_process_group("nccl", init_method=f"tcp://127.0.0.1:{port}", rank=0, world_size=1,
                            timeout=datetime.timedelta(seconds=120))
    try:
        side = torch.cuda.Stream()
        for stream in (None, side):
            _, g = lq.dp_train_step(step.layer, step.x, step.dy, step.w_dev, beta=0.01, stream=stream)
            torch.cuda.synchronize()
            assert abs(float(step.layer.balance()[0]) - loss) <= 2.0 ** -20 * loss
            step.layer.set_bias(torch.zeros(64, device="cuda"))
            for n in ref:
                # sums over K ranges in another order: the last bits
                assert torch.allclose(g[n], ref[n], rtol=1e-4, atol=1e-4 * float(ref[n].abs().max())), n
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("T,kernels", [(256, 1), (8300, 2)])
def test_launch_count_of_a_step(T, kernels):
    """The loss is one kernel up to 2^19 scores and two above; two more sum the offsets' gradient.  Eager,
    captured and replayed steps count alike."""
    step = Step(T=T)
    grads = step.run()

    def counts():
        out = []
        for _ in range(4):
            before = step.layer.launches()
            step.run(grads=grads)
            out.append(step.layer.launches() - before)
        return out

    without = counts()
    step.layer.set_balance(1.0)
    assert counts() == [n + kernels + 2 for n in without]
    step.layer.close()


def test_results_on_a_named_stream_belong_to_it(step):
    """balance(stream) writes into memory of that stream's: a block that the current stream has let go of may
    still be read there by work that is queued."""
    step.layer.set_balance(1.0)
    step.run()
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), None):
        loss, counts = step.layer.balance(stream=stream)
        torch.cuda.synchronize()
        assert int(counts.sum()) == 4 * 256 and float(loss) > 0
        for t in (loss, counts):
            owner = [s["stream"] for s in torch.cuda.memory_snapshot()
                     if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
            assert owner == [0 if stream is None else stream.cuda_stream]


def test_replayed_steps_of_large_batches_take_their_own_scores():
    """Above 2^19 scores (zeroed counts, counting, the pass: three nodes of the replayed backward), with inputs
    that change between the replays: loss and counts of the step's own scores and choice."""
    import oracle.balance as ob
    step = Step(T=8300)
    cu = [0, 1000, 1000, 5000, 8200]
    step.layer.set_balance(3.0, bounds(*cu))
    grads = step.run()
    x = step.x.clone()
    for i in range(4):
        step.x.copy_(x.roll(7 * i, 0))
        step.run(grads=grads)
        loss, counts = step.layer.balance()
        r = step.layer.routing()
        s, idx = r["scores"].double().cpu().numpy(), r["idx"].cpu().numpy()
        cnt = ob.counts(idx, 64, cu)
        assert np.array_equal(counts.cpu().numpy(), cnt)
        ref = ob.loss(s, cnt, 4, cu, 3.0)
        # each token's D to 84 u of its size and of 1, D near 1 here: 256 u of the mean
        assert abs(float(loss) - ref) <= 256 * 2.0 ** -24 * ref
    assert step.layer.status() == 0
    step.layer.close()
