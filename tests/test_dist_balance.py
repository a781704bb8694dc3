"""The data-parallel training step with the router's balance loss, two gloo ranks on CPU.

The ranks hold different numbers of sequences (one of them empty, and tokens outside every sequence).  The loss
is a mean over all ranks' sequences: every rank must end with the weight gradients of one rank that saw every
token, and the ranks' losses must add up to its loss (to fp64 rounding)."""
import os
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import datagen
import oracle
import oracle.backward as ob
import oracle.balance as bal
import latent_routing_quantile_b200 as lq

SHAPE = datagen.LayerShape("dp_bal", 96, 64, 32, 32, 4, 32, 0, "f32", seed=43, offset_var=0.5)
COEF = 500.0  # as large a gradient as the rest of the router's
# (tokens, bounds) of each rank: 4 sequences hold tokens, 0 .. 10, 10 .. 33, 33 .. 55 and 64 .. 96 of the batch
RANKS = [(60, [0, 10, 10, 33, 55]), (36, [4, 36])]
FILLED = 4


class BalanceLayer:
    """A CPU stand-in for lq.Layer: the oracle's gradients with the balance loss, S' as the layer takes it."""

    balance_sequences = lq.Layer.balance_sequences

    def __init__(self, w, cu):
        self.w, self.total = w, 0
        self._balance = (torch.tensor(cu, dtype=torch.int32), len(cu) - 1)

    def set_balance_total(self, total=None, stream=None):
        self.total = 0 if total is None else int(total)

    def forward_backward(self, x, dy, weights, record_stats=False, grads=None, stream=None):
        cu = self._balance[0].tolist()
        own = sum(b > a for a, b in zip(cu, cu[1:]))
        coef = COEF * own / (self.total or own)
        b = np.zeros(SHAPE.E)
        r = oracle.layer_routing(x, self.w, b, SHAPE.k)
        cnt = bal.counts(r["idx"], SHAPE.E, cu)
        ds, _ = bal.gradient(r["s"], cnt, SHAPE.k, cu, coef)
        self.loss = bal.loss(r["s"], cnt, SHAPE.k, cu, coef)
        g = ob.layer_backward(x, self.w, b, SHAPE.k, dy, dscores=ds)
        return None, {n: torch.from_numpy(np.ascontiguousarray(v)) for n, v in g.items() if n != "idx"}


def _weights():
    return {k: oracle.f64(v) for k, v in datagen.layer_weights(SHAPE, gain="random").items()}


def _inputs():
    return datagen.tokens(SHAPE), datagen.output_grad(SHAPE, seed=SHAPE.seed + 100)


def _rank(rank, world, port, out):
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        lo = sum(n for n, _ in RANKS[:rank])
        n, cu = RANKS[rank]
        x, dy = _inputs()
        layer = BalanceLayer(_weights(), cu)
        _, g = lq.dp_train_step(layer, x[lo:lo + n], dy[lo:lo + n], None)
        out[rank] = ({n: t.numpy() for n, t in g.items()}, layer.loss, layer.total)
    finally:
        dist.destroy_process_group()


def test_ranks_with_unequal_sequences_sum_to_one_rank():
    ctx = mp.get_context("spawn")
    with ctx.Manager() as mgr:
        out = mgr.dict()
        with socket.socket() as s:
            s.bind(("127.0.0.1", 0))
            port = s.getsockname()[1]
        procs = [ctx.Process(target=_rank, args=(r, 2, port, out)) for r in range(2)]
        for p in procs:
            p.start()
        for p in procs:
            p.join(timeout=300)
            assert p.exitcode == 0
        res = dict(out)
    w, b = _weights(), np.zeros(SHAPE.E)
    x, dy = _inputs()
    r = oracle.layer_routing(x, w, b, SHAPE.k)
    # one rank that saw every token: every sequence's loss by itself, over the 4 that hold tokens
    ds, loss = np.zeros_like(r["s"]), 0.0
    for lo, hi in ((0, 10), (10, 33), (33, 55), (64, 96)):
        cnt = bal.counts(r["idx"], SHAPE.E, [lo, hi])
        ds += bal.gradient(r["s"], cnt, SHAPE.k, [lo, hi], COEF / FILLED)[0]
        loss += bal.loss(r["s"], cnt, SHAPE.k, [lo, hi], COEF / FILLED)
    ref = ob.layer_backward(x, w, b, SHAPE.k, dy, dscores=ds)
    without = ob.layer_backward(x, w, b, SHAPE.k, dy)
    assert np.linalg.norm(ref["w_router"] - without["w_router"]) > 0.2 * np.linalg.norm(without["w_router"])
    for rank in range(2):
        g, _, total = res[rank]
        assert total == 0  # back to the step's own sequences
        for n in g:
            if n != "x":
                np.testing.assert_allclose(g[n], ref[n], rtol=1e-9, atol=1e-12 * np.max(np.abs(ref[n])))
    assert abs(res[0][1] + res[1][1] - loss) <= 1e-12 * loss


@pytest.mark.parametrize("cu,n", [([0, 3, 3, 9], 2), ([0, 0], 0), ([5, 5, 5, 6], 1)])
def test_sequences_with_tokens_are_counted(cu, n):
    got = BalanceLayer(None, cu).balance_sequences(9)
    assert got.dtype == torch.int32 and got.tolist() == [n]


def test_no_exchange_without_a_balance_loss():
    layer = BalanceLayer(None, [0, 1])
    layer._balance = None
    assert layer.balance_sequences(9) is None


def test_a_refused_step_leaves_the_layer_to_its_own_sequences(monkeypatch):
    """The other ranks' sequences are one step's: a step that raises does not leave them to the next."""
    layer = BalanceLayer(None, [0, 4])

    def refused(*args, **kw):
        assert layer.total == 1
        raise lq.LmoeError("refused")

    monkeypatch.setattr(dist, "all_reduce", lambda t, group=None: None)
    monkeypatch.setattr(layer, "forward_backward", refused)
    with pytest.raises(lq.LmoeError, match="refused"):
        lq.dp_train_step(layer, torch.zeros(4, 8), None, None)
    assert layer.total == 0


def test_collectives_follow_the_named_stream(monkeypatch):
    """On a stream that the caller names, every collective and every tensor made for one is issued with that
    stream current: the sums would otherwise not wait for the step that writes what they sum."""
    import contextlib
    current, seen = ["default"], []

    @contextlib.contextmanager
    def make_current(s):
        current.append(s)
        yield
        current.pop()

    class Recorder:
        def __getattr__(self, name):
            def call(*args, **kw):
                seen.append((name, current[-1], kw.get("stream", args[-1] if args else None)))
                if name == "forward_backward":
                    return None, {"x": torch.zeros(1), "w_up": torch.zeros(1)}
                if name in ("hist", "load"):
                    return (torch.zeros(1), torch.zeros(1)) if name == "hist" else torch.zeros(1)
                return torch.zeros(1)
            return call

    monkeypatch.setattr(torch.cuda, "stream", make_current)
    monkeypatch.setattr(dist, "all_reduce", lambda t, group=None: seen.append(("all_reduce", current[-1], "side")))
    lq.dp_train_step(Recorder(), torch.zeros(4, 8), None, None, beta=0.1, sign_rule=True, stream="side")
    assert [n for n, _, _ in seen].count("all_reduce") == 1 + 1 + 3
    assert all(c == "side" for _, c, _ in seen), seen
    seen.clear()
    lq.dp_train_step(Recorder(), torch.zeros(4, 8), None, None, beta=0.1)
    assert all(c == "default" for _, c, _ in seen)
