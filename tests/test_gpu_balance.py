"""The router's balance loss and its gradient on the GPU against the float64 oracle (oracle.balance).

Tolerances, in steps of u = 2^-24 (half a step of fp32).  R and D are sums of non-negative terms in at
most 32 + 5 additions, after at most three roundings a term (f) and one for the product: relative
errors under 40 u and 44 u; 1 / R and the products add a few.  So the loss, a sum of non-negative
terms w D, is within 128 u relative (its fp32 part adds at most 24 terms a warp here), and the
gradient w (f - D) / R, whose two terms cancel, within 128 u of w (f + D) / R.
"""
import numpy as np
import pytest
import torch

import datagen
import latent_routing_quantile_b200 as lq
import oracle
import oracle.backward
import oracle.balance as ob

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latent_routing_quantile_b200 import build
    build.build()
    yield


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert lq.op_status() == 0


def inputs(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    s = torch.sigmoid(torch.randn(T, E, generator=g) + 0.7 * torch.randn(E, generator=g))
    return s, s.topk(k, dim=1).indices.int()


def check(out, s, idx, k, cu, coef):
    s64, E = s.double().numpy(), s.shape[1]
    cnt = ob.counts(idx.numpy(), E, cu)
    assert np.array_equal(out["counts"].cpu().numpy(), cnt)
    ref = ob.loss(s64, cnt, k, cu, coef)
    assert abs(float(out["loss"]) - ref) <= 128 * U * abs(ref)
    if "dscores" in out:
        g, scale = ob.gradient(s64, cnt, k, cu, coef)
        err = np.abs(out["dscores"].cpu().double().numpy() - g)
        assert (err <= 128 * U * scale).all(), float((err - 128 * U * scale).max())


@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (1, 1, 1), (3, 33, 2), (37, 64, 4), (100, 100, 5), (257, 160, 6), (300, 256, 6),
                                   (129, 512, 8), (515, 896, 16), (64, 1024, 32), (70, 1023, 3), (9000, 256, 6)])
def test_one_sequence(T, E, k):
    s, idx = inputs(T, E, k, T + E)
    check(lq.balance_loss(s.cuda(), idx.cuda(), 0.01), s, idx, k, [0, T], 0.01)
    out = lq.balance_loss(s.cuda(), idx.cuda(), 0.5, grad=False)
    assert "dscores" not in out
    check(out, s, idx, k, [0, T], 0.5)


@pytest.mark.parametrize("E", [33, 64, 256, 896])
@pytest.mark.parametrize("cu", [[0, 100, 200, 300], [0, 0, 1, 299, 300, 300], [7, 9, 9, 260], [5, 5], [0, 300], [120, 121],
                                list(range(0, 301, 3))])
def test_sequences_empty_ones_and_tokens_outside(E, cu):
    T, k = 300, 4
    s, idx = inputs(T, E, k, E)
    out = lq.balance_loss(s.cuda(), idx.cuda(), 0.01, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    check(out, s, idx, k, cu, 0.01)
    g = out["dscores"]
    assert not g[:cu[0]].any() and not g[cu[-1]:].any()


def test_long_batch_of_many_sequences():
    T, E, k = 20000, 256, 6
    s, idx = inputs(T, E, k, 4)
    r = np.random.default_rng(8)
    cu = [0] + sorted(int(v) for v in r.integers(0, T - 100, 400)) + [T - 100]
    out = lq.balance_loss(s.cuda(), idx.cuda(), 0.01, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    check(out, s, idx, k, cu, 0.01)


def test_gradient_against_differences_of_the_loss():
    """The loss of the kernel itself moves as its gradient says: along one direction, central
    differences of the float64 oracle at the kernel's counts."""
    T, E, k = 50, 64, 4
    s, idx = inputs(T, E, k, 12)
    out = lq.balance_loss(s.cuda(), idx.cuda(), 1.0)
    cnt = out["counts"].cpu().numpy()
    d = np.random.default_rng(1).standard_normal((T, E))
    h = 1e-5
    num = (ob.loss(s.double().numpy() + h * d, cnt, k, [0, T], 1.0) -
           ob.loss(s.double().numpy() - h * d, cnt, k, [0, T], 1.0)) / (2 * h)
    ana = float((out["dscores"].cpu().double().numpy() * d).sum())
    _, scale = ob.gradient(s.double().numpy(), cnt, k, [0, T], 1.0)
    assert abs(num - ana) <= 128 * U * (scale * np.abs(d)).sum() + 1e-8


def test_scores_past_32_bit_offsets():
    """More than 2^31 scores, in a few long sequences and a short last one, which comes out as it does alone."""
    T, E, k = 2_150_000, 1024, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    s = torch.rand((T, E), generator=g, device="cuda")
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    cu = [0, 1_000_000, T - 300, T]
    out = lq.balance_loss(s, idx, 0.3, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    alone = lq.balance_loss(s[-300:], idx[-300:], 0.1)  # a third of the weight: three sequences share it
    assert torch.equal(out["counts"][2], alone["counts"][0]) and int(out["counts"].sum()) == T * k
    d, ref = out["dscores"][-300:], alone["dscores"]
    assert (d - ref).abs().max() <= 16 * U * ref.abs().max()
    assert abs(float(out["loss"]) - 0.3) < 1e-2  # uniform choices: balanced but for chance
    del s, idx, out, d
    torch.cuda.empty_cache()


def test_every_expert_chosen_is_balance():
    """k = E: f is 1 everywhere, so the loss is its weight and the gradient exactly zero."""
    T, E = 500, 8
    s, idx = inputs(T, E, E, 31)
    out = lq.balance_loss(s.cuda(), idx.cuda(), 0.3)
    assert not out["dscores"].any() and abs(float(out["loss"]) - 0.3) <= 8 * U * 0.3


def test_slots_without_an_expert_zero_rows_and_equal_experts():
    T, E, k = 40, 64, 4
    s, idx = inputs(T, E, k, 5)
    idx[3, 1:] = -1
    idx[10] = -1
    idx[11] = 7          # the same expert in every slot counts every slot
    s[12] = 0            # no probabilities: adds nothing, gradient zero
    out = lq.balance_loss(s.cuda(), idx.cuda(), 0.1)
    check(out, s, idx, k, [0, T], 0.1)
    assert not out["dscores"][12].any()


def test_no_tokens():
    s, idx = torch.empty(0, 64, device="cuda"), torch.empty(0, 4, dtype=torch.int32, device="cuda")
    out = lq.balance_loss(s, idx, 0.1)
    assert float(out["loss"]) == 0 and not out["counts"].any() and out["dscores"].shape == (0, 64)


def test_nan_scores_bad_experts_and_bad_bounds_are_reported():
    T, E, k = 40, 64, 4
    s, idx = inputs(T, E, k, 5)
    for v in (float("nan"), float("inf")):
        bad = s.clone()
        bad[9, 3] = v
        out = lq.balance_loss(bad.cuda(), idx.cuda(), 0.1)
        assert lq.op_status() == lq.STATUS_NAN_SCORE
        assert torch.isnan(out["loss"]).all() and torch.isnan(out["dscores"][9]).all()
        g = out["dscores"].cpu()
        keep = torch.arange(T) != 9
        assert torch.isfinite(g[keep]).all()
    wrong = idx.clone()
    wrong[2, 0], wrong[5, 1] = E, -7
    out = lq.balance_loss(s.cuda(), wrong.cuda(), 0.1)
    assert lq.op_status() == lq.STATUS_BAD_INDEX
    wrong[2, 0] = wrong[5, 1] = -1
    check(out, s, wrong, k, [0, T], 0.1)
    for cu in ([0, 50], [-3, 40], [0, 30, 20]):
        lq.balance_loss(s.cuda(), idx.cuda(), 0.1, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
        assert lq.op_status() == lq.STATUS_BAD_INDEX


def test_misaligned_buffers_and_given_outputs():
    T, E, k = 50, 64, 4
    s, idx = inputs(T, E, k, 6)
    sb = torch.empty(T * E + 1, device="cuda")[1:].view(T, E)
    sb.copy_(s)
    gb = torch.empty(T * E + 3, device="cuda")[3:].view(T, E)
    out = lq.balance_loss(sb, idx.cuda(), 0.1, out=dict(dscores=gb))
    assert out["dscores"] is gb
    check(out, s, idx, k, [0, T], 0.1)


def test_repeats_streams_and_graph_replay():
    T, E, k = 3000, 256, 6
    data = [inputs(T, E, k, 20 + i) for i in range(4)]
    dev = [(s.cuda(), i.cuda()) for s, i in data]
    cu = torch.tensor([0, 1000, 1700, 2900], dtype=torch.int32, device="cuda")
    ref = [lq.balance_loss(s, i, 0.01, cu_seqlens=cu) for s, i in dev]
    same = lambda a, b: all(torch.equal(a[n], b[n]) for n in ("loss", "counts", "dscores"))
    assert all(same(lq.balance_loss(s, i, 0.01, cu_seqlens=cu), r) for (s, i), r in zip(dev, ref))
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in dev]
    got = []
    for (s, i), st in zip(dev, ss):
        st.wait_stream(torch.cuda.current_stream())
        got.append(lq.balance_loss(s, i, 0.01, cu_seqlens=cu, stream=st))
    for st in ss:
        torch.cuda.current_stream().wait_stream(st)
    assert all(same(u, v) for u, v in zip(got, ref))
    s, i = dev[0][0].clone(), dev[0][1].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = lq.balance_loss(s, i, 0.01, cu_seqlens=cu)
    s.copy_(dev[2][0]); i.copy_(dev[2][1])
    g.replay()
    assert same(out, ref[2])


# ------------------------------------------------------------------ in the training step
def train_layer(shape, w_dev):
    return lq.Layer(shape.d, shape.l, shape.E, shape.k, shape.h, shape.hs, lq.BF16, shape.T, w_dev, rms_eps=shape.rms_eps)


def train_reference(shape, w, x, dy, cu, coef):
    r = oracle.layer_routing(x, w, np.zeros(shape.E), shape.k, shape.rms_eps)
    cnt = ob.counts(r["idx"], shape.E, cu)
    ds, _ = ob.gradient(r["s"], cnt, shape.k, cu, coef)
    return (oracle.backward.layer_backward(x, w, np.zeros(shape.E), shape.k, dy, shape.rms_eps, dscores=ds),
            ob.loss(r["s"], cnt, shape.k, cu, coef), cnt)


def check_train(grads, ref, names=("x", "w_router", "router_bias", "w_down", "rms_gain", "w_up")):
    """As for the backward's other gradients: at most 8 bf16 roundings on the longest chain, 2e-2 of the
    largest magnitude."""
    for n in names:
        err = np.abs(grads[n].cpu().double().numpy() - ref[n]).max() / np.abs(ref[n]).max()
        assert err <= 2e-2, (n, err)


@pytest.mark.parametrize("T,E,k,cu", [(300, 64, 4, None), (300, 128, 6, [0, 130, 130, 290]), (1, 64, 4, None),
                                      (200, 64, 4, [7, 150])])
def test_training_step_with_a_balance_loss(T, E, k, cu):
    """The weight makes the balance gradient as large as the rest of the router's (so that one left out, or
    taken twice, fails)."""
    shape = datagen.LayerShape("bal_train", T, 256, 128, E, k, 128, 256, "bf16", seed=91, offset_var=0.5)
    w = datagen.layer_weights(shape, gain="random")
    x, dy = datagen.tokens(shape), datagen.output_grad(shape, seed=191)
    w_dev = {n: t.cuda() for n, t in w.items()}
    layer = train_layer(shape, w_dev)
    y0, g0 = layer.forward_backward(x.cuda(), dy.cuda(), w_dev)
    bounds = [0, T] if cu is None else cu
    coef = 20.0 * T
    ref, loss, cnt = train_reference(shape, w, x, dy, bounds, coef)
    layer.set_balance(coef, None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"))
    y, g = layer.forward_backward(x.cuda(), dy.cuda(), w_dev)
    got_loss, got_cnt = layer.balance()
    assert torch.equal(y, y0)
    assert np.array_equal(got_cnt.cpu().numpy(), cnt)
    assert abs(float(got_loss) - loss) <= 1e-4 * loss  # the scores are within 2e-6 of the oracle's
    check_train(g, ref)
    assert (g["w_router"] - g0["w_router"]).norm() > 0.05 * g0["w_router"].norm()
    for n in ("w1", "w3", "w2", "w_up", "ws2"):
        # nothing on the experts' side of the choice changes (sums over K ranges may differ in the last bits)
        assert torch.allclose(g[n], g0[n], rtol=1e-4, atol=1e-4 * float(g0[n].abs().max())), n
    layer.set_balance(0.0)
    _, g1 = layer.forward_backward(x.cuda(), dy.cuda(), w_dev)
    for n in ("x", "w_router", "router_bias"):
        assert torch.allclose(g1[n], g0[n], rtol=1e-4, atol=1e-4 * float(g0[n].abs().max())), n
    with pytest.raises(lq.LmoeError):
        layer.balance()
    assert layer.status() == 0
    layer.close()


def test_training_steps_replay_with_new_bounds_and_more_sequences():
    shape = datagen.LayerShape("bal_replay", 256, 256, 128, 64, 4, 128, 0, "bf16", seed=92, offset_var=0.5)
    w = datagen.layer_weights(shape)
    x, dy = datagen.tokens(shape), datagen.output_grad(shape, seed=192)
    w_dev, xd, dyd = {n: t.cuda() for n, t in w.items()}, x.cuda(), dy.cuda()
    layer = train_layer(shape, w_dev)
    cu = torch.tensor([0, 100, 256], dtype=torch.int32, device="cuda")
    layer.set_balance(3000.0, cu)
    y, g = layer.forward_backward(xd, dyd, w_dev)
    for _ in range(3):  # eager, captured, replayed
        layer.forward_backward(xd, dyd, w_dev, y=y, grads=g)
    check_train(g, train_reference(shape, w, x, dy, [0, 100, 256], 3000.0)[0])
    cu.copy_(torch.tensor([0, 31, 200], dtype=torch.int32))  # other bounds, same graph
    layer.forward_backward(xd, dyd, w_dev, y=y, grads=g)
    check_train(g, train_reference(shape, w, x, dy, [0, 31, 200], 3000.0)[0])
    five = [0, 50, 100, 150, 200, 256]
    layer.set_balance(1000.0, torch.tensor(five, dtype=torch.int32, device="cuda"))
    layer.forward_backward(xd, dyd, w_dev, y=y, grads=g)
    ref, loss, cnt = train_reference(shape, w, x, dy, five, 1000.0)
    check_train(g, ref)
    assert np.array_equal(layer.balance()[1].cpu().numpy(), cnt)
    assert layer.status() == 0
    # bounds that do not fit the step: reported, and no balance loss
    layer.set_balance(1000.0, torch.tensor([0, 300], dtype=torch.int32, device="cuda"))
    layer.forward_backward(xd, dyd, w_dev, y=y, grads=g)
    assert layer.status() == lq.STATUS_BAD_INDEX
    check_train(g, oracle.backward.layer_backward(x, w, np.zeros(64), 4, dy, shape.rms_eps))
    layer.close()


def test_training_balance_is_refused_where_there_is_no_training():
    shape = datagen.LayerShape("bal_mx", 64, 256, 128, 64, 4, 128, 256, "bf16", seed=74)
    layer = lq.layer_from_weights(shape, datagen.layer_weights(shape), experts=lq.EXPERTS_MXFP4)
    with pytest.raises(lq.LmoeError, match="unsupported"):
        layer.set_balance(0.1)
    layer.close()
    layer = lq.layer_from_weights(shape, datagen.layer_weights(shape))
    with pytest.raises(lq.LmoeError, match="invalid"):
        layer.set_balance(float("nan"))
    layer.set_balance(0.0, torch.zeros(100, dtype=torch.int32, device="cuda"))  # off: nothing is kept of it
    layer.set_balance(0.1, torch.tensor([0, 64], dtype=torch.int32, device="cuda"))
    layer.close()
