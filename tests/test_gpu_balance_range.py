"""The router's balance loss over the whole range of scores, against float64 sums of its definition.

Tolerances, in u = 2^-24 (half a step of fp32), for the first-order terms; A = sum_e p |f - 1|.
f - 1 and f are off by 4 u relative (whole number to fp32, k n to fp32, its reciprocal, the product).
R is a sum of at most 32 terms a lane and 5 exchanges: 37 u.  sum s (f - 1): 4 + 32 + 5 roundings a term, so
45 u A R at most; divided by R: D - 1 is off by 45 u A + 39 u |D - 1| <= 84 u A.  w_q: 4 u.
  gradient w (f - D) / R:  u (4 |f - 1| + 84 A + (|f - 1| + A)) for the difference and 44 u (|f - 1| + A) for
  the factors: 136 u (|f - 1| + A) w / R covers it.
A form that takes D = sum p f as it is has 48 f + 123 D in that place, and where D < 1/2 (so A > 1/2, and
f <= |f - 1| + 2 A) that is at most 48 |f - 1| + 219 A: 224 u covers both.
  loss sum w D:  84 u A a token, a few roundings of the whole.
Where D < 1/2 alone, with D = sum p f a sum of non-negative terms: f 4 u, D 4 + 37 + 37 + 1 = 79 u, their
difference 4 f + 79 D + (f + D), the factors 44 (f + D): 128 u (f + D) w / R covers it, and 84 u of each
token's D the loss.
"""
import numpy as np
import pytest
import torch

import datagen
import latent_routing_quantile_b200 as lq
import oracle.balance as ob

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FMAX = float(np.finfo(np.float32).max)


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


def reference(s, idx, cu, coef):
    """Loss and gradient in float64 from f - 1, and the magnitudes A (a token) and w (|f - 1| + A) / R."""
    s, k, E = s.double().numpy(), idx.shape[1], s.shape[1]
    cnt = ob.counts(idx.numpy(), E, cu)
    filled = sum(hi > lo for lo, hi in zip(cu, cu[1:]))
    loss, slack, g, scale = 0.0, 0.0, np.zeros_like(s), np.zeros_like(s)
    for q, (lo, hi) in enumerate(zip(cu, cu[1:])):
        if hi == lo:
            continue
        f1 = (cnt[q] * E - k * (hi - lo)) / (k * (hi - lo))
        R = s[lo:hi].sum(axis=1, keepdims=True)
        some = R > 0
        p = np.divide(s[lo:hi], R, out=np.zeros_like(s[lo:hi]), where=some)
        D1, A = (p @ f1)[:, None], (p @ np.abs(f1))[:, None]
        wq = coef / (filled * (hi - lo))
        w = np.divide(wq, R, out=np.zeros_like(R), where=some)
        loss += wq * (1 + D1)[some].sum()
        slack += wq * A.sum()
        g[lo:hi] = w * (f1 - D1)
        scale[lo:hi] = w * (np.abs(f1) + A)
    return cnt, loss, slack, g, scale


def check(out, s, idx, cu, coef):
    cnt, loss, slack, g, scale = reference(s, idx, cu, coef)
    assert np.array_equal(out["counts"].cpu().numpy(), cnt)
    assert abs(float(out["loss"]) - loss) <= 16 * U * loss + 84 * U * slack
    got = out["dscores"].cpu().double().numpy()
    assert np.isfinite(got).all()
    # a value next to the largest may be on either side of it
    err = np.abs(got - np.clip(g, -FMAX, FMAX))
    tol = 224 * U * np.minimum(scale, FMAX * 4)
    # results below the normal range are rounded to steps of 2^-149
    assert (err <= tol + 2.0 ** -149).all(), float((err - tol).max())


def inputs(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    s = torch.sigmoid(torch.randn(T, E, generator=g) + 0.7 * torch.randn(E, generator=g))
    return s, s.topk(k, dim=1).indices.int()


@pytest.mark.parametrize("size", [1e-30, 1e-38, 1e-40, 3e-44, 1e30, 3e38])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (33, 2), (64, 4), (100, 5), (256, 6), (512, 8), (896, 16), (1024, 32)])
def test_rows_whose_sum_has_no_reciprocal(E, k, size):
    """Every row small or large, and every third one in a batch of ordinary rows (every lane layout)."""
    T = 70
    s, idx = inputs(T, E, k, E)
    check(lq.balance_loss((s * size).cuda(), idx.cuda(), 0.25), s * size, idx, [0, T], 0.25)
    s[::3] *= size
    for cu in ([0, T], [3, 20, 20, 61]):
        out = lq.balance_loss(s.cuda(), idx.cuda(), 0.25, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
        check(out, s, idx, cu, 0.25)


@pytest.mark.parametrize("E", [64, 100, 896])
def test_small_rows_in_a_batch_of_two_launches(E):
    T, k = (1 << 19) // E + 500, 4
    s, idx = inputs(T, E, k, 3 * E)
    s[5::7] *= 1e-40
    s[9] = 0
    check(lq.balance_loss(s.cuda(), idx.cuda(), 0.25), s, idx, [0, T], 0.25)


@pytest.mark.parametrize("T", [70, 0])
@pytest.mark.parametrize("small", [1e-3, 1e-7, 1e-12])
@pytest.mark.parametrize("E,k", [(8, 2), (33, 2), (64, 4), (100, 5), (256, 6), (512, 8), (896, 16), (1023, 3)])
def test_choices_of_experts_with_small_scores(E, k, small, T):
    """A batch whose choice (by its biases) fell on experts of small scores: D and the loss are near 0, and the
    gradient of every other expert is -w D / R.  T = 0: as many tokens as take two launches."""
    T = T or (1 << 19) // E + 300
    s, _ = inputs(T, E, k, 5 * E)
    idx = torch.arange(k, dtype=torch.int32).repeat(T, 1)
    s[:, :k] *= small
    out = lq.balance_loss(s.cuda(), idx.cuda(), 0.25)
    s64 = s.double().numpy()
    cnt = ob.counts(idx.numpy(), E, [0, T])
    loss = ob.loss(s64, cnt, k, [0, T], 0.25)
    g, scale = ob.gradient(s64, cnt, k, [0, T], 0.25)  # scale: w (f + D) / R
    D = (s64 / s64.sum(1, keepdims=True)) @ (cnt[0] * (E / (k * T)))
    assert D.max() < 0.49
    assert abs(float(out["loss"]) - loss) <= 128 * U * loss
    assert (np.abs(out["dscores"].cpu().double().numpy() - g) <= 128 * U * scale).all()


def test_tokens_on_both_sides_of_one_half():
    """D from 0 to 2 in one batch, its rows side by side in a warp."""
    T, E, k = 400, 64, 4
    s, _ = inputs(T, E, k, 77)
    idx = torch.arange(k, dtype=torch.int32).repeat(T, 1)
    s[:, :k] *= torch.linspace(0, 1, T)[:, None]
    for e in (64, 33, 16):
        part, cu = s[:, :e].contiguous(), [0, 150, T]
        out = lq.balance_loss(part.cuda(), idx.cuda(), 0.25, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
        check(out, part, idx, cu, 0.25)


@pytest.mark.parametrize("equal", [True, False])
def test_loss_of_tens_of_millions_of_tokens(equal):
    """A lane sums thousands of rows here: with rows all alike, roundings of a running sum would all fall the
    same way.  Against a float64 sum on the device, at the bounds of a short batch."""
    T, E = 1 << 26, 8
    g = torch.Generator(device="cuda").manual_seed(17)
    s = torch.rand((1 if equal else T, E), generator=g, device="cuda") + 0.01
    s = s.expand(T, E).contiguous()
    idx = torch.randint(0, 5, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    out = lq.balance_loss(s, idx, 0.25, grad=False)
    cnt = torch.bincount(idx.flatten(), minlength=E)
    assert torch.equal(out["counts"][0].long(), cnt)
    f1 = (cnt.double() * E - T) / T
    loss = slack = 0.0
    for part in s.split(1 << 22):
        p = part.double()
        p /= p.sum(1, keepdim=True)
        loss += 0.25 / T * float((1 + p @ f1).sum())
        slack += 0.25 / T * float((p @ f1.abs()).sum())
    assert abs(float(out["loss"]) - loss) <= 16 * U * loss + 84 * U * slack
    del s, idx, out, part, p
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,E,k", [(640, 64, 4), (512, 256, 6), (9000, 64, 4), (1792, 896, 16), (660, 33, 3)])
def test_next_to_balance(T, E, k):
    """Choices in turn with a few swaps: |f - 1| is some 1e-2 and less, and the gradient is held to that size, not
    to that of f and D (which an fp32 f - D would miss, as the last lines show)."""
    s, _ = inputs(T, E, k, 9 * E)
    idx = (torch.arange(T * k) % E).view(T, k).int()
    for t in range(0, T, T // 5):
        idx[t, 0] = idx[t, 1]
    out = lq.balance_loss(s.cuda(), idx.cuda(), 0.25)
    cnt, loss, slack, g, scale = reference(s, idx, [0, T], 0.25)
    assert np.array_equal(out["counts"].cpu().numpy(), cnt)
    assert abs(float(out["loss"]) - loss) <= 16 * U * loss + 84 * U * slack
    tol = 136 * U * scale
    assert (np.abs(out["dscores"].cpu().double().numpy() - g) <= tol).all()
    f = (cnt[0] * (E / (k * T))).astype(np.float32)
    R = s.numpy().sum(1, dtype=np.float32, keepdims=True)
    D = (s.numpy() / R) @ f
    cancelled = np.float32(0.25) / T * (f - D[:, None]) / R
    assert (np.abs(cancelled - g) > tol).any()


@pytest.mark.parametrize("where", ["before", "between", "behind"])
def test_runs_of_empty_sequences_are_stepped_over(where):
    """A million bounds alike: the results of the bounds without them, and no walk through each (which took a
    block 88 ms)."""
    T, E, k, n = 300, 64, 4, 1 << 20
    s, idx = inputs(T, E, k, 55)
    sd, id_ = s.cuda(), idx.cuda()
    short, at = [20, 100, 250], ["before", "between", "behind"].index(where)
    cu = short[:at] + [short[at]] * (n + 1) + short[at + 1:]
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ref = lq.balance_loss(sd, id_, 0.25, cu_seqlens=torch.tensor(short, dtype=torch.int32, device="cuda"))
    lq.balance_loss(sd, id_, 0.25, cu_seqlens=cud)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    out = lq.balance_loss(sd, id_, 0.25, cu_seqlens=cud)
    b.record()
    torch.cuda.synchronize()
    assert a.elapsed_time(b) < 20  # the bounds' checks, and 268 MB of counts set to zero
    full = out["counts"].sum(dim=1).nonzero().flatten()
    assert torch.equal(out["counts"][full], ref["counts"]) and len(full) == 2
    assert abs(float(out["loss"]) - float(ref["loss"])) <= 16 * U * float(ref["loss"])
    check({"counts": ref["counts"], "loss": out["loss"], "dscores": out["dscores"]}, s, idx, short, 0.25)


@pytest.mark.parametrize("cu", [[0, 0, 0, 5, 5, 5, 9, 9, 9], [3, 3, 4, 4, 4, 4], [7, 7, 7], [0, 0, 300, 300], [300, 300],
                                [0, 0, 0, 0], [5, 5, 290, 290, 290, 300]])
@pytest.mark.parametrize("E", [64, 1023])
def test_empty_sequences_anywhere(cu, E):
    T, k = 300, 4
    s, idx = inputs(T, E, k, 56)
    check(lq.balance_loss(s.cuda(), idx.cuda(), 0.25, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda")), s,
          idx, cu, 0.25)
    # the same in the form of two launches: the tokens behind are in no sequence
    T2 = (1 << 19) // E + 500
    s, idx = inputs(T2, E, k, 57)
    check(lq.balance_loss(s.cuda(), idx.cuda(), 0.25, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda")), s,
          idx, cu, 0.25)


def test_no_gradient_is_returned_that_was_not_made():
    """grad=False with the buffers of an earlier call: its gradient is left alone and not handed on."""
    s, idx = inputs(50, 64, 4, 41)
    out = lq.balance_loss(s.cuda(), idx.cuda(), 0.25)
    s2, idx2 = inputs(50, 64, 4, 42)
    old = out["dscores"].clone()
    again = lq.balance_loss(s2.cuda(), idx2.cuda(), 0.25, grad=False, out=out)
    assert sorted(again) == ["counts", "loss"] and torch.equal(out["dscores"], old)
    assert again["loss"] is out["loss"]
    check({**again, "dscores": lq.balance_loss(s2.cuda(), idx2.cuda(), 0.25)["dscores"]}, s2, idx2, [0, 50], 0.25)


def test_gradient_past_the_largest_value_is_held_there():
    s = torch.full((2, 8), 2.0 ** -149)
    s[0] = 0.5
    idx = torch.zeros(2, 1, dtype=torch.int32)
    out = lq.balance_loss(s.cuda(), idx.cuda(), 4.0)  # f = 8 for the first expert, D = 1
    g = out["dscores"].cpu()
    assert g[1, 0] == FMAX and (g[1, 1:] == -FMAX).all() and torch.isfinite(g[0]).all()
    assert float(out["loss"]) == 4.0


def test_training_step_with_small_scores():
    """Router offsets that leave every score near 1e-36: the balance loss's gradient in the scores is as large
    as 1 / R, and comes back to the ordinary range in the logits (here: summed into the offsets' gradient).
    The choice among such scores is the layer's own."""
    T, E, k = 130, 64, 4
    shape = datagen.LayerShape("bal_tiny", T, 256, 128, E, k, 128, 256, "bf16", seed=93, offset_var=0.5)
    w = datagen.layer_weights(shape, gain="random")
    w["router_bias"] = w["router_bias"] - 82.0
    x, dy = datagen.tokens(shape).cuda(), datagen.output_grad(shape, seed=193).cuda()
    w_dev = {n: t.cuda() for n, t in w.items()}
    layer = lq.Layer(shape.d, shape.l, E, k, shape.h, shape.hs, lq.BF16, T, w_dev, rms_eps=shape.rms_eps)
    _, g0 = layer.forward_backward(x, dy, w_dev)
    coef = 20.0 * T
    layer.set_balance(coef)
    _, g = layer.forward_backward(x, dy, w_dev)
    r = {n: t.cpu() for n, t in layer.routing().items()}
    s = r["scores"].double().numpy()
    assert 0 < s.min() and s.max() < 1e-32
    cnt, loss, slack, ds, scale = reference(r["scores"], r["idx"], [0, T], coef)
    got_loss, got_cnt = layer.balance()
    assert np.array_equal(got_cnt.cpu().numpy(), cnt)
    assert abs(float(got_loss) - loss) <= 16 * U * loss + 84 * U * slack
    want, size = (ds * s).sum(axis=0), (scale * s).sum(axis=0)
    moved = (g["router_bias"].double() - g0["router_bias"].double()).cpu().numpy()
    # 224 + T roundings of the aux sum; the rest of the gradient, summed in another order, to 1e-5
    assert (np.abs(moved - want) <= (224 + T) * U * size + 1e-5 * g0["router_bias"].abs().max().item()).all()
    assert np.abs(want).max() > 0.05 * g0["router_bias"].abs().max().item()
    assert all(torch.isfinite(t).all() for t in g.values())
    assert layer.status() == 0
    layer.close()
