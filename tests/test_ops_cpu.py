"""The balance-loss and MXFP4 entry points on the CPU: their oracles pinned to closed forms, brute force
and differences, sizes, and every refusal (the C entries check their arguments before they touch a
device, so the pointers here are never read)."""
import ctypes

import numpy as np
import pytest
import torch

import latent_routing_quantile_b200 as lq
import oracle.balance as ob
import oracle.mx4 as mx
from latent_routing_quantile_b200 import build as lbuild

EINVAL, EUNSUPPORTED = -1, -4


@pytest.fixture(scope="module")
def L():
    lbuild.build()
    return lq.lib()


# ------------------------------------------------------------------ oracles
def test_mx4_codes_are_the_nearest_values():
    rng = np.random.default_rng(5)
    a = rng.standard_normal((40, 64)) * np.exp2(rng.integers(-20, 20, (40, 1)))
    grid = np.concatenate([mx.E2M1, -mx.E2M1])
    v, sb = mx.values(a), mx.scale_bytes(a)
    for r in range(a.shape[0]):
        for b in range(2):
            blk = a[r, 32 * b:32 * b + 32]
            X = int(sb[r, b]) - 127
            assert 4 * 2.0 ** X <= np.abs(blk).max() < 8 * 2.0 ** X
            for i, x in enumerate(blk):
                d = np.abs(np.clip(x, -6 * 2.0 ** X, 6 * 2.0 ** X) - grid * 2.0 ** X)
                assert abs(v[r, 32 * b + i] - np.clip(x, -6 * 2.0 ** X, 6 * 2.0 ** X)) == d.min()


def test_mx4_ties_saturation_and_special_blocks():
    a = np.zeros((4, 32))
    a[0, :9] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25]  # X = 0: every midpoint
    a[1, :2] = [7.9, -7.9]                                          # saturates at 6
    a[2, 3] = np.nan
    a[3, 0] = 2.0 ** -140                                           # below the smallest scale
    v = mx.values(a)
    assert v[0, :9].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.0]
    assert v[1, :2].tolist() == [6.0, -6.0]
    assert np.isnan(v[2]).all() and mx.scale_bytes(a).ravel().tolist() == [127, 127, 255, 0]
    assert v[3, 0] == 0.0


@pytest.mark.parametrize("plant", ["ties_away", "scale_off", "no_clamp"])
def test_mx4_pins_catch_planted_mistakes(plant):
    a = np.zeros((1, 32))
    a[0, :3] = [4.0, 0.25, 1.25] if plant == "ties_away" else [7.9, 1.0, 0.5]
    good = mx.values(a)
    u = a / 2.0 ** (mx.scale_bytes(a)[0, 0] - 127 - (plant == "scale_off"))
    step = np.where(np.abs(u) < 2, 0.5, np.where(np.abs(u) < 4, 1.0, 2.0))
    q = np.floor(np.abs(u) / step + 0.5) * step if plant == "ties_away" else np.round(u / step) * step
    if plant != "no_clamp":
        q = np.clip(q, -6, 6)
    bad = q * 2.0 ** (mx.scale_bytes(a)[0, 0] - 127 - (plant == "scale_off"))
    assert not np.array_equal(good, bad)


def test_balance_oracle_closed_forms_and_differences():
    rng = np.random.default_rng(11)
    T, E, k = 12, 5, 2
    s = rng.uniform(0.05, 1, (T, E))
    idx = np.argsort(-s, axis=1)[:, :k]
    cu = [1, 4, 4, 11]
    cnt = ob.counts(idx, E, cu)
    assert cnt.sum(axis=1).tolist() == [3 * k, 0, 7 * k]
    g, _ = ob.gradient(s, cnt, k, cu, 0.3)
    for t in range(T):
        for e in range(E):
            h = 1e-6
            d = s.copy(); d[t, e] += h
            u = s.copy(); u[t, e] -= h
            num = (ob.loss(d, cnt, k, cu, 0.3) - ob.loss(u, cnt, k, cu, 0.3)) / (2 * h)
            assert abs(num - g[t, e]) < 1e-8
    # equal scores with a balanced choice: every f is 1, the loss is coef, the gradient zero
    s1 = np.full((E, E), 0.5)
    cnt1 = ob.counts(np.arange(E)[:, None], E, [0, E])
    assert abs(ob.loss(s1, cnt1, 1, [0, E], 0.7) - 0.7) < 1e-15
    assert np.abs(ob.gradient(s1, cnt1, 1, [0, E], 0.7)[0]).max() < 1e-15


# ------------------------------------------------------------------ sizes and refusals
def _bytes(L, rows, cols, groups, ragged):
    e, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    return L.lmoe_mx4_bytes(rows, cols, groups, ragged, ctypes.byref(e), ctypes.byref(s)), e.value, s.value


def test_mx4_sizes(L):
    assert _bytes(L, 1, 32, 1, 0) == (0, 16, 1024)
    assert _bytes(L, 129, 288, 1, 0) == (0, 129 * 144, 2 * 2 * 1024)
    assert _bytes(L, 6 * 100, 256, 6, 0) == (0, 600 * 128, 6 * 1024)     # a tile of its own for each group
    assert _bytes(L, 300, 256, 7, 1) == (0, 300 * 128, (3 + 7) * 1024)   # at most a partial tile a group
    assert _bytes(L, 0, 64, 1, 0) == (0, 0, 0)
    assert _bytes(L, 10, 48, 1, 0)[0] == EUNSUPPORTED
    assert _bytes(L, 10, 64, 3, 0)[0] == EINVAL                          # rows do not divide into groups
    assert _bytes(L, 10, 64, 1025, 1)[0] == EUNSUPPORTED
    assert _bytes(L, (1 << 30) + 1, 64, 1, 0)[0] == EUNSUPPORTED
    assert _bytes(L, -1, 64, 1, 0)[0] == EINVAL and _bytes(L, 1, 0, 1, 0)[0] == EINVAL


P = 1 << 20  # a pointer that is aligned and never read


@pytest.mark.parametrize("change,code", [
    (dict(cols=33), EUNSUPPORTED), (dict(rows=-1), EINVAL), (dict(groups=0), EINVAL), (dict(dtype=2), EINVAL),
    (dict(ld=63), EINVAL), (dict(x=None), EINVAL), (dict(x=P + 1), EINVAL), (dict(elems=P + 8), EINVAL),
    (dict(scales=None), EINVAL), (dict(status=None), EINVAL), (dict(groups=2, rows=5), EINVAL), (dict(rows=0), 0),
    (dict(status=P + 2), EINVAL), (dict(offsets=P + 1), EINVAL), (dict(index=P + 2), EINVAL),
    (dict(index=P, x_rows=-1), EINVAL), (dict(index=P, x_rows=1 << 31), EINVAL),
    (dict(rows=1 << 30, cols=1 << 20, ld=1 << 20), EUNSUPPORTED)])
def test_quant_refusals(L, change, code):
    a = dict(x=P, dtype=1, ld=64, index=None, x_rows=0, rows=4, cols=64, groups=1, offsets=None, elems=P, scales=P,
             status=P, stream=None)
    a.update(change)
    assert L.lmoe_mx4_quant(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(h=96), EUNSUPPORTED), (dict(h=0), EINVAL), (dict(w3=None), EINVAL), (dict(cols=40), EUNSUPPORTED),
    (dict(groups=1025), EUNSUPPORTED), (dict(dtype=3), EINVAL), (dict(elems=P + 4), EINVAL)])
def test_quant_w13_refusals(L, change, code):
    a = dict(w1=P, w3=P, dtype=1, groups=2, h=64, cols=64, elems=P, scales=P, status=P, stream=None)
    a.update(change)
    assert L.lmoe_mx4_quant_w13(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(cols=33), EUNSUPPORTED), (dict(dtype=2), EINVAL), (dict(ld=32), EINVAL), (dict(out=P + 1), EINVAL),
    (dict(flags=1), EINVAL), (dict(elems=None), EINVAL), (dict(status=P + 1), EINVAL), (dict(offsets=P + 2), EINVAL),
    (dict(rows=0), 0)])
def test_dequant_refusals(L, change, code):
    a = dict(elems=P, scales=P, rows=4, cols=64, groups=1, offsets=None, out=P, dtype=1, ld=64, flags=0, status=P,
             stream=None)
    a.update(change)
    assert L.lmoe_mx4_dequant(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(K=48), EUNSUPPORTED), (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(groups=2), EINVAL),
    (dict(flags=4), EINVAL), (dict(flags=1, N=64), EUNSUPPORTED), (dict(flags=1, N=128, dtype=0), EUNSUPPORTED),
    (dict(ldc=7), EINVAL), (dict(c=P + 1), EINVAL), (dict(c=P + 2, dtype=0), EINVAL), (dict(b_scales=P + 8), EINVAL),
    (dict(status=None), EINVAL), (dict(status=P + 2), EINVAL), (dict(offsets=P + 1), EINVAL),
    (dict(groups=1000, offsets=P, N=1 << 21), EUNSUPPORTED), (dict(M=0), 0)])
def test_gemm_refusals(L, change, code):
    a = dict(a_elems=P, a_scales=P, b_elems=P, b_scales=P, M=4, N=8, K=64, groups=1, offsets=None, c=P, dtype=1,
             ldc=64, flags=0, status=P, stream=None)
    a.update(change)
    assert L.lmoe_mx4_gemm(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(E=1025), EUNSUPPORTED), (dict(k=33, E=64), EUNSUPPORTED), (dict(k=9), EINVAL), (dict(T=-1), EINVAL),
    (dict(S=2), EINVAL), (dict(S=0), EINVAL), (dict(coef=float("nan")), EINVAL), (dict(counts=None), EINVAL),
    (dict(scratch=P + 8), EINVAL), (dict(scores=P + 2), EINVAL), (dict(idx=None), EINVAL), (dict(status=None), EINVAL),
    (dict(status=P + 1), EINVAL), (dict(cu=P + 2, S=2), EINVAL), (dict(S=(1 << 24) + 1, cu=P), EUNSUPPORTED)])
def test_balance_refusals(L, change, code):
    a = dict(scores=P, idx=P, T=4, E=8, k=2, cu=None, S=1, coef=0.1, counts=P, loss=P, dscores=P, scratch=P, status=P,
             stream=None)
    a.update(change)
    assert L.lmoe_balance_loss(*a.values()) == code


def test_binding_refuses_host_tensors_and_wrong_types():
    with pytest.raises(lq.LmoeError, match="CUDA"):
        lq.mx4_quant(torch.zeros(4, 64))
    with pytest.raises(lq.LmoeError, match="float32 or torch.bfloat16"):
        lq.mx4_quant(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(lq.LmoeError, match="rows, cols"):
        lq.mx4_quant(torch.zeros(64))
    with pytest.raises(lq.LmoeError, match="rows must not overlap"):
        lq.mx4_quant(torch.zeros(1, 64).expand(4, 64))
    with pytest.raises(lq.LmoeError, match="int32"):
        lq.mx4_quant(torch.zeros(4, 64), offsets=torch.zeros(3))
    with pytest.raises(lq.LmoeError, match="CUDA"):
        lq.balance_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), 0.1)
    with pytest.raises(lq.LmoeError, match="scores must be"):
        lq.balance_loss(torch.zeros(4), torch.zeros(4, 2, dtype=torch.int32), 0.1)


def test_layer_with_4_bit_experts_is_sized_and_checked():
    a = dict(d=1024, l=256, E=256, k=6, h=256, hs=2048, dtype=lq.BF16, max_tokens=8192)
    n4, n8 = (lq.workspace_bytes(**a, experts=e) for e in (lq.EXPERTS_MXFP4, lq.EXPERTS_MXFP8))
    assert 0 < n4 < n8
    lq.workspace_bytes(**{**a, "l": 192, "h": 64}, experts=lq.EXPERTS_MXFP4)
    with pytest.raises(lq.LmoeError, match="unsupported"):
        lq.workspace_bytes(256, 64, 32, 4, 128, 512, lq.F32, 256, experts=lq.EXPERTS_MXFP4)


def test_flag_constants_match_the_header():
    import os, re
    text = open(os.path.join(os.path.dirname(lq.__file__), "..", "include", "lmoe.h")).read()
    for name, v in (("MX4_SWIGLU", lq.MX4_SWIGLU), ("MX4_ZERO_REST", lq.MX4_ZERO_REST),
                    ("EXPERTS_MXFP4", lq.EXPERTS_MXFP4)):
        assert int(re.search(rf"#define LMOE_{name} (\d+)", text).group(1)) == v


def test_first_calls_of_two_threads_share_one_status_word(monkeypatch):
    """Both threads are past the look-up when the words are made: one word stays, and both get its address
    (the other's memory goes back to the allocator, so no kernel may have been given it)."""
    import threading
    both, zeros, got = threading.Barrier(2, timeout=30), torch.zeros, []

    def made_together(*shape, **kw):
        word = zeros(*shape, dtype=kw["dtype"])
        both.wait()
        return word

    monkeypatch.setattr(lq, "_status_words", {})
    monkeypatch.setattr(lq.torch, "zeros", made_together)
    monkeypatch.setattr(lq.torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(lq.torch.cuda, "synchronize", lambda index=None: None)
    threads = [threading.Thread(target=lambda: got.append(lq._status_word(0))) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got == [lq._status_words[0][1]] * 2
