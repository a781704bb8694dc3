"""The operators' fault bits: a device's shared word, and a word of the caller's own."""
import pytest
import torch

import latent_routing_quantile_b200 as lq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latent_routing_quantile_b200 import build
    build.build()
    yield


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def calls():
    """Every operator with a fault, as functions of a status word (and stream)."""
    x = torch.randn(20, 64, device="cuda")
    w = lq.mx4_quant(torch.randn(2, 8, 64, device="cuda"))
    bad = ints(0, 12, 21)
    q = lq.mx4_quant(x, offsets=ints(0, 12, 20))
    q.offsets = bad
    s, outside = torch.rand(20, 8, device="cuda"), torch.full((20, 1), 8, dtype=torch.int32, device="cuda")
    index = ints(0, 20)
    return {"quant": lambda **kw: lq.mx4_quant(x, offsets=bad, **kw),
            "index": lambda **kw: lq.mx4_quant(x, index=index, **kw),
            "dequant": lambda **kw: lq.mx4_dequant(q, **kw),
            "gemm": lambda **kw: lq.mx4_gemm(q, w, **kw),
            "balance": lambda **kw: lq.balance_loss(s, outside, 0.1, **kw)}


@pytest.mark.parametrize("name", ["quant", "index", "dequant", "gemm", "balance"])
@pytest.mark.parametrize("named", [False, True])
def test_a_call_with_its_own_word_leaves_the_shared_one(name, named):
    call = calls()[name]
    assert lq.op_status() == 0
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if named else None
    mine, other = ints(0), ints(0)
    torch.cuda.synchronize()
    call(status=mine, stream=stream)
    torch.cuda.synchronize()
    assert int(mine) == lq.STATUS_BAD_INDEX and int(other) == 0 and lq.op_status() == 0
    call(stream=stream)
    assert lq.op_status() == lq.STATUS_BAD_INDEX and lq.op_status() == 0
    assert int(mine) == lq.STATUS_BAD_INDEX  # kept: only the caller clears it


def test_weights_take_a_word_of_their_own():
    w1, w3 = (torch.randn(64, 64, device="cuda") for _ in range(2))
    mine = ints(0)
    a, b = lq.mx4_quant_w13(w1, w3, status=mine), lq.mx4_quant_w13(w1, w3)
    assert torch.equal(a.buf, b.buf) and int(mine) == 0


def test_a_first_call_can_be_captured_with_its_own_word(monkeypatch):
    x, mine = torch.randn(40, 64, device="cuda"), ints(0)
    lq.op_status()
    monkeypatch.setattr(lq, "_status_words", {})
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        v = lq.mx4_dequant(lq.mx4_quant(x, status=mine), status=mine)
        with pytest.raises(lq.LmoeError, match="pass a status word"):
            lq.mx4_quant(x)
    g.replay()
    assert torch.equal(v, lq.mx4_dequant(lq.mx4_quant(x))) and int(mine) == 0


def test_wrong_words_are_refused():
    x = torch.randn(4, 64, device="cuda")
    for bad in (torch.zeros(1, device="cuda"), ints(0, 0), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(lq.LmoeError):
            lq.mx4_quant(x, status=bad)
    assert lq.op_status() == 0


def test_first_calls_of_a_process_can_be_captured():
    """What a kernel asks the device once (its largest cluster, its shared memory) may be asked under a capture:
    the first calls of a process, in one graph, for every form."""
    import os
    import subprocess
    import sys
    code = """if True:
        import torch, latent_routing_quantile_b200 as lq
        cases = [(50, 64, 4), (700, 256, 6), (9000, 256, 6), (300, 33, 2), (200, 896, 16), (2048, 256, 6), (4000, 64, 4)]
        g = torch.Generator(device="cuda").manual_seed(1)
        s = [torch.rand(T, E, generator=g, device="cuda") for T, E, k in cases]
        i = [v.topk(c[2], dim=1).indices.int() for v, c in zip(s, cases)]
        x, w = torch.randn(70, 4128, generator=g, device="cuda"), torch.randn(256, 4128, generator=g, device="cuda")
        mine = torch.zeros(1, dtype=torch.int32, device="cuda")
        run = lambda: [lq.balance_loss(a, b, 0.1, status=mine) for a, b in zip(s, i)] + \\
            [dict(c=lq.mx4_gemm(lq.mx4_quant(x, status=mine), lq.mx4_quant(w, status=mine), status=mine))]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graph.replay()
        for a, b in zip(out, run()):
            assert all(torch.equal(a[n], b[n]) for n in b)
        assert int(mine) == 0
        print("same")
    """
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
