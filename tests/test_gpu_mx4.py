"""MXFP4 quantisation and products on the GPU against the float64 oracle (oracle.mx4), through the binding.

Tolerances.  Quantising, its scale bytes and dequantising are exact: the codes, the bytes and the
values must be equal.  A product's terms are exact (4-bit codes times powers of two), and a sum of K
terms in fp32, in any order, with each addition off by at most one step of 2^-23 (a tensor core may
truncate), is off by at most K 2^-23 sum|terms|.  bf16 results are rounded once more: 2^-8 |C|.  The
SwiGLU form adds silu's own error: relative 2^-15 covers the hardware exponential (2 + 1.16 |g| steps
of 2^-23 at |g| < 88; beyond that silu is 0 or g), and a change d of the gate moves silu by at most
1.1 |d|.
"""
import numpy as np
import pytest
import torch

import datagen
import latent_routing_quantile_b200 as lq
import oracle
import oracle.mx4 as mx

pytestmark = pytest.mark.gpu


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


def rows(shape, seed, dtype=torch.bfloat16, spread=3):
    """Rows of different sizes with a few large columns."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(shape, generator=g)
    v *= torch.exp2(torch.randint(-spread, spread + 1, shape[:-1] + (1,), generator=g).float())
    v[..., torch.randint(0, shape[-1], (max(1, shape[-1] // 64),), generator=g)] *= 10
    return v.to(dtype)


def np64(t):
    return t.detach().cpu().double().numpy()


def ragged(M, sizes, head=0):
    off = np.concatenate([[0], np.cumsum(sizes)]) + head
    assert off[-1] <= M
    return torch.tensor(off, dtype=torch.int32)


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (128, 256), (129, 160), (300, 1056), (2, 7168), (1000, 288)])
def test_quant_codes_scales_and_values(shape, dtype):
    x = rows(shape, shape[0] * 7 + shape[1], dtype)
    q = lq.mx4_quant(x.cuda())
    el = q.elems.cpu().numpy()
    code = np.stack([el & 15, el >> 4], axis=-1).reshape(shape)
    ref = mx.codes(np64(x))
    assert np.array_equal(code, ref)
    sb, sc = mx.scale_bytes(np64(x)), q.scales.cpu().numpy()
    want = np.zeros_like(sc)  # blocks past the last column, and rows past the last, hold 0
    r, b = np.meshgrid(np.arange(shape[0]), np.arange(shape[1] // 32), indexing="ij")
    nkb = (shape[1] + 255) // 256
    off = ((r // 128 * nkb + b // 8) * 2 + b // 4 % 2) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    want[off] = sb
    assert off[-1, -1] == mx.atom_offset((shape[0] - 1) // 128, (shape[0] - 1) % 128, shape[1] // 32 - 1, shape[1])
    assert np.array_equal(sc, want)
    for dt in (torch.bfloat16, torch.float32):
        assert np.array_equal(np64(lq.mx4_dequant(q, dtype=dt)), mx.values(np64(x)))


def special_rows(dtype):
    x = torch.zeros(12, 64, dtype=torch.float32)
    x[0, :9] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25])  # every midpoint
    x[1, :3] = torch.tensor([7.9375, -7.9375, 1.0])          # saturates
    x[2, 5] = float("nan")
    x[3, 6] = float("inf")
    x[4, 7] = -float("inf")
    x[4, 40] = float("nan")
    x[5, :3] = torch.tensor([2.0 ** -126, 2.0 ** -127, -2.0 ** -130])  # at and below the smallest scale
    x[6, :3] = torch.tensor([2.0 ** -140, 0.0, -0.0])
    x[7, :3] = torch.tensor([torch.finfo(torch.bfloat16).max, -1e38, 1.0])
    x[8, :4] = torch.tensor([2.0 ** -124, 2.0 ** -125, 1.5 * 2.0 ** -126, 2.0 ** -127])
    x[9] = -0.0
    x[10, 32:34] = torch.tensor([3.0, -3.0])
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_special_values(dtype):
    x = special_rows(dtype)
    q = lq.mx4_quant(x.cuda())
    ref = mx.values(np64(x))
    got = np64(lq.mx4_dequant(q, dtype=torch.float32))
    assert np.array_equal(got, ref, equal_nan=True)
    assert np.array_equal(np.signbit(got[~np.isnan(ref)]), np.signbit(ref[~np.isnan(ref)]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pitch,first", [(160, 0), (161, 0), (200, 3), (164, 4), (168, 8)])
def test_quant_strided_and_misaligned_rows(dtype, pitch, first):
    base = rows((70, pitch + 8), 3, dtype).cuda()
    x = base[:, first:first + 160]
    q = lq.mx4_quant(x)
    assert np.array_equal(np64(lq.mx4_dequant(q, dtype=torch.float32)), mx.values(np64(x)))
    for dt in (torch.bfloat16, torch.float32):
        for at in (1, 4, 8):  # off every boundary, and on 8, 16 and 32 bytes
            out = torch.empty(70 * 160 + at, dtype=dt, device="cuda")[at:].view(70, 160)
            assert np.array_equal(np64(lq.mx4_dequant(q, out=out)), mx.values(np64(x)))


@pytest.mark.parametrize("head,sizes,tail", [(0, [5, 0, 130, 1, 0, 256], 0), (3, [1, 1, 1], 9), (0, [0, 0], 4),
                                             (0, [200], 0), (7, [0, 129], 0)])
def test_ragged_groups_and_rows_of_none(head, sizes, tail):
    M = head + sum(sizes) + tail
    x = rows((M, 96), 17)
    off = ragged(M, sizes, head)
    q = lq.mx4_quant(x.cuda(), offsets=off.cuda())
    ref = mx.values(np64(x))
    inside = slice(head, M - tail)
    got = np64(lq.mx4_dequant(q, dtype=torch.float32))
    assert np.array_equal(got[inside], ref[inside])
    assert not got[:head].any() and not got[M - tail:].any()
    keep = torch.full((M, 96), 7.0, device="cuda")
    lq.mx4_dequant(q, out=keep)
    k = np64(keep)
    assert np.array_equal(k[inside], ref[inside]) and (k[:head] == 7).all() and (k[M - tail:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("grouped", [False, True])
def test_indexed_rows(dtype, grouped):
    x = rows((50, 352), 19, dtype)
    g = torch.Generator().manual_seed(2)
    idx = torch.randint(0, 50, (300,), generator=g).int()
    idx[7] = idx[8] = idx[250] = 3  # the same row again
    off = ragged(300, [10, 0, 150, 140]) if grouped else None
    q = lq.mx4_quant(x.cuda(), offsets=None if off is None else off.cuda(), index=idx.cuda())
    ref = mx.values(np64(x))[idx.numpy()]
    assert np.array_equal(np64(lq.mx4_dequant(q, dtype=torch.float32)), ref)
    bad = idx.clone()
    bad[4], bad[299] = 50, -1
    q = lq.mx4_quant(x.cuda(), offsets=None if off is None else off.cuda(), index=bad.cuda(), out=q)
    assert lq.op_status() == lq.STATUS_BAD_INDEX
    ref[4] = ref[299] = 0
    assert np.array_equal(np64(lq.mx4_dequant(q, dtype=torch.float32)), ref)


def test_many_groups_and_more_tiles_than_blocks():
    rng = np.random.default_rng(3)
    sizes = rng.integers(0, 40, 1024)
    M = int(sizes.sum())
    x = rows((M, 64), 23)
    q = lq.mx4_quant(x.cuda(), offsets=ragged(M, sizes).cuda())
    assert np.array_equal(np64(lq.mx4_dequant(q, dtype=torch.float32)), mx.values(np64(x)))


def test_stacked_and_interleaved_weights():
    w = rows((5, 100, 96), 29)
    q = lq.mx4_quant(w.cuda())
    assert np.array_equal(np64(lq.mx4_dequant(q, dtype=torch.float32)), mx.values(np64(w)))
    w1, w3 = rows((3, 128, 96), 31), rows((3, 128, 96), 37, spread=1)
    q = lq.mx4_quant_w13(w1.cuda(), w3.cuda())
    got = np64(lq.mx4_dequant(q, dtype=torch.float32)).reshape(3, 2, 2, 64, 96)
    assert np.array_equal(got[:, :, 0].reshape(3, 128, 96), mx.values(np64(w1)))
    assert np.array_equal(got[:, :, 1].reshape(3, 128, 96), mx.values(np64(w3)))


# ------------------------------------------------------------------ products
def check_product(got, c, mag, K, out):
    tol = K * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(c) if out == torch.bfloat16 else 0)
    err = np.abs(got - c)
    assert (err <= tol).all(), float((err - tol).max())


SIZES = [(1, 1, 32), (1, 7, 64), (1, 1000, 512), (7, 129, 96), (128, 128, 256), (129, 257, 288), (333, 1000, 992),
         (1025, 384, 544), (64, 2048, 2048), (513, 640, 1280),
         # K split over clusters of 2, 4 and 8 CTAs, their shares uneven
         (130, 4100, 3104), (70, 1000, 4128), (1, 130, 7200), (33, 250, 16416),
         # 256-wide tiles: a last one half outside, columns off the 16-byte grid, several tiles a CTA
         (2100, 2050, 96), (3001, 1700, 544), (5000, 2190, 288)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_dense_product(M, N, K, out):
    a, b = rows((M, K), M + K), rows((N, K), N + 5, spread=1)
    c = lq.mx4_gemm(lq.mx4_quant(a.cuda()), lq.mx4_quant(b.cuda()), dtype=out)
    assert c.dtype == out
    ref, mag = mx.product(mx.values(np64(a)), mx.values(np64(b)))
    check_product(np64(c), ref, mag, K, out)


@pytest.mark.parametrize("out,pitch,N", [(torch.bfloat16, 136, 130), (torch.bfloat16, 131, 130), (torch.float32, 132, 130),
                                         (torch.float32, 131, 130), (torch.bfloat16, 131, 1), (torch.bfloat16, 131, 65),
                                         (torch.bfloat16, 133, 64), (torch.bfloat16, 133, 127), (torch.float32, 67, 65),
                                         (torch.bfloat16, 2051, 2050), (torch.float32, 2051, 2051), (torch.float32, 2050, 2049),
                                         (torch.bfloat16, 132, 130), (torch.bfloat16, 132, 129), (torch.bfloat16, 132, 131),
                                         (torch.float32, 134, 130), (torch.float32, 134, 129)])
def test_product_into_strided_output_leaves_the_rest(out, pitch, N):
    M, K = 140 if N < 2000 else 2100, 320
    a, b = rows((M, K), 1), rows((N, K), 2)
    buf = torch.full((M + 2, pitch), 7.0, dtype=out, device="cuda")
    lq.mx4_gemm(lq.mx4_quant(a.cuda()), lq.mx4_quant(b.cuda()), out=buf[1:M + 1, :N])
    ref, mag = mx.product(mx.values(np64(a)), mx.values(np64(b)))
    check_product(np64(buf[1:M + 1, :N]), ref, mag, K, out)
    assert (buf[0] == 7).all() and (buf[M + 1] == 7).all() and (buf[:, N:] == 7).all()


GROUPS = [(0, [5, 0, 130, 1, 0, 256], 0), (3, [1, 1, 1], 9), (0, [0, 0], 4), (0, [200], 0),
          (2, [31, 33, 127, 128, 129], 1),
          (0, [1] * 16, 0), (0, [300, 0, 0, 290, 310, 33, 600, 2], 0),
          (5, list(range(0, 270, 3)), 6)]  # 90 groups: 256-wide tiles at N >= 257


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(96, 64), (257, 288), (512, 512)])
@pytest.mark.parametrize("head,sizes,tail", GROUPS)
def test_grouped_product(head, sizes, tail, N, K, out):
    M, G = head + sum(sizes) + tail, len(sizes)
    a, b = rows((M, K), 41 + M), rows((G, N, K), 43, spread=1)
    off = ragged(M, sizes, head)
    qa, qb = lq.mx4_quant(a.cuda(), offsets=off.cuda()), lq.mx4_quant(b.cuda())
    ref, mag = mx.product(mx.values(np64(a)), mx.values(np64(b)), off.numpy())
    check_product(np64(lq.mx4_gemm(qa, qb, dtype=out)), ref, mag, K, out)  # rows of no group: zeros
    keep = torch.full((M, N), 7.0, dtype=out, device="cuda")
    lq.mx4_gemm(qa, qb, out=keep)
    k = np64(keep)
    inside = slice(head, M - tail)
    check_product(k[inside], ref[inside], mag[inside], K, out)
    assert (k[:head] == 7).all() and (k[M - tail:] == 7).all()


def check_swiglu(got, c, mag, K):
    g, u = mx.swiglu_columns(c)
    mg, mu = mx.swiglu_columns(mag)
    ref = mx.silu(g) * u
    eg, eu = K * 2.0 ** -23 * mg, K * 2.0 ** -23 * mu
    s = np.abs(mx.silu(g))
    tol = (2.0 ** -8 + 2.0 ** -15) * np.abs(ref) + 1.1 * eg * (np.abs(u) + eu) + (s + 1.1 * eg) * eu + 1e-30
    err = np.abs(got - ref)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("pitch", [128, 129, 130, 132, 136])
def test_swiglu_into_strided_output_leaves_the_rest(pitch):
    M, h, K = 300, 128, 320
    a, w1, w3 = rows((M, K), 3), rows((h, K), 4, spread=0) / K ** 0.5, rows((h, K), 5, spread=0)
    buf = torch.full((M + 2, pitch), 7.0, dtype=torch.bfloat16, device="cuda")
    lq.mx4_gemm(lq.mx4_quant(a.cuda()), lq.mx4_quant_w13(w1.cuda(), w3.cuda()), swiglu=True, out=buf[1:M + 1, :h])
    b = np.stack([mx.values(np64(w1)).reshape(-1, 64, K), mx.values(np64(w3)).reshape(-1, 64, K)], 1).reshape(2 * h, K)
    check_swiglu(np64(buf[1:M + 1, :h]), *mx.product(mx.values(np64(a)), b), K)
    assert (buf[0] == 7).all() and (buf[M + 1] == 7).all() and (buf[:, h:] == 7).all()


@pytest.mark.parametrize("M,h,K", [(1, 64, 32), (5, 192, 288), (129, 128, 512), (300, 512, 2048), (1030, 320, 256),
                                   (70, 192, 4128), (3, 64, 7200), (3001, 1088, 288), (2300, 1984, 96)])
def test_dense_swiglu(M, h, K):
    a, w1, w3 = rows((M, K), 3), rows((h, K), 4, spread=0) / K ** 0.5, rows((h, K), 5, spread=0)
    act = lq.mx4_gemm(lq.mx4_quant(a.cuda()), lq.mx4_quant_w13(w1.cuda(), w3.cuda()), swiglu=True)
    assert act.shape == (M, h) and act.dtype == torch.bfloat16
    b = np.stack([mx.values(np64(w1)).reshape(-1, 64, K), mx.values(np64(w3)).reshape(-1, 64, K)], 1).reshape(2 * h, K)
    check_swiglu(np64(act), *mx.product(mx.values(np64(a)), b), K)


@pytest.mark.parametrize("head,sizes,tail", GROUPS)
def test_grouped_swiglu(head, sizes, tail):
    M, G, h, K = head + sum(sizes) + tail, len(sizes), 128, 320
    a, w1, w3 = rows((M, K), 3), rows((G, h, K), 4, spread=0) / K ** 0.5, rows((G, h, K), 5, spread=0)
    off = ragged(M, sizes, head)
    act = lq.mx4_gemm(lq.mx4_quant(a.cuda(), offsets=off.cuda()), lq.mx4_quant_w13(w1.cuda(), w3.cuda()), swiglu=True)
    b = np.stack([mx.values(np64(w1)).reshape(G, -1, 64, K), mx.values(np64(w3)).reshape(G, -1, 64, K)], 2)
    check_swiglu(np64(act), *mx.product(mx.values(np64(a)), b.reshape(G, 2 * h, K), off.numpy()), K)


def test_blocks_of_nan_reach_their_rows_and_columns_only():
    M, N, K = 140, 150, 320
    a, b = rows((M, K), 51), rows((N, K), 52)
    a[3, 100], a[130, 319], b[7, 0] = float("nan"), float("inf"), float("nan")
    c = np64(lq.mx4_gemm(lq.mx4_quant(a.cuda()), lq.mx4_quant(b.cuda()), dtype=torch.float32))
    bad = np.zeros((M, N), bool)
    bad[3] = bad[130] = True
    bad[:, 7] = True
    assert np.array_equal(np.isnan(c), bad)


def test_empty_and_bad_offsets():
    none = lq.mx4_quant(torch.empty(0, 64, device="cuda"))
    assert lq.mx4_gemm(none, lq.mx4_quant(rows((8, 64), 1).cuda())).shape == (0, 8)
    x, w = rows((20, 64), 1).cuda(), lq.mx4_quant(rows((2, 8, 64), 1).cuda())
    for off in ([0, 12, 21], [0, 12, 5], [-1, 3, 20]):
        q = lq.mx4_quant(x, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert lq.op_status() == lq.STATUS_BAD_INDEX
        assert not lq.mx4_gemm(q, w).any()
        assert lq.op_status() == lq.STATUS_BAD_INDEX and lq.op_status() == 0


def test_mismatched_operands_are_refused():
    x = lq.mx4_quant(rows((20, 64), 1).cuda())
    with pytest.raises(lq.LmoeError, match="disagree on K"):
        lq.mx4_gemm(x, lq.mx4_quant(rows((8, 96), 1).cuda()))
    with pytest.raises(lq.LmoeError, match="stacked"):
        lq.mx4_gemm(x, lq.mx4_quant(rows((2, 8, 64), 1).cuda()))
    with pytest.raises(lq.LmoeError, match="w13"):
        lq.mx4_gemm(x, lq.mx4_quant(rows((128, 64), 1).cuda()), swiglu=True)
    with pytest.raises(lq.LmoeError, match="shape"):
        lq.mx4_gemm(x, lq.mx4_quant(rows((8, 64), 1).cuda()), out=torch.empty(20, 9, device="cuda"))
    with pytest.raises(lq.LmoeError, match="another shape"):
        lq.mx4_quant(rows((21, 64), 1).cuda(), out=x)


def test_repeated_calls_give_the_same_bits_and_out_is_reused():
    a, b = rows((700, 1056), 61).cuda(), lq.mx4_quant(rows((520, 1056), 62).cuda())
    q = lq.mx4_quant(a)
    first = lq.mx4_gemm(q, b, dtype=torch.float32)
    ptr = q.elems.data_ptr()
    a2 = rows((700, 1056), 63).cuda()
    q2 = lq.mx4_quant(a2, out=q)
    assert q2 is q and q.elems.data_ptr() == ptr
    other = lq.mx4_gemm(q, b, dtype=torch.float32)
    assert not torch.equal(first, other)
    lq.mx4_quant(a, out=q)
    for _ in range(3):
        assert torch.equal(lq.mx4_gemm(q, b, dtype=torch.float32), first)


def test_streams_and_graph_replay():
    b = lq.mx4_quant(rows((4, 256, 512), 71).cuda())
    off = ragged(300, [100, 0, 150, 50]).cuda()
    a = [rows((300, 512), 72 + i).cuda() for i in range(4)]
    ref = [lq.mx4_gemm(lq.mx4_quant(x, offsets=off), b) for x in a]
    torch.cuda.synchronize()
    # two calls at once on streams of the caller's
    ss = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for x, s in zip(a, ss):
        s.wait_stream(torch.cuda.current_stream())
        got.append(lq.mx4_gemm(lq.mx4_quant(x, offsets=off, stream=s), b, stream=s))
    for s in ss:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(u, v) for u, v in zip(got, ref))
    # captured, and replayed on new rows and new offsets
    x, o = a[0].clone(), off.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lq.mx4_gemm(lq.mx4_quant(x, offsets=o), b)
    x.copy_(a[3])
    g.replay()
    assert torch.equal(y, ref[3])
    o.copy_(ragged(300, [0, 300, 0, 0]))
    g.replay()
    assert torch.equal(y, lq.mx4_gemm(lq.mx4_quant(a[3], offsets=o), b))


def test_matrices_past_32_bit_offsets():
    """More than 2^31 elements in the rows and in the result: the last rows come out as they do alone."""
    M, K, N = 270000, 8192, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for i in range(0, M, 30000):
        x[i:i + 30000].normal_(generator=g)
    w = lq.mx4_quant(torch.randn((N, K), generator=g, device="cuda", dtype=torch.bfloat16))
    q, last = lq.mx4_quant(x), lq.mx4_quant(x[-200:])
    c = lq.mx4_gemm(q, w)
    # the small product sums K in parts (too few tiles): fp32 sums in another order, rounded to bf16
    a, b = c[-200:].float(), lq.mx4_gemm(last, w).float()
    assert (a - b).abs().max() <= 2.0 ** -7 * b.abs().max()
    del c
    v = lq.mx4_dequant(q)
    assert torch.equal(v[-200:], lq.mx4_dequant(last)) and torch.equal(v[:200], lq.mx4_dequant(lq.mx4_quant(x[:200])))
    del x, q, v
    torch.cuda.empty_cache()


def test_two_graphs_at_once_and_alternating():
    """Two captured graphs of the operators, replayed on two streams at the same time and in turn: they share
    no workspace."""
    ws = [lq.mx4_quant(rows((256, 4128), 90 + i, spread=1).cuda()) for i in range(2)]
    xs = [rows((70, 4128), 95 + i).cuda() for i in range(2)]  # K split over clusters
    ss = [torch.sigmoid(torch.randn(400, 64, generator=torch.Generator().manual_seed(i))).cuda() for i in range(2)]
    ids = [s.topk(4, dim=1).indices.int() for s in ss]
    once = lambda i: (lq.mx4_gemm(lq.mx4_quant(xs[i]), ws[i], dtype=torch.float32),
                      *lq.balance_loss(ss[i], ids[i], 0.1).values())
    ref = [once(0), once(1)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(once(i))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], ref[i]))
    for i in (1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], ref[i]))


def test_experts_after_routing():
    """The operators as a serving step uses them: routing, the rows in expert order, both expert
    products in 4 bits."""
    T, E, k, l, h = 200, 64, 4, 256, 128
    g = torch.Generator().manual_seed(9)
    scores = torch.sigmoid(torch.randn(T, E, generator=g)).cuda()
    r = lq.route_noalloc(scores, torch.zeros(E, device="cuda"), k)
    x = rows((T, l), 81).cuda()
    w1, w3, w2 = (rows(s, 82 + i, spread=0) / s[2] ** 0.5 for i, s in enumerate(((E, h, l), (E, h, l), (E, l, h))))
    w13, wd = lq.mx4_quant_w13(w1.cuda(), w3.cuda()), lq.mx4_quant(w2.cuda())
    xp = x[r["perm"].long()]
    act = lq.mx4_gemm(lq.mx4_quant(x, offsets=r["offsets"], index=r["perm"]), w13, swiglu=True)
    o = lq.mx4_gemm(lq.mx4_quant(act, offsets=r["offsets"]), wd)
    off = r["offsets"].cpu().numpy()
    b = np.stack([mx.values(np64(w1)).reshape(E, -1, 64, l), mx.values(np64(w3)).reshape(E, -1, 64, l)], 2)
    check_swiglu(np64(act), *mx.product(mx.values(np64(xp)), b.reshape(E, 2 * h, l), off), l)
    c, mag = mx.product(mx.values(np64(act)), mx.values(np64(w2)), off)
    check_product(np64(o), c, mag, h, torch.bfloat16)


@pytest.mark.parametrize("name,T,d,l,E,k,h,hs", [
    ("mx4_small", 1000, 256, 128, 64, 4, 128, 256),
    ("mx4_ragged", 333, 256, 192, 64, 3, 64, 0),        # widths that fill no tile, no shared expert
    ("mx4_one", 1, 256, 128, 64, 4, 128, 256),          # a single token
    ("mx4_mini", 8192, 1024, 256, 256, 6, 256, 2048),   # mini_replica widths
])
def test_layer_with_4_bit_experts(name, T, d, l, E, k, h, hs):
    """Layer(experts=EXPERTS_MXFP4): routing identical to the oracle's; outputs within 1e-2 normwise of the
    float64 layer with MXFP4 experts (the bf16 roundings of o, z, a_s and y, at most 2^-8 each and
    independent, and the rare code that a rounding of h or of an activation moves), and at least five
    times as far from the bf16-expert oracle, so the 4-bit path is the one that ran."""
    shape = datagen.LayerShape(name, T, d, l, E, k, h, hs, "bf16", seed=83, offset_var=0.5)
    w, x = datagen.layer_weights(shape), datagen.tokens(shape)
    layer = lq.layer_from_weights(shape, w, experts=lq.EXPERTS_MXFP4)
    y = layer.forward(x.cuda(), record_stats=True)
    again = layer.forward(x.cuda(), y=torch.empty_like(y))
    r = layer.routing()
    torch.cuda.synchronize()
    assert torch.equal(y, again)
    pick = np.arange(T) if T <= 1000 else np.arange(0, T, 16)
    xs = x[torch.from_numpy(pick)]
    ro = oracle.layer_routing(xs, w, np.zeros(E), k, shape.rms_eps)
    assert np.array_equal(r["idx"].cpu().numpy()[pick], ro["idx"])
    yg = y.float().cpu().numpy()[pick]
    y4 = mx.layer_forward_mxfp4(xs, w, np.zeros(E), k, shape.rms_eps)
    y16 = oracle.layer_forward(xs, w, np.zeros(E), k, shape.rms_eps)["y"]
    norm = lambda a, b: float(np.linalg.norm(a - b) / np.linalg.norm(b))
    err4, err16 = norm(yg, y4), norm(yg, y16)
    print(name, err4, err16)
    assert err4 <= 1e-2 and err16 >= 5 * err4, (err4, err16)
    assert layer.status() == 0
    with pytest.raises(lq.LmoeError, match="unsupported"):
        layer.forward_backward(x.cuda(), x.cuda(), {n: t.cuda() for n, t in w.items()})
    layer.close()


def test_layer_with_4_bit_experts_replays_and_updates():
    """Repeated forwards (replayed as a graph), another T on the same handle, and the bias update inside."""
    shape = datagen.LayerShape("mx4_replay", 700, 256, 128, 64, 4, 128, 256, "bf16", seed=85, offset_var=0.5)
    w, x = datagen.layer_weights(shape), datagen.tokens(shape).cuda()
    layer = lq.layer_from_weights(shape, w, experts=lq.EXPERTS_MXFP4)
    y, x2 = torch.empty_like(x), x.clone()
    first = layer.forward(x2, y=y).clone()
    for _ in range(3):
        assert torch.equal(layer.forward(x2, y=y), first)
    x2.copy_(x.flip(0))
    assert torch.equal(layer.forward(x2, y=y), first.flip(0))
    part = layer.forward(x[:130].contiguous()).float()  # other tiles, and sums in another order
    assert (part - first[:130].float()).norm() <= 1e-2 * first[:130].float().norm()
    layer.set_update(0.05)
    layer.forward(x, update_bias=True)
    assert layer.bias().abs().max() > 0 and layer.status() == 0
    layer.close()


def test_full_sized_products_on_sampled_rows():
    """The wide layer's expert shape and a dense product large enough for every variant."""
    g = torch.Generator(device="cuda").manual_seed(5)
    for M, N, K, G in ((4096, 8192, 2048, 0), (9344, 1024, 2048, 32), (6000, 2048, 512, 64)):
        a = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)
        w = torch.randn((max(G, 1), N, K), generator=g, device="cuda", dtype=torch.bfloat16)
        cuts = torch.sort(torch.randint(0, M + 1, (max(G - 1, 0),), generator=g, device="cuda")).values.int()
        off = None
        if G:
            off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), M)])
        for out in (torch.bfloat16, torch.float32):
            c = lq.mx4_gemm(lq.mx4_quant(a, offsets=off), lq.mx4_quant(w if G else w[0]), dtype=out)
            pick = torch.randint(0, M, (48,), generator=g, device="cuda")
            av = lq.mx4_dequant(lq.mx4_quant(a[pick]), dtype=torch.float32).double()
            grp = torch.searchsorted(off, pick.int(), right=True) - 1 if G else torch.zeros_like(pick)
            wv = lq.mx4_dequant(lq.mx4_quant(w), dtype=torch.float32)
            ref = torch.stack([wv[e].double() @ v for e, v in zip(grp.tolist(), av)])
            mag = torch.stack([wv[e].double().abs() @ v.abs() for e, v in zip(grp.tolist(), av)])
            check_product(np64(c[pick]), np64(ref), np64(mag), K, out)
