"""bench.py's algorithmic bytes of the routed experts follow their format."""
import bench
import datagen


def test_expert_bytes_by_format():
    s = datagen.WORKLOADS["wide_stress"]
    T, TK = s.T, s.T * s.k
    work = {f: bench.stage_work(s, T, n) for f, n in bench.EXPERT_FORMATS.items()}
    assert work["bf16"] == bench.stage_work(s, T)
    # rows, gate and linear weights, activations; 17 bytes for 32 values in 4 bits, 33 in 8
    values = TK * s.l + 2 * s.E * s.h * s.l + TK * s.h
    assert work["bf16"]["expert_swiglu"][1] == 2 * values
    assert work["mxfp8"]["expert_swiglu"][1] == 33 * values / 32
    assert work["mxfp4"]["expert_swiglu"][1] == 17 * values / 32
    for f, n in (("bf16", 64), ("mxfp8", 33), ("mxfp4", 17)):
        assert work[f]["expert_down"][1] == (TK * s.h + s.E * s.l * s.h) * n / 32 + 2 * TK * s.l
        assert work[f]["gather"][1] == 2 * T * s.l + TK * (s.l * n / 32 + 12)
    # the other stages, and every stage's operations, are the same in all
    for f in ("mxfp8", "mxfp4"):
        for stage, (flops, by) in work[f].items():
            assert flops == work["bf16"][stage][0]
            assert by == work["bf16"][stage][1] or stage in ("expert_swiglu", "expert_down", "gather")
