"""Arguments of the operators' entry points that their sizes or their callers make unusual, on the CPU (no call
here reaches a device)."""
import ctypes

import pytest
import torch

import latent_routing_quantile_b200 as lq
from latent_routing_quantile_b200 import build as lbuild

EINVAL, EUNSUPPORTED = -1, -4
P = 1 << 20  # a pointer that is aligned and never read


@pytest.fixture(scope="module")
def L():
    lbuild.build()
    return lq.lib()


def test_set_balance_refuses_more_sequences_than_its_steps_take(L):
    assert L.lmoe_set_balance(None, 0.1, P, (1 << 24) + 1) == EUNSUPPORTED
    assert L.lmoe_set_balance(None, 0.1, P, 1 << 24) == EINVAL  # no handle


def _bytes(L, rows, cols, groups, ragged):
    e, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    return L.lmoe_mx4_bytes(rows, cols, groups, ragged, ctypes.byref(e), ctypes.byref(s)), e.value, s.value


def test_sizes_of_the_widest_rows(L):
    """cols up to the last multiple of 32 that an int32 holds: k-blocks of 256 are counted without overflow."""
    cols = (1 << 31) - 32
    assert _bytes(L, 1, cols, 1, 0) == (0, cols // 2, 1024 * (1 << 23))
    assert _bytes(L, 128, cols - 192, 1, 1) == (0, 128 * ((cols - 192) // 2), 2 * 1024 * ((1 << 23) - 1) + 2 * 1024)
    # 2^23 k-blocks of 8 slices a tile: 31 tiles stay below 2^31 slices, 32 do not
    assert _bytes(L, 31 * 128, cols, 1, 0)[0] == 0
    assert _bytes(L, 31 * 128 + 1, cols, 1, 0)[0] == EUNSUPPORTED


def _of(shape, dtype):
    """A tensor of any shape on the meta device: no memory."""
    return torch.empty(shape, dtype=dtype, device="meta")


def test_sizes_past_32_bits_are_refused_not_cut():
    """2^32 + 32 columns are not 32 columns."""
    big, bf = (1 << 32) + 32, torch.bfloat16
    calls = [lambda: lq.mx4_quant(_of((1, big), bf)),
             lambda: lq.mx4_quant(_of((big, 1, 64), bf)),
             lambda: lq.mx4_quant(_of((1, 64), bf), offsets=_of((big,), torch.int32)),
             lambda: lq.mx4_quant_w13(*(_CudaLike((64, big)) for _ in range(2))),
             lambda: lq.mx4_quant_w13(*(_CudaLike((big, 32)) for _ in range(2))),
             lambda: lq.balance_loss(_of((big, 8), torch.float32), _of((big, 2), torch.int32), 0.1),
             lambda: lq.balance_loss(_of((8, 8), torch.float32), _of((8, 2), torch.int32), 0.1,
                                     cu_seqlens=_of((big,), torch.int32)),
             lambda: lq.Layer.set_balance(lq.Layer.__new__(lq.Layer), 0.1, _of((big,), torch.int32))]
    for call in calls:
        with pytest.raises(lq.LmoeError, match="unsupported shape"):
            call()


class _CudaLike:
    """What mx4_quant_w13 looks at before its sizes."""
    dtype, is_cuda = torch.bfloat16, True

    def __init__(self, shape):
        self.shape = torch.Size(shape)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True


def test_op_status_clears_only_the_bits_it_returns(monkeypatch):
    """A bit that another thread's call sets between the read and the clearing is there for the next read."""
    class Word(torch.Tensor):
        def item(self):
            v = super().item()
            self.bitwise_or_(lq.STATUS_BAD_INDEX)
            return v

    word = torch.tensor([lq.STATUS_NAN_SCORE], dtype=torch.int32).as_subclass(Word)
    monkeypatch.setattr(lq, "_status_words", {0: (word, word.data_ptr())})
    monkeypatch.setattr(torch.cuda, "synchronize", lambda index=None: None)
    assert lq.op_status(torch.device("cuda", 0)) == lq.STATUS_NAN_SCORE
    assert lq.op_status(torch.device("cuda", 0)) == lq.STATUS_BAD_INDEX
