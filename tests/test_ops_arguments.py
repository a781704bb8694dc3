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
