"""How the cache library's calls take the tensors that programs have: copied
caches, layouts whose strides differ, sizes at the interface's limits."""

import copy
import sys

import numpy as np
import pytest

from tests import gpu_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    print("\n[gpu] %s" % request.node.nodeid, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def K():
    from bit_nf4_quantized_04_amd import nf4kv

    return nf4kv


def i32(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(U.dev())


def normal(seed, *shape):
    import torch

    g = torch.Generator(device=U.dev()).manual_seed(seed)
    return torch.randn(shape, generator=g, device=U.dev()).bfloat16()


def test_a_copied_cache_is_written_and_read_by_itself(K):
    import torch

    c = K.nf4_kv_cache_alloc(4, 2, 128, 16)
    slots = torch.arange(20, device=U.dev())
    K.nf4_kv_append(c, normal(1, 20, 2, 128), normal(2, 20, 2, 128), slots)
    first = K.nf4_kv_read(c, slots)
    d = copy.deepcopy(c)
    K.nf4_kv_append(d, normal(3, 20, 2, 128), normal(4, 20, 2, 128), slots)
    second = K.nf4_kv_read(d, slots)
    assert all(torch.equal(a, b) for a, b in zip(first, K.nf4_kv_read(c, slots)))
    assert not any(torch.equal(a, b) for a, b in zip(first, second))
    args = (normal(5, 1, 4, 128), i32([0, 1]), i32([20]), i32([[0, 1]]))
    out = K.nf4_kv_attention(d, *args, max_q=1)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):  # the other's buffers from here on
        setattr(c, n, getattr(d, n))
    assert all(torch.equal(a, b) for a, b in zip(second, K.nf4_kv_read(c, slots)))
    assert torch.equal(out, K.nf4_kv_attention(c, *args, max_q=1))
