"""How the cache library's calls take the tensors that programs have: copied
caches, layouts whose strides differ, sizes at the interface's limits."""

import copy
import sys

import numpy as np
import pytest

from tests import gpu_util as U
from tests.test_gpu_kv_attention import Setup

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


def one_token(seed, heads, dim):
    """[1, heads, dim] as a transpose leaves it: contiguous, with another token
    stride than a row's length."""
    t = normal(seed, heads, 1, dim).transpose(0, 1)
    assert t.is_contiguous() and t.stride(0) < heads * dim
    return t


def test_single_tokens_of_any_stride(K):
    import torch

    c, d = (K.nf4_kv_cache_alloc(3, 2, 128, 16) for _ in range(2))
    k, v, q = one_token(1, 2, 128), one_token(2, 2, 128), one_token(3, 8, 128)
    slots, positions, table = torch.tensor([17], device=U.dev()), i32([5]), K.nf4_rope_table(9, 128)
    plain = [t.clone(memory_format=torch.contiguous_format).view(-1).view(t.shape) for t in (k, v, q)]
    assert all(t.stride(0) == t[0].numel() for t in plain)
    room = torch.zeros_like(q).view(-1)[: 8 * 128].view(8, 1, 128).transpose(0, 1)
    want = K.nf4_kv_append(c, *plain[:2], slots, positions, table, q=plain[2])
    assert torch.equal(want, K.nf4_kv_append(d, k, v, slots, positions, table, q=q))
    assert torch.equal(want, K.nf4_kv_append(d, k, v, slots, positions, table, q=q, q_out=room))
    assert all(torch.equal(a, b) for a, b in zip(K.nf4_kv_read(c, slots), K.nf4_kv_read(d, slots)))
    args = (i32([0, 1]), i32([2]), i32([[1]]))
    want = K.nf4_kv_attention(c, plain[2], *args, max_q=1)
    assert torch.equal(want, K.nf4_kv_attention(d, q, *args, max_q=1))
    room.zero_()
    K.nf4_kv_attention(d, q, *args, max_q=1, out=room)
    assert torch.equal(want, room)


@pytest.mark.parametrize("fn", ["nf4_rope_forward", "nf4_rope_backward"])
def test_rotations_of_single_tokens_and_heads(K, fn):
    import torch

    fn, table = getattr(K, fn), K.nf4_rope_table(40, 64)
    x = one_token(4, 6, 64)
    want = fn(x.reshape(-1).view(1, 6, 64), i32([7]), table)
    assert torch.equal(want, fn(x, i32([7]), table))
    room = torch.zeros(6, 1, 64, dtype=torch.bfloat16, device=U.dev()).transpose(0, 1)
    fn(x, i32([7]), table, out=room)
    assert torch.equal(want, room)
    assert torch.equal(want, fn(x, i32([7]), table, out=x))
    # one head of many tokens, its stride shorter than a head and of no whole vectors
    y = normal(5, 33, 64)
    odd = torch.as_strided(y, (33, 1, 64), (64, 3, 1))
    positions = i32(np.arange(33))
    assert torch.equal(fn(y.view(33, 1, 64), positions, table), fn(odd, positions, table))
    room = torch.zeros_like(y)
    fn(y.view(33, 1, 64), positions, table, out=torch.as_strided(room, (33, 1, 64), (64, 3, 1)))
    assert torch.equal(room.view(33, 1, 64), fn(y.view(33, 1, 64), positions, table))


def test_as_many_heads_as_a_cache_may_have(K):
    """Single tokens and blocks of rows of 1024 heads."""
    for lens, new in (([300, 40], [1, 1]), ([500], [100])):
        s = Setup(K, lens, new, 1024, 1024, 64, 16, "nf4", seed=40).device()
        s.check(s.run(), heads=(0, 511, 1023))


@pytest.mark.parametrize("lens,new,qh,kh", [([700, 90], [150, 97], 256, 256), ([50, 9000], [60, 60], 2, 1),
                                            ([2, 9, 40] * 4, [5, 1, 3] * 4, 256, 256), ([2, 90], [6, 1], 8, 2)])
def test_the_largest_windows(K, lens, new, qh, kh):
    """Windows around 2^31 hide nothing, also from requests with more queries than
    tokens, whose first ones stand before the first token: in blocks of many rows,
    in tokens that are split, with a wave for each request and with a workgroup."""
    import torch

    s = Setup(K, lens, new, qh, kh, 64, 16, "nf4", seed=41).device()
    want = s.run()
    s.check(want, heads=(0, kh - 1))
    for window in (max(lens), 2 ** 31 - 100, 2 ** 31 - 2, 2 ** 31 - 1):
        for sinks in (0, 5, 2 ** 31 - 1):
            assert torch.equal(want, s.run(window=window, sinks=sinks)), (window, sinks)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rot,gap", [(9, 5, 64, 64, 0), (700, 40, 128, 96, 0), (33, 3, 72, 20, 8),
                                                      (2, 2, 8, 8, 16)])
def test_rotations_of_tensors_with_the_heads_outside(K, tokens, heads, dim, rot, gap, layout, dtype):
    """[heads, tokens, dim] transposed, as inputs, as outputs and in place, with
    what lies between the heads left alone."""
    import torch

    table, positions = K.nf4_rope_table(64, rot), i32(np.arange(tokens) * 7 % 64)
    x = normal(6, tokens, heads, dim).to(getattr(torch, dtype))
    wide = torch.full((heads, tokens * dim + gap), 3.0, dtype=x.dtype, device=U.dev())
    outside = wide[:, : tokens * dim].unflatten(1, (tokens, dim)).transpose(0, 1)
    assert outside.shape == x.shape and outside.stride(0) == dim
    for fn in (K.nf4_rope_forward, K.nf4_rope_backward):
        want = fn(x, positions, table, layout)
        outside.zero_()
        fn(x, positions, table, layout, out=outside)
        assert torch.equal(want, outside)
        outside.copy_(x)
        assert torch.equal(want, fn(outside, positions, table, layout))
        fn(outside, positions, table, layout, out=outside)
        assert torch.equal(want, outside)
    assert bool((wide[:, tokens * dim:] == 3).all())


def after_sevens(shape, call):
    """The call's result in memory that held sevens before."""
    import torch

    torch.cuda.synchronize()
    torch.full(shape, 7.0, dtype=torch.bfloat16, device=U.dev())  # freed at once: the next of its size
    return call()


@pytest.mark.parametrize("lens,new,qh,kh,dim", [
    ([40, 70, 9], [1, 1, 1], 8, 2, 128), ([40, 70, 9], [6, 1, 3], 8, 2, 64), ([9000, 3000], [1, 1], 8, 2, 256),
    ([300, 40, 90] * 30, [1, 2, 3] * 30, 128, 64, 64), ([500, 300], [150, 97], 256, 256, 64), ([2500], [256], 64, 64, 128)])
def test_rows_that_nobody_computes(K, lens, new, qh, kh, dim):
    """Rows in front of the first request and behind the last, and queries past
    max_q, are zeros in an output that the call makes and stay in a given one."""
    import torch

    s = Setup(K, lens, new, qh, kh, dim, 16, "nf4", seed=42).device()
    want = s.run()
    n, before, behind = len(s.q), 5, 37
    s.qd = torch.cat((s.qd[:1].expand(before, -1, -1), s.qd, s.qd[:1].expand(behind, -1, -1)))
    s.args = (s.args[0] + before, *s.args[1:])
    full = torch.zeros_like(s.qd)
    full[before: before + n] = want
    assert torch.equal(full, after_sevens(full.shape, s.run))
    given = torch.full_like(full, 7.0)
    s.run(out=given)
    assert torch.equal(given[before: before + n], want)
    assert bool((given[:before] == 7).all()) and bool((given[before + n:] == 7).all())
    # fewer queries than a request has
    most = max(new) - 1
    if most:
        got = after_sevens(full.shape, lambda: s.run(max_q=most))
        given.fill_(7.0)
        s.run(max_q=most, out=given)
        for i, m in enumerate(new):
            rows = slice(before + s.cu[i] + min(most, m), before + s.cu[i] + m)
            assert not got[rows].any() and bool((given[rows] == 7).all()), i
            rows = slice(before + s.cu[i], before + s.cu[i] + min(most, m))
            assert torch.equal(got[rows], given[rows])
        assert not got[:before].any() and not got[before + n:].any()
    assert not after_sevens(full.shape, lambda: s.run(max_q=0)).any()


def test_rows_that_nobody_computes_in_strided_outputs(K):
    """The C function that makes zeros, on a slice of wider rows."""
    import ctypes as C

    import torch

    s = Setup(K, [40, 70], [3, 1], 8, 2, 64, 16, "nf4", seed=43).device()
    want, c = s.run(), s.cache.c_struct()
    for max_q in (0, 2, 3):
        wide = torch.full((9, 11, 64), 7.0, dtype=torch.bfloat16, device=U.dev())
        q = torch.cat((s.qd, s.qd, s.qd[:1]))
        assert K._lib.nf4_kv_attention_padded(
            C.byref(c), q.data_ptr(), q.stride(0), 9, 8, *(t.data_ptr() for t in s.args), s.args[2].shape[1], 2, max_q, 70,
            0.125, 0, 0, wide[:, 2:].data_ptr(), wide.stride(0), None, 0, torch.cuda.current_stream().cuda_stream) == 0
        out = wide[:, 2:10]
        assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 10:] == 7).all()) and not out[4:].any()
        assert torch.equal(out[:min(max_q, 3)], want[:min(max_q, 3)]) and not out[max_q:3].any()
        assert torch.equal(out[3], want[3]) if max_q else not out.any()
