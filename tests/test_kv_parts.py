"""Host checks of how the cache library's Python layer takes its arguments (no GPU)."""

import copy
import ctypes as C
import os
import pickle

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(
    not os.path.exists(os.path.join(ROOT, "bit_nf4_quantized_04_amd", "libnf4kv.so")), reason="libnf4kv.so not built")
EINVAL, ELAUNCH = 1, 5
PARTS = ("k_codes", "k_scales", "v_codes", "v_scales")


@pytest.fixture(scope="module")
def K():
    from bit_nf4_quantized_04_amd import nf4kv

    return nf4kv


def of(c):
    """What the C functions get is what the attributes hold."""
    s = c.c_struct()
    assert tuple(getattr(s, n) for n in PARTS) == tuple(getattr(c, n).data_ptr() for n in PARTS)
    assert (s.n_pages, s.n_heads, s.head_dim, s.page_size) == (c.n_pages, c.n_heads, c.head_dim, c.page_size)
    assert s.quant_type == {"nf4": 0, "fp4": 1}[c.quant_type]
    return {getattr(c, n).data_ptr() for n in PARTS}


@pytest.mark.parametrize("quant", ["nf4", "fp4"])
def test_a_cache_that_is_copied_has_its_own_buffers(K, quant):
    c = K.nf4_kv_cache_alloc(3, 2, 128, 16, quant, device="cpu")
    mine = of(c)
    assert of(copy.copy(c)) == mine
    assert not of(copy.deepcopy(c)) & mine
    assert not of(pickle.loads(pickle.dumps(c))) & mine
    assert of(c) == mine


def test_a_cache_whose_buffers_are_replaced(K):
    c = K.nf4_kv_cache_alloc(3, 2, 128, 16, device="cpu")
    other = K.nf4_kv_cache_alloc(5, 4, 64, 32, "fp4", device="cpu")
    before, keep = of(c), [getattr(c, n) for n in PARTS]  # (kept: freed addresses come back)
    for n in PARTS:
        setattr(c, n, getattr(c, n).clone())
        of(c)
    assert not of(c) & before and len(keep) == 4
    c.k_codes.resize_(3, 2, 16, 32)
    with pytest.raises(ValueError):  # the others no longer fit
        c.c_struct()
    for n in (*PARTS, "quant_type"):
        setattr(c, n, getattr(other, n))
    assert of(c) == of(other)
    for n, wrong in (("k_codes", other.k_scales), ("v_scales", None), ("quant_type", "int4"), ("quant_type", 0)):
        keep = getattr(c, n)
        setattr(c, n, wrong)
        with pytest.raises(ValueError):
            c.c_struct()
        setattr(c, n, keep)
    del c.v_codes
    with pytest.raises(ValueError):
        c.c_struct()


def test_calls_want_a_cache(K):
    import torch

    slots = torch.zeros(4, dtype=torch.int64)
    for wrong in (None, 3, b"0" * 64, slots):
        with pytest.raises(ValueError):
            K.nf4_kv_read(wrong, slots)


def test_a_rope_table_is_made_on_the_current_gpu_only(K, monkeypatch):
    """With tensors that say they are on GPU 1 while GPU 0 is current, and the
    other way round, nothing is launched; with both the same it is, on the
    tensor's address and the current stream."""
    import types

    calls = []
    for where, current in ((1, 0), (0, 1), (1, 1)):
        t = types.SimpleNamespace(is_cuda=True, device=types.SimpleNamespace(index=where), data_ptr=lambda: 4096)
        cuda = types.SimpleNamespace(current_device=lambda: current,
                                     current_stream=lambda: types.SimpleNamespace(cuda_stream=77))
        monkeypatch.setattr(K, "torch", types.SimpleNamespace(empty=lambda *a, **k: t, float32=None, cuda=cuda))
        monkeypatch.setattr(K, "_lib", types.SimpleNamespace(nf4_rope_table=lambda *a: calls.append(a) or 0))
        if where != current:
            with pytest.raises(ValueError):
                K.nf4_rope_table(8, 64, device="cuda:%d" % where)
            assert not calls
        else:
            assert K.nf4_rope_table(8, 64, device="cuda:1") is t
            assert calls[0][:3] == (4096, 8, 64) and calls[0][-1] == 77


@pytest.mark.parametrize("heads,batch,max_q", [(1024, 8191, 256), (1024, 4096, 512), (1, 65535, 32768), (8, 65535, 4096),
                                               (1000, 40, 2048)])
def test_blocks_of_many_rows_up_to_what_a_grid_holds(K, heads, batch, max_q):
    """batch * n_heads * blocks of 256 rows: below 2^23 a call gets as far as the
    launch, which fails without a GPU; from 2^23 on it is refused."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    fake, other = C.c_void_p(0x100000), C.c_void_p(0x200000)
    c = K.nf4_kv_cache(fake, fake, fake, fake, 10, heads, 64, 32, 0)

    def call(batch, max_q, max_len=4096):
        return K._lib.nf4_kv_attention(C.byref(c), fake, heads * 64, 1, heads, fake, fake, fake, 1 << 20, batch, max_q,
                                       max_len, 1.0, 0, 0, other, heads * 64, None, 0, None)

    blocks = lambda b, n: b * heads * -(-n // 256)  # noqa: E731
    assert call(1, 128, 1 << 20) != EINVAL
    b = min(batch, ((1 << 23) - 1) // blocks(1, max_q))
    assert blocks(b, max_q) < 1 << 23 and call(b, max_q) == ELAUNCH
    over = -(-(1 << 23) // (b * heads)) * 256
    assert blocks(b, over) >= 1 << 23 and call(b, over) == EINVAL


def test_rotations_whose_outputs_would_overlap_are_refused(K):
    fake, other = C.c_void_p(0x100000), C.c_void_p(0x200000)

    def call(yt, yh, tokens=7, heads=5, dim=64):
        return K._lib.nf4_rope_forward(fake, heads * dim, dim, other, yt, yh, tokens, heads, dim, 1, fake, fake, 9, 64, 0, None)

    for yt, yh in ((64, 64), (4 * 64, 64), (64, 6 * 64), (64 + 32, 7 * 64), (0, 1 << 40), (-64, 1 << 40), (56, 1 << 20),
                   (1 << 62, 1 << 61)):
        assert call(yt, yh) == EINVAL, (yt, yh)
    assert call(64, 64, tokens=1 << 40) == EINVAL


def test_attention_with_zeros_refuses_what_attention_does(K):
    fake, other = C.c_void_p(0x100000), C.c_void_p(0x200000)
    c = K.nf4_kv_cache(fake, fake, fake, fake, 10, 8, 128, 32, 0)

    def call(fn, q=fake, qs=4096, n=1, qh=32, w=64, b=1, mq=1, ml=2048, sc=1.0, win=0, out=other, os_=4096, ws=None, cu=fake):
        return fn(C.byref(c), q, qs, n, qh, cu, fake, fake, w, b, mq, ml, sc, win, 0, out, os_, ws, 0, None)

    for code, kw in ((0, dict(n=0, q=None)), (EINVAL, dict(n=-1)), (EINVAL, dict(b=0)), (2, dict(qh=30)), (EINVAL, dict(ml=2049)),
                     (EINVAL, dict(win=-1)), (EINVAL, dict(q=None)), (EINVAL, dict(out=fake)), (EINVAL, dict(cu=None)),
                     (2, dict(qs=4100)), (EINVAL, dict(os_=2048)), (EINVAL, dict(sc=float("inf"))),
                     (4, dict(w=4096, ml=100000, b=2))):
        assert call(K._lib.nf4_kv_attention, **kw) == call(K._lib.nf4_kv_attention_padded, **kw) == code, kw
    assert call(K._lib.nf4_kv_attention, mq=0, out=None) == 0
    assert call(K._lib.nf4_kv_attention_padded, mq=0, out=None) == EINVAL  # rows to fill


def test_rope_tables_of_more_threads_than_a_grid_has(K):
    """A thread for each pair of each position: more than 2^31 are refused, as by
    the other calls."""
    import torch

    scaling = K.nf4_rope_scaling(0, 1.0, 1.0, 4.0, 8192.0, 1.0)
    call = lambda max_pos, rot: K._lib.nf4_rope_table(C.c_void_p(0x100000), max_pos, rot, 10000.0, C.byref(scaling), None)  # noqa: E731
    for max_pos, rot in ((1 << 35, 2), ((1 << 31) + 1, 2), ((1 << 25) + 1, 128), (1 << 24, 512), (1 << 62, 2)):
        assert call(max_pos, rot) == EINVAL, (max_pos, rot)
    if not torch.cuda.is_available():  # (the address is made up)
        assert call((1 << 25) - 256, 128) == call((1 << 31) - 256, 2) == ELAUNCH


@pytest.mark.parametrize("tokens", [1 << 62, 1 << 60, 1 << 56, (1 << 61) + 1, 1 << 40, 1 << 31])
def test_numbers_of_tokens_whose_products_do_not_fit(K, tokens):
    fake, other = C.c_void_p(0x100000), C.c_void_p(0x200000)
    c = K.nf4_kv_cache(fake, fake, fake, fake, 10, 8, 128, 32, 0)
    for fn in (K._lib.nf4_rope_forward, K._lib.nf4_rope_backward):
        assert fn(fake, 1024, 128, other, 1024, 128, tokens, 8, 128, 1, fake, fake, 64, 128, 0, None) == EINVAL
    assert K._lib.nf4_kv_append(C.byref(c), fake, 1024, fake, 1024, fake, tokens, fake, 4096, other, 4096, 32, fake, fake, 64,
                                128, 0, None) == EINVAL
    assert K._lib.nf4_kv_read(C.byref(c), fake, tokens, fake, fake, None) == EINVAL


def test_tiles_are_shared_while_their_sums_fit(K):
    """Shares are laid out in sums of all units' tiles (16 more for each): a
    workspace, which a call that shares them has, is asked for up to where a
    share's rounded end still fits 31 bits."""
    size = lambda tiles: K._lib.nf4_kv_attention_ws_bytes(64, 1, 1, 64, 1, 32 * tiles, 0, 0)  # noqa: E731
    assert 64 * (33554398 + 18) == (1 << 31) - 1024 and size(33554398) == size(33554399) == 0
    assert size(33554397) > 0
