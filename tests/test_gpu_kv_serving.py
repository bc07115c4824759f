"""Which rows belong to which request when the example's server turns some of
them away, and in steps with more rows than tokens."""

import importlib.util
import os
import sys

import numpy as np
import pytest

from oracle import nf4_oracle as O
from tests import gpu_util as U
from tests import kv_ref as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _announce(request):
    print("\n[gpu] %s" % request.node.nodeid, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def E():
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def i32(v):
    import torch

    return torch.tensor(v, dtype=torch.int32).to(U.dev())


def tokens(rng, n, hidden):
    return U.bf(O.rne_bf16_bits(rng.standard_normal((n, hidden)).astype(np.float32)).reshape(n, hidden))


def test_rows_stay_with_their_requests(E):
    """Each request's entries and outputs come from its own rows, laid out by
    new_lens, with refused and ending requests between those that go on."""
    import torch

    rng = np.random.default_rng(8)
    hidden, heads, kv_heads, dim, page, max_len, batch = 256, 4, 2, 64, 16, 128, 4
    layer = E.AttentionLayer(hidden, heads, kv_heads, dim, r=8, max_pos=max_len, seed=3)
    server = E.Server(layer, batch, 8, max_len, page)
    rope = layer.rope.cpu().numpy()
    held = [[] for _ in range(batch)]  # each request's (k, v) tokens
    steps = [  # new, done, what the requests are expected to be granted
        ([20, 16, 30, 17], [0, 0, 0, 0], [20, 16, 30, 17]),
        ([1, 20, 40, 1], [0, 0, 0, 0], [1, 0, 0, 1]),    # one free page: the two in the middle have to wait
        ([1, 7, 1, 1], [0, 1, 0, 0], [1, 0, 1, 1]),      # the second ends, whatever it asks for
        ([-2, 3, 50, 9], [0, 0, 0, 0], [0, 3, 0, 9]),    # a negative length is none
        ([2, 1, 1, 1], [1, 0, 0, 0], [0, 1, 1, 1]),
    ]
    for new, done, granted in steps:
        asked = [max(a, 0) for a in new]
        n, first = sum(asked), np.concatenate(([0], np.cumsum(asked)))
        x = tokens(rng, n, hidden)
        y, plan = server.step(x, i32(new), max(asked), i32(done))
        lens, cu = plan.kv_lens.cpu().numpy(), plan.cu_new.cpu().numpy()
        assert np.diff(cu).tolist() == granted
        rows = np.concatenate([np.arange(first[i], first[i] + granted[i]) for i in range(batch)])
        q, k, v = layer.project(x)
        positions = plan.positions.cpu().numpy()[: len(rows)]
        at = torch.from_numpy(rows).to(U.dev())
        k_rot = O.rne_bf16(R.rotate(U.bf16_to_f64(k[at]).astype(np.float32), positions, rope, "half")
                           ).reshape(len(rows), kv_heads, dim)
        vf = U.bf16_to_f64(v[at]).astype(np.float32)
        table = server.table.cpu().numpy()
        for i in range(batch):
            held[i] = [] if done[i] else held[i] + [(k_rot[t], vf[t]) for t in range(cu[i], cu[i + 1])]
            assert lens[i] == len(held[i])
            if not held[i]:
                continue
            t = np.arange(lens[i])
            for side, (codes, scales) in enumerate(((server.cache.k_codes, server.cache.k_scales),
                                                    (server.cache.v_codes, server.cache.v_scales))):
                c, a = R.store(np.stack([e[side] for e in held[i]]), "nf4")
                where = (table[i, t // page], slice(None), t % page)
                assert np.array_equal(codes.cpu().numpy()[where], c), (i, side)
                assert np.array_equal(U.bf16_to_f64(scales)[where], a), (i, side)
        att = torch.zeros((n, heads, dim), dtype=torch.bfloat16, device=U.dev())
        att[: len(rows)] = E.nf4kv.nf4_kv_attention(
            server.cache, E.nf4kv.nf4_rope_forward(q[at], plan.positions[: len(rows)], layer.rope), plan.cu_new,
            plan.kv_lens, server.table, max_q=max(asked), max_len=max_len)
        want = E.nf4qlora.qlora_linear_forward(layer.out, att.view(n, -1), layer.a_out, layer.b_out, layer.scale)
        assert np.array_equal(U.bits_of(y[: len(rows)]), U.bits_of(want[: len(rows)]))
