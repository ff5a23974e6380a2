"""Calls of the compiled functions from three threads at once, each on a stream of its
own: products, the fused store with the load behind it, and the backward pass with
its workspace. A call that fails fails the test."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import int8_ref as I  # noqa: E402
from test_gpu_int8 import operands  # noqa: E402
from test_gpu_qkv import Case, cache, slots_of  # noqa: E402
from threads import together  # noqa: E402

ROUNDS = 40


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_three_threads():
    say("products, stores and gradients from three threads")
    product = operands(300, 2501, 4112)
    want = I.linear(*product)
    c, rows = Case(300, 8, 2, 80, 16), 320
    slots, before = slots_of(c.t, rows), cache(rows, c.hk, c.d)
    g = Case(700, 4, 4, 64, None, 3, True)

    def store(after):
        q = F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, slots, *after, **c.how)
        return (q, *after, *F.fp8_kv_load(*after, slots))

    def gradients():
        return F.fp8_qk_norm_rope_backward(g.dq, g.dk, g.q, g.k, *g.table, **g.how)

    stored, grads = store([x.clone() for x in before]), gradients()
    torch.cuda.synchronize()

    def on_a_stream(call, equal):
        def work():
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got = [call() for _ in range(ROUNDS)]
            stream.synchronize()
            return sum(bool(equal(y)) for y in got)
        return work

    counts = together(on_a_stream(lambda: F.int8_linear(*product[:4], bias=product[4]), lambda y: I.same_bits(y, want)),
                      on_a_stream(lambda: store([x.clone() for x in before]), lambda y: same(y, stored)),
                      on_a_stream(gradients, lambda y: same(y, grads)))
    assert counts == [ROUNDS] * 3
