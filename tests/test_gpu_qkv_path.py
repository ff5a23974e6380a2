"""The new operators as they are used together: a block's attention input from its
activation to the cache and back, prompt and single tokens; the same projection
in a training step, with its gradients; and sizes drawn over the whole range."""

from __future__ import annotations

import os
import random
import re

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import int8_ref as I  # noqa: E402
import layers_ref as LR  # noqa: E402
import qkv_ref as R  # noqa: E402

BF = torch.bfloat16
HQ, HK, D, WIDTH = 8, 2, 64, 512


def block(seed):
    gen = torch.Generator().manual_seed(seed)
    w = torch.randn((HQ + 2 * HK) * D, WIDTH, generator=gen).cuda() * 0.05
    weights = [(1 + 0.2 * torch.randn(D, generator=gen)).to(BF).cuda() for _ in range(2)]
    freq = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
    return gen, w, weights, freq, tuple(i % 3 for i in range(D // 2))


def split(qkv):
    t = qkv.shape[0]
    q, k, v = qkv.split([HQ * D, HK * D, HK * D], 1)
    return q.view(t, HQ, D), k.view(t, HK, D), v.view(t, HK, D)


def test_prompt_then_single_tokens():
    """Two sequences in pages of 16 rows, a padded batch: what is read back at the
    end is each token's own k and v, whatever stored it."""
    gen, w, (qw, kw), freq, axes = block(0)
    wq, ws = F.int8_row_quantize(w.to(BF))
    assert torch.equal(wq, I.quantize(w.to(BF))[0])
    rows, page = 160, 16
    cache = [torch.zeros(rows, HK, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.ones(rows, HK, device="cuda") for _ in range(2)]
    tables = torch.randperm(rows // page, generator=gen).view(2, 5)
    lengths, expected = [37, 21], ([], [])

    def run(tokens):
        """tokens: (sequence, position) of each row, None for padding."""
        t = len(tokens)
        x = torch.randn(t, WIDTH, generator=gen).to(BF).cuda()
        slots = torch.tensor([-1 if u is None else int(tables[u[0], u[1] // page]) * page + u[1] % page for u in tokens],
                             dtype=torch.int32)
        p = torch.tensor([0 if u is None else u[1] for u in tokens], dtype=torch.int32)
        positions = torch.stack([p, p // 3, p % 3]).cuda()
        qkv = F.int8_linear_bf16(x, wq, ws)
        assert I.same_bits(qkv, I.linear(*I.quantize(x), wq, ws))
        q, k, v = split(qkv)
        out = F.fp8_qk_norm_rope_store(q, k, v, qw, kw, positions, freq, slots.cuda(), *cache, axes=axes)
        ref, bound = R.forward(q, qw, positions, freq, axes, 1e-6, False)
        assert R.outside(out, ref, bound) <= 1
        kref, kbound = R.forward(k, kw, positions, freq, axes, 1e-6, False)
        for i, u in enumerate(tokens):
            if u is not None:
                expected[u[0]].append((kref[i], kbound[i], v[i].clone()))

    run([(0, i) for i in range(37)] + [None] * 3 + [(1, i) for i in range(21)] + [None] * 11)
    for step in range(9):
        run([(0, lengths[0]), None, (1, lengths[1])])
        lengths = [n + 1 for n in lengths]
    for s in range(2):
        i = torch.arange(lengths[s])
        slots = (tables[s][i // page] * page + i % page).to(torch.int32).cuda()
        k, v = F.fp8_kv_load(*cache, slots)
        ref, bound, values = (torch.stack(z) for z in zip(*expected[s]))
        scale = ref.abs().amax(-1, keepdim=True) / 448
        most = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * scale) * 1.001 + 2.0 ** -8 * 1.07 * ref.abs() + 3 * bound
        assert bool(((k.double() - ref).abs() <= most).all())
        codes, scales = R.stored(values)
        assert torch.equal(v, (codes * scales.double()[..., None]).float().to(BF))


class Projection(torch.autograd.Function):
    """q, k, v = split(x W^T) on a frozen block-FP8 weight; q and k normed and turned."""

    @staticmethod
    def forward(ctx, x, q8, s8, qw, kw, positions, freq, axes):
        qkv = F.fp8_block_linear(x, q8, s8)
        q, k, v = split(qkv)
        ctx.save_for_backward(qkv, q8, s8, qw, kw, positions, freq)
        ctx.axes = axes
        return (*F.fp8_qk_norm_rope(q, k, qw, kw, positions, freq, axes), v.clone())

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk, dv):
        qkv, q8, s8, qw, kw, positions, freq = ctx.saved_tensors
        grad = torch.empty_like(qkv)
        gq, gk, gv = split(grad)
        q, k, _ = split(qkv)
        _, _, dqw, dkw = F.fp8_qk_norm_rope_backward(dq.contiguous(), dk.contiguous(), q, k, qw, kw, positions, freq,
                                                     ctx.axes, q_grad=gq, k_grad=gk)
        gv.copy_(dv)
        dx, _ = F.fp8_block_linear_act_backward(grad, q8, s8)
        return dx, None, None, dqw.to(BF), dkw.to(BF), None, None, None


def test_training_step():
    """Gradients of the activation and of both norm weights through the projection,
    each stage against its own 64-bit form from the stage before."""
    gen, w, (qw, kw), freq, axes = block(1)
    t = 150
    q8, s8 = F.fp8_block_quantize(w)
    x = torch.randn(t, WIDTH, generator=gen).to(BF).cuda().requires_grad_(True)
    qw, kw = qw.requires_grad_(True), kw.requires_grad_(True)
    positions = torch.randint(0, 500, (3, t), generator=gen, dtype=torch.int32).cuda()
    out = Projection.apply(x, q8, s8, qw, kw, positions, freq, axes)
    grads = [torch.randn(o.shape, generator=gen).to(BF).cuda() for o in out]
    torch.autograd.backward(out, grads)
    with torch.no_grad():
        q, k, v = split(F.fp8_block_linear(x, q8, s8))
        packed = []
        for got, dy, heads, weight in ((qw.grad, grads[0], q, qw), (kw.grad, grads[1], k, kw)):
            dx, bound, dw, dw_bound = R.backward(dy, heads, weight, positions, freq, axes, 1e-6, False, 1)
            packed.append(F.fp8_qk_norm_rope_backward(*grads[:2], q, k, qw, kw, positions, freq, axes)[len(packed)])
            assert R.outside(packed[-1], dx, bound) <= 1
            assert bool(((got.double() - dw).abs() <= 2.0 ** -8 * 1.01 * dw.abs() + 1.01 * dw_bound).all())
        dz = torch.cat([packed[0].reshape(t, -1), packed[1].reshape(t, -1), grads[2].reshape(t, -1)], 1)
        LR.check_linear_act_backward(dz, None, q8, s8, "none", x.grad, dz, None, "projection")
    with pytest.raises(RuntimeError, match="autograd"):
        F.fp8_qk_norm_rope(q, k, qw, kw, positions, freq, axes)


def printed(name):
    """What the README's Python block that defines `name` defines."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), flags=re.S)
    scope = {"torch": torch, "F": F}
    exec(next(b for b in blocks if re.search(rf"(def|class) {name}\b", b)), scope)
    return scope


def test_printed_serving_example():
    gen, w, weights, freq, axes = block(2)
    scope = printed("attention_inputs")
    x = torch.randn(50, WIDTH, generator=gen).to(BF).cuda()
    wq, ws = F.int8_row_quantize(w)
    cache = [torch.zeros(64, HK, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.ones(64, HK, device="cuda") for _ in range(2)]
    slots = torch.randperm(64, generator=gen)[:50].to(torch.int32).cuda()
    positions = torch.randint(0, 99, (3, 50), generator=gen, dtype=torch.int32).cuda()
    out = scope["attention_inputs"](x, wq, ws, *weights, positions, freq, axes, slots, cache, (HQ, HK), D)
    q, k, v = split(I.linear(*I.quantize(x), wq, ws))
    assert R.outside(out, *R.forward(q, weights[0], positions, freq, axes, 1e-6, False)) <= 1
    _, loaded = scope["context"](slots, cache)
    codes, scale = R.stored(v)
    assert torch.equal(loaded, (codes * scale.double()[..., None]).float().to(BF))


def test_printed_training_example():
    """Gradients through the printed function, from an expanded output gradient too."""
    gen, _, weights, freq, axes = block(3)
    turn = printed("QkNormRope")["QkNormRope"].apply
    q, k = (torch.randn(40, h, D, generator=gen).to(BF).cuda().requires_grad_(True) for h in (HQ, HK))
    weights = [x.requires_grad_(True) for x in weights]
    positions = torch.randint(0, 99, (3, 40), generator=gen, dtype=torch.int32).cuda()
    out = turn(q, k, *weights, positions, freq, axes)
    (out[0].sum() + out[1].float().square().sum()).backward()
    for x, w, dy in ((q, weights[0], torch.ones_like(q)), (k, weights[1], (2 * out[1].float()).to(BF))):
        with torch.no_grad():
            dx, bound, dw, dw_bound = R.backward(dy, x, w, positions, freq, axes, 1e-6, False, 1)
            assert R.outside(x.grad, dx, bound) <= 1
            assert bool(((w.grad.double() - dw).abs() <= 2.0 ** -8 * 1.01 * dw.abs() + 1.01 * dw_bound).all())


def test_outputs_are_ordinary_tensors():
    """What the functions allocate: contiguous, without a gradient, usable by recorded
    operations, inference tensors in inference mode, from the pool of a capture."""
    x = torch.randn(4, 64, device="cuda").to(BF)
    wq, ws = F.int8_row_quantize(torch.randn(32, 64, device="cuda"))
    y = F.int8_linear_bf16(x, wq, ws)
    assert wq.dtype == torch.int8 and ws.dtype == torch.float32 and y.dtype == BF and y.shape == (4, 32)
    assert y.is_contiguous() and not y.requires_grad and not y.is_inference() and y.device == x.device
    leaf = torch.ones_like(y).requires_grad_(True)
    (leaf * y).sum().backward()
    assert torch.equal(leaf.grad, y)
    with torch.inference_mode():
        z = F.int8_linear_bf16(x, wq, ws)
        assert z.is_inference() and torch.equal(z, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = F.int8_linear_bf16(x, wq, ws)
    for _ in range(3):
        x.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, F.int8_linear_bf16(x, wq, ws))


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(40))
def test_drawn_int8(seed):
    rng = random.Random(seed)
    while True:
        m, n, k = _log(rng, 1, 3000), _log(rng, 1, 9000), 16 * _log(rng, 1, 1000)
        if m * n * k <= 2e10 and n * k <= 3e7:
            break
    say("int8", m, n, k)
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(m, k, generator=gen) * torch.exp(torch.randn(m, 1, generator=gen))).to(BF).cuda()
    wq = torch.randint(-128, 128, (n, k), generator=gen, dtype=torch.int8).cuda()
    ws = (torch.rand(n, generator=gen) * 0.01).cuda()
    bias = torch.randn(n, generator=gen).to(BF).cuda() if rng.random() < 0.5 else None
    q, s = F.int8_row_quantize(x)
    eq, es = I.quantize(x)
    assert torch.equal(q, eq) and I.same_bits(s, es)
    y = F.int8_linear_bf16(x, wq, ws, bias=bias)
    assert I.same_bits(y, I.linear(q, s, wq, ws, bias)) and I.same_bits(y, F.int8_linear(q, s, wq, ws, bias=bias))


@pytest.mark.parametrize("seed", range(40))
def test_drawn_heads(seed):
    rng = random.Random(100 + seed)
    inter = rng.random() < 0.5
    d = 8 * rng.randint(2, 32)
    step = 4 if inter else 8
    pairs = step * rng.randint(1, d // 2 // step) if d // 2 >= step else None
    hq, hk = _log(rng, 1, 70), _log(rng, 1, 40)
    t = max(1, min(_log(rng, 1, 6000), 1500000 // ((hq + hk) * d)))
    axes_count = rng.randint(1, 8)
    say("heads", t, hq, hk, d, pairs, axes_count, inter)
    gen = torch.Generator().manual_seed(seed)
    q, k, v, dq, dk = (torch.randn(t, h, d, generator=gen).to(BF).cuda() for h in (hq, hk, hk, hq, hk))
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=gen)).to(BF).cuda() for _ in range(2))
    positions = torch.randint(-1000, 300000, (axes_count, t), generator=gen, dtype=torch.int32).cuda()
    freq = (1e4 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()
    axes = bytes(rng.randrange(axes_count) for _ in range(pairs))
    eps = 10.0 ** -rng.randint(3, 8)
    how = {"axes": axes, "eps": eps, "interleaved": inter}
    refs = [R.forward(x, w, positions, freq, axes, eps, inter) for x, w in ((q, qw), (k, kw))]
    for got, ref in zip(F.fp8_qk_norm_rope(q, k, qw, kw, positions, freq, **how), refs):
        assert R.outside(got, *ref) <= 1
    lanes = next(l for l in (2, 4, 8, 16, 32) if 8 * l >= d)
    got = F.fp8_qk_norm_rope_backward(dq, dk, q, k, qw, kw, positions, freq, **how)
    for i, (dy, x, w) in enumerate(((dq, q, qw), (dk, k, kw))):
        steps = -(-x.shape[1] * lanes // 64) * -(-t // 4096)
        dx, bound, dw, dw_bound = R.backward(dy, x, w, positions, freq, axes, eps, inter, steps)
        assert R.outside(got[i], dx, bound) <= 1
        assert bool(((got[2 + i].double() - dw).abs() <= dw_bound + R.U * dw.abs()).all())
    rows = t + rng.randint(0, 100)
    slots = torch.randperm(rows, generator=gen)[:t].to(torch.int32)
    if rng.random() < 0.5:                     # padding, and tokens that share a slot
        slots[torch.rand(t, generator=gen) < 0.2] = -1
        slots[torch.rand(t, generator=gen) < 0.2] = int(slots[0])
    slots = slots.cuda()
    live = R.last_ones(slots.cpu(), rows).cuda()
    cache = [torch.zeros(rows, hk, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.ones(rows, hk, device="cuda") for _ in range(2)]
    fused = [c.clone() for c in cache]
    F.fp8_kv_store(k, v, slots, *cache)
    qo = F.fp8_qk_norm_rope_store(q, k, v, qw, kw, positions, freq, slots, *fused, **how)
    assert R.outside(qo, *refs[0]) <= 1
    at = slots[live].long()
    for i, x in enumerate((k, v)):
        values, scale = R.stored(x)
        assert torch.equal(R.values(cache[i][at]), values[live]) and torch.equal(cache[2 + i][at], scale[live])
    assert torch.equal(fused[1], cache[1]) and torch.equal(fused[3], cache[3])
    ref, bound = (z[live] for z in refs[1])
    scale = fused[2][at].double()[..., None]
    most = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * scale) * 1.001 + 3 * bound
    assert bool(((R.values(fused[0][at]) * scale - ref).abs() <= most).all())
    for side in (cache, fused):
        kl, vl = F.fp8_kv_load(*side, slots)
        assert torch.equal(kl, R.loaded(side[0], side[2], slots)) and torch.equal(vl, R.loaded(side[1], side[3], slots))
