"""The plain forms that the GPU tests compare with, against other ways to the
same numbers: complex products, differences, and whole tables."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import int8_ref as I  # noqa: E402
import qkv_ref as R  # noqa: E402


def case(interleaved, pairs, d=32, t=5, h=3):
    gen = torch.Generator().manual_seed(pairs + d)
    x = torch.randn(t, h, d, generator=gen, dtype=torch.float64)
    w = torch.randn(d, generator=gen, dtype=torch.float64)
    positions = torch.randint(-50, 1000, (3, t), generator=gen)
    freq = 100.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    return x, w, positions, freq, tuple(i % 3 for i in range(pairs)), 1e-3, interleaved


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pairs", [8, 16])
def test_turn_is_a_complex_product(interleaved, pairs):
    x, w, positions, freq, axes, eps, _ = case(interleaved, pairs)
    out, _ = R.forward(x, w, positions, freq, axes, eps, interleaved)
    n = x * w / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps)
    for t in range(x.shape[0]):
        for i in range(pairs):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
            angle = float(positions[axes[i], t]) * float(freq[i])
            z = torch.complex(n[t, :, a], n[t, :, b]) * complex(torch.tensor(1j * angle, dtype=torch.complex128).exp())
            assert torch.allclose(out[t, :, a], z.real, atol=1e-12) and torch.allclose(out[t, :, b], z.imag, atol=1e-12)
    assert torch.equal(out[..., 2 * pairs:], n[..., 2 * pairs:]) or torch.allclose(out[..., 2 * pairs:], n[..., 2 * pairs:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_by_differences(interleaved):
    x, w, positions, freq, axes, eps, _ = case(interleaved, 8, d=24, t=2, h=2)
    gen = torch.Generator().manual_seed(1)
    dy = torch.randn(x.shape, generator=gen, dtype=torch.float64)
    dx, _, dw, _ = R.backward(dy, x, w, positions, freq, axes, eps, interleaved, 1)

    def loss(x, w):
        return (R.forward(x, w, positions, freq, axes, eps, interleaved)[0] * dy).sum()

    step = 1e-6
    for _ in range(6):
        ex = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        ew = torch.randn(w.shape, generator=gen, dtype=torch.float64)
        diff = (loss(x + step * ex, w + step * ew) - loss(x - step * ex, w - step * ew)) / (2 * step)
        assert abs(float(diff - (dx * ex).sum() - (dw * ew).sum())) < 1e-6 * float((dx.abs() * ex.abs()).sum() + 1)


def test_bounds_reject_a_wrong_axis_and_a_wrong_sign():
    x, w, positions, freq, axes, eps, inter = case(False, 16)
    x, w, freq = x.to(torch.bfloat16), w.to(torch.bfloat16), freq.float()
    ref, bound = R.forward(x, w, positions, freq, axes, eps, inter)
    assert R.outside(ref.to(torch.bfloat16), ref, bound) <= 1
    for other in (R.forward(x, w, positions, freq, (0,) * 16, eps, inter), R.forward(x, w, positions, -freq, axes, eps, inter),
                  R.forward(x, w, positions, freq, axes, 2 * eps, inter), R.forward(x, w, positions, freq, axes, eps, True)):
        assert R.outside(other[0].to(torch.bfloat16), ref, bound) > 1
    gen = torch.Generator().manual_seed(1)
    dy = torch.randn(x.shape, generator=gen).to(torch.bfloat16)
    dx, db, dw, dwb = R.backward(dy, x, w, positions, freq, axes, eps, inter, 3)
    assert R.outside(dx.to(torch.bfloat16), dx, db) <= 1
    less = R.backward(dy[:-1], x[:-1], w, positions[:, :-1], freq, axes, eps, inter, 3)
    assert float(((less[2] - dw).abs() / dwb).max()) > 1
    other = R.backward(dy, x, w, positions, -freq, axes, eps, inter, 3)
    assert R.outside(other[0].to(torch.bfloat16), dx, db) > 1


def test_nearest_code_against_the_table():
    table = R.VALUES[:127]
    mid = (table[1:] + table[:-1]) / 2
    for x, code in ((mid, [i if i % 2 == 0 else i + 1 for i in range(126)]), (mid * (1 - 1e-9), range(126)),
                    (mid * (1 + 1e-9), range(1, 127))):
        got = R.nearest(x)
        assert torch.equal(got, table[torch.tensor(list(code))])
        assert torch.equal(R.nearest(-x), -got)
    assert float(R.nearest(torch.tensor(460.0, dtype=torch.float64))) == 448


def test_last_of_equal_slots():
    slots = torch.tensor([3, 5, 3, -1, 5, 9, 3])
    assert R.last_ones(slots, 9).tolist() == [False, False, False, False, True, False, True]


def test_quantizer_by_whole_numbers():
    x = torch.tensor([[127.0, -63.5, 62.5, 0.5, -1.5, 0.25], [0.0] * 6, [2.0 ** -149] * 6])
    q, s = I.quantize(x)
    assert s.tolist() == [1.0, 1.0, 1.0]
    assert q.tolist() == [[127, -64, 62, 0, -2, 0], [0] * 6, [0] * 6]


def test_linear_by_whole_numbers():
    gen = torch.Generator().manual_seed(0)
    xq = torch.randint(-128, 128, (3, 64), generator=gen, dtype=torch.int8)
    wq = torch.randint(-128, 128, (5, 64), generator=gen, dtype=torch.int8)
    xs, ws, bias = torch.rand(3), torch.rand(5), torch.randn(5).to(torch.bfloat16)
    acc = (xq.long()[:, None] * wq.long()[None]).sum(-1)
    ref = acc.double() * xs.double()[:, None] * ws.double() + bias.double()
    size = (acc.double() * xs.double()[:, None] * ws.double()).abs() + bias.double().abs()
    assert bool(((I.linear(xq, xs, wq, ws, bias).double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -21 * size).all())
