"""The 8-bit integer linear and its quantizer on the GPU: every output bit is
determined by the definition (tests/int8_ref.py), so everything is compared bit
for bit."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import int8_ref as R  # noqa: E402

BF = torch.bfloat16


def codes(gen, rows, k):
    return torch.randint(-128, 128, (rows, k), generator=gen, dtype=torch.int8).cuda()


def scales(gen, rows):
    return (torch.rand(rows, generator=gen) * 0.02 + 1e-3).cuda()


def operands(m, n, k, bias=True):
    gen = torch.Generator().manual_seed(m + 3 * n + 7 * k)
    b = torch.randn(n, generator=gen).to(BF).cuda() if bias else None
    return codes(gen, m, k), scales(gen, m), codes(gen, n, k), scales(gen, n), b


# Smallest sizes, odd ones, K tails, rows and columns below, at and past tile
# edges, columns that are no multiple of 8, few rows and many.
SHAPES = [
    (1, 1, 16), (1, 8, 16), (1, 129, 400), (1, 2048, 2064), (1, 8000, 8192), (2, 7, 80), (3, 130, 48), (4, 4099, 336),
    (5, 1000, 272), (8, 33, 4368), (15, 64, 128), (16, 520, 1040), (17, 64, 4096), (31, 300, 8208), (32, 257, 512),
    (32, 8193, 272), (33, 256, 528), (48, 40, 2064), (63, 65, 64), (64, 384, 256), (65, 129, 192), (77, 1003, 656),
    (128, 128, 128), (129, 257, 144), (130, 300, 1040), (192, 256, 256), (193, 264, 400), (200, 1288, 144),
    (256, 256, 1024), (257, 520, 784), (300, 36, 2320), (333, 4300, 1168), (512, 5120, 2576), (513, 1028, 336),
    (1025, 264, 80), (2304, 2056, 272), (4100, 1300, 400),
]


@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_linear(shape):
    say("int8_linear", *shape)
    xq, xs, wq, ws, bias = operands(*shape)
    y = F.int8_linear(xq, xs, wq, ws, bias=bias)
    plain = F.int8_linear(xq, xs, wq, ws)
    assert R.same_bits(y, R.linear(xq, xs, wq, ws, bias))
    assert R.same_bits(plain, R.linear(xq, xs, wq, ws))


# Large tiles in one round of workgroups and in several (whole and cut off, with
# few steps and many, rows of whole lines and not), splits of K of every tile and of
# few rows, and of the smallest last range.
LARGE = [
    (2048, 5120, 2064), (2045, 5117, 528), (1999, 8001, 1040), (1280, 13000, 1040), (8192, 8192, 400), (8190, 8200, 1024),
    (16385, 5120, 272), (16300, 5121, 144), (500, 5000, 25600), (1500, 1203, 40960), (500, 2000, 12304), (300, 2501, 20496),
    (1000, 1000, 30000), (64, 1000, 25600), (200, 136, 131056), (1, 300, 32784), (1, 5000, 32784), (1, 4500, 16400),
    (9, 500, 16400), (16, 300, 25600), (16, 5000, 20480), (32, 1000, 8208), (20, 4500, 8208), (29, 100, 131056),
]


@pytest.mark.parametrize("shape", LARGE, ids=["x".join(map(str, s)) for s in LARGE])
def test_large_tiles_and_splits(shape):
    say("int8_linear", *shape)
    xq, xs, wq, ws, bias = operands(*shape)
    want = R.linear(xq, xs, wq, ws, bias)
    for _ in range(3):
        assert R.same_bits(F.int8_linear(xq, xs, wq, ws, bias=bias), want)


def test_two_threads():
    """Calls from two threads at once, each on a stream of its own."""
    import threading
    say("int8_linear from two threads")
    shapes = [(300, 2501, 4112), (17, 700, 8208)]
    data = [operands(*s) for s in shapes]
    want = [R.linear(*d) for d in data]
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [F.int8_linear(*data[i][:4], bias=data[i][4]) for _ in range(40)]
        stream.synchronize()
        wrong.extend(i for y in got if not R.same_bits(y, want[i]))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("m,n", [(1, 40), (16, 40), (100, 300)])
def test_largest_sums(m, n):
    """k at its limit with every code -128: sums of 2^31 - 2^18."""
    k = 131056
    say("int8_linear", m, n, k)
    xq = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    wq[1::2] = 127
    xs, ws = torch.full((m,), 2.0 ** -10, device="cuda"), torch.full((n,), 2.0 ** -9, device="cuda")
    assert R.same_bits(F.int8_linear(xq, xs, wq, ws), R.linear(xq, xs, wq, ws))


ROWS = [(1, 16), (1, 8192), (2, 48), (3, 2064), (7, 4096), (16, 5120), (33, 272), (100, 1040), (257, 8208), (1000, 32),
        (3, 131056)]


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("m,k", ROWS)
def test_quantize(m, k, dtype):
    say("int8_row_quantize", m, k, dtype)
    gen = torch.Generator().manual_seed(m + k)
    x = torch.randn(m, k, generator=gen) * torch.exp(4 * torch.randn(m, 1, generator=gen))
    x = x.to(dtype).cuda()
    q, s = F.int8_row_quantize(x)
    eq, es = R.quantize(x)
    assert R.same_bits(s, es) and torch.equal(q, eq)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_quantize_special_rows(dtype):
    """Rows of zeros (both signs), subnormals, the largest values, ties of the
    rounding, one value among zeros, and scales of few bits."""
    k = 64
    rows = [torch.zeros(k), -torch.zeros(k), torch.full((k,), 2.0 ** -133), torch.linspace(-127, 127, k).round() * 2.0 ** -133,
            torch.full((k,), torch.finfo(dtype).max), torch.arange(k) - 31.5, (torch.arange(k) * 4 - 127) * 0.5,
            torch.cat([torch.ones(1), torch.zeros(k - 1)]), torch.cat([torch.zeros(k - 1), -torch.ones(1)]),
            torch.linspace(-1, 1, k) * 190 * 2.0 ** -133, torch.linspace(-1, 1, k) * 2.0 ** -100]
    if dtype == torch.float32:
        rows += [torch.full((k,), 2.0 ** -149), (torch.arange(k) - 32.0) * 2.0 ** -149, torch.arange(k) * 3 * 2.0 ** -149,
                 torch.linspace(-190, 190, k).round() * 2.0 ** -149]
    x = torch.stack(rows).to(dtype)
    q, s = F.int8_row_quantize(x.cuda())
    eq, es = R.quantize(x)
    assert R.same_bits(s.cpu(), es) and torch.equal(q.cpu(), eq)


def test_quantize_every_bf16_quotient():
    """Every bf16 maximum with every bf16 below it would be 2^30 pairs; here each
    maximum of one binade and each value of the nine binades below."""
    top = (torch.arange(128) / 128 + 1).to(BF)
    low = torch.cat([top * 2.0 ** -e for e in range(0, 9)]).to(BF)
    x = low.repeat(128, 1)
    x = torch.where(x > top[:, None], torch.zeros_like(x), x)
    x = torch.cat([top[:, None], x, -x, torch.zeros(128, 15, dtype=BF)], 1)
    q, s = F.int8_row_quantize(x.cuda())
    eq, es = R.quantize(x)
    assert R.same_bits(s.cpu(), es) and torch.equal(q.cpu(), eq)


@pytest.mark.parametrize("shape", [(1, 520, 8192), (2, 40, 48), (4, 1000, 5120), (5, 72, 4096), (16, 2056, 1040), (40, 300, 272),
                                   (300, 520, 1040)])
def test_from_bf16(shape):
    """The same bits as the two calls, which are the definition's."""
    m, n, k = shape
    say("int8_linear_bf16", *shape)
    _, _, wq, ws, bias = operands(m, n, k)
    gen = torch.Generator().manual_seed(m)
    x = (torch.randn(m, k, generator=gen) * torch.exp(torch.randn(m, 1, generator=gen))).to(BF).cuda()
    for b in (None, bias):
        y = F.int8_linear_bf16(x, wq, ws, bias=b)
        q, s = F.int8_row_quantize(x)
        assert R.same_bits(y, F.int8_linear(q, s, wq, ws, bias=b))
        assert R.same_bits(y, R.linear(*R.quantize(x), wq, ws, b))


def test_rows_that_are_not_finite_stay_their_own():
    m, n, k = 40, 72, 272
    _, _, wq, ws, bias = operands(m, n, k)
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    ref = F.int8_linear_bf16(x, wq, ws, bias=bias)
    x[3, 5], x[17, 0], x[31, 271] = float("nan"), float("inf"), float("-inf")
    y = F.int8_linear_bf16(x, wq, ws, bias=bias)
    others = [i for i in range(m) if i not in (3, 17, 31)]
    assert R.same_bits(y[others], ref[others])


@pytest.mark.parametrize("shape", [(1, 300, 400), (16, 4099, 2064), (33, 257, 528), (300, 1003, 656), (1025, 264, 80)])
def test_writes_only_its_output_and_workspace(shape):
    """Output and a workspace of exactly the queried size between guards, the
    workspace full of NaNs before."""
    m, n, k = shape
    xq, xs, wq, ws, bias = operands(m, n, k)
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    for from_bf16 in (False, True):
        size = F.int8_workspace_size(m, n, k, from_bf16=from_bf16)
        assert size % 256 == 0
        buf = torch.full((size + 512,), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.full((m * n + 256,), 3.0, dtype=BF, device="cuda")
        y, work = out[128:128 + m * n].view(m, n), buf[256:256 + size]
        if from_bf16:
            F.int8_linear_bf16(x, wq, ws, bias=bias, out=y, workspace=work)
            ref = R.linear(*R.quantize(x), wq, ws, bias)
        else:
            F.int8_linear(xq, xs, wq, ws, bias=bias, out=y, workspace=work if size else None)
            ref = R.linear(xq, xs, wq, ws, bias)
        assert R.same_bits(y, ref)
        assert bool((out[:128] == 3).all()) and bool((out[128 + m * n:] == 3).all())
        assert bool((buf[:256] == 0xFF).all()) and bool((buf[256 + size:] == 0xFF).all())


def test_other_streams_and_two_at_once():
    shapes = [(1, 2056, 4096), (16, 1000, 5120), (300, 520, 2064), (700, 1288, 1040)]
    cases = [(operands(*s), torch.cuda.Stream()) for s in shapes]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for (xq, xs, wq, ws, bias), stream in cases:
            with torch.cuda.stream(stream):
                got.append(F.int8_linear(xq, xs, wq, ws, bias=bias))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert R.same_bits(y, R.linear(*cases[i % len(cases)][0]))


@pytest.mark.parametrize("shape", [(1, 2056, 4096), (16, 1000, 5120), (300, 520, 2064)])
def test_captured_and_replayed(shape):
    m, n, k = shape
    _, _, wq, ws, bias = operands(m, n, k)
    gen = torch.Generator().manual_seed(9)
    x = torch.empty(m, k, dtype=BF, device="cuda")
    y = torch.empty(m, n, dtype=BF, device="cuda")
    work = torch.empty(F.int8_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        F.int8_linear_bf16(x.zero_(), wq, ws, bias=bias, out=y, workspace=work)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.int8_linear_bf16(x, wq, ws, bias=bias, out=y, workspace=work)
    for _ in range(4):
        x.copy_(torch.randn(m, k, generator=gen).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        assert R.same_bits(y, F.int8_linear_bf16(x, wq, ws, bias=bias))
        work.fill_(0xFF)
        torch.cuda.synchronize()


def test_past_32_bit_offsets():
    """Arrays past 2^32 bytes: codes of 40000 x 112000, rows at their far end."""
    m, n, k = 40000, 24, 112000
    say("int8_linear", m, n, k)
    gen = torch.Generator().manual_seed(2)
    xq = torch.zeros(m, k, dtype=torch.int8, device="cuda")
    rows = torch.tensor([0, 1, 19173, 19174, m - 2, m - 1])
    xq[rows] = codes(gen, len(rows), k)
    xs, wq, ws = scales(gen, m), codes(gen, n, k), scales(gen, n)
    y = F.int8_linear(xq, xs, wq, ws)
    assert R.same_bits(y[rows], R.linear(xq[rows], xs[rows], wq, ws))
    assert int(y.count_nonzero()) <= len(rows) * n
    q, s = F.int8_row_quantize(xq.to(BF))
    eq, es = R.quantize(xq[rows].float())
    assert torch.equal(q[rows], eq) and R.same_bits(s[rows], es)
    del xq, q
    wide = torch.zeros(50000, k, dtype=torch.int8, device="cuda")
    at = torch.tensor([0, 38347, 38348, 49999])
    wide[at] = codes(gen, 4, k)
    ws, xq, xs = scales(gen, 50000), codes(gen, 3, k), scales(gen, 3)
    assert R.same_bits(F.int8_linear(xq, xs, wide, ws)[:, at], R.linear(xq, xs, wide[at], ws[at]))
    xq, xs = codes(gen, 70, k), scales(gen, 70)
    assert R.same_bits(F.int8_linear(xq, xs, wide, ws)[:, at], R.linear(xq, xs, wide[at], ws[at]))


def test_empty():
    xq, xs, wq, ws, bias = operands(3, 8, 32)
    assert F.int8_linear(xq[:0], xs[:0], wq, ws).shape == (0, 8)
    assert F.int8_linear(xq, xs, wq[:0], ws[:0]).shape == (3, 0)
    q, s = F.int8_row_quantize(torch.empty(0, 32, dtype=BF, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0,)
