"""The layer operators on the GPU, through the package's functions, against
their plain 64-bit forms (tests/layers_ref.py has the forms and the bounds)."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import layers_ref as R  # noqa: E402

BF = torch.bfloat16


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(BF).cuda()


def weight(gen, n, k, std=0.05):
    """A quantized weight whose scales differ from block to block."""
    w = torch.randn(n, k, generator=gen) * std
    w *= torch.exp(0.5 * torch.randn(n, 1, generator=gen))
    return F.fp8_block_quantize(w.cuda())


def fenced(t, fill):
    """The same matrix inside a larger buffer, 128 elements of `fill` on
    either side (the address stays 16-byte aligned)."""
    buf = torch.full((t.numel() + 256,), fill, dtype=t.dtype, device=t.device)
    view = buf[128:128 + t.numel()].view(t.shape)
    view.copy_(t)
    return view, buf


def fence_kept(buf, fill):
    ends = torch.cat([buf[:128], buf[-128:]])
    return bool((ends == fill).all())


# Smallest sizes, odd ones, K tails (K % 64 and K % 256), N below, at and past
# tile edges and no multiple of 8, rows on both sides of every kernel's limit.
SHAPES = [
    (1, 1, 16), (1, 8, 16), (1, 129, 400), (1, 2048, 2064), (2, 7, 80), (3, 130, 48), (5, 1000, 272),
    (16, 520, 1040), (17, 64, 4096), (31, 300, 8208), (32, 257, 512), (33, 256, 528), (64, 384, 256),
    (77, 1003, 656), (128, 128, 128), (130, 300, 1040), (200, 1288, 144), (257, 520, 784),
    (300, 36, 2320), (513, 1028, 336), (1025, 264, 80),
    # few rows in grids of up to and past 256 workgroups, whose X takes different ways
    (3, 8200, 400), (4, 72, 1296), (6, 299, 1168), (11, 4112, 336), (15, 33, 4368), (16, 8193, 144),
    (16, 8225, 272), (18, 8225, 144), (29, 4112, 912), (32, 40, 2064),
]
IDS = ["x".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear_act(shape):
    m, n, k = shape
    gen = torch.Generator().manual_seed(m + 3 * n + 7 * k)
    x, (q, s) = normal(gen, m, k), weight(gen, n, k)
    bias, residual = normal(gen, n), normal(gen, m, n)
    for act, b, r, save in (("none", None, residual, False), ("gelu_tanh", bias, None, True),
                            ("silu", None, None, False), ("gelu", bias, residual, True),
                            ("relu", bias, residual, False)):
        say("linear_act", m, n, k, act)
        z = torch.empty(m, n, dtype=BF, device="cuda") if save else None
        y = F.fp8_block_linear_act(x, q, s, bias=b, residual=r, act=R.ACTS[act], z=z)
        torch.cuda.synchronize()
        R.check_linear_act(x, q, s, b, r, act, y, z, f"{shape} {act}")


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear_act_backward(shape):
    m, n, k = shape
    gen = torch.Generator().manual_seed(m + 5 * n + 11 * k)
    q, s = weight(gen, n, k)
    dy, z = normal(gen, m, n), normal(gen, m, n, std=2.0)
    for act, db in (("none", False), ("none", True), ("silu", True), ("gelu", False), ("gelu_tanh", True),
                    ("relu", True)):
        say("linear_act_backward", m, n, k, act, db)
        dbias = torch.empty(n, device="cuda") if db else None
        dx, dz = F.fp8_block_linear_act_backward(dy, q, s, z=None if act == "none" else z,
                                                 act=R.ACTS[act], dbias=dbias)
        torch.cuda.synchronize()
        assert act != "none" or dz is dy
        R.check_linear_act_backward(dy, z, q, s, act, dx, dz, dbias, f"{shape} {act}")


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_glu(shape):
    m, n, k = shape
    gen = torch.Generator().manual_seed(m + 13 * n + 17 * k)
    x, (qg, sg), (qu, su) = normal(gen, m, k), weight(gen, n, k), weight(gen, n, k)
    for act, save in (("silu", True), ("silu", False), ("gelu_tanh", False), ("gelu", True), ("relu", False),
                      ("none", True)):
        say("glu", m, n, k, act, save)
        g = torch.empty(m, n, dtype=BF, device="cuda") if save else None
        u = torch.empty(m, n, dtype=BF, device="cuda") if save else None
        h = F.fp8_block_glu(x, qg, sg, qu, su, act=R.ACTS[act], g=g, u=u)
        torch.cuda.synchronize()
        R.check_glu(x, qg, sg, qu, su, act, h, g, u, f"{shape} {act}")


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_glu_backward(shape):
    m, n, k = shape
    gen = torch.Generator().manual_seed(m + 19 * n + 23 * k)
    (qg, sg), (qu, su) = weight(gen, n, k), weight(gen, n, k)
    dh, g, u = normal(gen, m, n), normal(gen, m, n, std=2.0), normal(gen, m, n)
    for act in ("silu", "gelu_tanh", "gelu", "relu", "none"):
        say("glu_backward", m, n, k, act)
        dx, dg, du = F.fp8_block_glu_backward(dh, g, u, qg, sg, qu, su, act=R.ACTS[act])
        torch.cuda.synchronize()
        R.check_glu_backward(dh, g, u, qg, sg, qu, su, act, dx, dg, du, f"{shape} {act}")


# Sizes whose tiles fill the chip: workgroups that walk several units, 256-row
# tiles with and without K splits, and plans that run whole rounds unsplit and
# the tile columns left over in splits. Compared in full.
LARGE = [
    (2304, 8200, 4112),     # 9 x 33 tiles of 256 rows, a ragged last column tile, 65 K steps
    (700, 5120, 2576),      # row tiles partly filled
    (4100, 1300, 400),      # many row tiles, few steps
    (520, 10001, 1552),     # rows of odd length
]


@pytest.mark.parametrize("shape", LARGE, ids=["x".join(map(str, s)) for s in LARGE])
def test_large(shape):
    m, n, k = shape
    gen = torch.Generator().manual_seed(n + k)
    x, (qg, sg), (qu, su) = normal(gen, m, k), weight(gen, n, k, std=0.02), weight(gen, n, k, std=0.02)
    dy, bias = normal(gen, m, n), normal(gen, n)
    z, g, u = (torch.empty_like(dy) for _ in range(3))
    dbias = torch.empty(n, device="cuda")
    say("large linear", shape)
    y = F.fp8_block_linear_act(x, qg, sg, bias=bias, residual=dy, act=F.ACT_GELU, z=z)
    torch.cuda.synchronize()
    R.check_linear_act(x, qg, sg, bias, dy, "gelu", y, z, f"{shape}")
    say("large glu", shape)
    h = F.fp8_block_glu(x, qg, sg, qu, su, g=g, u=u)
    torch.cuda.synchronize()
    R.check_glu(x, qg, sg, qu, su, "silu", h, g, u, f"{shape}")
    say("large linear backward", shape)
    dx, dz = F.fp8_block_linear_act_backward(dy, qg, sg, z=z, act=F.ACT_GELU_TANH, dbias=dbias)
    torch.cuda.synchronize()
    R.check_linear_act_backward(dy, z, qg, sg, "gelu_tanh", dx, dz, dbias, f"{shape}")
    say("large glu backward", shape)
    dx, dg, du = F.fp8_block_glu_backward(dy, g, u, qg, sg, qu, su)
    torch.cuda.synchronize()
    R.check_glu_backward(dy, g, u, qg, sg, qu, su, "silu", dx, dg, du, f"{shape}")


def test_large_columns_left_over():
    """The input gradient over 8448 columns (8 x 33 tiles, 33 columns of tiles
    being one more than whole rounds hold) and its join beside columns that
    are not split; the same for the forward over as many weight rows."""
    m, n, k = 2048, 4096, 8448
    gen = torch.Generator().manual_seed(4)
    q, s = weight(gen, n, k, std=0.02)
    dy = normal(gen, m, n)
    assert F.layer_workspace_size("linear_act_backward", m, n, k) > 0
    say("columns left over, gradient")
    dx, _ = F.fp8_block_linear_act_backward(dy, q, s)
    torch.cuda.synchronize()
    R.check_linear_act_backward(dy, None, q, s, "none", dx, dy, None, "left over")
    m, n, k = 2048, 8448, 4096
    x, (q, s), res = normal(gen, m, k), weight(gen, n, k, std=0.02), normal(gen, m, n)
    assert F.layer_workspace_size("linear_act", m, n, k) > 0
    say("columns left over, forward")
    y = F.fp8_block_linear_act(x, q, s, residual=res, act=F.ACT_SILU)
    torch.cuda.synchronize()
    R.check_linear_act(x, q, s, None, res, "silu", y, None, "left over")


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activation_values(act):
    """Each activation and derivative over the whole range of bf16: z walks
    through every finite bf16 value (dy = 1), and through a one-hot product
    the forward does the same for the values E4M3 times a scale reaches."""
    bits = torch.arange(1 << 16, dtype=torch.int32)
    z = bits.to(torch.int16).view(BF)
    z = z[torch.isfinite(z.float())].view(-1, 128).contiguous().cuda()     # 510 x 128
    q = torch.zeros(128, 16, dtype=torch.uint8, device="cuda")
    s = torch.ones(1, 1, device="cuda")
    say("activation derivative", act)
    _, dz = F.fp8_block_linear_act_backward(torch.ones_like(z), q, s, z=z, act=R.ACTS[act])
    torch.cuda.synchronize()
    t = z.double()
    want = R.grad64(t.clamp(-1e4, 1e4), act)         # flat beyond; t^3 overflows there in the plain form
    off = (dz.double() - want).abs()
    assert bool((off <= R.HALF * want.abs() + R.EVAL * (1 + t.abs().clamp_max(100)) + R.TINY).all()), float(off.max())
    # forward: bias holds every value, the product is zero
    zb = z.view(-1)
    x = torch.zeros(1, 16, dtype=BF, device="cuda")
    q = torch.zeros(zb.numel(), 16, dtype=torch.uint8, device="cuda")
    s = torch.ones((zb.numel() + 127) // 128, 1, device="cuda")
    say("activation", act)
    y = F.fp8_block_linear_act(x, q, s, bias=zb.contiguous(), act=R.ACTS[act])
    torch.cuda.synchronize()
    t = zb.double()
    big = t.abs() > 1e4
    want = torch.where(big, t.clamp_min(0), R.act64(t.clamp(-1e4, 1e4), act))
    off = (y[0].double() - want).abs()
    assert bool((off <= R.HALF * want.abs() + R.EVAL * t.abs().clamp_max(100) + R.TINY).all()), float(off.max())


ROUTES = [(1, 264, 512), (7, 299, 1168), (3, 8200, 144), (20, 136, 1040), (77, 1003, 656), (300, 264, 528)]


@pytest.mark.parametrize("shape", ROUTES, ids=["x".join(map(str, s)) for s in ROUTES])
def test_neighbouring_memory(shape):
    """Inputs lie between NaNs and outputs between sentinels: nothing outside
    the arrays is read into a result or written."""
    m, n, k = shape
    gen = torch.Generator().manual_seed(n)
    nan, mark = float("nan"), 7.0
    x, _ = fenced(normal(gen, m, k), nan)
    qg, sg = weight(gen, n, k)
    qu, su = weight(gen, n, k)
    qg, _ = fenced(qg, 0x7F)      # the E4M3 NaN
    qu, _ = fenced(qu, 0x7F)
    bias, _ = fenced(normal(gen, n), nan)
    res, _ = fenced(normal(gen, m, n), nan)
    z0, zbuf = fenced(torch.zeros(m, n, dtype=BF, device="cuda"), mark)
    y0, ybuf = fenced(torch.zeros(m, n, dtype=BF, device="cuda"), mark)
    say("fences", shape)
    F.fp8_block_linear_act(x, qg, sg, bias=bias, residual=res, act=F.ACT_SILU, z=z0, out=y0)
    torch.cuda.synchronize()
    R.check_linear_act(x, qg, sg, bias, res, "silu", y0, z0, "fenced")
    assert fence_kept(zbuf, mark) and fence_kept(ybuf, mark)
    g, gbuf = fenced(z0 * 0, mark)
    u, ubuf = fenced(z0 * 0, mark)
    F.fp8_block_glu(x, qg, sg, qu, su, g=g, u=u, out=y0)
    torch.cuda.synchronize()
    R.check_glu(x, qg, sg, qu, su, "silu", y0, g, u, "fenced")
    assert fence_kept(gbuf, mark) and fence_kept(ubuf, mark) and fence_kept(ybuf, mark)
    gbuf[:128] = ubuf[:128] = gbuf[-128:] = ubuf[-128:] = nan
    dh, _ = fenced(normal(gen, m, n), nan)
    dg, dgb = fenced(z0 * 0, mark)
    du, dub = fenced(z0 * 0, mark)
    dx, dxb = fenced(torch.zeros(m, k, dtype=BF, device="cuda"), mark)
    F.fp8_block_glu_backward(dh, g, u, qg, sg, qu, su, dg=dg, du=du, dx=dx)
    torch.cuda.synchronize()
    R.check_glu_backward(dh, g, u, qg, sg, qu, su, "silu", dx, dg, du, "fenced")
    assert fence_kept(dgb, mark) and fence_kept(dub, mark) and fence_kept(dxb, mark)
    dbias, dbb = fenced(torch.zeros(n, device="cuda"), mark)
    F.fp8_block_linear_act_backward(dh, qg, sg, z=g, act=F.ACT_GELU, dz=dg, dx=dx, dbias=dbias)
    torch.cuda.synchronize()
    R.check_linear_act_backward(dh, g, qg, sg, "gelu", dx, dg, dbias, "fenced")
    assert fence_kept(dgb, mark) and fence_kept(dxb, mark) and fence_kept(dbb, mark)


@pytest.mark.parametrize("shape", ROUTES, ids=["x".join(map(str, s)) for s in ROUTES])
def test_same_bits_and_residual_in_place(shape):
    m, n, k = shape
    gen = torch.Generator().manual_seed(k)
    x, (q, s) = normal(gen, m, k), weight(gen, n, k)
    qu, su = weight(gen, n, k)
    res, dy = normal(gen, m, n), normal(gen, m, n)
    say("repeat", shape)
    ws = torch.empty(max(1, F.layer_workspace_size("linear_act", m, n, k)), dtype=torch.uint8, device="cuda")
    y = F.fp8_block_linear_act(x, q, s, residual=res, act=F.ACT_GELU)
    inplace = res.clone()
    F.fp8_block_linear_act(x, q, s, residual=inplace, act=F.ACT_GELU, out=inplace,
                           workspace=ws if ws.numel() > 1 else None)
    g1, u1 = torch.empty_like(dy), torch.empty_like(dy)
    h1, h2 = (F.fp8_block_glu(x, q, s, qu, su, g=g1, u=u1) for _ in range(2))
    b1 = F.fp8_block_glu_backward(dy, g1, u1, q, s, qu, su)
    b2 = F.fp8_block_glu_backward(dy, g1, u1, q, s, qu, su)
    d1, d2 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    c1 = F.fp8_block_linear_act_backward(dy, q, s, z=g1, act=F.ACT_SILU, dbias=d1)
    c2 = F.fp8_block_linear_act_backward(dy, q, s, z=g1, act=F.ACT_SILU, dbias=d2)
    torch.cuda.synchronize()
    assert torch.equal(y, inplace)
    assert torch.equal(h1, h2) and torch.equal(d1, d2)
    assert all(torch.equal(a, b) for a, b in zip(b1 + c1, b2 + c2))


@pytest.mark.parametrize("m,n", [(0, 40), (5, 0), (0, 0)])
def test_empty(m, n):
    """Empty sums are zeros and are written; empty outputs are left alone."""
    k = 32
    q = torch.zeros(n, k, dtype=torch.uint8, device="cuda")
    s = torch.zeros(F.scale_grid_shape(n, k), device="cuda")
    x, dy = torch.ones(m, k, dtype=BF, device="cuda"), torch.ones(m, n, dtype=BF, device="cuda")
    say("empty", m, n)
    assert F.fp8_block_linear_act(x, q, s, bias=torch.ones(n, dtype=BF, device="cuda")).shape == (m, n)
    assert F.fp8_block_glu(x, q, s, q, s).shape == (m, n)
    dbias = torch.full((n,), 3.0, device="cuda")
    dx, dz = F.fp8_block_linear_act_backward(dy, q, s, z=dy, act=F.ACT_RELU, dbias=dbias,
                                             dx=torch.full((m, k), 3.0, dtype=BF, device="cuda"))
    dx2, dg, du = F.fp8_block_glu_backward(dy, dy, dy, q, s, q, s,
                                           dx=torch.full((m, k), 3.0, dtype=BF, device="cuda"))
    torch.cuda.synchronize()
    assert not dbias.any() and not dx.any() and not dx2.any()
    assert dx.shape == dx2.shape == (m, k) and dz.shape == dg.shape == du.shape == (m, n)


@pytest.mark.parametrize("shape", ROUTES, ids=["x".join(map(str, s)) for s in ROUTES])
def test_not_finite_rows_stay_rows(shape):
    """A NaN or an infinity in one row of the activations or gradients reaches
    that row's results alone (and the column sums), and none of the others."""
    m, n, k = shape
    gen = torch.Generator().manual_seed(m + k)
    x, (q, s), (qu, su) = normal(gen, m, k), weight(gen, n, k), weight(gen, n, k)
    dy, z, u = normal(gen, m, n), normal(gen, m, n), normal(gen, m, n)
    bad = m // 2
    keep = torch.arange(m, device="cuda") != bad
    say("not finite", shape)
    for value in (float("nan"), float("inf")):
        xb, dyb = x.clone(), dy.clone()
        xb[bad, k - 1] = value
        dyb[bad, n - 1] = value
        y0, y1 = (F.fp8_block_linear_act(t, q, s, residual=z, act=F.ACT_GELU_TANH) for t in (x, xb))
        h0, h1 = (F.fp8_block_glu(t, q, s, qu, su) for t in (x, xb))
        a0, a1 = (F.fp8_block_glu_backward(t, z, u, q, s, qu, su)[0] for t in (dy, dyb))
        b0, b1 = (F.fp8_block_linear_act_backward(t, q, s, z=z, act=F.ACT_SILU)[0] for t in (dy, dyb))
        torch.cuda.synchronize()
        for clean, dirty in ((y0, y1), (h0, h1), (a0, a1), (b0, b1)):
            assert torch.equal(clean[keep], dirty[keep])
            assert not bool(torch.isfinite(dirty[bad].float()).all())


@pytest.mark.parametrize("shape", ROUTES, ids=["x".join(map(str, s)) for s in ROUTES])
def test_other_stream_and_captured_graph(shape):
    """The calls follow torch's current stream, and a captured graph of all
    four replays on new inputs, with eager work between the replays."""
    m, n, k = shape
    gen = torch.Generator().manual_seed(9)
    (qg, sg), (qu, su) = weight(gen, n, k), weight(gen, n, k)
    x, dy = normal(gen, m, k), normal(gen, m, n)
    bias = normal(gen, n)
    out = {name: torch.empty(m, n, dtype=BF, device="cuda") for name in ("y", "z", "h", "g", "u", "dg", "du", "dz")}
    out["dx"], out["dx2"] = torch.empty_like(x), torch.empty_like(x)
    out["dbias"] = torch.empty(n, device="cuda")

    def step(o):
        F.fp8_block_linear_act(x, qg, sg, bias=bias, act=F.ACT_GELU, z=o["z"], out=o["y"])
        F.fp8_block_glu(x, qg, sg, qu, su, g=o["g"], u=o["u"], out=o["h"])
        F.fp8_block_glu_backward(dy, o["g"], o["u"], qg, sg, qu, su, dx=o["dx"], dg=o["dg"], du=o["du"])
        F.fp8_block_linear_act_backward(dy, qg, sg, z=o["z"], act=F.ACT_GELU, dz=o["dz"], dx=o["dx2"],
                                        dbias=o["dbias"])

    say("graph", shape)
    eager = {name: torch.empty_like(t) for name, t in out.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out)
    torch.cuda.current_stream().wait_stream(side)
    step(eager)
    torch.cuda.synchronize()
    assert all(torch.equal(out[i], eager[i]) for i in out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for turn in range(4):
        x.copy_(normal(gen, m, k))
        dy.copy_(normal(gen, m, n))
        for t in out.values():
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(out[i], eager[i]) for i in out), turn


@pytest.mark.parametrize("m", [1, 24, 200])
def test_feed_forward_block_and_its_gradient(m):
    """The operators as a block runs them: a gated pair and the down
    projection added to the residual stream, then the whole backward pass,
    against the formulas in 64 bits on the kernels' own intermediates and
    against differences of the 64-bit block."""
    hidden, inner = 384, 784
    gen = torch.Generator().manual_seed(m)
    (qg, sg), (qu, su), (qd, sd) = weight(gen, inner, hidden), weight(gen, inner, hidden), weight(gen, hidden, inner)
    x, dy = normal(gen, m, hidden), normal(gen, m, hidden)
    g, u = (torch.empty(m, inner, dtype=BF, device="cuda") for _ in range(2))
    say("block", m)
    h = F.fp8_block_glu(x, qg, sg, qu, su, g=g, u=u)
    y = F.fp8_block_linear_act(h, qd, sd, residual=x)
    dh, _ = F.fp8_block_linear_act_backward(dy, qd, sd)
    dx, dg, du = F.fp8_block_glu_backward(dh, g, u, qg, sg, qu, su)
    dx = dx + dy
    torch.cuda.synchronize()
    R.check_glu(x, qg, sg, qu, su, "silu", h, g, u, "block")
    R.check_linear_act(h, qd, sd, None, x, "none", y, None, "block")
    R.check_linear_act_backward(dy, None, qd, sd, "none", dh, dy, None, "block")

    wg, wu, wd = R.weight64(qg, sg), R.weight64(qu, su), R.weight64(qd, sd)

    def loss(t):
        return ((R.act64(t @ wg.t(), "silu") * (t @ wu.t())) @ wd.t() + t).mul(dy.double()).sum()

    # Differences of the 64-bit block along four directions. The gradient the
    # kernels give carries the roundings of g, u, h, dh, dg, du and dx (seven
    # half steps of 2^-8 a term, counted over absolute values).
    xd = x.double()
    gr, ur = xd @ wg.t(), xd @ wu.t()
    dhr = dy.double() @ wd
    size = (dhr * ur).abs() * 1.13 @ wg.abs() + (dhr * R.act64(gr, "silu")).abs() @ wu.abs() + dy.double().abs()
    size += (dy.double().abs() @ wd.abs() * (ur.abs() + 1)) @ wg.abs() + (dy.double().abs() @ wd.abs() * (gr.abs() + 1)) @ wu.abs()
    for i in range(4):
        v = torch.randn(m, hidden, generator=gen, dtype=torch.float64).cuda()
        step = 1e-4
        want = float((loss(xd + step * v) - loss(xd - step * v)) / (2 * step))
        got = float((dx.double() * v).sum())
        room = 7 * R.HALF * float((size * v.abs()).sum())
        # errors of single terms are independent: their sum stays far inside
        # the count over absolute values
        assert abs(got - want) <= room, (i, got, want, room)
        norm = math.sqrt(float((size * v).pow(2).sum()))
        assert abs(got - want) <= 7 * R.HALF * 6 * norm, (i, got, want, norm)


def test_two_streams_at_once():
    """Calls on two streams, each with its own (implicit) workspace, overlap
    without touching each other: several rounds against results alone."""
    gen = torch.Generator().manual_seed(12)
    (qg, sg), (qu, su) = weight(gen, 1032, 2064), weight(gen, 1032, 2064)
    xs = [normal(gen, m, 2064) for m in (70, 200)]
    dys = [normal(gen, m, 1032) for m in (70, 200)]

    def step(i):
        g, u = torch.empty_like(dys[i]), torch.empty_like(dys[i])
        h = F.fp8_block_glu(xs[i], qg, sg, qu, su, g=g, u=u)
        y = F.fp8_block_linear_act(xs[i], qg, sg, residual=h, act=F.ACT_GELU)
        return (h, y) + F.fp8_block_glu_backward(dys[i], g, u, qg, sg, qu, su)

    say("two streams")
    alone = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(step(i))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(p, r) for p, r in zip(a, b))


@pytest.mark.parametrize("n", [32776, 32771])
def test_offsets_past_32_bits(n):
    """Arrays of more than 2^32 bytes (and 2^31 elements), rows of whole
    chunks and of odd length: rows at both ends and around 2^31 bytes and
    elements against the formulas, and the column sums in full."""
    m, k = 67000, 64
    gen = torch.Generator().manual_seed(n)
    (qg, sg), (qu, su) = weight(gen, n, k), weight(gen, n, k)
    x = normal(gen, m, k)
    rows = sorted({0, 1, 255, 256, (1 << 30) // n, (1 << 30) // n + 1, (1 << 31) // n, (1 << 31) // n + 1, m - 2, m - 1})
    at = torch.tensor(rows, device="cuda")
    z, g, u = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(3))
    say("past 32 bits", n, "forward")
    y = F.fp8_block_linear_act(x, qg, sg, act=F.ACT_SILU, z=z)
    h = F.fp8_block_glu(x, qg, sg, qu, su, g=g, u=u)
    torch.cuda.synchronize()
    R.check_linear_act(x[at], qg, sg, None, None, "silu", y[at], z[at], "past 32 bits")
    R.check_glu(x[at], qg, sg, qu, su, "silu", h[at], g[at], u[at], "past 32 bits")
    del y
    say("past 32 bits", n, "backward")
    dbias = torch.empty(n, device="cuda")
    dx, dz = F.fp8_block_linear_act_backward(h, qg, sg, z=z, act=F.ACT_SILU, dbias=dbias)
    torch.cuda.synchronize()
    R.check_linear_act_backward(h[at], z[at], qg, sg, "silu", dx[at], dz[at], None, "past 32 bits")
    # dz as returned, summed in 64 bits; each of its roundings is a half step
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(total)
    for part in dz.split(4096):
        total += part.double().sum(0)
        size += part.double().abs().sum(0)
    assert bool(((dbias.double() - total).abs() <= (R.HALF + (m + 8) * 2.0 ** -23) * size + R.TINY).all())
    del dz, z
    dx, dg, du = F.fp8_block_glu_backward(h, g, u, qg, sg, qu, su)
    torch.cuda.synchronize()
    R.check_glu_backward(h[at], g[at], u[at], qg, sg, qu, su, "silu", dx[at], dg[at], du[at], "past 32 bits")


def test_long_rows():
    """x and dx of more than 2^32 bytes (long rows of the reduction)."""
    m, n, k = 70000, 24, 32768
    gen = torch.Generator().manual_seed(3)
    q, s = weight(gen, n, k)
    x = normal(gen, 1000, k).repeat(70, 1)
    at = torch.tensor([0, 999, 32767, 32768, 65535, 65536, m - 1], device="cuda")
    say("long rows")
    y = F.fp8_block_linear_act(x, q, s, act=F.ACT_RELU)
    dx, _ = F.fp8_block_linear_act_backward(y, q, s)
    torch.cuda.synchronize()
    R.check_linear_act(x[at], q, s, None, None, "relu", y[at], None, "long rows")
    R.check_linear_act_backward(y[at], None, q, s, "none", dx[at], y[at], None, "long rows")


def test_everything_given_allocates_nothing_and_dx_is_optional():
    """With outputs and workspaces given a call allocates nothing; the C entry
    points take a null dx (an adapter's first layer needs none)."""
    m, n, k = 100, 1003, 656
    gen = torch.Generator().manual_seed(8)
    (qg, sg), (qu, su) = weight(gen, n, k), weight(gen, n, k)
    x, dy, z = normal(gen, m, k), normal(gen, m, n), normal(gen, m, n)
    ws = torch.empty(max(F.layer_workspace_size(op, m, n, k) for op in
                         ("linear_act", "linear_act_backward", "glu", "glu_backward")), dtype=torch.uint8, device="cuda")
    y, dz, du, dx, db = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(x), torch.empty(n, device="cuda")
    say("no allocation")
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    F.fp8_block_linear_act(x, qg, sg, act=F.ACT_SILU, out=y, workspace=ws)
    F.fp8_block_glu(x, qg, sg, qu, su, out=y, workspace=ws)
    F.fp8_block_linear_act_backward(dy, qg, sg, z=z, act=F.ACT_SILU, dz=dz, dx=dx, dbias=db, workspace=ws)
    F.fp8_block_glu_backward(dy, z, y, qg, sg, qu, su, dg=dz, du=du, dx=dx, workspace=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    torch.cuda.synchronize()
    R.check_glu_backward(dy, z, y, qg, sg, qu, su, "silu", dx, dz, du, "given")
    want, wantb = dz.clone(), db.clone()
    F.fp8_block_linear_act_backward(dy, qg, sg, z=z, act=F.ACT_SILU, dz=want, dx=dx, dbias=wantb, workspace=ws)
    L, st = F._lib, torch.cuda.current_stream().cuda_stream
    dz.zero_()
    db.zero_()
    assert L.linear_act_backward_raw(dy.data_ptr(), z.data_ptr(), 0, 0, dz.data_ptr(), db.data_ptr(), 0, m, n, k,
                                     F.ACT_SILU, ws.data_ptr(), ws.numel(), st) == 0
    du2, dg2 = torch.empty_like(du), torch.empty_like(du)
    assert L.glu_backward_raw(dy.data_ptr(), z.data_ptr(), y.data_ptr(), 0, 0, 0, 0, dg2.data_ptr(), du2.data_ptr(), 0,
                              m, n, k, F.ACT_SILU, ws.data_ptr(), ws.numel(), st) == 0
    torch.cuda.synchronize()
    assert torch.equal(dz, want) and torch.equal(db, wantb) and torch.equal(du2, du)


def test_refusals_on_the_device():
    x = torch.zeros(4, 32, dtype=BF, device="cuda")
    q = torch.zeros(24, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, 1, device="cuda")
    y = torch.zeros(4, 24, dtype=BF, device="cuda")
    with pytest.raises(F.Fp8blError):
        F.fp8_block_linear_act(x, q, s, act=9)
    with pytest.raises(F.Fp8blError):                       # z over y
        F.fp8_block_linear_act(x, q, s, z=y, out=y)
    with pytest.raises(F.Fp8blError):                       # residual overlaps y without being y
        both = torch.zeros(5, 24, dtype=BF, device="cuda")
        F.fp8_block_linear_act(x, q, s, residual=both[:4], out=both[1:])
    with pytest.raises(ValueError):
        F.fp8_block_linear_act(x, q, s, residual=y.t().contiguous().t())
    with pytest.raises(TypeError):
        F.fp8_block_linear_act(x, q, s, residual=y.cpu())
    with pytest.raises(ValueError):
        F.fp8_block_linear_act(x, q, s, bias=torch.zeros(23, dtype=BF, device="cuda"))
    with pytest.raises(TypeError):
        F.fp8_block_linear_act(x.half(), q, s)
    with pytest.raises(ValueError):
        F.fp8_block_glu(x, q, s, q, s, g=y)
    with pytest.raises(ValueError):
        F.fp8_block_linear_act_backward(y, q, s, act=F.ACT_SILU)
    with pytest.raises(ValueError):
        F.fp8_block_linear_act_backward(y, q, s, z=y)
    with pytest.raises(F.Fp8blError):
        F.fp8_block_glu_backward(y, y.clone(), y.clone(), q, s, q, s, dg=y)
    torch.cuda.synchronize()
