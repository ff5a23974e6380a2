"""Norm and rotation of query and key heads, their gradients, and the E4M3 cache
on the GPU, against the definitions in 64 bits (tests/qkv_ref.py, with the
bounds' derivation)."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from gpu_util import say  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

import block_scaled_fp8_linear_amd as F  # noqa: E402
import qkv_ref as R  # noqa: E402

BF = torch.bfloat16


def heads(gen, t, h, d, std=1.0):
    x = torch.randn(t, h, d, generator=gen) * std
    x[..., 3::17] *= 5
    return x.to(BF).cuda()


class Case:
    """Inputs of one size; `axes` of them, dealt to the pairs in turn."""

    def __init__(self, t, hq, hk, d, pairs=None, axes=1, interleaved=False, base=1e4, far=1000, seed=0):
        gen = torch.Generator().manual_seed(t + 3 * hq + 5 * hk + 7 * d + seed)
        self.t, self.hq, self.hk, self.d = t, hq, hk, d
        pairs = d // 2 if pairs is None else pairs
        self.q, self.k, self.v = heads(gen, t, hq, d), heads(gen, t, hk, d), heads(gen, t, hk, d, 2.0)
        self.dq, self.dk = heads(gen, t, hq, d, 0.1), heads(gen, t, hk, d, 0.1)
        self.qw, self.kw = ((1 + 0.3 * torch.randn(d, generator=gen)).to(BF).cuda() for _ in range(2))
        self.positions = torch.randint(-far // 8, far, (axes, t), generator=gen, dtype=torch.int32).cuda()
        self.freq = (base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()
        self.axes = None if axes == 1 else tuple(i % axes for i in range(pairs))
        self.how = {"axes": self.axes, "interleaved": interleaved}

    @property
    def table(self):
        return self.qw, self.kw, self.positions, self.freq

    def ref(self, x, w, eps=1e-6):
        return R.forward(x, w, self.positions, self.freq, self.axes, eps, self.how["interleaved"])

    def stored_turned(self, eps=1e-6):
        return R.stored_turned(self.k, self.kw, self.positions, self.freq, self.axes, eps, self.how["interleaved"])

    def ref_back(self, dy, x, w, eps=1e-6):
        # one wave's steps of 64 / L heads; its units, where there are more than
        # 1024 workgroups of 4 waves
        lanes = next(l for l in (2, 4, 8, 16, 32) if 8 * l >= self.d)
        steps = -(-x.shape[1] * lanes // 64) * -(-self.t // 4096)
        return R.backward(dy, x, w, self.positions, self.freq, self.axes, eps, self.how["interleaved"], steps)


def check_forward(c, q, k, name, eps=1e-6):
    for got, x, w in ((q, c.q, c.qw), (k, c.k, c.kw)):
        worst = R.outside(got, *c.ref(x, w, eps))
        assert worst <= 1, (name, worst)


def check_backward(c, got, name, eps=1e-6):
    dq, dk, dqw, dkw = got
    for dx, dw, dy, x, w in ((dq, dqw, c.dq, c.q, c.qw), (dk, dkw, c.dk, c.k, c.kw)):
        ref, bound, wref, wbound = c.ref_back(dy, x, w, eps)
        worst = R.outside(dx, ref, bound)
        assert worst <= 1, (name, worst)
        off = (dw.double() - wref).abs()
        assert bool((off <= wbound + R.U * wref.abs()).all()), (name, float((off / (wbound + 1e-30)).max()))


# t, hq, hk, d, pairs, axes, interleaved: one token, odd counts, more heads than a
# wave holds, every lane count of a head, heads that fill their lanes in part,
# rotations of a part of the head.
CASES = [
    (1, 1, 1, 16, None, 1, False), (1, 64, 8, 128, None, 3, False), (2, 3, 1, 16, 4, 2, True), (3, 5, 5, 24, 4, 1, True),
    (3, 7, 2, 32, 8, 3, False), (5, 2, 2, 32, 16, 8, True), (7, 9, 3, 48, None, 3, False), (4, 33, 1, 64, None, 1, False),
    (9, 16, 2, 80, 16, 1, False), (6, 14, 2, 80, None, 3, True), (5, 6, 6, 96, None, 3, False), (33, 12, 4, 128, None, 3, True),
    (17, 40, 8, 128, 16, 1, False), (3, 5, 3, 136, 64, 2, False), (11, 7, 1, 192, None, 3, False), (2, 3, 3, 248, 120, 2, False),
    (13, 4, 2, 256, None, 3, False), (5, 8, 8, 256, None, 4, True), (130, 3, 1, 64, None, 3, False), (515, 8, 2, 128, None, 3, False),
    (2, 4096, 2, 16, 8, 1, False), (5000, 2, 1, 16, 8, 1, False),
]
IDS = ["-".join(str(int(v)) if v is not None else "all" for v in c) for c in CASES]


@pytest.mark.parametrize("size", CASES, ids=IDS)
def test_norm_rope(size):
    say("qk_norm_rope", size)
    c = Case(*size)
    check_forward(c, *F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how), size)


@pytest.mark.parametrize("size", CASES, ids=IDS)
def test_backward(size):
    say("qk_norm_rope_backward", size)
    c = Case(*size)
    got = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)
    check_backward(c, got, size)
    again = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    dq, dk, none, none2 = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how, need_weights=False)
    assert none is None and none2 is None and torch.equal(dq, got[0]) and torch.equal(dk, got[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_by_differences(interleaved):
    """The gradients along random directions against central differences of the
    64-bit forward. A step of 2^-17 leaves the difference good to about 2^-34."""
    c = Case(20, 6, 2, 64, 16, 3, interleaved)
    dq, dk, dqw, dkw = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)
    gen = torch.Generator().manual_seed(3)
    for dx, dw, dy, x, w in ((dq, dqw, c.dq, c.q, c.qw), (dk, dkw, c.dk, c.k, c.kw)):
        ref, bound, wref, wbound = c.ref_back(dy, x, w)
        for _ in range(5):
            ex = torch.randn(x.shape, generator=gen, dtype=torch.float64).cuda()
            ew = torch.randn(w.shape, generator=gen, dtype=torch.float64).cuda()
            h = 2.0 ** -17
            up, _ = c.ref(x.double() + h * ex, w.double() + h * ew)
            down, _ = c.ref(x.double() - h * ex, w.double() - h * ew)
            diff = float(((up - down) * dy.double()).sum()) / (2 * h)
            got = float((dx.double() * ex).sum() + (dw.double() * ew).sum())
            most = float(((R.HALF_BF16 * ref.abs() + bound) * ex.abs()).sum() + (wbound * ew.abs()).sum())
            size = float((ref * ex).abs().sum() + (wref * ew).abs().sum())
            assert abs(got - diff) <= most + 2.0 ** -26 * size
            assert most < 2.0 ** -6 * size


@pytest.mark.parametrize("far", [200000, 2 ** 31 - 1])
def test_far_positions(far):
    """Positions whose angles fp32 holds to no better than 2^-8 of a turn, and
    the largest ones there are."""
    c = Case(40, 2, 2, 128, None, 3, False, far=far)
    c.positions[0, 0], c.positions[1, 1], c.positions[2, 2] = 2 ** 31 - 1, -2 ** 31, 0
    check_forward(c, *F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how), far)
    check_backward(c, F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how), far)


def test_zero_heads_and_large_ones():
    c = Case(6, 3, 2, 64)
    c.q[0, 1], c.q[1], c.k[2, 0] = 0, 0, 0
    c.q[3] *= 2.0 ** 40
    c.k[4] *= 2.0 ** -40
    for eps in (1e-6, 1e-2):
        check_forward(c, *F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how, eps=eps), eps, eps)
        check_backward(c, F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how, eps=eps), eps, eps)
    q, _ = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)
    assert not q[0, 1].any() and not q[1].any()


def test_values_that_are_not_finite_stay_in_their_head():
    c = Case(9, 6, 2, 80, 16)
    q, k = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)
    back = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)
    c.q[2, 3, 7], c.k[5, 1, 79] = float("nan"), float("inf")
    q2, k2 = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)
    back2 = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)
    for a, b, at in ((q, q2, (2, 3)), (k, k2, (5, 1)), (back[0], back2[0], (2, 3)), (back[1], back2[1], (5, 1))):
        same = (a == b).all(-1)
        same[at] = True
        assert bool(same.all())


def packed(c, *arrays):
    """The arrays beside each other in one row a token, as a projection writes
    them, with 8 elements of 7.0 behind each."""
    parts = []
    for a in arrays:
        parts += [a.reshape(c.t, -1), torch.full((c.t, 8), 7.0, dtype=BF, device="cuda")]
    buf = torch.cat(parts, 1).contiguous()
    views, at = [], 0
    for a in arrays:
        n = a.shape[1] * a.shape[2]
        views.append(buf[:, at:at + n].view(c.t, a.shape[1], c.d))
        at += n + 8
    return buf, views


def fences_kept(buf, arrays):
    at = 0
    for a in arrays:
        at += a.shape[1] * a.shape[2]
        if not bool((buf[:, at:at + 8] == 7).all()):
            return False
        at += 8
    return True


@pytest.mark.parametrize("size", [(5, 6, 2, 80, None, 3, True), (130, 8, 2, 128, None, 3, False)])
def test_views_and_in_place(size):
    """Views of one packed projection, outputs in place and into another packed
    array, heads-first arrays: the same bits as from arrays of their own."""
    c = Case(*size)
    q0, k0 = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)
    back0 = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)

    buf, (q, k, v) = packed(c, c.q, c.k, c.v)
    out, (qo, ko, vo) = packed(c, c.q, c.k, c.v)
    F.fp8_qk_norm_rope(q, k, *c.table, **c.how, q_out=qo, k_out=ko)
    assert torch.equal(qo, q0) and torch.equal(ko, k0) and torch.equal(vo, c.v) and fences_kept(out, (c.q, c.k, c.v))
    grad, (gq, gk, gv) = packed(c, c.q, c.k, c.v)
    back = F.fp8_qk_norm_rope_backward(c.dq, c.dk, q, k, *c.table, **c.how, q_grad=gq, k_grad=gk)
    assert torch.equal(gq, back0[0]) and torch.equal(gk, back0[1]) and torch.equal(gv, c.v)
    assert fences_kept(grad, (c.q, c.k, c.v)) and torch.equal(back[2], back0[2]) and torch.equal(back[3], back0[3])

    F.fp8_qk_norm_rope(q, k, *c.table, **c.how, q_out=q, k_out=k)
    assert torch.equal(q, q0) and torch.equal(k, k0) and torch.equal(v, c.v) and fences_kept(buf, (c.q, c.k, c.v))
    dq, dk = c.dq.clone(), c.dk.clone()
    F.fp8_qk_norm_rope_backward(dq, dk, c.q, c.k, *c.table, **c.how, q_grad=dq, k_grad=dk)
    assert torch.equal(dq, back0[0]) and torch.equal(dk, back0[1])

    first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (c.q, c.k)]
    outs = [torch.empty_like(x) for x in first]
    assert outs[0].stride(0) == c.d
    F.fp8_qk_norm_rope(*first, *c.table, **c.how, q_out=outs[0], k_out=outs[1])
    assert torch.equal(outs[0], q0) and torch.equal(outs[1], k0)
    # every other head of a larger array, and one key head read as many
    wide = torch.zeros(c.t, 2 * c.hq, c.d, dtype=BF, device="cuda")
    wide[:, ::2] = c.q
    one = c.k[:, :1].expand(c.t, 3, c.d)
    q1, k1 = F.fp8_qk_norm_rope(wide[:, ::2], one, *c.table, **c.how)
    assert torch.equal(q1, q0) and all(torch.equal(k1[:, i], k0[:, 0]) for i in range(3))


# ---- the cache ----------------------------------------------------------

def cache(rows, h, d, seed=0):
    """A cache in use: every row holds something."""
    gen = torch.Generator().manual_seed(seed)
    codes = [(torch.randint(0, 127, (rows, h, d), generator=gen) + 128 * torch.randint(0, 2, (rows, h, d), generator=gen))
             .to(torch.uint8).cuda() for _ in range(2)]
    scales = [(torch.rand(rows, h, generator=gen) + 0.5).cuda() for _ in range(2)]
    return codes[0], codes[1], scales[0], scales[1]


def slots_of(t, rows, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randperm(rows, generator=gen)[:t].to(torch.int32).cuda()


def check_store(before, after, slots, k, v):
    """k, v: (E4M3 values, scales) of every token."""
    live = R.last_ones(slots.cpu(), before[0].shape[0]).cuda()
    rows = slots[live].long()
    for i, (values, scale) in enumerate((k, v)):
        codes, scales = before[i].clone(), before[2 + i].clone()
        got = R.values(after[i][rows])
        assert torch.equal(got, values[live]) and torch.equal(torch.signbit(got), torch.signbit(values[live]))
        assert torch.equal(after[2 + i][rows], scale[live])
        codes[rows], scales[rows] = after[i][rows], after[2 + i][rows]
        assert torch.equal(codes, after[i]) and torch.equal(scales, after[2 + i]), "another row was written"


STORE = [(1, 1, 16), (1, 8, 128), (2, 3, 24), (5, 2, 32), (7, 9, 64), (16, 8, 128), (33, 2, 80), (65, 5, 96), (100, 1, 256),
         (64, 3, 248), (300, 4, 128), (2049, 2, 64), (2500, 3, 128), (8193, 1, 32), (9000, 2, 16)]


@pytest.mark.parametrize("t,h,d", STORE)
def test_store_and_load(t, h, d):
    say("kv_store", t, h, d)
    c = Case(t, 1, h, d, 4, interleaved=True)
    rows = t + 37
    before = cache(rows, h, d)
    slots = slots_of(t, rows)
    after = [x.clone() for x in before]
    F.fp8_kv_store(c.k, c.v, slots, *after)
    check_store(before, after, slots, R.stored(c.k), R.stored(c.v))
    k, v = F.fp8_kv_load(*after, slots)
    assert torch.equal(k, R.loaded(after[0], after[2], slots)) and torch.equal(v, R.loaded(after[1], after[3], slots))
    # back within half a step of E4M3, its smallest step 2^-9 of the scale
    for got, x in ((k, c.k), (v, c.v)):
        x, s = x.double(), R.scales(x).double()[..., None]
        most = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s) * (1 + 2.0 ** -7) + 2.0 ** -8 * x.abs()
        assert bool(((got.double() - x).abs() <= most).all())


@pytest.mark.parametrize("t,h,d", [(6, 2, 64), (40, 3, 32), (200, 1, 16), (2100, 2, 16), (9001, 1, 16)])
def test_padding_and_equal_slots(t, h, d):
    """Slots outside the cache, and many tokens with one slot: the last is
    stored, its codes and its scale together."""
    say("kv_store", t, h, d, "equal slots")
    c = Case(t, 1, h, d, 4, interleaved=True)
    rows = max(3, t // 5)
    gen = torch.Generator().manual_seed(t)
    slots = torch.randint(-2, rows + 3, (t,), generator=gen, dtype=torch.int32)
    slots[0], slots[-1], slots[1] = 2 ** 31 - 1, 1, -2 ** 31
    slots = slots.cuda()
    before = cache(rows, h, d)
    after = [x.clone() for x in before]
    F.fp8_kv_store(c.k, c.v, slots, *after)
    check_store(before, after, slots, R.stored(c.k), R.stored(c.v))
    k, v = F.fp8_kv_load(*after, slots)
    assert torch.equal(k, R.loaded(after[0], after[2], slots)) and torch.equal(v, R.loaded(after[1], after[3], slots))


def test_one_slot_for_all():
    for t in (3, 64, 2500, 9000):
        c = Case(t, 1, 2, 16, 4, interleaved=True)
        before = cache(5, 2, 16)
        after = [x.clone() for x in before]
        slots = torch.full((t,), 3, dtype=torch.int32, device="cuda")
        F.fp8_kv_store(c.k, c.v, slots, *after)
        check_store(before, after, slots, R.stored(c.k), R.stored(c.v))


def test_store_every_bf16_quotient():
    """Every pair of mantissas of a value and its head's largest, the values down
    to 2^-12 of it: codes of the IEEE quotient, ties among them."""
    m = torch.arange(128, 256, dtype=torch.float64)
    x = (m[:, None] * 2.0 ** -torch.arange(13, dtype=torch.float64)).reshape(-1)
    x = torch.cat([x, torch.zeros(-len(x) % 255)])
    heads = len(x) // 255
    a = m[:, None, None, None].expand(128, heads, 1, 1)
    values = torch.minimum(x.view(1, heads, 255, 1).expand(128, heads, 255, 1), a)
    v = torch.cat([a, values], 2).squeeze(-1)
    for scale in (1.0, 2.0 ** -40, 2.0 ** 90):
        k = (v * scale).to(BF).cuda()
        assert torch.equal(k.double().cpu(), v * scale)
        after = cache(128, heads, 256)
        before = [c.clone() for c in after]
        slots = torch.arange(128, dtype=torch.int32, device="cuda")
        F.fp8_kv_store(k, -k, slots, *after)
        check_store(before, after, slots, R.stored(k), R.stored(-k))


def test_special_heads():
    """Heads of zeros of both signs, subnormals, the largest values, ties."""
    d = 32
    rows = [torch.zeros(d), -torch.zeros(d), torch.full((d,), 2.0 ** -133), torch.linspace(-127, 127, d).round() * 2.0 ** -133,
            torch.full((d,), torch.finfo(BF).max), torch.linspace(-448, 448, d), (torch.arange(d) + 0.5) * 2, torch.eye(d)[5],
            torch.linspace(-1, 1, d) * 2.0 ** -100, torch.linspace(-1, 1, d) * 900 * 2.0 ** -133]
    x = torch.stack(rows).to(BF)[:, None].contiguous().cuda()
    t = x.shape[0]
    before = cache(t, 1, d)
    after = [y.clone() for y in before]
    slots = torch.arange(t, dtype=torch.int32, device="cuda")
    F.fp8_kv_store(x, -x, slots, *after)
    check_store(before, after, slots, R.stored(x), R.stored(-x))
    k, v = F.fp8_kv_load(*after, slots)
    assert torch.equal(k, R.loaded(after[0], after[2], slots)) and torch.equal(v, R.loaded(after[1], after[3], slots))


def test_heads_that_are_not_finite_stay_their_own():
    c = Case(20, 2, 3, 64)
    slots = slots_of(20, 30)
    clean, dirty = ([x for x in cache(30, 3, 64)] for _ in range(2))
    F.fp8_kv_store(c.k, c.v, slots, *clean)
    c.k[4, 1, 9], c.v[7, 2, 0] = float("nan"), float("inf")
    F.fp8_kv_store(c.k, c.v, slots, *dirty)
    for i, (token, head) in enumerate(((4, 1), (7, 2))):
        same = (clean[i] == dirty[i]).all(-1)
        same[int(slots[token]), head] = True
        assert bool(same.all())


def check_fused(c, before, after, q, slots, name):
    worst = R.outside(q, *c.ref(c.q, c.qw))
    assert worst <= 1, (name, worst)
    ref, bound = c.ref(c.k, c.kw)
    live = R.last_ones(slots.cpu(), before[0].shape[0]).cuda()
    rows = slots[live].long()
    # k: the scale within the bound of its largest element, each value within
    # half a step of E4M3 (2^-10 of the scale at its smallest) on top
    s_ref = (ref.abs().amax(-1) / 448)[live]
    s_off = (after[2][rows].double() - s_ref).abs()
    assert bool((s_off <= bound.amax(-1)[live] / 448 + 2 * R.U * s_ref).all()), name
    got = R.values(after[0][rows]) * after[2][rows].double()[..., None]
    most = torch.maximum(2.0 ** -4 * ref.abs()[live], 2.0 ** -10 * s_ref[..., None]) * (1 + 2.0 ** -10) + 2 * bound[live]
    assert bool(((got - ref[live]).abs() <= most).all()), name
    # and the very codes and scales, but within fp64's own error of a border
    codes, scale, sure, sure_scale = (x[live] for x in c.stored_turned())
    assert float(sure.double().mean()) > 0.99, name
    assert bool(((R.values(after[0][rows]) == codes) | ~sure).all()), name
    assert bool(((after[2][rows] == scale) | ~sure_scale).all()), name
    untouched = torch.ones(before[0].shape[0], dtype=torch.bool, device="cuda")
    untouched[rows] = False
    assert all(torch.equal(a[untouched], b[untouched]) for a, b in zip(before, after)), name
    values, scale = R.stored(c.v)
    assert torch.equal(R.values(after[1][rows]), values[live]) and torch.equal(after[3][rows], scale[live]), name


@pytest.mark.parametrize("size", CASES, ids=IDS)
def test_fused_store(size):
    say("qk_norm_rope_store", size)
    c = Case(*size)
    rows = c.t + 5
    slots = slots_of(c.t, rows)
    if c.t > 4:
        slots[2], slots[c.t - 1] = -1, slots[0]
    before = cache(rows, c.hk, c.d)
    after = [x.clone() for x in before]
    q = F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, slots, *after, **c.how)
    check_fused(c, before, after, q, slots, size)
    assert torch.equal(q, F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)[0])


def test_rolling_cache():
    """A cache of a window's rows that a sequence runs through twice over: slot =
    position % window, a prompt longer than the window in one call, then token by
    token."""
    window, h, d = 48, 2, 64
    c = Case(130, 4, h, d, None, 1, False)
    after = list(cache(window, h, d))
    position = torch.arange(130, dtype=torch.int32, device="cuda")
    c.positions = position[None].contiguous()
    slots = position % window
    F.fp8_qk_norm_rope_store(c.q[:120], c.k[:120], c.v[:120], c.qw, c.kw, c.positions[:, :120].contiguous(), c.freq,
                             slots[:120], *after, **c.how)
    for i in range(120, 130):
        F.fp8_qk_norm_rope_store(c.q[i:i + 1], c.k[i:i + 1], c.v[i:i + 1], c.qw, c.kw, c.positions[:, i:i + 1].contiguous(),
                                 c.freq, slots[i:i + 1], *after, **c.how)
    k, v = F.fp8_kv_load(*after, slots[130 - window:])
    kept = slice(130 - window, 130)
    ref, bound = c.ref(c.k, c.kw)
    most = (2.0 ** -4 + 2.0 ** -8) * 1.01 * ref.abs() + 2.0 ** -9 * (ref.abs().amax(-1, keepdim=True) / 448) + 3 * bound
    assert bool(((k.double() - ref[kept]).abs() <= most[kept]).all())
    assert torch.equal(v, R.loaded(after[1], after[3], slots[kept]))


def test_load_into_views_and_the_same_slot_often():
    h, d = 3, 80
    codes = cache(50, h, d)
    slots = torch.tensor([4, 4, 49, -1, 0, 50, 4, 2 ** 31 - 1, -2 ** 31] * 9, dtype=torch.int32, device="cuda")
    t = slots.numel()
    buf = torch.full((t, 2 * h * d + 16), 5.0, dtype=BF, device="cuda")
    k_out, v_out = buf[:, :h * d].view(t, h, d), buf[:, h * d + 8:2 * h * d + 8].view(t, h, d)
    F.fp8_kv_load(*codes, slots, k_out=k_out, v_out=v_out)
    assert torch.equal(k_out, R.loaded(codes[0], codes[2], slots)) and torch.equal(v_out, R.loaded(codes[1], codes[3], slots))
    assert bool((buf[:, h * d:h * d + 8] == 5).all()) and bool((buf[:, 2 * h * d + 8:] == 5).all())
    turned = torch.empty(h, t, d, dtype=BF, device="cuda").transpose(0, 1)
    F.fp8_kv_load(*codes, slots, k_out=turned, v_out=v_out)
    assert torch.equal(turned, k_out)


def test_cache_past_32_bit_offsets():
    """A cache of 2^33 bytes a side, slots on both sides of 2^31 and 2^32."""
    h, d = 8, 128
    rows = (1 << 23) + 64
    say("cache of", rows, "rows")
    k_cache, v_cache = (torch.zeros(rows, h, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    k_scale, v_scale = (torch.ones(rows, h, device="cuda") for _ in range(2))
    at = [0, (1 << 21) - 1, 1 << 21, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, (1 << 23) - 1, 1 << 23, rows - 1]
    slots = torch.tensor(at, dtype=torch.int32, device="cuda")
    c = Case(len(at), 4, h, d)
    F.fp8_kv_store(c.k, c.v, slots, k_cache, v_cache, k_scale, v_scale)
    values, scale = R.stored(c.k)
    assert torch.equal(R.values(k_cache[slots.long()]), values) and torch.equal(k_scale[slots.long()], scale)
    assert int(k_cache.view(torch.int64).count_nonzero()) <= len(at) * h * d // 8
    k, v = F.fp8_kv_load(k_cache, v_cache, k_scale, v_scale, slots)
    assert torch.equal(k, R.loaded(k_cache, k_scale, slots)) and torch.equal(v, R.loaded(v_cache, v_scale, slots))


def test_heads_past_32_bit_offsets():
    """Tokens a long stride apart: an array of 2^33 bytes read in place."""
    t, h, d = 9, 2, 64
    buf = torch.zeros(t, 1 << 29, dtype=BF, device="cuda")
    c = Case(t, h, h, d)
    q, k = buf[:, :h * d].view(t, h, d), buf[:, -h * d:].view(t, h, d)
    q.copy_(c.q)
    k.copy_(c.k)
    ref = F.fp8_qk_norm_rope(c.q, c.k, *c.table, **c.how)
    got = F.fp8_qk_norm_rope(q, k, *c.table, **c.how, q_out=q, k_out=k)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [16, 24, 64, 120, 256])
def test_sizes_past_the_caches(d, interleaved):
    """Calls that move more than 256 MB go past the caches: token by token the bits of
    the same call on a quarter of the tokens."""
    say("past the caches", d, interleaved)
    gen = torch.Generator(device="cuda").manual_seed(d)
    t = 40000
    hq, hk = 2 ** 26 // (t * d) + 1, 3
    q, dq = (torch.randn(t, hq, d, generator=gen, device="cuda").to(BF) for _ in range(2))
    k, v, dk = (torch.randn(t, hk, d, generator=gen, device="cuda").to(BF) for _ in range(3))
    w = [(1 + 0.3 * torch.randn(d, generator=gen, device="cuda")).to(BF) for _ in range(2)]
    positions = torch.randint(0, 100000, (t,), generator=gen, device="cuda", dtype=torch.int32)
    freq = torch.rand(8, generator=gen, device="cuda")
    slots = torch.randperm(t, generator=gen, device="cuda").to(torch.int32)
    how = {"interleaved": interleaved}

    def calls(a, b, store):
        part = [x[a:b] for x in (q, k, v, dq, dk, positions, slots)]
        table = (*w, part[5], freq)
        turned = F.fp8_qk_norm_rope(part[0], part[1], *table, **how)
        grads = F.fp8_qk_norm_rope_backward(part[3], part[4], part[0], part[1], *table, **how)[:2]
        stored = F.fp8_qk_norm_rope_store(part[0], part[1], part[2], *table, part[6], *store, **how)
        return (*turned, *grads, stored)

    whole, parts = cache(t, hk, d), cache(t, hk, d)
    got = calls(0, t, whole)
    for a in range(0, t, t // 4):
        for x, y in zip(got, calls(a, a + t // 4, parts)):
            assert torch.equal(x[a:a + t // 4].view(torch.int16), y.view(torch.int16))
    assert all(torch.equal(x, y) for x, y in zip(whole, parts))
    # a long context: each row of the cache many times
    again = -(-2 ** 28 // (6 * t * hk * d)) + 1
    out = F.fp8_kv_load(*whole, slots.repeat(again))
    once = F.fp8_kv_load(*whole, slots)
    for x, y in zip(out, once):
        assert all(torch.equal(x[i * t:(i + 1) * t], y) for i in range(again))


def test_writes_only_its_workspace():
    c = Case(515, 8, 2, 128, None, 3, False)
    ref = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)
    size = F.qk_norm_rope_backward_workspace_size(c.t, c.hq, c.hk, c.d)
    buf = torch.full((size + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    got = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how, workspace=buf[256:256 + size])
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    assert bool((buf[:256] == 0xFF).all()) and bool((buf[256 + size:] == 0xFF).all())


def test_other_streams_and_two_at_once():
    cases = [Case(16, 16, 4, 128), Case(300, 8, 2, 80, 16), Case(700, 4, 4, 64, None, 3, True)]
    caches = [cache(c.t + 8, c.hk, c.d) for c in cases]
    refs = []
    for c, before in zip(cases, caches):
        after = [x.clone() for x in before]
        q = F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, slots_of(c.t, c.t + 8), *after, **c.how)
        refs.append((q, *after, *F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how)))
    streams = [torch.cuda.Stream() for _ in cases]
    sets = [(slots_of(c.t, c.t + 8), [x.clone() for x in before]) for c, before in zip(cases, caches)]
    torch.cuda.synchronize()
    got = [None] * len(cases)
    for _ in range(3):
        for i, (c, stream) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(stream):
                q = F.fp8_qk_norm_rope_store(c.q, c.k, c.v, *c.table, sets[i][0], *sets[i][1], **c.how)
                got[i] = (q, *sets[i][1], *F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table, **c.how))
    torch.cuda.synchronize()
    for a, b in zip(refs, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed():
    """A block's step in one graph: quantised projection, norm, turn, store and
    load, replayed on new inputs with eager work between."""
    t, hq, hk, d, width = 16, 8, 2, 64, 256
    gen = torch.Generator().manual_seed(4)
    wq, ws = F.int8_row_quantize(torch.randn((hq + 2 * hk) * d, width, generator=gen).cuda() * 0.05)
    c = Case(t, hq, hk, d, None, 3, False)
    x = torch.zeros(t, width, dtype=BF, device="cuda")
    slots = slots_of(t, 40)
    store = list(cache(40, hk, d))

    def step(store):
        qkv = F.int8_linear_bf16(x, wq, ws)
        q, k, v = (p.view(t, -1, d) for p in qkv.split([hq * d, hk * d, hk * d], 1))
        q = F.fp8_qk_norm_rope_store(q, k, v, *c.table, slots, *store, **c.how)
        return (q, *F.fp8_kv_load(*store, slots), *F.fp8_qk_norm_rope_backward(q, k, q, k, *c.table, **c.how))

    with torch.cuda.stream(torch.cuda.Stream()):
        step(store)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(store)
    for _ in range(4):
        x.copy_(torch.randn(t, width, generator=gen).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        eager = [y.clone() for y in store]
        ref = step(eager)
        assert all(torch.equal(a, b) for a, b in zip(outs, ref)) and all(torch.equal(a, b) for a, b in zip(store, eager))


def test_empty():
    c = Case(4, 2, 2, 64)
    q, k = F.fp8_qk_norm_rope(c.q[:0], c.k[:0], c.qw, c.kw, c.positions[:, :0].contiguous(), c.freq)
    assert q.shape == (0, 2, 64) and k.shape == (0, 2, 64)
    _, _, dqw, dkw = F.fp8_qk_norm_rope_backward(c.dq[:0], c.dk[:0], c.q[:0], c.k[:0], c.qw, c.kw,
                                                 c.positions[:, :0].contiguous(), c.freq)
    assert not dqw.any() and not dkw.any() and dqw.shape == (64,)
    # no key heads: their weight's gradient is zero
    none = c.k[:, :0]
    got = F.fp8_qk_norm_rope_backward(c.dq, none, c.q, none, *c.table)
    ref = F.fp8_qk_norm_rope_backward(c.dq, c.dk, c.q, c.k, *c.table)
    assert torch.equal(got[0], ref[0]) and not got[3].any() and got[1].shape == (4, 0, 64)
    store = cache(3, 2, 64)
    F.fp8_kv_store(c.k[:0], c.v[:0], torch.empty(0, dtype=torch.int32, device="cuda"), *store)
    empty = [x[:0] for x in store]
    slots = torch.zeros(4, dtype=torch.int32, device="cuda")
    F.fp8_kv_store(c.k, c.v, slots, *empty)
    k, v = F.fp8_kv_load(*empty, slots)
    assert not k.any() and not v.any()
