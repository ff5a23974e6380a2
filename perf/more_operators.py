"""What is measured of the 8-bit integer linear and of the operators between a
block's QKV projection and its cache.

  int8_linear          y = (sum_k xq wq) xs ws + bias: codes of 8-bit integers, a
                       scale for each token (xs) and each output channel (ws).
                       From a bf16 x the codes come first: s = fl32(max|x| / 127)
                       of the row, 1 where that is 0, xq = x / s to the nearest
                       integer, ties to even.
  qk_norm_rope         each head of q and k through n = x / sqrt(mean(x^2) + eps) * w,
                       then pairs (a, b) of n turned by theta = position * inv_freq:
                       (a cos - b sin, b cos + a sin). Pair i goes by the position
                       on the axis axes[i]; pair i is (i, i + P) of the first 2 P
                       elements, or (2 i, 2 i + 1) where `interleaved`.
  qk_norm_rope_backward  gradients of q, k and of both norm weights.
  kv_store             k and v of each token into rows `slots` of a cache of E4M3
                       codes with one scale for each token and head:
                       s = fl32(max|x| / 448) over the head, 1 where that is 0,
                       code = E4M3 nearest to x / s. `fused`: q and k go through
                       qk_norm_rope in the same pass, and k is stored unrounded.
  kv_load              rows `slots` of the cache back as bf16(code * s).

A token whose slot is negative is padding: nothing is stored for it, and zeros
are read. `run` computes all this in elementary torch operations; with `own`
set it makes the calls a user of the package makes.
"""

import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # One token through a wide projection with a bias: quantised, then the
        # weight is streamed once; latency counts.
        {"name": "token_int8", "op": "int8_linear", "m": 1, "n": 8000, "k": 8192, "codes": False, "bias": True},
        # A decode batch of 16 through the gate projection.
        {"name": "batch_int8", "op": "int8_linear", "m": 16, "n": 25600, "k": 5120, "codes": False, "bias": False},
        # Everything ragged, on codes that an earlier layer wrote: rows,
        # columns that are no multiple of 8, a K tail.
        {"name": "ragged_int8", "op": "int8_linear", "m": 333, "n": 4300, "k": 1168, "codes": True, "bias": True},
        # A long prompt's feed-forward projection.
        {"name": "prompt_int8", "op": "int8_linear", "m": 8192, "n": 12288, "k": 4096, "codes": False, "bias": True},
        # The heads of a 512-token prompt with text and an image: three axes
        # dealt to the pairs in turn, eight query heads to a key head.
        {"name": "prompt_rope", "op": "qk_norm_rope", "t": 512, "hq": 64, "hk": 8, "d": 128, "pairs": 64,
         "axes": "woven", "interleaved": False},
        # A video's tokens on time, height and width: as many key heads as
        # query heads, neighbouring elements turned together.
        {"name": "video_rope", "op": "qk_norm_rope", "t": 16384, "hq": 40, "hk": 40, "d": 128, "pairs": 64,
         "axes": "sections", "interleaved": True},
        # A short training sequence, an odd length, heads of 80 of which a part
        # is turned.
        {"name": "back_short", "op": "qk_norm_rope_backward", "t": 77, "hq": 16, "hk": 2, "d": 80, "pairs": 16,
         "axes": "one", "interleaved": False},
        # A training step's long sequence.
        {"name": "back_long", "op": "qk_norm_rope_backward", "t": 8192, "hq": 64, "hk": 8, "d": 128, "pairs": 64,
         "axes": "sections", "interleaved": False},
        # One token of each of 16 sequences, normed, turned and stored.
        {"name": "decode_store", "op": "kv_store", "t": 16, "hq": 64, "hk": 8, "d": 128, "pairs": 64,
         "axes": "one", "interleaved": False, "fused": True, "padding": 3},
        # A prompt's keys and values, stored as they are.
        {"name": "prompt_store", "op": "kv_store", "t": 8192, "hq": 0, "hk": 8, "d": 128, "fused": False,
         "padding": 100},
        # The cache of a short sequence read back.
        {"name": "short_load", "op": "kv_load", "t": 129, "hk": 8, "d": 128, "padding": 0},
        # Long sequences read back through their pages.
        {"name": "long_load", "op": "kv_load", "t": 131071, "hk": 8, "d": 128, "padding": 1000},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: 1 to 8192 rows, 16 to 25600 outputs of any
    remainder, K from 64 to 25600 in steps of 16; 1 to 16384 tokens (131072
    read back) of 1 to 64 heads of 64 to 256."""
    op = rng.choice(("int8_linear", "qk_norm_rope", "qk_norm_rope_backward", "kv_store", "kv_load"))
    if op == "int8_linear":
        while True:
            m = _log_uniform(rng, 1, 8192)
            n = _log_uniform(rng, 16, 25600)
            step = rng.choice((1, 8, 128))
            n = max(step, n // step * step)
            k = 16 * _log_uniform(rng, 4, 1600)
            if m * n * k <= 4.0e11 and n * k <= 2.0e8:
                return {"op": op, "m": m, "n": n, "k": k, "codes": rng.random() < 0.3, "bias": rng.random() < 0.5}
    case = {"op": op}
    d = rng.choice((64, 80, 96, 128, 128, 256))
    if op == "kv_load":
        t, hk = _log_uniform(rng, 1, 131072), _log_uniform(rng, 1, 32)
        while t * hk * d > 131071 * 8 * 128:
            t = max(1, t // 2)
        return {"op": op, "t": t, "hk": hk, "d": d, "padding": rng.choice((0, 0, t // 7))}
    t, hk = _log_uniform(rng, 1, 16384), _log_uniform(rng, 1, 40)
    hq = min(64, hk * rng.choice((1, 1, 2, 4, 7, 8)))
    most = {"qk_norm_rope": 16384 * 80 * 128, "qk_norm_rope_backward": 8192 * 72 * 128, "kv_store": 8192 * 80 * 128}[op]
    while t * (hq + hk) * d > most:
        t = max(1, t // 2)
    case.update(t=t, hq=hq, hk=hk, d=d)
    if op == "kv_store":
        case["fused"] = rng.random() < 0.6
        case["padding"] = rng.choice((0, 0, t // 5))
        if not case["fused"]:
            case["hq"] = 0
            return case
    case["pairs"] = rng.choice((d // 2, d // 2, 16))
    case["axes"] = rng.choice(("one", "sections", "woven"))
    case["interleaved"] = rng.random() < 0.4
    return case


# ---- inputs -------------------------------------------------------------

def _axes_of(case):
    """The axis that each pair turns by: one axis; or time, height and width
    in three runs of pairs; or the three dealt out in turn."""
    p = case["pairs"]
    if case["axes"] == "one":
        return (0,) * p
    if case["axes"] == "woven":
        return tuple(i % 3 for i in range(p))
    first, second = p - 2 * (p * 5 // 16), p * 5 // 16
    return tuple(0 if i < first else 1 if i < first + second else 2 for i in range(p))


def _positions(case, gen):
    """Where each token stands: [axes, t] int32. A third of the tokens is text,
    counted on from wherever the context has got to; the others are a grid of
    frames, rows and columns behind it."""
    t = case["t"]
    start = int(torch.randint(0, 200000, (), generator=gen, device="cuda"))
    i = torch.arange(t, device="cuda")
    if case["axes"] == "one":
        return (start + i).to(torch.int32)[None].contiguous()
    text, wide = t // 3, max(1, int(math.sqrt(t) / 2))
    j = (i - text).clamp_min(0)
    grid = torch.stack((j // (wide * wide), j // wide % wide, j % wide))
    return (start + torch.where(i < text, i[None], text + grid)).to(torch.int32).contiguous()


def _heads(gen, t, heads, d):
    """A projection's output [t, heads * d] in which a few elements of each
    head carry most of its size, as bf16."""
    x = torch.randn(t, heads, d, generator=gen, device="cuda")
    x[:, :, 5::31] *= 6.0
    return x.to(torch.bfloat16).view(t, heads * d)


def _slots(case, gen, count):
    """A slot for each token: sequences in pages of 64 that lie anywhere in the
    cache; padding at the end."""
    t = case["t"]
    pages = torch.randperm(count // 64, generator=gen, device="cuda")
    i = torch.arange(t, device="cuda")
    slots = pages[i // 64] * 64 + i % 64
    slots[t - case["padding"]:] = -1
    return slots.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, state = case["op"], {"case": dict(case)}
    if op == "int8_linear":
        m, n, k = case["m"], case["n"], case["k"]
        w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
        state["ws"] = w.abs().amax(1) / 127
        state["wq"] = torch.round(w / state["ws"][:, None]).to(torch.int8)
        x = torch.randn(m, k, generator=gen, device="cuda")
        x[:, 3::97] *= 4.0          # a few channels carry most of an activation's size
        if case["codes"]:
            state["xs"] = x.abs().amax(1) / 127
            state["xq"] = torch.round(x / state["xs"][:, None]).to(torch.int8)
        else:
            state["x"] = x.to(torch.bfloat16)
        bias = torch.randn(n, generator=gen, device="cuda") * 0.5
        state["bias"] = bias.to(torch.bfloat16) if case["bias"] else None
        return state
    t, hk, d = case["t"], case["hk"], case["d"]
    hq = case.get("hq", 0)
    if op != "kv_load":
        # views of one packed projection output
        qkv = _heads(gen, t, hq + 2 * hk, d)
        state["q"] = qkv[:, :hq * d].view(t, hq, d)
        state["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        state["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
    if case.get("pairs"):
        state["qw"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        state["kw"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        state["positions"] = _positions(case, gen)
        base = 5.0e6 if case["axes"] != "sections" else 1.0e4
        p = case["pairs"]
        state["inv_freq"] = (base ** (-torch.arange(p, dtype=torch.float64, device="cuda") / p)).float()
        state["axes"] = _axes_of(case)
    if op == "qk_norm_rope_backward":
        state["dq"] = (torch.randn(t, hq, d, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
        state["dk"] = (torch.randn(t, hk, d, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    if op in ("kv_store", "kv_load"):
        # a cache of pages, a third more than the tokens here take, in use
        # already; one row more lies behind it
        count = 64 * (-(-t // 64) * 4 // 3 + 1)
        state["slots"] = _slots(case, gen, count)
        for name in ("kc", "vc"):
            codes = torch.randint(0, 127, (count + 1, hk, d), generator=gen, device="cuda", dtype=torch.uint8)
            sign = torch.randint(0, 2, (count + 1, hk, d), generator=gen, device="cuda", dtype=torch.uint8)
            state[name] = codes + 128 * sign
        for name in ("ks", "vs"):
            state[name] = torch.rand(count + 1, hk, generator=gen, device="cuda") * 0.01 + 1e-3
    return state


# ---- the plain form -----------------------------------------------------

def _angles(state):
    """cos and sin [t, 1, pairs], the angle in 64 bits: at far positions 32
    hold it to no better than a hundredth."""
    axes = torch.tensor(state["axes"], device="cuda")
    theta = state["positions"][axes].t().double() * state["inv_freq"].double()
    return theta.cos().float()[:, None], theta.sin().float()[:, None]


def _split(x, pairs, interleaved):
    """The two members of each pair, and the elements behind them."""
    turned, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    if interleaved:
        return turned[..., 0::2], turned[..., 1::2], rest
    return turned[..., :pairs], turned[..., pairs:], rest


def _join(a, b, rest, interleaved):
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1)


def _turn(x, cos, sin, interleaved):
    a, b, rest = _split(x, cos.shape[-1], interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, rest, interleaved)


def _norm_rope(x, w, cos, sin, interleaved):
    x = x.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return _turn(n, cos, sin, interleaved)


def _norm_rope_backward(x, w, dy, cos, sin, interleaved):
    x, w = x.float(), w.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    dn = _turn(dy.float(), cos, -sin, interleaved)
    u = dn * w
    dx = r * (u - x * (r * r * (u * x).mean(-1, keepdim=True)))
    return dx.to(torch.bfloat16), (dn * x * r).double().sum((0, 1)).float()


def _scale(x, most):
    """fl32(max|x| / most) of each row, 1 where that is 0. Many quotients x / s
    are ties, so s has to be the nearest fp32: it is divided in 64 bits."""
    s = (x.abs().amax(-1).double() / most).float()
    return torch.where(s == 0, 1.0, s)


def _put(x, slots, cache, scales):
    """Rows of x into the cache; a negative slot's go to the row behind it."""
    x = x.float()
    s = _scale(x, 448)
    codes = (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    at = torch.where(slots < 0, cache.shape[0] - 1, slots).long()
    cache[at] = codes
    scales[at] = s


def _get(slots, cache, scales):
    at = slots.clamp_min(0).long()
    x = cache[at].view(torch.float8_e4m3fn).float() * scales[at][..., None]
    return torch.where(slots[:, None, None] < 0, 0.0, x).to(torch.bfloat16)


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "int8_linear":
        if case["codes"]:
            xq, xs = state["xq"].float(), state["xs"]
        else:
            x = state["x"].float()
            xs = _scale(x, 127)
            xq = torch.round(x / xs[:, None])
        y = (xq @ state["wq"].float().t()) * (xs[:, None] * state["ws"])
        if case["bias"]:
            y = y + state["bias"].float()
        return {"y": y.to(torch.bfloat16)}
    if op == "kv_load":
        return {"k": _get(state["slots"], state["kc"], state["ks"]),
                "v": _get(state["slots"], state["vc"], state["vs"])}
    if op == "kv_store" and not case["fused"]:
        _put(state["k"], state["slots"], state["kc"], state["ks"])
        _put(state["v"], state["slots"], state["vc"], state["vs"])
        return _caches(state)
    cos, sin = _angles(state)
    inter = case["interleaved"]
    if op == "qk_norm_rope_backward":
        dq, dqw = _norm_rope_backward(state["q"], state["qw"], state["dq"], cos, sin, inter)
        dk, dkw = _norm_rope_backward(state["k"], state["kw"], state["dk"], cos, sin, inter)
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    q = _norm_rope(state["q"], state["qw"], cos, sin, inter)
    k = _norm_rope(state["k"], state["kw"], cos, sin, inter)
    if op == "qk_norm_rope":
        return {"q": q.to(torch.bfloat16), "k": k.to(torch.bfloat16)}
    _put(k, state["slots"], state["kc"], state["ks"])
    _put(state["v"], state["slots"], state["vc"], state["vs"])
    return {"q": q.to(torch.bfloat16), **_caches(state)}


def _caches(state):
    """The updated cache whole: the codes as E4M3 values, and the scales."""
    return {"kc": state["kc"][:-1].view(torch.float8_e4m3fn), "vc": state["vc"][:-1].view(torch.float8_e4m3fn),
            "ks": state["ks"][:-1], "vs": state["vs"][:-1]}


# ---- the framework's calls ----------------------------------------------

def _own(state):
    import block_scaled_fp8_linear_amd as F

    case = state["case"]
    op = case["op"]
    if op == "int8_linear":
        if case["codes"]:
            y = F.int8_linear(state["xq"], state["xs"], state["wq"], state["ws"], bias=state["bias"])
        else:
            y = F.int8_linear_bf16(state["x"], state["wq"], state["ws"], bias=state["bias"])
        return {"y": y}
    if op == "kv_load":
        k, v = F.fp8_kv_load(state["kc"][:-1], state["vc"][:-1], state["ks"][:-1], state["vs"][:-1], state["slots"])
        return {"k": k, "v": v}
    cache = ()
    if op == "kv_store":
        cache = (state["slots"], state["kc"][:-1], state["vc"][:-1], state["ks"][:-1], state["vs"][:-1])
        if not case["fused"]:
            F.fp8_kv_store(state["k"], state["v"], *cache)
            return _caches(state)
    turn = {"axes": state["axes"], "eps": EPS, "interleaved": case["interleaved"]}
    heads = (state["q"], state["k"])
    table = (state["qw"], state["kw"], state["positions"], state["inv_freq"])
    if op == "qk_norm_rope":
        q, k = F.fp8_qk_norm_rope(*heads, *table, **turn)
        return {"q": q, "k": k}
    if op == "qk_norm_rope_backward":
        dq, dk, dqw, dkw = F.fp8_qk_norm_rope_backward(state["dq"], state["dk"], *heads, *table, **turn)
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    q = F.fp8_qk_norm_rope_store(*heads, state["v"], *table, *cache, **turn)
    return {"q": q, **_caches(state)}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---- what a pass cannot do without --------------------------------------

def work(case):
    op = case["op"]
    if op == "int8_linear":
        m, n, k = case["m"], case["n"], case["k"]
        x = m * k + 4 * m if case["codes"] else 2 * m * k
        return {"bytes": x + n * k + 4 * n + 2 * m * n + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    t, hk, d = case["t"], case["hk"], case["d"]
    hq = case.get("hq", 0)
    kept = t - case.get("padding", 0)
    turned = t * (hq + hk) * d          # elements of q and k
    table = 4 * t * (1 if case.get("axes") == "one" else 3) + 4 * case.get("pairs", 0) + 4 * d
    if op == "qk_norm_rope":
        return {"bytes": 4 * turned + table, "flops": 7 * turned}
    if op == "qk_norm_rope_backward":
        return {"bytes": 6 * turned + table + 8 * d, "flops": 17 * turned}
    cache = 2 * kept * hk * d + 8 * kept * hk       # codes and scales of k and v
    if op == "kv_load":
        return {"bytes": cache + 4 * t + 4 * t * hk * d, "flops": 2 * kept * hk * d}
    if not case["fused"]:
        return {"bytes": 4 * kept * hk * d + 4 * t + cache, "flops": 6 * kept * hk * d}
    # q of every token in and out, k and v of those that are stored
    return {"bytes": 4 * t * hq * d + 4 * kept * hk * d + table + 4 * t + cache,
            "flops": 7 * turned + 6 * kept * hk * d}


# ---- the definition in 64 bits ------------------------------------------

def _e4m3_table():
    """The 256 values of OCP E4M3: sign, 4 exponent bits (bias 7), 3 mantissa
    bits; exponent 0 is subnormal, S.1111.111 is NaN."""
    values = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = math.nan if (c & 127) == 127 else f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        values.append(-v if c >= 128 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _nearest_e4m3(x):
    """x to the nearest multiple of its binade's step, ties to even, at most 448."""
    _, e = torch.frexp(x)
    step = (((e - 4).clamp_min(-9).long() + 1023) << 52).view(torch.float64)     # 2^(e - 4), from its bits
    return (torch.round(x / step) * step).clamp(-448, 448)


def _fp32(x):
    return x.to(torch.float32).double()


def _rope64(x, w, state, backward=None):
    """One of q and k as complex numbers: the norm, and a turn by e^(i theta);
    with `backward`, the gradients from that of the result."""
    case = state["case"]
    p, inter = case["pairs"], case["interleaved"]
    x, w = x.double(), w.double()
    order = torch.arange(2 * p, device="cuda")
    order = order.view(p, 2) if inter else order.view(2, p).t()
    where = state["positions"].double()[torch.tensor(state["axes"], device="cuda")]
    turn = torch.exp(1j * (where * state["inv_freq"].double()[:, None])).t()[:, None]

    def turned(n, by):
        z = torch.complex(n[..., order[:, 0]], n[..., order[:, 1]]) * by
        out = n.clone()
        out[..., order[:, 0]], out[..., order[:, 1]] = z.real, z.imag
        return out

    size = (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    if backward is None:
        return turned(x / size * w, turn)
    dn = turned(backward.double(), turn.conj())
    unit = x / size
    dw = (dn * unit).sum(dim=(0, 1))
    u = dn * w / size
    along = (u * unit).sum(-1, keepdim=True) / x.shape[-1]
    return u - unit * along, dw


def _store64(x, slots, codes, scales):
    x = x.double()
    s = _fp32(x.abs().max(dim=-1).values / 448)
    s[s == 0] = 1.0
    values = _nearest_e4m3(_fp32(x / s[..., None]))
    live = slots >= 0
    codes[slots[live].long()] = values[live]
    scales[slots[live].long()] = s[live]
    return codes, scales


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "int8_linear":
        if case["codes"]:
            xq, xs = state["xq"].double(), state["xs"].double()
        else:
            x = state["x"].double()
            xs = _fp32(x.abs().max(dim=1).values / 127)
            xs[xs == 0] = 1.0
            xq = torch.round(_fp32(x / xs[:, None]))
        y = torch.matmul(xq, state["wq"].double().T)      # below 2^53: exact
        y = y * xs[:, None] * state["ws"].double()
        if case["bias"]:
            y = y + state["bias"].double()
        return {"y": y}
    table = _e4m3_table()
    if op == "kv_load":
        out = {}
        live = (state["slots"] >= 0)[:, None, None]
        rows = state["slots"].clamp(min=0).long()
        for name, codes, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
            x = table[state[codes][rows].int()] * state[scales][rows].double()[..., None]
            out[name] = x * live
        return out
    if op == "qk_norm_rope":
        return {"q": _rope64(state["q"], state["qw"], state), "k": _rope64(state["k"], state["kw"], state)}
    if op == "qk_norm_rope_backward":
        dq, dqw = _rope64(state["q"], state["qw"], state, state["dq"])
        dk, dkw = _rope64(state["k"], state["kw"], state, state["dk"])
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    slots, out = state["slots"], {}
    k = state["k"]
    if case["fused"]:
        out["q"] = _rope64(state["q"], state["qw"], state)
        k = _rope64(k, state["kw"], state)
    for x, codes, scales in ((k, "kc", "ks"), (state["v"], "vc", "vs")):
        out[codes], out[scales] = _store64(x, slots, table[state[codes][:-1].int()], state[scales][:-1].double())
    return out
