"""What is measured of the layer operators: linears against block-FP8 weights
with the epilogue of a transformer block, the gated feed-forward pair, and the
backward pass of both through the frozen weight.

A weight is E4M3 bytes Q[N,K] with one fp32 scale per 128x128 block
S[ceil(N/128), ceil(K/128)], and stands for W = bf16(fl32(e4m3(Q) * S)).

  linear_act           z = x W^T + bias,  y = act(z) + residual
  linear_act_backward  dz = dy act'(z),  dbias = sum over rows of dz,  dx = dz W
  glu                  g = x Wg^T,  u = x Wu^T,  h = act(g) u
  glu_backward         dg = dh u act'(g),  du = dh act(g),  dx = dg Wg + du Wu

`run` computes them in elementary torch operations in fp32, rounded once at
the end; with `own` set it makes the calls a user of the package makes.
"""

import math

import torch

own = False

BLOCK = 128
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # One token through a wide projection with bias and activation: the
        # weight is streamed once, latency counts.
        {"name": "token_fc1", "op": "linear_act", "m": 1, "n": 8000, "k": 8192, "act": "gelu_tanh",
         "bias": True, "residual": False, "save": False},
        # A decode batch through an attention output projection, added to the
        # residual stream.
        {"name": "batch_proj", "op": "linear_act", "m": 16, "n": 5120, "k": 5120, "act": "none",
         "bias": False, "residual": True, "save": False},
        # The same projection for a prompt of 512 tokens.
        {"name": "prompt_proj", "op": "linear_act", "m": 512, "n": 5120, "k": 5120, "act": "none",
         "bias": False, "residual": True, "save": False},
        # The down projection of the feed-forward block for that prompt: a long
        # reduction with few output tiles.
        {"name": "prompt_down", "op": "linear_act", "m": 512, "n": 5120, "k": 25600, "act": "none",
         "bias": False, "residual": True, "save": False},
        # Everything ragged: rows, columns that are no multiple of 8, a K tail,
        # and every part of the epilogue at once.
        {"name": "ragged_fc1", "op": "linear_act", "m": 333, "n": 4300, "k": 1168, "act": "gelu",
         "bias": True, "residual": True, "save": True},
        # A training step's first feed-forward projection, which keeps z for
        # its backward pass.
        {"name": "train_fc1", "op": "linear_act", "m": 8192, "n": 12288, "k": 4096, "act": "gelu_tanh",
         "bias": True, "residual": False, "save": True},
        # Its backward pass on half the rows.
        {"name": "back_fc1", "op": "linear_act_backward", "m": 4096, "n": 12288, "k": 4096,
         "act": "gelu_tanh", "bias": True},
        # A short, odd-sized backward pass: an adapter's narrow layer.
        {"name": "back_ragged", "op": "linear_act_backward", "m": 77, "n": 1003, "k": 656, "act": "silu",
         "bias": True},
        # One token through the gated feed-forward pair: two weights streamed.
        {"name": "token_glu", "op": "glu", "m": 1, "n": 25600, "k": 5120, "act": "silu", "save": False},
        # The pair for a 512-token prompt, kept for the backward pass.
        {"name": "train_glu", "op": "glu", "m": 512, "n": 25600, "k": 5120, "act": "silu", "save": True},
        # Its backward pass.
        {"name": "back_glu", "op": "glu_backward", "m": 512, "n": 25600, "k": 5120, "act": "silu"},
        # A long sequence through a narrower pair, backward.
        {"name": "back_glu_long", "op": "glu_backward", "m": 4096, "n": 12800, "k": 5120,
         "act": "gelu_tanh"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: 1 to 8192 rows, 16 to 25600 outputs of any
    remainder, K from 64 to 25600 in steps of 16 (what the format takes)."""
    op = rng.choice(("linear_act", "linear_act_backward", "glu", "glu_backward"))
    while True:
        m = _log_uniform(rng, 1, 8192)
        n = _log_uniform(rng, 16, 25600)
        step = rng.choice((1, 8, 128))
        n = max(step, n // step * step)
        k = 16 * _log_uniform(rng, 4, 1600)
        weights = 2 if op.startswith("glu") else 1
        if m * n * k * weights <= 3.0e11 and n * k * weights <= 2.0e8:
            break
    case = {"op": op, "m": m, "n": n, "k": k, "act": rng.choice(ACTS)}
    if op == "linear_act":
        case.update(bias=rng.random() < 0.5, residual=rng.random() < 0.5, save=rng.random() < 0.5)
    elif op == "linear_act_backward":
        case.update(bias=rng.random() < 0.5)
    else:
        case["act"] = rng.choice(("silu", "gelu_tanh", "gelu", "relu"))
        if op == "glu":
            case.update(save=rng.random() < 0.5)
    return case


# ---- inputs -------------------------------------------------------------

def _quantized(gen, n, k):
    """A weight N(0, 0.02^2) in the block format: S = amax / 448 per block,
    Q the nearest E4M3 code of w / S."""
    w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    gn, gk = -(-n // BLOCK), -(-k // BLOCK)
    padded = torch.zeros(gn * BLOCK, gk * BLOCK, device="cuda")
    padded[:n, :k] = w
    blocks = padded.view(gn, BLOCK, gk, BLOCK)
    s = (blocks.abs().amax(dim=(1, 3)) / 448).contiguous()
    q = (blocks / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).view(gn * BLOCK, gk * BLOCK)[:n, :k].contiguous()
    return q, s


def _normal(gen, rows, cols, std=1.0):
    return (torch.randn(rows, cols, generator=gen, device="cuda") * std).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    state = {"case": dict(case)}
    if op in ("linear_act", "linear_act_backward"):
        state["q"], state["s"] = _quantized(gen, n, k)
    else:
        state["qg"], state["sg"] = _quantized(gen, n, k)
        state["qu"], state["su"] = _quantized(gen, n, k)
    if op in ("linear_act", "glu"):
        # a few channels carry most of an activation's size
        x = torch.randn(m, k, generator=gen, device="cuda")
        x[:, 3::97] *= 4.0
        state["x"] = x.to(torch.bfloat16)
    z_std = 0.02 * math.sqrt(k)
    if op == "linear_act":
        state["bias"] = _normal(gen, 1, n, 0.5).view(n) if case["bias"] else None
        state["residual"] = _normal(gen, m, n) if case["residual"] else None
    elif op == "linear_act_backward":
        state["dy"] = _normal(gen, m, n, 0.05)
        state["z"] = _normal(gen, m, n, z_std) if case["act"] != "none" else None
    elif op == "glu_backward":
        state["dh"] = _normal(gen, m, n, 0.05)
        state["g"] = _normal(gen, m, n, z_std)
        state["u"] = _normal(gen, m, n, z_std)
    return state


# ---- the plain form -----------------------------------------------------

def _weight(q, s):
    n, k = q.shape
    wide = s.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return (q.view(torch.float8_e4m3fn).float() * wide).to(torch.bfloat16).float()


_TANH_A, _TANH_B = math.sqrt(2 / math.pi), 0.044715


def _act(t, act):
    if act == "none":
        return t
    if act == "relu":
        return t.clamp_min(0)
    if act == "silu":
        return t * torch.sigmoid(t)
    if act == "gelu":
        return 0.5 * t * torch.erfc(t * -math.sqrt(0.5))
    # 1 + tanh(v) = 2 sigmoid(2 v): no cancellation where tanh is near -1
    return t * torch.sigmoid(2 * _TANH_A * (t + _TANH_B * t * t * t))


def _act_grad(t, act):
    if act == "none":
        return torch.ones_like(t)
    if act == "relu":
        return (t > 0).to(t.dtype)
    if act == "silu":
        p = torch.sigmoid(t)
        return p + t * p * torch.sigmoid(-t)
    if act == "gelu":
        return 0.5 * torch.erfc(t * -math.sqrt(0.5)) + t * torch.exp(-0.5 * t * t) / math.sqrt(2 * math.pi)
    v = 2 * _TANH_A * (t + _TANH_B * t * t * t)
    p = torch.sigmoid(v)
    return p + t * p * torch.sigmoid(-v) * (2 * _TANH_A * (1 + 3 * _TANH_B * t * t))


def _plain(state):
    case = state["case"]
    op, act = case["op"], case["act"]
    bf = torch.bfloat16
    if op == "linear_act":
        z = state["x"].float() @ _weight(state["q"], state["s"]).t()
        if state["bias"] is not None:
            z = z + state["bias"].float()
        y = _act(z, act)
        if state["residual"] is not None:
            y = y + state["residual"].float()
        return {"y": y.to(bf), "z": z.to(bf)} if case["save"] else {"y": y.to(bf)}
    if op == "linear_act_backward":
        dz = state["dy"].float()
        if act != "none":
            dz = dz * _act_grad(state["z"].float(), act)
        out = {"dx": (dz @ _weight(state["q"], state["s"])).to(bf)}
        if act != "none":
            out["dz"] = dz.to(bf)
        if case["bias"]:
            out["dbias"] = dz.sum(0)
        return out
    if op == "glu":
        x = state["x"].float()
        g = x @ _weight(state["qg"], state["sg"]).t()
        u = x @ _weight(state["qu"], state["su"]).t()
        h = (_act(g, act) * u).to(bf)
        return {"h": h, "g": g.to(bf), "u": u.to(bf)} if case["save"] else {"h": h}
    dh, g, u = state["dh"].float(), state["g"].float(), state["u"].float()
    dg = dh * u * _act_grad(g, act)
    du = dh * _act(g, act)
    dx = dg @ _weight(state["qg"], state["sg"]) + du @ _weight(state["qu"], state["su"])
    return {"dx": dx.to(bf), "dg": dg.to(bf), "du": du.to(bf)}


# ---- the framework's calls ----------------------------------------------

def _own(state):
    import block_scaled_fp8_linear_amd as F

    case = state["case"]
    op, m, n = case["op"], case["m"], case["n"]
    act = getattr(F, "ACT_" + case["act"].upper())
    if op == "linear_act":
        x = state["x"]
        z = x.new_empty((m, n)) if case["save"] else None
        y = F.fp8_block_linear_act(x, state["q"], state["s"], bias=state["bias"],
                                   residual=state["residual"], act=act, z=z)
        return {"y": y, "z": z} if case["save"] else {"y": y}
    if op == "linear_act_backward":
        dy = state["dy"]
        dbias = torch.empty(n, dtype=torch.float32, device=dy.device) if case["bias"] else None
        dx, dz = F.fp8_block_linear_act_backward(dy, state["q"], state["s"], z=state["z"], act=act,
                                                 dbias=dbias)
        out = {"dx": dx}
        if case["act"] != "none":
            out["dz"] = dz
        if case["bias"]:
            out["dbias"] = dbias
        return out
    weights = (state["qg"], state["sg"], state["qu"], state["su"])
    if op == "glu":
        x = state["x"]
        g = x.new_empty((m, n)) if case["save"] else None
        u = x.new_empty((m, n)) if case["save"] else None
        h = F.fp8_block_glu(x, *weights, act=act, g=g, u=u)
        return {"h": h, "g": g, "u": u} if case["save"] else {"h": h}
    dx, dg, du = F.fp8_block_glu_backward(state["dh"], state["g"], state["u"], *weights, act=act)
    return {"dx": dx, "dg": dg, "du": du}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---- what a pass cannot do without --------------------------------------

def work(case):
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    weight = n * k + 4 * -(-n // BLOCK) * -(-k // BLOCK)
    mn, mk = 2 * m * n, 2 * m * k          # bytes of a bf16 [M,N] and [M,K]
    if op == "linear_act":
        arrays = 1 + bool(case["residual"]) + bool(case["save"])
        return {"bytes": weight + mk + arrays * mn + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if op == "linear_act_backward":
        arrays = 3 if case["act"] != "none" else 1
        return {"bytes": weight + mk + arrays * mn + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if op == "glu":
        return {"bytes": 2 * weight + mk + (3 if case["save"] else 1) * mn, "flops": 4 * m * n * k}
    return {"bytes": 2 * weight + mk + 5 * mn, "flops": 4 * m * n * k}


# ---- the definition in 64 bits ------------------------------------------

def _e4m3_values():
    """The 256 values of OCP E4M3: sign, 4 exponent bits (bias 7), 3 mantissa
    bits; exponent 0 is subnormal, S.1111.111 is NaN."""
    values = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = math.nan if (c & 127) == 127 else f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        values.append(-v if c >= 128 else v)
    return values


def _weight64(q, s):
    """W in 64 bits. The format itself rounds twice (the product to fp32, then
    to bf16); the fp64 product of a 4-bit and a 24-bit significand is exact."""
    table = torch.tensor(_e4m3_values(), dtype=torch.float64, device=q.device)
    n, k = q.shape
    rows = torch.arange(n, device=q.device) // BLOCK
    cols = torch.arange(k, device=q.device) // BLOCK
    w = table[q.int()]
    w *= s.double()[rows][:, cols]
    return w.to(torch.float32).to(torch.bfloat16).double()


def _cdf64(t):
    return torch.special.ndtr(t)


def _act64(t, act):
    """(act(t), act'(t)) in 64 bits."""
    if act == "none":
        return t, torch.ones_like(t)
    if act == "relu":
        on = torch.where(t > 0, 1.0, 0.0).double()
        return t * on, on
    if act == "silu":
        p = 1 / (1 + torch.exp(-t))
        return t * p, p * (1 + t * (1 - p))
    if act == "gelu":
        density = torch.exp(-t ** 2 / 2) / (2 * math.pi) ** 0.5
        return t * _cdf64(t), _cdf64(t) + t * density
    a, b = (2 / math.pi) ** 0.5, 0.044715
    h = torch.tanh(a * (t + b * t ** 3))
    return t * (1 + h) / 2, (1 + h) / 2 + t * (1 - h ** 2) * a * (1 + 3 * b * t ** 2) / 2


def exact(case, seed):
    state = prepare(case, seed)
    op, act = case["op"], case["act"]
    if op == "linear_act":
        z = torch.matmul(state["x"].double(), _weight64(state["q"], state["s"]).T)
        if case["bias"]:
            z += state["bias"].double()
        y = _act64(z, act)[0]
        if case["residual"]:
            y = y + state["residual"].double()
        return {"y": y, "z": z} if case["save"] else {"y": y}
    if op == "linear_act_backward":
        dz = state["dy"].double()
        if act != "none":
            dz = dz * _act64(state["z"].double(), act)[1]
        out = {"dx": torch.matmul(dz, _weight64(state["q"], state["s"]))}
        if act != "none":
            out["dz"] = dz
        if case["bias"]:
            out["dbias"] = dz.sum(dim=0)
        return out
    if op == "glu":
        x = state["x"].double()
        g = torch.matmul(x, _weight64(state["qg"], state["sg"]).T)
        u = torch.matmul(x, _weight64(state["qu"], state["su"]).T)
        h = _act64(g, act)[0] * u
        return {"h": h, "g": g, "u": u} if case["save"] else {"h": h}
    dh, g, u = state["dh"].double(), state["g"].double(), state["u"].double()
    value, slope = _act64(g, act)
    dg, du = dh * u * slope, dh * value
    dx = torch.matmul(dg, _weight64(state["qg"], state["sg"]))
    dx += torch.matmul(du, _weight64(state["qu"], state["su"]))
    return {"dx": dx, "dg": dg, "du": du}
