"""What is measured of the gated linear recurrence (prompt, training step, single token) and
of the microscaled 4-bit format (quantiser with the way back, matrix product).

A block of these is  4-bit in-projections -> conv + SiLU -> gated recurrence -> 4-bit
quantiser -> out-projection.  The sizes are this repository's workloads: the fp32 block
(d_model 768, d_inner 1536, 2 x 8192 tokens, one sequence of 131072) and the 2.8B-scale layer
(d_model 2560, d_inner 5120, 8 x 2048 tokens, 256 sequences in decode).  `own` selects the
library's kernels; otherwise run() computes the plain form, elementary torch operations in 32
bits, rounded once.

The recurrence, per channel, with v = c softplus(lam) sigmoid(r + r_bias) and a = exp(-v), or
a = 0 at a step with `reset` (the first of a packed sequence):
    h_t = a_t h_(t-1) + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t,   y_t = h_t SiLU(z_t)

The 4-bit format holds elements of {0, .5, 1, 1.5, 2, 3, 4, 6} and a sign, two a byte (the
first in the low half), with a power of two for every 32 of the inner axis, stored as its
exponent + 127.  Rows are filled up with zeros to whole groups of 256; scales lie by group:
[groups, rows, 8].  What is held in 4 bits comes back as the numbers it stands for.
"""
import math

import torch

own = False

C = 8.0
GROUP = 256  # elements a row is filled up to a multiple of
BLOCK = 32   # elements of a scale
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ---------------------------------------------------------------------------

def listed():
    def scan(name, op, batch, channels, length, io, gate, packed):
        return {"name": name, "op": op, "batch": batch, "channels": channels, "length": length,
                "io": io, "gate": gate, "packed": packed}

    def quant(name, batch, length, width, order, io):
        return {"name": name, "op": "quantize", "batch": batch, "length": length,
                "width": width, "order": order, "io": io}

    def matmul(name, batch, shared, m, n, k, out):
        return {"name": name, "op": "matmul", "batch": batch, "shared": shared, "m": m, "n": n,
                "k": k, "out": out}

    return [
        # the large layer's prompts, gated
        scan("scan_layer", "scan", 8, 5120, 2048, "bf16", True, False),
        # one long sequence
        scan("scan_long", "scan", 1, 1536, 131072, "bf16", False, False),
        # packed sequences of odd lengths, odd sizes
        scan("scan_ragged", "scan", 3, 771, 1001, "f32", True, True),
        # training step of the fp32 block on packed sequences
        scan("train_block", "train", 2, 1536, 8192, "f32", False, True),
        # training step of the large layer
        scan("train_layer", "train", 8, 5120, 2048, "bf16", True, False),
        # one decoded token: latency
        scan("step_token", "step", 1, 2560, 1, "bf16", False, False),
        # one decode step over 256 sequences
        scan("step_batch", "step", 256, 5120, 1, "bf16", True, False),
        # the recurrence's output of one decode step, before the out-projection
        quant("quant_step", 1, 256, 5120, "token", "bf16"),
        # the recurrence's output over the prompts, channel-major as the scans write it
        quant("quant_layer", 8, 2048, 5120, "channel", "bf16"),
        # in-projection of one decoded token (the weight is the right operand)
        matmul("matmul_token", 1, "none", 1, 5120, 2560, "bf16"),
        # odd in every size
        matmul("matmul_ragged", 1, "none", 333, 515, 1001, "f32"),
        # in-projection over the prompts, written channel-major for the scan (weight on the left)
        matmul("matmul_layer", 8, "a", 5120, 2048, 2560, "bf16"),
    ]


MOST = {"scan": 1536 * 131072, "train": 8 * 5120 * 2048, "step": 256 * 5120}  # elements drawn
MOST_QUANTISED = 8 * 2048 * 5120
MOST_PRODUCTS = 8 * 5120 * 2048 * 2560


def draw(rng):
    def spread(low, high):
        return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))

    def size(low, high, step):  # half of them multiples of `step`, as models have them
        v = spread(low, high)
        return max(step, v // step * step) if rng.random() < 0.5 else v

    op = rng.choice(["scan", "train", "step", "quantize", "matmul", "matmul"])
    io = rng.choice(["bf16", "f32"])
    if op in MOST:
        channels = size(32, 8192, 64)
        batch = (spread(1, min(256, MOST[op] // channels)) if op == "step" else
                 rng.choice([1, 1, 2, 3, 8]))
        length = (1 if op == "step" else
                  spread(2, max(2, min(131072, MOST[op] // (channels * batch)))))
        return {"op": op, "batch": batch, "channels": channels, "length": length, "io": io,
                "gate": rng.random() < 0.5, "packed": op != "step" and rng.random() < 0.5}
    if op == "quantize":
        width = size(32, 8192, 64)
        batch = rng.randint(1, 8)
        length = spread(1, max(1, min(131072, MOST_QUANTISED // (width * batch))))
        return {"op": op, "batch": batch, "length": length, "width": width,
                "order": rng.choice(["token", "channel"]), "io": io}
    k = size(32, 8192, 64)
    n = size(16, 8192, 64)
    batch = rng.choice([1, 1, 2, 8])
    m = spread(1, max(1, min(131072, MOST_PRODUCTS // (k * n * batch))))
    shared = rng.choice(["a", "b"]) if batch > 1 else "none"
    if rng.random() < 0.5:  # either side may be the weight
        m, n = n, m
    return {"op": op, "batch": batch, "shared": shared, "m": m, "n": n, "k": k,
            "out": rng.choice(["bf16", "f32"])}


# ---- inputs ------------------------------------------------------------------------------

def _activations(shape, channel_axis, gen, dtype):
    """N(0, 1) values with one channel in 64 ten times as large, as hidden states have them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    width = shape[channel_axis]
    loud = 1.0 + 9.0 * (torch.rand(width, generator=gen, device="cuda") < 1 / 64)
    view = [1] * len(shape)
    view[channel_axis] = width
    return x.mul_(loud.view(view)).to(dtype)


def _operand(lead, rows, k, gen):
    """N(0, 1) rows in 4 bits: (packed [*lead, rows, padded / 2], scales [groups, *lead, rows, 8]);
    the largest of 32 such values is 1 to 4, a row's size varies by powers of two."""
    padded = -(-k // GROUP) * GROUP
    x = torch.randn((*lead, rows, padded), generator=gen, device="cuda")
    x[..., k:] = 0
    x = x.mul_(torch.exp2(torch.randint(-3, 4, (*lead, rows, 1), generator=gen, device="cuda").float()))
    exponent, elements = _to_elements(x)
    sign = (elements < 0) * 8
    code = torch.zeros(x.shape, dtype=torch.uint8, device="cuda")
    for border in BORDERS:
        code += elements.abs() > border
    code += sign.to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, _scale_layout((exponent + 127).to(torch.uint8))


VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]  # between the values; used on exact values only


def _scale_layout(codes):
    """[*lead, padded / 32] -> [groups, *lead, 8]."""
    lead = codes.shape[:-1]
    return codes.view(*lead, -1, 8).movedim(-2, 0).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case)
    op = case["op"]
    if op in MOST:
        b, d, length = case["batch"], case["channels"], case["length"]
        shape = (b, d) if op == "step" else (b, d, length)
        io = TYPES[case["io"]]
        normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        state["x"], state["r"], state["i"] = (normal(*shape).to(io) for _ in range(3))
        state["z"] = normal(*shape).to(io) if case["gate"] else None
        # a at r = 0 between 0.9 and 0.999, as such layers are initialised
        keep = 0.9 + 0.099 * torch.rand(d, generator=gen, device="cuda")
        state["lam"] = torch.log(torch.expm1(-2.0 * torch.log(keep) / C))
        state["r_bias"], state["i_bias"] = 0.1 * normal(d), 0.1 * normal(d)
        if op == "step":
            state["h"] = normal(b, d)
        else:
            state["reset"] = None
            if case["packed"]:  # sequences of about 300 tokens
                state["reset"] = torch.rand((b, length), generator=gen, device="cuda") < 1 / 300
                state["reset"][:, 0] = True
            if op == "train":
                state["dout"] = normal(*shape).to(io)
            else:
                state["h0"] = normal(b, d)
    elif op == "quantize":
        b, length, width = case["batch"], case["length"], case["width"]
        if case["order"] == "token":
            state["x"] = _activations((b, length, width), 2, gen, TYPES[case["io"]])
        else:
            state["x"] = _activations((b, width, length), 1, gen, TYPES[case["io"]])
    else:
        b, k = case["batch"], case["k"]
        lead = (b,) if b > 1 else ()
        for name, rows in (("a", case["m"]), ("b", case["n"])):
            state[name], state[name + "_scale"] = _operand(() if case["shared"] == name else lead,
                                                           rows, k, gen)
    return state


# ---- one pass ----------------------------------------------------------------------------

def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def _own(s):
    import selective_state_space_80_amd as mamba
    op = s["op"]
    if op == "matmul":
        return mamba.mxfp4_matmul(s["a"], s["b"], s["a_scale"], s["b_scale"], out_dtype=TYPES[s["out"]])
    if op == "quantize":
        q, scale = mamba.quantize_mxfp4(s["x"], channel_major=s["order"] == "channel")
        return mamba.dequantize_mxfp4(q, scale, s["width"]), _scale_values(scale)
    gates = {"r_bias": s["r_bias"], "i_bias": s["i_bias"], "z": s["z"], "c": C}
    inputs = (s["x"], s["r"], s["i"], s["lam"])
    if op == "step":
        h = torch.empty_like(s["h"])  # beside the state, so that every pass starts from the same one
        return mamba.gated_state_update(s["h"], *inputs, h_out=h, **gates), h
    gates["reset"] = s["reset"]
    if op == "scan":
        return mamba.gated_scan_fwd(*inputs, h0=s["h0"], return_last_state=True, **gates)
    y, kept = mamba.gated_scan_fwd(*inputs, return_checkpoints=True, **gates)
    grads = mamba.gated_scan_bwd(*inputs, s["dout"], checkpoints=kept, **gates)
    return (y,) + tuple(grads[name] for name in _gradients(s))


def _gradients(s):
    return ("dx", "dr", "di", "dlam", "dr_bias", "di_bias") + (("dz",) if s["gate"] else ())


def _scale_values(code):
    """2^(code - 127) in fp32."""
    return code.view(torch.float8_e8m0fnu).to(torch.float32)


def _coefficients(s, seq):
    """(v, a, m, gate of the input) in fp32; seq: a trailing axis of steps."""
    per_channel = (lambda p: p[:, None]) if seq else (lambda p: p)
    rate = C * torch.log1p(torch.exp(s["lam"]))
    v = per_channel(rate) * torch.sigmoid(s["r"].float() + per_channel(s["r_bias"]))
    a, m = torch.exp(-v), torch.sqrt(-torch.expm1(-2.0 * v))
    if seq and s["reset"] is not None:
        first = s["reset"][:, None, :]
        a, m = torch.where(first, 0.0, a), torch.where(first, 1.0, m)
    return v, a, m, torch.sigmoid(s["i"].float() + per_channel(s["i_bias"]))


def _linear(a, b):
    """h_t = a_t h_(t-1) + b_t along the last axis, spans doubled."""
    span, length = 1, b.shape[-1]
    while span < length:
        b = torch.cat([b[..., :span], b[..., span:] + a[..., span:] * b[..., :-span]], -1)
        if 2 * span < length:
            a = torch.cat([a[..., :span], a[..., span:] * a[..., :-span]], -1)
        span *= 2
    return b


def _plain_scan(s):
    io = s["x"].dtype
    _, a, m, gate = _coefficients(s, True)
    b = m * gate * s["x"].float()
    b[..., 0] += a[..., 0] * s["h0"]
    h = _linear(a, b)
    y = h if s["z"] is None else h * (s["z"].float() * torch.sigmoid(s["z"].float()))
    return y.to(io), h[..., -1].contiguous()


def _plain_train(s):
    io = s["x"].dtype
    v, a, m, gate = _coefficients(s, True)
    x, dout = s["x"].float(), s["dout"].float()
    h = _linear(a, m * gate * x)
    y, dh, dz = h, dout, ()
    if s["z"] is not None:
        z = s["z"].float()
        sz = torch.sigmoid(z)
        y, dh = h * z * sz, dout * z * sz
        dz = ((dout * h * sz * (1.0 + z * (1.0 - sz))).to(io),)
    nothing = torch.zeros_like(a[..., :1])
    # g_t = dh_t + a_(t+1) g_(t+1): the same recurrence from the end
    g = _linear(torch.cat([a[..., 1:], nothing], -1).flip(-1), dh.flip(-1)).flip(-1)
    before = torch.cat([nothing, h[..., :-1]], -1)
    dv = g * (a * a / m.clamp_min(1e-30) * gate * x - a * before)
    if s["reset"] is not None:
        dv = torch.where(s["reset"][:, None, :], 0.0, dv)
    dgate = g * m * x * gate * (1.0 - gate)
    rate = C * torch.log1p(torch.exp(s["lam"]))
    dr = dv * v * (1.0 - v / rate[:, None])
    dlam = (dv * v).sum(dim=(0, 2)) * C * torch.sigmoid(s["lam"]) / rate
    return (y.to(io), (g * m * gate).to(io), dr.to(io), dgate.to(io), dlam, dr.sum(dim=(0, 2)),
            dgate.sum(dim=(0, 2))) + dz


def _plain_step(s):
    _, a, m, gate = _coefficients(s, False)
    h = a * s["h"] + m * gate * s["x"].float()
    y = h if s["z"] is None else h * (s["z"].float() * torch.sigmoid(s["z"].float()))
    return y.to(s["x"].dtype), h


def _to_elements(x):
    """(exponents [..., padded / 32], elements [..., padded]) of fp32 rows of whole groups."""
    blocks = x.view(*x.shape[:-1], -1, BLOCK)
    top = blocks.abs().amax(dim=-1)
    exponent = (torch.frexp(top).exponent - 3).clamp_min(-127)  # top = f 2^n, f in [1/2, 1)
    exponent = torch.where(top > 0, exponent, -127)
    y = torch.ldexp(blocks, -exponent.unsqueeze(-1))
    size = y.abs()
    step = torch.where(size < 2.0, 0.5, torch.where(size < 4.0, 1.0, 2.0))
    size = (torch.round(size / step) * step).clamp_max(6.0)  # round: ties to even
    return exponent, torch.copysign(size, y).view(x.shape)


def _plain_quantize(s):
    x = s["x"].float()
    x = x if s["order"] == "token" else x.transpose(1, 2)
    width = s["width"]
    x = torch.nn.functional.pad(x, (0, -width % GROUP))
    exponent, elements = _to_elements(x)
    values = torch.ldexp(elements.view(*exponent.shape, BLOCK), exponent.unsqueeze(-1))
    values = values.view(x.shape)[..., :width].to(torch.bfloat16)
    return values, torch.exp2(_scale_layout(exponent.float()))


def _unpack(q, scale):
    """Packed rows and their scales as fp32 values."""
    table = torch.tensor(VALUES + [-v for v in VALUES], device=q.device)
    elements = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1).view(*q.shape[:-1], -1, BLOCK)
    exponent = scale.movedim(0, -2).reshape(*q.shape[:-1], -1).float() - 127.0
    return (elements * torch.exp2(exponent).unsqueeze(-1)).view(*q.shape[:-1], -1)


def _plain_matmul(s):
    a, b = _unpack(s["a"], s["a_scale"]), _unpack(s["b"], s["b_scale"])
    return torch.matmul(a, b.transpose(-1, -2)).to(TYPES[s["out"]])


_PLAIN = {"scan": _plain_scan, "train": _plain_train, "step": _plain_step,
          "quantize": _plain_quantize, "matmul": _plain_matmul}


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    size = {"bf16": 2, "f32": 4}
    op = case["op"]
    if op in MOST:
        b, d, n = case["batch"], case["channels"], case["batch"] * case["channels"] * case["length"]
        io, gate = size[case["io"]], 1 if case["gate"] else 0
        marks = b * case["length"] if case["packed"] else 0
        if op == "train":  # x, r, i, dout (z) in; y, dx, dr, di (dz) out
            return {"bytes": n * io * (8 + 2 * gate) + 24 * d + marks, "flops": n * (70 + 15 * gate)}
        # x, r, i (z) in, y out; the state in and out; three parameters a channel
        return {"bytes": n * io * (4 + gate) + 8 * b * d + 12 * d + marks, "flops": n * (30 + 5 * gate)}
    if op == "quantize":  # the 4-bit rows are written, then read back as values in bf16
        rows, width = case["batch"] * case["length"], case["width"]
        groups = -(-width // GROUP)
        return {"bytes": rows * (width * (size[case["io"]] + 2) + 2 * groups * (GROUP // 2 + 8) + 32 * groups),
                "flops": 4 * rows * width}
    b, m, n, k = case["batch"], case["m"], case["n"], case["k"]
    rows = m * (1 if case["shared"] == "a" else b) + n * (1 if case["shared"] == "b" else b)
    return {"bytes": rows * (-(-k // BLOCK)) * (BLOCK // 2 + 1) + b * m * n * size[case["out"]],
            "flops": 2 * b * m * n * k}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantised(s)
    if op == "matmul":
        values = [_exact_values(s[n], s[n + "_scale"]) for n in ("a", "b")]
        return values[0] @ values[1].mT
    lead = s["x"].shape[:2]
    rows = lead[0] * lead[1]

    def steps(t):  # [B, D, L] -> [L, B * D] in 64 bits: one row a step
        return None if t is None else t.reshape(rows, -1).t().to(torch.float64).contiguous()

    def channels(t):
        return t.to(torch.float64).repeat(lead[0])

    lam = channels(s["lam"])
    softplus = torch.nn.functional.softplus(lam, threshold=1000.0)
    gate_r = 1 / (1 + torch.exp(-(steps(s["r"]) + channels(s["r_bias"]))))
    v = C * softplus * gate_r
    gate_i = 1 / (1 + torch.exp(-(steps(s["i"]) + channels(s["i_bias"]))))
    a = torch.exp(-v)
    m = torch.sqrt(-torch.expm1(-2 * v))
    first = None
    if s.get("reset") is not None:
        first = s["reset"].t().repeat_interleave(lead[1], dim=1)  # [L, B * D]
        a.masked_fill_(first, 0.0)
        m.masked_fill_(first, 1.0)
    x = steps(s["x"])
    into = m * gate_i * x
    h0 = s["h"] if op == "step" else s.get("h0")
    state = torch.zeros(rows, dtype=torch.float64, device=a.device) if h0 is None else h0.reshape(-1).double()
    h = into
    for t in range(h.shape[0]):  # h_t = a_t h_(t-1) + b_t, step by step in place
        state = h[t].addcmul_(a[t], state)
    z = steps(s["z"])
    shape = lambda t: t.t().reshape(s["x"].shape)  # noqa: E731
    silu = None if z is None else z / (1 + torch.exp(-z))
    y = h if z is None else h * silu
    if op != "train":
        return shape(y), h[-1].view(lead)
    dout = steps(s["dout"])
    g = dout.clone() if z is None else dout * silu
    for t in range(g.shape[0] - 2, -1, -1):
        g[t].addcmul_(a[t + 1], g[t + 1])
    # h_t depends on v_t by a (da/dv = -a) and by m (dm/dv = a^2 / m)
    dm = g * gate_i * x
    da = torch.zeros_like(g)
    da[1:] = g[1:] * h[:-1]
    dv = torch.where(m > 0, dm * a.square() / m, 0.0) - da * a
    if first is not None:
        dv.masked_fill_(first, 0.0)
    dr = dv * v * (1 - gate_r)
    di = g * m * x * gate_i * (1 - gate_i)
    total = lambda t: t.sum(dim=0).view(lead).sum(dim=0)  # noqa: E731
    dlam = total(dv * C * gate_r) / (1 + torch.exp(-s["lam"].double()))
    out = (shape(y), shape(g * m * gate_i), shape(dr), shape(di), dlam, total(dr), total(di))
    if z is None:
        return out
    sz = 1 / (1 + torch.exp(-z))
    return out + (shape(dout * h * (sz + z * sz * (1 - sz))),)


def _exact_values(q, scale):
    """Sign, exponent and fraction of each 4-bit element, times its block's power of two."""
    nibbles = torch.stack([q.bitwise_and(15), q.bitwise_right_shift(4)], dim=-1).flatten(-2).long()
    power, half = nibbles.bitwise_right_shift(1).bitwise_and(3), nibbles.bitwise_and(1).double()
    size = torch.where(power > 0, (1 + half / 2) * 2.0 ** (power - 1).double(), half / 2)
    size = torch.where(nibbles >= 8, -size, size)
    exponents = scale.double().sub(127).movedim(0, -2).flatten(-2)
    return size * torch.pow(2.0, exponents).repeat_interleave(BLOCK, dim=-1)


def _exact_quantised(s):
    x = s["x"].double()
    x = x if s["order"] == "token" else x.permute(0, 2, 1)
    width = x.shape[-1]
    groups = -(-width // GROUP)
    full = torch.zeros((*x.shape[:-1], groups * GROUP), dtype=torch.float64, device=x.device)
    full[..., :width] = x
    blocks = full.unflatten(-1, (-1, BLOCK))
    top = torch.linalg.vector_norm(blocks, ord=math.inf, dim=-1)
    exponent = torch.floor(torch.log2(top.clamp_min(1e-300)))
    exponent += (torch.pow(2.0, exponent + 1) <= top).double() - (torch.pow(2.0, exponent) > top).double()
    scale = torch.pow(2.0, (exponent - 2).clamp_min(-127.0))
    y = blocks / scale.unsqueeze(-1)
    # nearest of the values, ties to the one with an even code: counted by the borders passed
    size, code = y.abs(), torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    for place, border in enumerate(BORDERS):
        code += (size > border) if place % 2 == 0 else (size >= border)
    values = torch.tensor(VALUES, dtype=torch.float64, device=y.device)[code.int()] * torch.sign(y)
    values = (values * scale.unsqueeze(-1)).flatten(-2)[..., :width]
    return values, scale.unflatten(-1, (groups, 8)).movedim(-2, 0)
