"""The cases on which the gated feed-forward operators and the 4-bit matrix-vector operators are measured.

Four operators:

  gated_f16            H = act(X Wg^T) * (X Wu^T), 16-bit operands; for training it also returns G = X Wg^T and U = X Wu^T
  gated_f16_backward   dX, dWg, dWu from dH and what the forward pass kept
  gemv_fp4             Y = X W^T for up to 16 rows of X, W in MXFP4 or NVFP4 (the tables that quantize_fp4 writes)
  gated_gemv_fp4       H = act(X Wg^T) * (X Wu^T) for up to 16 rows of X, both weights in MXFP4 or NVFP4

With `own` false, run() computes them in elementary torch operations in 32 bits; with `own` true it calls this
package.  The gated_f16 weights are (inter, hidden), X is (tokens, hidden); gemv_fp4 weights are (rows, cols).
"""
import math

import torch

own = False

BF16, F16 = "bf16", "fp16"


# --------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token through an expert's gate and up projections (the 7168 x 2048 expert shape of the benchmark): the
        # smallest call, bound by reading the weights and by latency
        _gated("gated_1_token", 1, 7168, 2048, BF16, "silu", False),
        # a short prompt, sizes that fill no tile
        _gated("gated_331_tokens_odd", 331, 1800, 2744, F16, "gelu_tanh", False),
        # a training step's forward pass, keeping G and U
        _gated("gated_8192_tokens_train", 8192, 7168, 2048, BF16, "silu", True),
        # gradients of a small batch, sizes that fill no tile
        _backward("backward_67_tokens_odd", 67, 2048, 1368, F16, "gelu_tanh"),
        # gradients of an expert that was sent few of a batch's tokens
        _backward("backward_1000_tokens", 1000, 4096, 4096, BF16, "silu"),
        # a training step's backward pass
        _backward("backward_4096_tokens_train", 4096, 7168, 2048, BF16, "silu"),
        # one token through an expert's down projection: the smallest 4-bit call
        _gemv("gemv_nv_1_token_down", 1, 7168, 2048, "nv", BF16),
        # one token through a square projection (the benchmark's 7168 x 7168)
        _gemv("gemv_mx_1_token_square", 1, 7168, 7168, "mx", BF16),
        # a batch of 16 sequences through an output layer
        _gemv("gemv_nv_16_tokens_wide", 16, 32768, 7168, "nv", BF16),
        # one token through an expert's gate and up projections in 4 bits
        _gated_gemv("gated_gemv_mx_1_token", 1, 7168, 2048, "mx", BF16, "silu"),
        # a few drafted tokens, odd sizes
        _gated_gemv("gated_gemv_nv_5_tokens_odd", 5, 1856, 1501, "nv", F16, "gelu_tanh"),
        # a batch of 8 sequences through a wide dense block
        _gated_gemv("gated_gemv_mx_8_tokens_wide", 8, 7168, 16384, "mx", BF16, "silu"),
    ]


def _gated(name, tokens, hidden, inter, dtype, act, save):
    return {"name": name, "op": "gated_f16", "tokens": tokens, "hidden": hidden, "inter": inter, "dtype": dtype, "act": act, "save": save}


def _backward(name, tokens, hidden, inter, dtype, act):
    return {"name": name, "op": "gated_f16_backward", "tokens": tokens, "hidden": hidden, "inter": inter, "dtype": dtype, "act": act}


def _gemv(name, tokens, rows, cols, fmt, dtype):
    return {"name": name, "op": "gemv_fp4", "tokens": tokens, "rows": rows, "cols": cols, "fmt": fmt, "dtype": dtype}


def _gated_gemv(name, tokens, hidden, inter, fmt, dtype, act):
    return {"name": name, "op": "gated_gemv_fp4", "tokens": tokens, "hidden": hidden, "inter": inter, "fmt": fmt, "dtype": dtype, "act": act}


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9))))


def draw(rng):
    """One more case.  16-bit rows are multiples of 8 elements, 4-bit rows of 64 (what the formats need); the rest is any number."""
    op = rng.choice(["gated_f16", "gated_f16_backward", "gemv_fp4", "gated_gemv_fp4"])
    dtype, act, fmt = rng.choice([BF16, F16]), rng.choice(["silu", "gelu_tanh"]), rng.choice(["mx", "nv"])
    if op.startswith("gated_f16"):
        hidden, inter = 8 * _spread(rng, 32, 1024), 8 * _spread(rng, 16, 1024)
        most = 8192 * 7168 * 2048 // (2 if op.endswith("backward") else 1)
        tokens = _spread(rng, 1, max(1, min(8192, most // (hidden * inter))))
        if op == "gated_f16":
            return _drawn(_gated(None, tokens, hidden, inter, dtype, act, rng.random() < 0.5))
        return _drawn(_backward(None, tokens, hidden, inter, dtype, act))
    tokens, cols = rng.randint(1, 16), 64 * _spread(rng, 4, 256)
    if op == "gemv_fp4":
        return _drawn(_gemv(None, tokens, _spread(rng, 64, min(32768, 32768 * 7168 // cols)), cols, fmt, dtype))
    return _drawn(_gated_gemv(None, tokens, cols, _spread(rng, 64, min(16384, 16384 * 7168 // cols)), fmt, dtype, act))


def _drawn(case):
    del case["name"]
    return case


# --------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float16


def _normal(gen, shape, scale, dtype, outliers=False):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if outliers:  # a few large channels, as activations have
        x[:, torch.randint(0, shape[1], (max(1, shape[1] // 512),), generator=gen, device="cuda")] *= 20.0
    return (x * scale).to(dtype)


def _quantized(gen, rows, cols, fmt):
    """Normal weights in the layout of quantize_fp4: codes uint8 (rows, cols / 2), scales int32 (ceil(groups / 4), rows padded to 4)."""
    sv = 32 if fmt == "mx" else 16
    w = torch.randn((rows, cols // sv, sv), generator=gen, device="cuda", dtype=torch.float32) / math.sqrt(cols)
    w *= torch.exp2(torch.randn((rows, 1, 1), generator=gen, device="cuda"))  # rows of unlike size
    want = w.abs().amax(-1, keepdim=True) / 6.0
    if fmt == "mx":
        e = torch.ceil(torch.log2(want)).clamp(-127, 127)
        scale, byte = torch.exp2(e), (e + 127).to(torch.uint8)
    else:
        q = want.to(torch.float8_e4m3fn)
        scale, byte = q.float(), q.view(torch.uint8)
    r = w / scale.clamp_min(1e-30)
    steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(r.abs(), steps).to(torch.uint8) + 8 * (r < 0).to(torch.uint8)
    code = code.view(rows, cols // 2, 2)
    packed = (code[..., 0] + 16 * code[..., 1]).contiguous()
    words = (cols // sv + 3) // 4
    table = torch.zeros((words, (rows + 3) // 4 * 4, 4), dtype=torch.uint8, device="cuda")
    per_row = torch.zeros((rows, words * 4), dtype=torch.uint8, device="cuda")
    per_row[:, : cols // sv] = byte.view(rows, -1)
    table[:, :rows] = per_row.view(rows, words, 4).permute(1, 0, 2)
    return packed, table.view(torch.int32).squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    dt = _dtype(case)
    if case["op"] in ("gated_f16", "gated_f16_backward"):
        t, h, i = case["tokens"], case["hidden"], case["inter"]
        st["x"] = _normal(gen, (t, h), 1.0, dt, outliers=True)
        st["wg"] = _normal(gen, (i, h), 1.0 / math.sqrt(h), dt)
        st["wu"] = _normal(gen, (i, h), 1.0 / math.sqrt(h), dt)
        if case["op"] == "gated_f16_backward":
            # what the forward pass kept, and a gradient of the size that a mean loss sends back
            st["g"], st["u"] = st["x"] @ st["wg"].t(), st["x"] @ st["wu"].t()
            st["dh"] = _normal(gen, (t, i), 0.05, dt)
        return st
    rows, cols = (case["rows"], case["cols"]) if case["op"] == "gemv_fp4" else (case["inter"], case["hidden"])
    st["x"] = _normal(gen, (case["tokens"], cols), 1.0, dt, outliers=True)
    if case["op"] == "gemv_fp4":
        st["wq"], st["sf"] = _quantized(gen, rows, cols, case["fmt"])
    else:
        st["wgq"], st["sfg"] = _quantized(gen, rows, cols, case["fmt"])
        st["wuq"], st["sfu"] = _quantized(gen, rows, cols, case["fmt"])
    return st


# --------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    return _own(case, st) if own else _plain(case, st)


def _own(case, st):
    import fine_grained_fp8_persistent_gb300 as fg
    if case["op"] == "gated_f16":
        return fg.gated_f16(st["x"], st["wg"], st["wu"], case["act"], save=case["save"])
    if case["op"] == "gated_f16_backward":
        return fg.gated_f16_backward(st["dh"], st["x"], st["wg"], st["wu"], st["g"], st["u"], case["act"])
    if case["op"] == "gemv_fp4":
        return fg.gemv_fp4(st["x"], st["wq"], st["sf"], case["fmt"])
    return fg.gated_gemv_fp4(st["x"], st["wgq"], st["sfg"], st["wuq"], st["sfu"], case["fmt"], case["act"])


_GELU_A, _GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(_GELU_A * (g + _GELU_B * g * g * g)))


def _act_slope(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    t = torch.tanh(_GELU_A * (g + _GELU_B * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _GELU_A * (1.0 + 3.0 * _GELU_B * g * g)


def _weights32(packed, table, fmt):
    """The values of a quantize_fp4 matrix in 32 bits, by arithmetic on the codes and the scale bytes."""
    rows, cols = packed.shape[0], 2 * packed.shape[1]
    code = torch.stack((packed & 15, packed >> 4), dim=-1).view(rows, cols).int()
    e, m = (code >> 1) & 3, (code & 1).float()
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(e.float() - 1.0))
    value = torch.where(code > 7, -mag, mag)
    sv = 32 if fmt == "mx" else 16
    byte = table.view(torch.uint8).view(table.shape[0], table.shape[1], 4)[:, :rows].permute(1, 0, 2).reshape(rows, -1)[:, : cols // sv].int()
    if fmt == "mx":
        scale = torch.exp2(byte.float() - 127.0)
    else:
        se, sm = byte >> 3, (byte & 7).float()
        scale = torch.where(se == 0, sm * 2.0 ** -9, (1.0 + sm / 8.0) * torch.exp2(se.float() - 7.0))
    return (value.view(rows, cols // sv, sv) * scale.unsqueeze(-1)).view(rows, cols)


def _plain(case, st):
    dt, x = _dtype(case), st["x"].float()
    if case["op"] == "gated_f16":
        g, u = x @ st["wg"].float().t(), x @ st["wu"].float().t()
        h = (_act(g, case["act"]) * u).to(dt)
        return (h, g.to(dt), u.to(dt)) if case["save"] else h
    if case["op"] == "gated_f16_backward":
        g, u, dh = st["g"].float(), st["u"].float(), st["dh"].float()
        dg, du = dh * u * _act_slope(g, case["act"]), dh * _act(g, case["act"])
        dx = dg @ st["wg"].float() + du @ st["wu"].float()
        return dx.to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
    if case["op"] == "gemv_fp4":
        return (x @ _weights32(st["wq"], st["sf"], case["fmt"]).t()).to(dt)
    g = x @ _weights32(st["wgq"], st["sfg"], case["fmt"]).t()
    u = x @ _weights32(st["wuq"], st["sfu"], case["fmt"]).t()
    return (_act(g, case["act"]) * u).to(dt)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    t = case["tokens"]
    if case["op"] in ("gated_f16", "gated_f16_backward"):
        h, i = case["hidden"], case["inter"]
        if case["op"] == "gated_f16":
            return {"bytes": 2 * (t * h + 2 * i * h + t * i * (3 if case["save"] else 1)), "flops": 4 * t * h * i}
        return {"bytes": 2 * (3 * t * i + 2 * t * h + 4 * i * h), "flops": 8 * t * h * i}
    mats = 1 if case["op"] == "gemv_fp4" else 2
    rows, cols = (case["rows"], case["cols"]) if mats == 1 else (case["inter"], case["hidden"])
    scales = rows * cols // (32 if case["fmt"] == "mx" else 16)
    return {"bytes": mats * (rows * cols // 2 + scales) + 2 * t * (rows + cols), "flops": 2 * mats * t * rows * cols}


# --------------------------------------------------------------------------- the definition in 64 bits
def _weights64(packed, table, fmt):
    """The values of a quantize_fp4 matrix by table, in 64 bits."""
    e2m1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    values = torch.tensor(e2m1 + [-v for v in e2m1], dtype=torch.float64, device="cuda")
    pairs = torch.stack((values.repeat(16), values.repeat_interleave(16)), dim=-1)  # both elements of each byte
    rows = packed.shape[0]
    w = pairs[packed.long()].view(rows, -1)
    sv = 32 if fmt == "mx" else 16
    if fmt == "mx":
        scales = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), torch.arange(256, dtype=torch.float64, device="cuda") - 127)
    else:
        scales = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    groups = w.shape[1] // sv
    k = torch.arange(groups, device="cuda")
    words = table[(k // 4).unsqueeze(0), torch.arange(rows, device="cuda").unsqueeze(1)].long()
    byte = (words >> (8 * (k % 4)).unsqueeze(0)) & 255
    return w.view(rows, groups, sv).mul_(scales[byte].unsqueeze(-1)).view(rows, -1)


def _act64(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return g * torch.sigmoid(2.0 * _GELU_A * (g + _GELU_B * g ** 3))  # (1 + tanh z) / 2 is sigmoid(2 z)


def _slope64(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return s + g * s * (1.0 - s)
    s = torch.sigmoid(2.0 * _GELU_A * (g + _GELU_B * g ** 3))
    return s + g * s * (1.0 - s) * 2.0 * _GELU_A * (1.0 + 3.0 * _GELU_B * g ** 2)


def exact(case, seed):
    st = prepare(case, seed)
    x = st["x"].double()
    if case["op"] == "gated_f16":
        g, u = torch.mm(x, st["wg"].double().t()), torch.mm(x, st["wu"].double().t())
        h = _act64(g, case["act"]) * u
        return (h, g, u) if case["save"] else h
    if case["op"] == "gated_f16_backward":
        g, u, dh = st["g"].double(), st["u"].double(), st["dh"].double()
        dg, du = dh * u * _slope64(g, case["act"]), dh * _act64(g, case["act"])
        dx = torch.mm(dg, st["wg"].double()) + torch.mm(du, st["wu"].double())
        return dx, torch.mm(dg.t(), x), torch.mm(du.t(), x)
    if case["op"] == "gemv_fp4":
        return torch.mm(x, _weights64(st["wq"], st["sf"], case["fmt"]).t())
    g = torch.mm(x, _weights64(st["wgq"], st["sfg"], case["fmt"]).t())
    u = torch.mm(x, _weights64(st["wuq"], st["sfu"], case["fmt"]).t())
    return _act64(g, case["act"]) * u
