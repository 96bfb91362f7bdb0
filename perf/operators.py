"""Workloads of the norm, activation-checkpoint and weight-gradient operators.

Each case is one pass of one operator (or of the few that a training step
calls in a row), in the plain form of elementary torch operations or, where
``own`` is true, through the package's entry points.

Checkpoint format: 8-bit codes [T][ldc] (E4M3 or E5M2, ldc = d rounded up to
32) and one power-of-two scale per token and 32 columns, held as the biased
exponent e in bscales [ceil(T / 8)][ldc / 32][8] (the last index is the token
within its group of eight).  e is the smallest integer >= 32 with
amax <= FMAX 2^(e - 127); a value is code 2^(e - 127).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def listed():
    return [
        # one token of a decoding step, width of the 600M-class model: launch latency
        {"name": "norm_fwd_token", "op": "norm_fwd", "T": 1, "d": 1536, "dtype": "bf16", "kind": "rms"},
        # a short prompt in fp32 with an odd row length (no row but the first is aligned)
        {"name": "norm_fwd_odd", "op": "norm_fwd", "T": 1000, "d": 1023, "dtype": "fp32", "kind": "layer"},
        # the training batch of the 600M-class layer (8 sequences of 2048 tokens)
        {"name": "norm_fwd_batch", "op": "norm_fwd", "T": 16384, "d": 1536, "dtype": "bf16", "kind": "layer"},
        # a micro-batch of 256 tokens at the 300M-class width, fp16
        {"name": "norm_bwd_micro", "op": "norm_bwd", "T": 256, "d": 1024, "dtype": "fp16", "kind": "layer"},
        # a training batch at the stress width
        {"name": "norm_bwd_wide", "op": "norm_bwd", "T": 8192, "d": 4096, "dtype": "bf16", "kind": "rms"},
        # forward keeping the input in 8 bits, then backward from it: one norm of a training step
        {"name": "norm_step_batch", "op": "norm_step", "T": 16384, "d": 1536, "dtype": "bf16", "kind": "layer",
         "fmt": "e4m3"},
        # a ragged fp32 activation (config 1 keeps fp32 activations), E5M2
        {"name": "act_odd", "op": "act", "T": 333, "d": 1001, "dtype": "fp32", "fmt": "e5m2"},
        # the input of the 600M-class fc2 layer over a training batch
        {"name": "act_fc2", "op": "act", "T": 16384, "d": 6144, "dtype": "bf16", "fmt": "e4m3"},
        # the smallest layer of the test configurations, fp32 output gradients
        {"name": "wgrad_tiny", "op": "wgrad", "T": 1024, "m": 64, "d": 256, "dtype": "fp32", "fmt": "e4m3"},
        # odd sizes on every axis, fp16 output gradients
        {"name": "wgrad_odd", "op": "wgrad", "T": 1537, "m": 1001, "d": 2731, "dtype": "fp16", "fmt": "e5m2"},
        # the 300M-class fc2 layer over a training batch
        {"name": "wgrad_300m", "op": "wgrad", "T": 8192, "m": 1024, "d": 4096, "dtype": "bf16", "fmt": "e4m3"},
        # the 600M-class fc2 layer: the product that makes the gradient the codec is measured on
        {"name": "wgrad_600m", "op": "wgrad", "T": 16384, "m": 1536, "d": 6144, "dtype": "bf16", "fmt": "e4m3"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi):
    """Half of the widths are multiples of 64, the others anything."""
    n = _log(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_step", "act", "wgrad"])
    c = {"op": op, "T": _log(rng, 1, 16384), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    if op == "wgrad":
        c["m"], c["d"] = _width(rng, 16, 4096), _width(rng, 16, 8192)
        c["T"] = max(16, c["T"])
        while c["T"] * c["m"] * c["d"] > 16384 * 1536 * 6144:
            c["T"] = (c["T"] + 1) // 2
    else:
        c["d"] = _width(rng, 64, 12288)
        while c["T"] * c["d"] * SIZES[c["dtype"]] > 16384 * 6144 * 2:
            c["T"] = (c["T"] + 1) // 2
    if op in ("norm_fwd", "norm_bwd", "norm_step"):
        c["kind"] = rng.choice(["layer", "rms"])
    if op in ("norm_step", "act", "wgrad"):
        c["fmt"] = rng.choice(["e4m3", "e4m3", "e5m2"])
    return c


# -- inputs -----------------------------------------------------------------

def _activation(g, T, d, dtype, dev):
    """Hidden states: columns of different size and offset, a few of them
    twenty times as large, and tokens of different size."""
    col = torch.exp(0.5 * torch.randn(d, generator=g, device=dev))
    col = torch.where(torch.rand(d, generator=g, device=dev) < 0.005, 20 * col, col)
    tok = torch.exp(0.3 * torch.randn(T, 1, generator=g, device=dev))
    off = 0.2 * torch.randn(d, generator=g, device=dev)
    x = torch.randn(T, d, generator=g, device=dev)
    return x.mul_(col).mul_(tok).add_(off).to(dtype)


def _gradient(g, T, m, dtype, dev):
    """Output gradients: small, tokens of different size."""
    tok = 0.05 * torch.exp(0.7 * torch.randn(T, 1, generator=g, device=dev))
    return torch.randn(T, m, generator=g, device=dev).mul_(tok).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op, T, d, dt = case["op"], case["T"], case["d"], DTYPES[case["dtype"]]
    s = dict(case)
    if op == "wgrad":
        s["delta"] = _gradient(g, T, case["m"], dt, dev)
        # what the forward pass kept: the checkpoint of a bf16 activation
        s["codes"], s["bscales"] = _pack(_activation(g, T, d, torch.bfloat16, dev), case["fmt"])
        return s
    s["x"] = _activation(g, T, d, dt, dev)
    if op == "act":
        return s
    s["weight"] = (1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(dt)
    s["bias"] = (0.1 * torch.randn(d, generator=g, device=dev)).to(dt) if case["kind"] == "layer" else None
    if op != "norm_fwd":
        s["dy"] = _gradient(g, T, d, dt, dev)
    if op == "norm_bwd":
        # what the forward pass kept
        s["mean"], s["rstd"] = _moments(s["x"].float(), case["kind"])
    return s


def work(case):
    T, d, n = case["T"], case["d"], SIZES[case["dtype"]]
    op = case["op"]
    ck = T * d + T * -(-d // 32)
    if op == "wgrad":
        m = case["m"]
        return {"bytes": T * m * n + ck + 4 * m * d, "flops": 2 * m * d * T}
    if op == "act":
        return {"bytes": 2 * T * d * n + 2 * ck, "flops": 4 * T * d}
    layer = case["kind"] == "layer"
    stats = 4 * T * (2 if layer else 1)
    w = d * n * (2 if layer else 1)
    fwd = {"bytes": 2 * T * d * n + stats + w, "flops": 8 * T * d}
    bwd = {"bytes": 3 * T * d * n + stats + d * n + 4 * d * (2 if layer else 1), "flops": 14 * T * d}
    if op == "norm_fwd":
        return fwd
    if op == "norm_bwd":
        return bwd
    # x read once by the forward; the backward reads the checkpoint instead
    return {"bytes": fwd["bytes"] + bwd["bytes"] - T * d * n + 2 * ck, "flops": fwd["flops"] + bwd["flops"] + 4 * T * d}


# -- the plain form -----------------------------------------------------------

FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _exponent(amax, fmt):
    """Smallest e >= 32 with amax <= FMAX 2^(e - 127).  frexp: amax = f 2^p
    with f in [0.5, 1), and FMAX = 0.875 2^(9 or 16)."""
    f, p = torch.frexp(amax)
    e = p - (9 if fmt == "e4m3" else 16) + (f > 0.875).to(torch.int32) + 127
    return torch.where(amax > 0, e, torch.zeros_like(e)).clamp_(min=32)


def _pack(x, fmt):
    """Codes [T][ldc] and bscales [ceil(T / 8)][ldc / 32][8] of finite x."""
    T, d = x.shape
    nb = -(-d // 32)
    u = torch.nn.functional.pad(x.float(), (0, nb * 32 - d)).view(T, nb, 32)
    e = _exponent(u.abs().amax(2), fmt)
    q = torch.ldexp(u, (127 - e).unsqueeze(2))
    codes = q.to(FP8[fmt]).view(torch.uint8).view(T, nb * 32)
    b = torch.nn.functional.pad(e.to(torch.uint8), (0, 0, 0, -T % 8))
    return codes, b.view(-1, 8, nb).transpose(1, 2).contiguous()


def _unpack(codes, bscales, T, d, fmt):
    nb = bscales.shape[1]
    e = bscales.transpose(1, 2).reshape(-1, nb)[:T].to(torch.int32) - 127
    v = codes.view(FP8[fmt]).float().view(T, nb, 32)
    return torch.ldexp(v, e.unsqueeze(2)).view(T, nb * 32)[:, :d]


def _moments(x, kind):
    mean = x.mean(1) if kind == "layer" else None
    c = x - mean.unsqueeze(1) if kind == "layer" else x
    return mean, (c.square().mean(1) + EPS).rsqrt()


def _normal(x, mean, rstd):
    c = x if mean is None else x - mean.unsqueeze(1)
    return c * rstd.unsqueeze(1)


def _forward(x, weight, bias, kind):
    u = x.float()
    mean, rstd = _moments(u, kind)
    y = _normal(u, mean, rstd) * weight.float()
    if bias is not None:
        y = y + bias.float()
    return y.to(x.dtype), mean, rstd


def _backward(dy, x, mean, rstd, weight):
    xh = _normal(x, mean, rstd)
    t = dy.float()
    g = t * weight.float()
    r = g - xh * (g * xh).mean(1, keepdim=True)
    if mean is not None:
        r = r - g.mean(1, keepdim=True)
    dx = (r * rstd.unsqueeze(1)).to(dy.dtype)
    return dx, (t * xh).sum(0), t.sum(0) if mean is not None else None


def _plain(s):
    op = s["op"]
    if op == "wgrad":
        a = _unpack(s["codes"], s["bscales"], s["T"], s["d"], s["fmt"])
        return {"dW": (s["delta"].float().t() @ a) * (1.0 / s["T"])}
    if op == "act":
        codes, bscales = _pack(s["x"], s["fmt"])
        return {"x": _unpack(codes, bscales, s["T"], s["d"], s["fmt"]).to(s["x"].dtype)}
    out = {}
    if op in ("norm_fwd", "norm_step"):
        out["y"], mean, rstd = _forward(s["x"], s["weight"], s["bias"], s["kind"])
        out["mean"], out["rstd"] = mean, rstd
    if op == "norm_bwd":
        out["dx"], out["dweight"], out["dbias"] = _backward(s["dy"], s["x"].float(), s["mean"], s["rstd"], s["weight"])
    if op == "norm_step":
        codes, bscales = _pack(s["x"], s["fmt"])
        x = _unpack(codes, bscales, s["T"], s["d"], s["fmt"])
        out["dx"], out["dweight"], out["dbias"] = _backward(s["dy"], x, mean, rstd, s["weight"])
    return out


# -- the package's entry points -------------------------------------------------

def _own(s):
    import fac_whitening_amd as fw

    op = s["op"]
    if op == "wgrad":
        ck = fw.ActCheckpoint(s["T"], s["d"], s["fmt"], codes=s["codes"], bscales=s["bscales"])
        return {"dW": fw.weight_grad(s["delta"], ck, alpha=1.0 / s["T"])}
    if op == "act":
        ck = fw.ActCheckpoint(s["T"], s["d"], s["fmt"], device=s["x"].device)
        ck.save(s["x"])
        return {"x": ck.restore(s["x"].dtype)}
    if op == "norm_bwd":
        dx, dw, db = fw.norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], kind=s["kind"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    ck = fw.ActCheckpoint(s["T"], s["d"], s["fmt"], device=s["x"].device) if op == "norm_step" else None
    y, mean, rstd = fw.norm_forward(s["x"], s["weight"], s["bias"], eps=EPS, kind=s["kind"], ckpt=ck)
    out = {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_step":
        out["dx"], out["dweight"], out["dbias"] = fw.norm_backward(s["dy"], ck, mean, rstd, s["weight"],
                                                                  kind=s["kind"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# -- 64 bits, from the definitions -----------------------------------------------

def _values64(fmt):
    """Value of each of the 256 codes, from the format's fields."""
    eb, mb, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    out = []
    for c in range(256):
        e, f = (c & 127) >> mb, c & ((1 << mb) - 1)
        v = math.ldexp(f, 1 - bias - mb) if e == 0 else math.ldexp((1 << mb) + f, e - bias - mb)
        if e == (1 << eb) - 1 and (fmt == "e5m2" or f == (1 << mb) - 1):
            v = math.inf if fmt == "e5m2" and f == 0 else math.nan
        out.append(-v if c & 128 else v)
    return out


def _stored64(x, fmt):
    """The values a checkpoint of x stands for: x rounded to the format's
    grid under its block's scale."""
    T, d = x.shape
    mb, low, top = (3, -6, 8) if fmt == "e4m3" else (2, -14, 15)
    v = torch.nn.functional.pad(x.double(), (0, -d % 32)).view(T, -1, 32)
    amax = v.abs().amax(2, keepdim=True)
    # scale 2^k: amax / 2^k in (FMAX / 2, FMAX], FMAX = 1.75 2^top
    k = torch.ceil(torch.log2(amax / 1.75)) - top
    k = torch.where(amax > torch.exp2(k + top) * 1.75, k + 1, k)
    k = torch.where(amax <= torch.exp2(k - 1 + top) * 1.75, k - 1, k)
    k = torch.where(amax > 0, k, torch.full_like(k, -95.0)).clamp(min=-95.0)
    w = v / torch.exp2(k)
    # spacing of the grid around w
    p = torch.floor(torch.log2(w.abs().clamp(min=2.0 ** low))).clamp(min=low)
    p = torch.where(w.abs() >= torch.exp2(p + 1), p + 1, p)
    h = torch.exp2(p - mb)
    return (torch.round(w / h) * h * torch.exp2(k)).view(T, -1)[:, :d]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "wgrad":
        T, d = s["T"], s["d"]
        lut = torch.tensor(_values64(s["fmt"]), dtype=torch.float64, device=s["codes"].device)
        col = torch.arange(d, device=s["codes"].device)
        tok = torch.arange(T, device=s["codes"].device)
        e = s["bscales"][tok[:, None] // 8, col[None, ::32] // 32, tok[:, None] % 8].double() - 127
        a = lut[s["codes"][:, :d].int()] * torch.exp2(e).repeat_interleave(32, 1)[:, :d]
        return {"dW": torch.mm(s["delta"].double().t(), a) / T}
    x = s["x"].double()
    if op == "act":
        return {"x": _stored64(s["x"], s["fmt"])}
    d, w = s["d"], s["weight"].double()
    layer = s["kind"] == "layer"
    out = {}
    if op == "norm_bwd":
        mean, rstd = s["mean"], s["rstd"].double()
        mean = mean.double() if layer else torch.zeros_like(rstd)
    else:
        mean = x.sum(1) / d if layer else torch.zeros(s["T"], dtype=torch.float64, device=x.device)
        rstd = 1.0 / torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / d + EPS)
        y = (x - mean[:, None]) * rstd[:, None] * w
        out = {"y": y + s["bias"].double() if layer else y, "mean": mean if layer else None, "rstd": rstd}
    if op == "norm_fwd":
        return out
    if op == "norm_step":
        x = _stored64(s["x"], s["fmt"])
    t = s["dy"].double()
    xh = (x - mean[:, None]) * rstd[:, None]
    g = t * w
    dx = g - xh * ((g * xh).sum(1) / d)[:, None]
    if layer:
        dx = dx - (g.sum(1) / d)[:, None]
    out["dx"] = dx * rstd[:, None]
    out["dweight"] = (t * xh).sum(0)
    out["dbias"] = t.sum(0) if layer else None
    return out
