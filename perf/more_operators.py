"""Workloads of the gated feed-forward, dropout and whole-activation
weight-gradient operators.

Each case is one pass of one operator, in the plain form of elementary torch
operations or, where ``own`` is true, through the package's entry points.

    glu_fwd   z = x Wg^T, u = x Wu^T, h = D(act(z) u); z and u are also
              returned where the backward pass will need them ("keep")
    glu_bwd   e = D'(dh): dgate = e u act'(z), dup = e act(z),
              dx = dgate Wg + dup Wu
    wgrad     alpha delta^T x in fp32
    drop_fwd  y = residual + D(x), or D(x)
    drop_bwd  dx = D'(dy)

D keeps element (t, j) of a matrix where its 16 random bits are at least
thr = round(65536 p), and scales it by 65536 / (65536 - thr).  The bits are
half j % 2 of word j % 8 / 2 of Philox4x32-10 (Salmon et al., "Parallel random
numbers: as easy as 1, 2, 3", 2011) at the counter (j / 8, t, offset low,
offset high) under the key (seed low, seed high).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]


def listed():
    return [
        # one token of a decoding step, 600M-class widths: latency
        {"name": "glu_token", "op": "glu_fwd", "T": 1, "d": 1536, "f": 6144, "dtype": "bf16", "act": "silu", "p": 0.0,
         "keep": False},
        # sixteen requests decoded together at the stress widths: the weights' bytes
        {"name": "glu_tokens", "op": "glu_fwd", "T": 16, "d": 4096, "f": 16384, "dtype": "bf16", "act": "gelu_tanh",
         "p": 0.0, "keep": False},
        # a short batch of odd sizes in fp16, pre-activations kept
        {"name": "glu_fwd_odd", "op": "glu_fwd", "T": 1000, "d": 1001, "f": 2731, "dtype": "fp16", "act": "gelu",
         "p": 0.0, "keep": True},
        # the training batch of the 600M-class block (8 sequences of 2048 tokens) with hidden dropout
        {"name": "glu_fwd_batch", "op": "glu_fwd", "T": 16384, "d": 1536, "f": 6144, "dtype": "bf16", "act": "silu",
         "p": 0.1, "keep": True},
        # backward of a micro-batch of 256 tokens at the 300M-class widths
        {"name": "glu_bwd_micro", "op": "glu_bwd", "T": 256, "d": 1024, "f": 4096, "dtype": "fp16", "act": "gelu_tanh",
         "p": 0.0},
        # backward in fp32, odd on every axis
        {"name": "glu_bwd_odd", "op": "glu_bwd", "T": 333, "d": 1001, "f": 2731, "dtype": "fp32", "act": "gelu",
         "p": 0.25},
        # backward of the training batch
        {"name": "glu_bwd_batch", "op": "glu_bwd", "T": 16384, "d": 1536, "f": 6144, "dtype": "bf16", "act": "silu",
         "p": 0.1},
        # weight gradient of an odd layer in fp32
        {"name": "wgrad_odd", "op": "wgrad", "T": 1537, "m": 2731, "d": 1001, "dtype": "fp32"},
        # weight gradient of one projection of the training batch
        {"name": "wgrad_batch", "op": "wgrad", "T": 16384, "m": 6144, "d": 1536, "dtype": "bf16"},
        # one token's hidden state onto the residual stream: latency
        {"name": "drop_token", "op": "drop_fwd", "T": 1, "d": 1536, "dtype": "bf16", "p": 0.1, "residual": True},
        # the block's output onto the residual stream over the training batch
        {"name": "drop_fwd_batch", "op": "drop_fwd", "T": 16384, "d": 1536, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # its backward in fp32 over a ragged batch (no row but the first is aligned)
        {"name": "drop_bwd_odd", "op": "drop_bwd", "T": 8191, "d": 1023, "dtype": "fp32", "p": 0.25},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, lo, hi):
    """Half of the widths are multiples of 64, the others anything."""
    n = _log(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["glu_fwd", "glu_fwd", "glu_bwd", "glu_bwd", "wgrad", "drop_fwd", "drop_bwd"])
    c = {"op": op, "T": _log(rng, 1, 16384), "d": _width(rng, 64, 4096), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    if op in ("drop_fwd", "drop_bwd"):
        c["p"] = rng.choice([0.05, 0.1, 0.25, 0.5])
        if op == "drop_fwd":
            c["residual"] = rng.random() < 0.7
        return c
    # half of the work for fp32, whose products cost several times as much
    most = 16384 * 1536 * 6144 // (2 if c["dtype"] == "fp32" else 1)
    n = _width(rng, 64, 16384)
    while c["T"] * c["d"] * n > most or c["T"] * n > 16384 * 6144:
        c["T"] = (c["T"] + 1) // 2
    if op == "wgrad":
        c["m"] = n
        return c
    c["f"], c["act"], c["p"] = n, rng.choice(ACTS + ["silu"]), rng.choice([0.0, 0.0, 0.1, 0.25])
    if op == "glu_fwd":
        c["keep"] = rng.random() < 0.6
    return c


# -- inputs -----------------------------------------------------------------

def _hidden(g, T, d, dtype, dev):
    """Normalised hidden states: rows of about one size, columns of different
    size, a few of them ten times as large."""
    col = torch.exp(0.4 * torch.randn(d, generator=g, device=dev))
    col = torch.where(torch.rand(d, generator=g, device=dev) < 0.003, 10 * col, col)
    return torch.randn(T, d, generator=g, device=dev).mul_(col).to(dtype)


def _gradient(g, T, n, dtype, dev):
    """Output gradients: small, tokens of different size."""
    tok = 0.05 * torch.exp(0.7 * torch.randn(T, 1, generator=g, device=dev))
    return torch.randn(T, n, generator=g, device=dev).mul_(tok).to(dtype)


def _weight(g, m, d, dtype, dev):
    return torch.randn(m, d, generator=g, device=dev).mul_(0.8 * d ** -0.5).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op, T, d, dt = case["op"], case["T"], case["d"], DTYPES[case["dtype"]]
    s = dict(case)
    if case.get("p"):
        # this step's key and draw number; both halves of each are in use
        s["seed"] = (int(seed) * 0x9E3779B97F4A7C15 + 0x1234567) % (1 << 64)
        s["offset"] = (int(seed) * 0xD1B54A32D192ED03 + 11) % (1 << 64)
        if own:
            import fac_whitening_amd as fw
            s["drop"] = fw.Dropout(s["p"], s["seed"], s["offset"])
    if op == "wgrad":
        s["delta"], s["x"] = _gradient(g, T, case["m"], dt, dev), _hidden(g, T, d, dt, dev)
    elif op == "drop_fwd":
        s["x"] = _hidden(g, T, d, dt, dev)
        s["r"] = _hidden(g, T, d, dt, dev).mul_(2) if case["residual"] else None
    elif op == "drop_bwd":
        s["dy"] = _gradient(g, T, d, dt, dev)
    else:
        f = case["f"]
        s["w_gate"], s["w_up"] = _weight(g, f, d, dt, dev), _weight(g, f, d, dt, dev)
        if op == "glu_fwd":
            s["x"] = _hidden(g, T, d, dt, dev)
        else:
            # what the forward pass kept, and the gradient of its output
            s["gate"], s["up"] = (torch.randn(T, f, generator=g, device=dev).mul_(1.2).to(dt) for _ in range(2))
            s["dh"] = _gradient(g, T, f, dt, dev)
    return s


def work(case):
    T, d, n = case["T"], case["d"], SIZES[case["dtype"]]
    op = case["op"]
    if op == "wgrad":
        m = case["m"]
        return {"bytes": T * (m + d) * n + 4 * m * d, "flops": 2 * T * m * d}
    if op == "drop_fwd":
        return {"bytes": T * d * n * (3 if case["residual"] else 2), "flops": 3 * T * d}
    if op == "drop_bwd":
        return {"bytes": 2 * T * d * n, "flops": 2 * T * d}
    f = case["f"]
    if op == "glu_fwd":
        return {"bytes": n * (T * d + 2 * f * d + T * f * (3 if case["keep"] else 1)), "flops": 4 * T * d * f + 8 * T * f}
    return {"bytes": n * (5 * T * f + 2 * f * d + T * d), "flops": 4 * T * d * f + 16 * T * f}


# -- the plain form -----------------------------------------------------------

M32 = 0xFFFFFFFF


def _mulhilo(a, m):
    """High and low 32 bits of a m, a an int64 tensor of 32-bit values."""
    return (a * (m >> 16) + ((a * (m & 0xFFFF)) >> 16)) >> 16, (a * m) & M32


def _keep(T, d, p, seed, offset, dev):
    """[T][d]: whether an element is kept; and the scale."""
    thr = round(65536 * p)
    nb = -(-d // 8)
    c0 = torch.arange(nb, device=dev).expand(T, nb)
    c1 = torch.arange(T, device=dev).unsqueeze(1).expand(T, nb)
    c2 = torch.full((T, nb), offset & M32, device=dev)
    c3 = torch.full((T, nb), offset >> 32, device=dev)
    k0, k1 = seed & M32, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    bits = torch.stack([v for w in (c0, c1, c2, c3) for v in (w & 0xFFFF, w >> 16)], 2).view(T, nb * 8)[:, :d]
    return bits >= thr, 65536.0 / (65536 - thr) if thr < 65536 else 0.0


def _drop(v, s):
    """D of a float tensor."""
    if not s.get("p"):
        return v
    keep, scale = _keep(*v.shape, s["p"], s["seed"], s["offset"], v.device)
    return torch.where(keep, v * scale, torch.zeros_like(v))


def _act(z, act):
    """act(z) and act'(z)."""
    if act == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if act in ("silu", "sigmoid"):
        g = 1 / (1 + torch.exp(-z))
        return (z * g, g * (1 + z * (1 - g))) if act == "silu" else (g, g * (1 - g))
    if act == "gelu":
        phi = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def _plain(s):
    op = s["op"]
    if op == "wgrad":
        return {"dW": (s["delta"].float().t() @ s["x"].float()) * (1.0 / s["T"])}
    if op == "drop_fwd":
        y = _drop(s["x"].float(), s)
        return {"y": (y if s["r"] is None else s["r"].float() + y).to(s["x"].dtype)}
    if op == "drop_bwd":
        return {"dx": _drop(s["dy"].float(), s).to(s["dy"].dtype)}
    wg, wu = s["w_gate"].float(), s["w_up"].float()
    if op == "glu_fwd":
        dt, x = s["x"].dtype, s["x"].float()
        z, u = x @ wg.t(), x @ wu.t()
        h = _drop(_act(z, s["act"])[0] * u, s).to(dt)
        return {"h": h, "gate": z.to(dt), "up": u.to(dt)} if s["keep"] else {"h": h}
    dt, z, u = s["dh"].dtype, s["gate"].float(), s["up"].float()
    e = _drop(s["dh"].float(), s)
    a, da = _act(z, s["act"])
    dz, du = e * u * da, e * a
    return {"dx": (dz @ wg + du @ wu).to(dt), "dgate": dz.to(dt), "dup": du.to(dt)}


# -- the package's entry points -------------------------------------------------

def _own(s):
    import fac_whitening_amd as fw

    op = s["op"]
    if op == "wgrad":
        return {"dW": fw.weight_grad(s["delta"], s["x"], alpha=1.0 / s["T"])}
    if op == "drop_fwd":
        return {"y": fw.dropout_forward(s["x"], s["drop"], residual=s["r"])}
    if op == "drop_bwd":
        return {"dx": fw.dropout_backward(s["dy"], s["drop"])}
    if op == "glu_fwd":
        h, gate, up = fw.glu_forward(s["x"], s["w_gate"], s["w_up"], act=s["act"], keep=s["keep"], drop=s.get("drop"))
        return {"h": h, "gate": gate, "up": up} if s["keep"] else {"h": h}
    dx, dgate, dup = fw.glu_backward(s["dh"], s["gate"], s["up"], s["w_gate"], s["w_up"], act=s["act"],
                                     drop=s.get("drop"))
    return {"dx": dx, "dgate": dgate, "dup": dup}


def run(state):
    return _own(state) if own else _plain(state)


# -- 64 bits, from the definitions -----------------------------------------------

def _philox64(ctr, key):
    """Philox4x32-10 on the host: four arrays of 32-bit words in uint64."""
    m0, m1, low, s32 = (np.uint64(v) for v in (0xD2511F53, 0xCD9E8D57, M32, 32))
    x0, x1, x2, x3 = ctr
    for r in range(10):
        k0, k1 = (np.uint64((key[i] + r * w) % (1 << 32)) for i, w in ((0, 0x9E3779B9), (1, 0xBB67AE85)))
        a, b = x0 * m0, x2 * m1
        x0, x1, x2, x3 = (b >> s32) ^ x1 ^ k0, b & low, (a >> s32) ^ x3 ^ k1, a & low
    return x0, x1, x2, x3


def _factor64(T, d, s, dev):
    """What D multiplies each element of a [T][d] matrix by."""
    if not s.get("p"):
        return None
    thr = round(65536 * s["p"])
    nb = -(-d // 8)
    out = np.empty((T, nb, 8), np.float64)
    rows = max(1, (1 << 20) // nb)
    for t0 in range(0, T, rows):
        n = min(rows, T - t0)
        c0 = np.tile(np.arange(nb, dtype=np.uint64), n)
        c1 = np.repeat(np.arange(t0, t0 + n, dtype=np.uint64), nb)
        c2, c3 = (np.full(n * nb, v, np.uint64) for v in (s["offset"] % (1 << 32), s["offset"] // (1 << 32)))
        w = _philox64((c0, c1, c2, c3), (s["seed"] % (1 << 32), s["seed"] // (1 << 32)))
        for i in range(8):
            r = (w[i // 2] // np.uint64(1 << 16 * (i % 2))) % np.uint64(65536)
            out[t0:t0 + n, :, i] = np.where(r < np.uint64(thr), 0.0, 65536.0 / max(65536 - thr, 1)).reshape(n, nb)
    return torch.from_numpy(out.reshape(T, nb * 8)[:, :d]).to(dev)


def _act64(z, act):
    if act == "relu":
        return z.clamp(min=0), torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
    if act in ("silu", "sigmoid"):
        e = torch.exp(-z.abs())
        g = torch.where(z >= 0, 1 / (1 + e), e / (1 + e))
        dg = e / (1 + e) ** 2
        return (g, dg) if act == "sigmoid" else (z * g, g + z * dg)
    if act == "gelu":
        phi = torch.erfc(-z / math.sqrt(2)) / 2
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # (1 + tanh v) / 2 = 1 / (1 + exp(-2 v))
    w = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    e = torch.exp(-w.abs())
    g = torch.where(w >= 0, 1 / (1 + e), e / (1 + e))
    return z * g, g + z * (e / (1 + e) ** 2) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op, T, d = s["op"], s["T"], s["d"]
    if op == "wgrad":
        return {"dW": torch.mm(s["delta"].double().t(), s["x"].double()) / T}
    if op in ("drop_fwd", "drop_bwd"):
        v = s["x" if op == "drop_fwd" else "dy"].double()
        v = v * _factor64(T, d, s, v.device)
        return {"dx": v} if op == "drop_bwd" else {"y": v if s["r"] is None else v + s["r"].double()}
    wg, wu = s["w_gate"].double(), s["w_up"].double()
    k = _factor64(T, s["f"], s, wg.device)
    if op == "glu_fwd":
        x = s["x"].double()
        z, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        h = _act64(z, s["act"])[0] * u
        h = h if k is None else h * k
        return {"h": h, "gate": z, "up": u} if s["keep"] else {"h": h}
    e, u = s["dh"].double(), s["up"].double()
    e = e if k is None else e * k
    a, da = _act64(s["gate"].double(), s["act"])
    dz, du = e * u * da, e * a
    return {"dx": torch.mm(dz, wg) + torch.mm(du, wu), "dgate": dz, "dup": du}
