"""Cases of the 8-bit linear layer's operators: what a pass of each takes, gives and costs.

The operators quantise bf16 rows to FP8 E4M3 codes in blocks of 128 consecutive
columns, each block with one power-of-two scale held as an E8M0 byte (2^(byte - 127)).
A row's codes are padded with zeros to whole blocks, its scale bytes with 127 (scale
one) to a multiple of four.  A block's scale is the smallest power of two that brings
its largest magnitude to 448 or less; a block of zeros has scale one.  Weights have one
scale for each 128 x 128 block.  The operators:

* norm, norm_grad: residual addition, root-mean-square norm, quantised output; its gradient.
* weight, matmul: a weight's codes (as stored and transposed), and the product of
  quantised rows with quantised weights.
* linear_grad: both gradients of a linear layer whose input was kept in 8 bits.
* gate, gate_grad: SiLU-gated unit with a quantised output and an 8-bit checkpoint of
  its input; its gradient from that checkpoint.

Sizes: 4096, 1600 and 3584 columns and 4096 and 8192 tokens are this repository's
workloads; four times the columns is the usual inner width.
"""
import math
import random

import torch

own = False

BLOCK = 128
EPS = 1e-5


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one step of decoding for 8 sequences: latency
        {"name": "norm_decode", "op": "norm", "tokens": 8, "hidden": 4096, "residual": True},
        # a training step's norm between two layers
        {"name": "norm_train", "op": "norm", "tokens": 4096, "hidden": 4096, "residual": True},
        # a short ragged batch, columns that end inside a block
        {"name": "norm_grad_ragged", "op": "norm_grad", "tokens": 1021, "hidden": 1600, "residual": True},
        # the largest activation of the workloads, backward
        {"name": "norm_grad_train", "op": "norm_grad", "tokens": 8192, "hidden": 3584, "residual": True},
        # one step of decoding for 4 sequences: the weight is read, hardly anything is computed
        {"name": "matmul_decode", "op": "matmul", "tokens": 4, "outputs": 4096, "hidden": 4096},
        # a prompt's prefill, ragged in every dimension
        {"name": "matmul_ragged", "op": "matmul", "tokens": 777, "outputs": 1601, "hidden": 1600},
        # the inner product of a training step, forward
        {"name": "matmul_train", "op": "matmul", "tokens": 8192, "outputs": 14336, "hidden": 3584},
        # laying out that weight after an optimizer step, for both directions
        {"name": "weight_train", "op": "weight", "outputs": 14336, "hidden": 3584},
        # backward of a projection on a short ragged batch
        {"name": "linear_grad_ragged", "op": "linear_grad", "tokens": 1021, "outputs": 1601, "hidden": 1600},
        # backward of a training step's inner projection
        {"name": "linear_grad_train", "op": "linear_grad", "tokens": 4096, "outputs": 16384, "hidden": 4096},
        # a training step's gated unit, both directions
        {"name": "gate_train", "op": "gate", "tokens": 4096, "inner": 8192},
        {"name": "gate_grad_train", "op": "gate_grad", "tokens": 4096, "inner": 8192},
    ]


def _size(rng, low, high, odd=0.3):
    """Log-uniform in [low, high]; mostly multiples of 64 above that, else any number."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v > 64 and rng.random() > odd:
        v = v // 64 * 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "matmul", "matmul", "weight", "linear_grad", "linear_grad", "gate", "gate_grad"])
    tokens = _size(rng, 1, 8192, 0.5)
    if op in ("norm", "norm_grad"):
        return {"op": op, "tokens": tokens, "hidden": _size(rng, 100, 8192), "residual": rng.random() < 0.7}
    if op == "matmul":
        case = {"op": op, "tokens": tokens, "outputs": _size(rng, 100, 16384), "hidden": _size(rng, 100, 8192)}
        while case["tokens"] * case["outputs"] * case["hidden"] > 8192 * 14336 * 3584:
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    if op == "weight":
        return {"op": op, "outputs": _size(rng, 100, 14336), "hidden": _size(rng, 100, 3584)}
    if op == "linear_grad":
        case = {"op": op, "tokens": tokens, "outputs": _size(rng, 100, 16384), "hidden": _size(rng, 100, 8192)}
        while case["tokens"] * case["outputs"] * case["hidden"] > 4096 * 16384 * 4096:
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    return {"op": op, "tokens": min(tokens, 4096), "inner": _size(rng, 100, 8192)}


# --------------------------------------------------------------------------- sizes

def _padded(cols):
    return -(-cols // BLOCK) * BLOCK


def _scale_cols(cols):
    return -(-(_padded(cols) // BLOCK) // 4) * 4


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        t, h = case["tokens"], case["hidden"]
        extra = 2 * t * h if case["residual"] else 0
        if op == "norm":       # x read, the codes, their scales and 1/rms written; with a residual it is read and the sum written
            return {"bytes": 3 * t * h + 2 * extra + t * h / BLOCK + 4 * t + 2 * h, "flops": 8 * t * h}
        # dy, z (and the residual's gradient) read, dx written, the weight's gradient once
        return {"bytes": 6 * t * h + extra + 4 * t + 6 * h, "flops": 10 * t * h}
    if op == "matmul":
        m, n, k = case["tokens"], case["outputs"], case["hidden"]
        return {"bytes": m * k + n * k + 2 * m * n, "flops": 2 * m * n * k}
    if op == "weight":
        return {"bytes": 4 * case["outputs"] * case["hidden"], "flops": 2 * case["outputs"] * case["hidden"]}
    if op == "linear_grad":    # dy, the weight's codes and the input's codes read; dx and dw written
        m, n, k = case["tokens"], case["outputs"], case["hidden"]
        return {"bytes": 2 * m * n + n * k + m * k + 2 * m * k + 4 * n * k, "flops": 4 * m * n * k}
    t, f = case["tokens"], case["inner"]
    if op == "gate":           # gate and up read (bf16); codes of the product and of both inputs written
        return {"bytes": 7 * t * f, "flops": 12 * t * f}
    # the output's gradient and the checkpoint read; both inputs' gradients written, bf16 and codes
    return {"bytes": 10 * t * f, "flops": 16 * t * f}


# --------------------------------------------------------------------------- inputs

def _activation(g, rows, cols):
    """Activations: dense near zero with a long tail, a few outlier columns, rows of differing
    magnitude, and every 97th row zero (a padding token)."""
    x = torch.empty(rows, cols, device="cuda").exponential_(100.0, generator=g)
    x *= torch.randint(0, 2, (rows, cols), device="cuda", generator=g, dtype=torch.int8) * 2 - 1
    hot = torch.randint(0, cols, (max(1, cols // 200),), device="cuda", generator=g)
    x[:, hot] *= 20.0
    x *= torch.exp(torch.randn(rows, 1, device="cuda", generator=g))
    x[96::97] = 0.0
    return x.to(torch.bfloat16)


def _gradient(g, rows, cols):
    x = torch.randn(rows, cols, device="cuda", generator=g)
    x *= 1e-4 * torch.exp(torch.randn(rows, 1, device="cuda", generator=g))
    x[96::97] = 0.0
    return x.to(torch.bfloat16)


def _matrix(g, rows, cols):
    return (torch.randn(rows, cols, device="cuda", generator=g) * cols ** -0.5).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("norm", "norm_grad"):
        t, h = case["tokens"], case["hidden"]
        s["weight"] = (1 + 0.1 * torch.randn(h, device="cuda", generator=g)).to(torch.bfloat16)
        x = _activation(g, t, h)
        if op == "norm":
            s["x"] = x
            s["residual"] = _activation(g, t, h) if case["residual"] else None
        else:
            s["z"] = x
            s["rstd"] = torch.rsqrt(x.float().square().mean(1) + EPS)
            s["dy"] = _gradient(g, t, h)
            s["dz"] = _gradient(g, t, h) if case["residual"] else None
    elif op == "weight":
        s["w"] = _matrix(g, case["outputs"], case["hidden"])
    elif op in ("matmul", "linear_grad"):
        m, n, k = case["tokens"], case["outputs"], case["hidden"]
        s["xq"], s["xs"] = _plain_rows(_activation(g, m, k).float())
        wq, ws, wqt, wst = _plain_weight(_matrix(g, n, k).float())
        if op == "matmul":
            s["wq"], s["ws"] = wq, ws
        else:
            s["wqt"], s["wst"] = wqt, wst
            s["dy"] = _gradient(g, m, n)
    else:
        t, f = case["tokens"], case["inner"]
        gu = (torch.randn(t, 2 * f, device="cuda", generator=g) * 1.5).to(torch.bfloat16)
        gu[96::97] = 0.0
        if op == "gate":
            s["gu"] = gu
        else:
            s["cq"], s["cs"] = _plain_checkpoint(gu.float(), f)
            s["dh"] = _gradient(g, t, f)
    return s


# --------------------------------------------------------------------------- plain forms

def _exponents(amax):
    """E8M0 byte of the smallest power of two that brings amax to 448 or less; one for zero."""
    bits = amax.contiguous().view(torch.int32)
    up = ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)          # 448 = 1.75 * 2^8
    byte = torch.clamp((bits >> 23) - 8 + up, 1, 254)
    return torch.where(amax == 0, torch.full_like(byte, 127), byte)


def _power(byte):
    return torch.ldexp(torch.ones((), device=byte.device), byte.to(torch.int32) - 127)


def _pad_scales(byte, cols):
    out = torch.full((byte.shape[0], _scale_cols(cols)), 127, dtype=torch.uint8, device=byte.device)
    out[:, :byte.shape[1]] = byte.to(torch.uint8)
    return out


def _plain_rows(x):
    """fp32 rows -> codes (uint8, padded to whole blocks) and scale bytes."""
    t, cols = x.shape
    x = torch.nn.functional.pad(x, (0, _padded(cols) - cols)).reshape(t, -1, BLOCK)
    byte = _exponents(x.abs().amax(2))
    q = (x / _power(byte)[:, :, None]).to(torch.float8_e4m3fn)
    return q.reshape(t, -1).view(torch.uint8), _pad_scales(byte, cols)


def _plain_weight(w):
    n, k = w.shape
    w = torch.nn.functional.pad(w, (0, _padded(k) - k, 0, _padded(n) - n))
    blocks = w.reshape(w.shape[0] // BLOCK, BLOCK, w.shape[1] // BLOCK, BLOCK)
    byte = _exponents(blocks.abs().amax((1, 3)))
    q = (blocks / _power(byte)[:, None, :, None]).to(torch.float8_e4m3fn).reshape(w.shape).view(torch.uint8)
    return q[:n].contiguous(), _pad_scales(byte, k), q[:, :k].t().contiguous(), _pad_scales(byte.t(), n)


def _plain_values(q, scale):
    """Codes and scale bytes -> fp32 values, padded columns included."""
    t, cols = q.shape
    v = q.view(torch.float8_e4m3fn).float().reshape(t, -1, BLOCK)
    return (v * _power(scale[:, :cols // BLOCK])[:, :, None]).reshape(t, cols)


def _plain_weight_values(q, scale):
    n, cols = q.shape
    s = _power(scale[:, :cols // BLOCK]).repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)
    return q.view(torch.float8_e4m3fn).float() * s


def _plain_checkpoint(gu, f):
    gq, gs = _plain_rows(gu[:, :f])
    uq, us = _plain_rows(gu[:, f:])
    blocks = _padded(f) // BLOCK
    both = torch.cat([gs[:, :blocks], us[:, :blocks]], 1)
    return torch.cat([gq, uq], 1), _pad_scales(both, 2 * _padded(f))


def _codes(q):
    return q.view(torch.float8_e4m3fn)


def _scales(s):
    return s.view(torch.float8_e8m0fnu)


def _run_plain(s):
    op, case = s["case"]["op"], s["case"]
    if op == "norm":
        z = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
        zf = z.float()
        rstd = torch.rsqrt((zf * zf).mean(1) + EPS)
        q, scale = _plain_rows(zf * rstd[:, None] * s["weight"].float())
        return {"z": z, "rstd": rstd, "q": _codes(q), "scale": _scales(scale)}
    if op == "norm_grad":
        xhat = s["z"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        dxhat = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True))
        if s["dz"] is not None:
            dx = dx + s["dz"].float()
        return {"dx": dx.to(torch.bfloat16), "dw": (dy * xhat).sum(0)}
    if op == "weight":
        q, scale, qt, st = _plain_weight(s["w"].float())
        return {"q": _codes(q), "scale": _scales(scale), "qt": _codes(qt), "scale_t": _scales(st)}
    if op == "matmul":
        return {"y": (_plain_values(s["xq"], s["xs"]) @ _plain_weight_values(s["wq"], s["ws"]).t()).to(torch.bfloat16)}
    if op == "linear_grad":
        dy = s["dy"].float()
        dq, ds = _plain_rows(dy)
        dx = _plain_values(dq, ds) @ _plain_weight_values(s["wqt"], s["wst"]).t()
        dw = dy.t() @ _plain_values(s["xq"], s["xs"])[:, :case["hidden"]]
        return {"dx": dx.to(torch.bfloat16), "dw": dw}
    f = case["inner"]
    if op == "gate":
        gu = s["gu"].float()
        h = gu[:, :f] / (1 + torch.exp(-gu[:, :f])) * gu[:, f:]
        hq, hs = _plain_rows(h)
        cq, cs = _plain_checkpoint(gu, f)
        return {"hq": _codes(hq), "hs": _scales(hs), "cq": _codes(cq), "cs": _scales(cs)}
    gu = _plain_values(s["cq"], s["cs"])
    gate, up = gu[:, :f], gu[:, _padded(f):_padded(f) + f]
    dh = s["dh"].float()
    sig = 1 / (1 + torch.exp(-gate))
    dgu = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1)
    dq, ds = _plain_rows(dgu)
    return {"dgu": dgu.to(torch.bfloat16), "dq": _codes(dq), "ds": _scales(ds)}


# --------------------------------------------------------------------------- the framework's operators

def _run_own(s):
    import fp8_compression_tensor_taco_amd as taco
    op, case = s["case"]["op"], s["case"]
    if op == "norm":
        z, rstd, q, scale = taco.rmsnorm_quantize(s["x"], s["weight"], EPS, residual=s["residual"])
        return {"z": z, "rstd": rstd, "q": _codes(q), "scale": _scales(scale)}
    if op == "norm_grad":
        dx, dw = taco.rmsnorm_backward(s["dy"], s["z"], s["rstd"], s["weight"], dz=s["dz"])
        return {"dx": dx, "dw": dw}
    if op == "weight":
        q, scale, qt, st = taco.quantize_weight(s["w"])
        return {"q": _codes(q), "scale": _scales(scale), "qt": _codes(qt), "scale_t": _scales(st)}
    if op == "matmul":
        return {"y": taco.matmul_fp8(s["xq"], s["xs"], s["wq"], s["ws"])}
    if op == "linear_grad":
        dq, ds = taco.quantize_rows(s["dy"])
        dx = taco.matmul_fp8(dq, ds, s["wqt"], s["wst"])
        return {"dx": dx, "dw": taco.wgrad_fp8(s["dy"], s["xq"], s["xs"], case["hidden"])}
    if op == "gate":
        hq, hs, cq, cs = taco.swiglu_quantize(s["gu"])
        return {"hq": _codes(hq), "hs": _scales(hs), "cq": _codes(cq), "cs": _scales(cs)}
    dgu, dq, ds = taco.swiglu_backward(s["dh"], s["cq"], s["cs"])
    return {"dgu": dgu, "dq": _codes(dq), "ds": _scales(ds)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- 64 bits

def _code_value(q):
    """E4M3: a sign, four bits of exponent with bias 7, three of mantissa."""
    q = q.to(torch.int64)
    exponent, mantissa = (q >> 3) & 15, (q & 7).double()
    size = torch.where(exponent == 0, mantissa * 2.0 ** -9, (1 + mantissa / 8) * torch.exp2(exponent.double() - 7))
    return torch.where(q >> 7 == 1, -size, size)


def _scale_value(s):
    return torch.exp2(s.double() - 127)


def _to_grid(v):
    """The E4M3 value nearest to v, |v| <= 448, ties to the even one."""
    _, e = torch.frexp(v)
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)
    return torch.round(v / step) * step


def _power_for(amax):
    m, e = torch.frexp(amax)                     # amax = m * 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-126)
    return torch.where(amax == 0, torch.ones_like(amax), torch.exp2(e.double()))


def _exact_rows(x):
    t, cols = x.shape
    wide = torch.zeros(t, _padded(cols), dtype=torch.float64, device=x.device)
    wide[:, :cols] = x
    blocks = wide.view(t, -1, BLOCK)
    power = _power_for(blocks.abs().amax(2))
    scales = torch.ones(t, _scale_cols(cols), dtype=torch.float64, device=x.device)
    scales[:, :power.shape[1]] = power
    return _to_grid(blocks / power[:, :, None]).reshape(t, -1), scales


def _decoded(q, s, weight=False):
    v, p = _code_value(q), _scale_value(s)[:, :q.shape[1] // BLOCK]
    rows = torch.arange(q.shape[0], device=q.device) // (BLOCK if weight else 1)
    return v * p[rows].repeat_interleave(BLOCK, 1)


def exact(case, seed):
    if case["op"] in ("matmul", "linear_grad"):
        if work(case)["flops"] > 3e14:           # over about 20 seconds in 64 bits
            return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        # the sum of the residual is stored, and normalised, in bf16: one rounding of the exact sum
        z = s["x"].double()
        if s["residual"] is not None:
            z = (z + s["residual"].double()).float().to(torch.bfloat16).double()
        rstd = 1 / torch.sqrt((z ** 2).sum(1) / z.shape[1] + EPS)
        q, scale = _exact_rows(s["weight"].double() * (z * rstd[:, None]))
        return {"z": z, "rstd": rstd, "q": q, "scale": scale}
    if op == "norm_grad":
        z, r, w, dy = s["z"].double(), s["rstd"].double()[:, None], s["weight"].double(), s["dy"].double()
        inner = (dy * w * z).sum(1, keepdim=True)
        dx = r * w * dy - z * r ** 3 * inner / z.shape[1]
        if s["dz"] is not None:
            dx += s["dz"].double()
        return {"dx": dx, "dw": (dy * z * r).sum(0)}
    if op == "weight":
        w = s["w"].double()
        n, k = w.shape
        wide = torch.zeros(_padded(n), _padded(k), dtype=torch.float64, device=w.device)
        wide[:n, :k] = w
        nb, kb = wide.shape[0] // BLOCK, wide.shape[1] // BLOCK
        blocks = wide.view(nb, BLOCK, kb, BLOCK).transpose(1, 2)
        power = _power_for(blocks.abs().amax((2, 3)))
        q = _to_grid(blocks / power[:, :, None, None]).transpose(1, 2).reshape(wide.shape)
        scale = torch.ones(nb, _scale_cols(k), dtype=torch.float64, device=w.device)
        scale[:, :kb] = power
        scale_t = torch.ones(kb, _scale_cols(n), dtype=torch.float64, device=w.device)
        scale_t[:, :nb] = power.t()
        return {"q": q[:n], "scale": scale, "qt": q[:, :k].t(), "scale_t": scale_t}
    if op == "matmul":
        return {"y": _decoded(s["xq"], s["xs"]) @ _decoded(s["wq"], s["ws"], True).t().contiguous()}
    if op == "linear_grad":
        dy, k = s["dy"].double(), case["hidden"]
        q, scale = _exact_rows(dy)
        dq = (q.view(dy.shape[0], -1, BLOCK) * scale[:, :q.shape[1] // BLOCK, None]).reshape(q.shape)
        return {"dx": dq @ _decoded(s["wqt"], s["wst"], True).t().contiguous(),
                "dw": dy.t().contiguous() @ _decoded(s["xq"], s["xs"])[:, :k].contiguous()}
    f = case["inner"]
    if op == "gate":
        gate, up = s["gu"][:, :f].double(), s["gu"][:, f:].double()
        hq, hs = _exact_rows(up * gate * torch.sigmoid(gate))
        (gq, gs), (uq, us) = _exact_rows(gate), _exact_rows(up)
        blocks = _padded(f) // BLOCK
        cs = torch.ones(gq.shape[0], _scale_cols(2 * _padded(f)), dtype=torch.float64, device=gq.device)
        cs[:, :2 * blocks] = torch.cat([gs[:, :blocks], us[:, :blocks]], 1)
        return {"hq": hq, "hs": hs, "cq": torch.cat([gq, uq], 1), "cs": cs}
    both = _decoded(s["cq"], s["cs"])
    gate, up = both[:, :f], both[:, _padded(f):_padded(f) + f]
    dh, sig = s["dh"].double(), torch.sigmoid(gate)
    dgu = torch.cat([dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig], 1)
    dq, ds = _exact_rows(dgu)
    return {"dgu": dgu, "dq": dq, "ds": ds}


if __name__ == "__main__":
    for one in listed() + [draw(random.Random(k)) for k in range(6)]:
        print(one, work(one))
