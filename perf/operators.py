"""Cases for the 8-bit block products: what a linear layer trained with 8-bit
operands runs beside the optimizer step, from the layer's sizes up.

The 8-bit format.  Values are E4M3 codes, one power-of-two scale 2^e for each
block of 128: along a row for activations and gradients ("rows"), 128 x 128
for weights.  e is the smallest integer with max|block| <= 448 * 2^e, clamped
to [-117, 120] and stored as the byte e + 127; a code is value * 2^-e rounded
to nearest even.

  rows      codes [T, Kp] and scales [Kp / 128, T4] of x [T, K]; Kp is K
            rounded up to 128 (zero codes behind K), T4 is T rounded up to 4
            (the scale bytes of zero rows behind T)
  weights   per matrix w [N, K]: codes [N, Kp], scales [Np / 128, Kp / 128],
            and the same codes transposed, [K, Np], with their scales
  product   out = a b^T of rows a and weights b: y = x w^T, or with the
            transposed codes the gradient of the input, dx = dy w
  wgrad     out = base + dy^T x of a bf16 gradient dy [T, N] and the 8-bit
            copy of x that the forward pass kept

``own`` chooses between the plain torch form and the framework's calls.
"""

import torch

own = False

BLOCK = 128
LO, HI = -117, 120

# projections of one layer: q, k, v, o, gate, up, down
LLAMA31_8B_LAYER = ("4096x4096,1024x4096,1024x4096,4096x4096,"
                    "14336x4096,14336x4096,4096x14336")


def listed():
    return [
        # the activation of one generated token: pure latency
        {"name": "rows 1x4096 bf16", "op": "rows", "T": 1, "K": 4096, "dtype": "bf16"},
        # a training micro-batch's activations, kept in 8 bits for the backward pass
        {"name": "rows 8192x4096 bf16", "op": "rows", "T": 8192, "K": 4096, "dtype": "bf16"},
        # fp32 values with rows that no vector access divides
        {"name": "rows 777x1001 f32", "op": "rows", "T": 777, "K": 1001, "dtype": "f32"},
        # the projections of a Llama-3.1-8B layer after an optimizer step
        {"name": "weights 8B layer bf16", "op": "weights", "shapes": LLAMA31_8B_LAYER, "dtype": "bf16"},
        # small and ragged fp32 matrices
        {"name": "weights ragged f32", "op": "weights", "shapes": "300x200,129x1,1000x1001,1x513,128x256", "dtype": "f32"},
        # one generated token through a gate projection: the weight's bytes
        {"name": "product 1 14336x4096", "op": "product", "T": 1, "N": 14336, "K": 4096, "transpose": False, "dtype": "bf16"},
        # a batch of 24 generated tokens through a down projection
        {"name": "product 24 4096x14336", "op": "product", "T": 24, "N": 4096, "K": 14336, "transpose": False, "dtype": "bf16"},
        # the forward pass of a training micro-batch
        {"name": "product 8192 14336x4096", "op": "product", "T": 8192, "N": 14336, "K": 4096, "transpose": False, "dtype": "bf16"},
        # the gradient of the input of a Qwen2.5-7B gate projection, fp32 out, a ragged token count
        {"name": "dgrad 2001 18944x3584 f32", "op": "product", "T": 2001, "N": 18944, "K": 3584, "transpose": True, "dtype": "f32"},
        # the weight gradient of the same micro-batch
        {"name": "wgrad 8192 14336x4096", "op": "wgrad", "T": 8192, "N": 14336, "K": 4096, "add": False, "dtype": "bf16"},
        # a k projection's gradient added to an earlier micro-batch's: few output tiles, many tokens
        {"name": "wgrad 4096 1024x4096 f32 add", "op": "wgrad", "T": 4096, "N": 1024, "K": 4096, "add": True, "dtype": "f32"},
        # odd sizes everywhere
        {"name": "wgrad 333 1001x513 f32", "op": "wgrad", "T": 333, "N": 1001, "K": 513, "add": False, "dtype": "f32"},
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(lo * (hi / lo) ** rng.random()))
        kind = rng.randrange(3)  # any size, a multiple of 8, a multiple of 128
        return max(1, v if kind == 0 else (v + 7) // 8 * 8 if kind == 1 else (v + 127) // 128 * 128)

    op = rng.choice(["rows", "weights", "product", "product", "wgrad", "wgrad"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "rows":
        k = size(16, 16384)
        return {"op": op, "T": max(1, min(size(1, 16384), 8192 * 4096 // (k * (2 if dtype == "f32" else 1)))), "K": k, "dtype": dtype}
    if op == "weights":
        return {"op": op, "shapes": ",".join("%dx%d" % (size(1, 8192), size(1, 8192)) for _ in range(rng.randrange(1, 4))), "dtype": dtype}
    n, k = size(32, 16384), size(32, 16384)
    t = max(1, min(size(1, 16384), 8192 * 14336 * 4096 // (2 * n * k)))
    if op == "product":
        return {"op": op, "T": t, "N": n, "K": k, "transpose": rng.random() < 0.5, "dtype": dtype}
    return {"op": op, "T": t, "N": n, "K": k, "add": rng.random() < 0.5, "dtype": dtype}


# ---------------------------------------------------------------- inputs --

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _up(n, a):
    return (n + a - 1) // a * a


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _tokens(gen, t, k, std, dtype):
    """Rows of differing size with a few large channels; one row in 16 is a
    padding token's zeros."""
    x = _normal(gen, t, k) * std * torch.exp(0.5 * _normal(gen, t, 1))
    large = torch.rand(k, generator=gen, device="cuda") < 0.01
    x = x * torch.where(large, 30.0, 1.0)
    if t >= 16:
        x[15::16] = 0
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dtype = case["op"], _type(case["dtype"])
    state = {"case": case, "dtype": dtype}
    if op == "rows":
        state["x"] = _tokens(gen, case["T"], case["K"], 1.0, dtype)
    elif op == "weights":
        state["w"] = [(0.02 * _normal(gen, r, c)).to(dtype) for r, c in _shapes(case)]
    elif op == "product":
        n, k = case["N"], case["K"]
        inner = n if case["transpose"] else k
        state["a"] = _rows(_tokens(gen, case["T"], inner, 1e-3 if case["transpose"] else 1.0, torch.bfloat16))
        state["b"] = _weights((0.02 * _normal(gen, n, k)).to(torch.bfloat16))
        state["inner"] = inner
    else:
        t, n, k = case["T"], case["N"], case["K"]
        state["dy"] = _tokens(gen, t, n, 1e-3, torch.bfloat16)
        state["x"] = _rows(_tokens(gen, t, k, 1.0, torch.bfloat16))
        state["base"] = (0.05 * _normal(gen, n, k)).to(dtype) if case["add"] else None
    return state


# ------------------------------------------------------------ plain forms --

def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, 448 = 1.75 * 2^8, from the bits
    of the fp32 amax."""
    bits = amax.view(torch.int32)
    e = (bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return e.clamp(LO, HI)


def _power(e):
    """2^e as fp32, for e in the format's range."""
    return ((e + 127) << 23).view(torch.float32)


def _rows(x):
    t, k = x.shape
    kp, t4 = _up(k, BLOCK), _up(t, 4)
    v = torch.nn.functional.pad(x.float(), (0, kp - k)).view(t, kp // BLOCK, BLOCK)
    e = _exponent(v.abs().amax(2))
    codes = (v * _power(-e)[:, :, None]).to(torch.float8_e4m3fn).view(t, kp)
    scales = torch.nn.functional.pad((e + 127).to(torch.uint8).t(), (0, t4 - t), value=LO + 127).contiguous()
    return {"codes": codes, "scales": scales}


def _weights(w):
    n, k = w.shape
    np_, kp = _up(n, BLOCK), _up(k, BLOCK)
    v = torch.nn.functional.pad(w.float(), (0, kp - k, 0, np_ - n)).view(np_ // BLOCK, BLOCK, kp // BLOCK, BLOCK)
    e = _exponent(v.abs().amax((1, 3)))
    q = (v * _power(-e)[:, None, :, None]).view(np_, kp)
    scales = (e + 127).to(torch.uint8)
    return {"codes": q[:n].to(torch.float8_e4m3fn), "scales": scales,
            "codes_t": q.t()[:k].contiguous().to(torch.float8_e4m3fn), "scales_t": scales.t().contiguous()}


def _row_values(q):
    t, kp = q["codes"].shape
    s = _power(q["scales"][:, :t].t().to(torch.int32) - 127)
    return (q["codes"].float().view(t, kp // BLOCK, BLOCK) * s[:, :, None]).view(t, kp)


def _weight_values(codes, scales):
    n, kp = codes.shape
    s = _power(scales.to(torch.int32) - 127).repeat_interleave(BLOCK, 0)[:n]
    return (codes.float().view(n, kp // BLOCK, BLOCK) * s[:, :, None]).view(n, kp)


def _plain(s):
    case = s["case"]
    if case["op"] == "rows":
        return _rows(s["x"])
    if case["op"] == "weights":
        return [_weights(w) for w in s["w"]]
    if case["op"] == "product":
        b = _weight_values(s["b"]["codes_t"], s["b"]["scales_t"]) if case["transpose"] else _weight_values(s["b"]["codes"], s["b"]["scales"])
        return (_row_values(s["a"]) @ b.t()).to(s["dtype"])
    out = s["dy"].float().t() @ _row_values(s["x"])[:, :case["K"]]
    return (out if s["base"] is None else s["base"].float() + out).to(s["dtype"])


# ---------------------------------------------------- the framework's calls --

def _own(s):
    import newton_schulz_dmuon_amd as nsd
    case = s["case"]
    if case["op"] == "rows":
        q = nsd.q8_quantize(s["x"])
        return {"codes": q.codes, "scales": q.scales}
    if case["op"] == "weights":
        return [{"codes": q.codes, "scales": q.scales, "codes_t": q.codes_t, "scales_t": q.scales_t}
                for q in nsd.q8_quantize_weights(s["w"])]
    if case["op"] == "product":
        a = nsd.Q8Rows(s["a"]["codes"], s["a"]["scales"], s["inner"])
        b = s["b"]
        w = nsd.Q8Weight(b["codes"], b["scales"], b["codes_t"], b["scales_t"])
        return nsd.q8_matmul(a, w, transpose=case["transpose"], dtype=s["dtype"])
    x = nsd.Q8Rows(s["x"]["codes"], s["x"]["scales"], case["K"])
    return nsd.q8_weight_grad(s["dy"], x, dtype=s["dtype"], base=s["base"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work --

def work(case):
    item = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rows":
        t, k = case["T"], case["K"]
        return {"bytes": t * k * (item + 1) + t * _up(k, BLOCK) // BLOCK, "flops": 2 * t * k}
    if case["op"] == "weights":
        elems = sum(r * c for r, c in _shapes(case))
        return {"bytes": elems * (item + 2), "flops": 2 * elems}
    t, n, k = case["T"], case["N"], case["K"]
    if case["op"] == "product":
        inner, outer = (n, k) if case["transpose"] else (k, n)
        return {"bytes": t * inner + n * k + (t + n / BLOCK) * inner / BLOCK + item * t * outer, "flops": 2 * t * n * k}
    return {"bytes": 2 * t * n + t * k + t * k / BLOCK + item * n * k * (2 if case["add"] else 1), "flops": 2 * t * n * k}


# --------------------------------------------- the definition in 64 bits --

def _exact_power(e):
    """2^e as fp64 (pow is not exact on the device)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quantize(v, dims):
    """(rounded value * 2^-e, 2^e) of blocks of fp64 values, the block along ``dims``."""
    amax = v.abs().amax(dims, keepdim=True)
    _, p = torch.frexp(amax)
    e = p - 9
    e = e + (amax > 448 * _exact_power(e)).to(e.dtype)
    scale = _exact_power(torch.where(amax > 0, e, LO).clamp(LO, HI))
    q = v / scale
    _, p = torch.frexp(q.abs().clamp(min=2.0 ** -6))
    step = _exact_power(p - 4)  # four significant bits; below 2^-6 a fixed step
    return torch.round(q / step) * step, scale


def _exact_padded(x, rows):
    n, k = x.shape
    out = torch.zeros(_up(n, rows), _up(k, BLOCK), dtype=torch.float64, device=x.device)
    out[:n, :k] = x
    return out


def _exact_rows(x):
    v = _exact_padded(x, 1)
    q, scale = _exact_quantize(v.view(v.shape[0], -1, BLOCK), 2)
    return q.reshape(v.shape), (q * scale).reshape(v.shape)


def _exact_weights(w):
    n, k = w.shape
    v = _exact_padded(w, BLOCK)
    q, scale = _exact_quantize(v.view(v.shape[0] // BLOCK, BLOCK, -1, BLOCK), (1, 3))
    return q.reshape(v.shape), (q * scale).reshape(v.shape)


def _exact_inputs(case, seed):
    """The inputs of prepare() before they were quantised, in its order of draws."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "product":
        n, k = case["N"], case["K"]
        a = _tokens(gen, case["T"], n if case["transpose"] else k, 1e-3 if case["transpose"] else 1.0, torch.bfloat16)
        return a, (0.02 * _normal(gen, n, k)).to(torch.bfloat16)
    dy = _tokens(gen, case["T"], case["N"], 1e-3, torch.bfloat16)
    x = _tokens(gen, case["T"], case["K"], 1.0, torch.bfloat16)
    base = (0.05 * _normal(gen, case["N"], case["K"])).to(_type(case["dtype"])) if case["add"] else None
    return dy, x, base


def exact(case, seed):
    if case["op"] == "rows":
        return {"codes": _exact_rows(prepare(case, seed)["x"])[0], "scales": None}
    if case["op"] == "weights":
        got = [(w.shape, _exact_weights(w)[0]) for w in prepare(case, seed)["w"]]
        return [{"codes": q[:n], "scales": None, "codes_t": q.t()[:k], "scales_t": None} for (n, k), q in got]
    if case["op"] == "product":
        a, w = _exact_inputs(case, seed)
        av, wv = _exact_rows(a)[1], _exact_weights(w)[1]
        n, k = case["N"], case["K"]
        return av[:, :n] @ wv[:n, :k] if case["transpose"] else av[:, :k] @ wv[:n, :k].t()
    dy, x, base = _exact_inputs(case, seed)
    out = dy.double().t() @ _exact_rows(x)[1][:, :case["K"]]
    return out if base is None else base.double() + out
