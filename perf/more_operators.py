"""Cases for the 4-bit block products: a linear layer trained or served with
microscaled 4-bit operands, from quantisation to the weight gradient.

The 4-bit format.  Values are E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives), two to a byte, with one power-of-two scale 2^e for each block of 32
along the direction that a product sums over.  e is the smallest integer with
max|block| <= 6 * 2^e, clamped to [-125, 126] and stored as the byte e + 127; a
code is value * 2^-e rounded to nearest even, or, given a random byte n,
up iff the part of a step that is left is at least (255.5 - n) / 256.

  codes    [R, Cp / 2] and scales [Cp / 32, R16] of x [R, C], blocks along a
           row; Cp is C rounded up to 256 (zero codes behind C), R16 is R
           rounded up to 16 (the scale bytes of zero rows behind R)
  codes_t  the same of x transposed, blocks along a column of x

  quantise  x to codes and, where asked for, codes_t; read back as values
  weights   the same for a list of matrices
  product   out = a b^T of 4-bit a and b: y = x w^T, or with the transposed
            codes the gradient of the input, dx = dy w
  bf16rows  the same with a in bf16
  wgrad     out = base + dy^T x of the transposed codes of dy and x

``own`` chooses between the plain torch form and the framework's calls.
"""

import torch

own = False

BLOCK = 32
PAD = 256
LO, HI = -125, 126

# projections of one layer: q, k, v, o, gate, up, down
LLAMA31_8B_LAYER = ("4096x4096,1024x4096,1024x4096,4096x4096,"
                    "14336x4096,14336x4096,4096x14336")


def listed():
    return [
        # the activation of one generated token, for the forward product alone: pure latency
        {"name": "quantise 1x4096 bf16", "op": "quantise", "T": 1, "K": 4096, "dtype": "bf16", "transposed": False, "random": False},
        # a micro-batch's output gradient, rounded by given random bytes, for both backward products
        {"name": "quantise 8192x4096 bf16 random", "op": "quantise", "T": 8192, "K": 4096, "dtype": "bf16", "transposed": True, "random": True},
        # fp32 activations whose rows no vector access divides
        {"name": "quantise 777x1001 f32", "op": "quantise", "T": 777, "K": 1001, "dtype": "f32", "transposed": True, "random": False},
        # the projections of a Llama-3.1-8B layer after an optimizer step
        {"name": "weights 8B layer bf16", "op": "weights", "shapes": LLAMA31_8B_LAYER, "dtype": "bf16"},
        # small and ragged fp32 matrices
        {"name": "weights ragged f32", "op": "weights", "shapes": "300x200,129x1,1000x1001,1x513,128x256", "dtype": "f32"},
        # one generated token through a gate projection, its activation in 4 bits too: the weight's bytes
        {"name": "product 1 14336x4096", "op": "product", "T": 1, "N": 14336, "K": 4096, "transpose": False, "dtype": "bf16"},
        # the forward pass of a training micro-batch
        {"name": "product 8192 14336x4096", "op": "product", "T": 8192, "N": 14336, "K": 4096, "transpose": False, "dtype": "bf16"},
        # the gradient of the input of a Qwen2.5-7B gate projection, fp32 out, a ragged token count
        {"name": "dgrad 2001 18944x3584 f32", "op": "product", "T": 2001, "N": 18944, "K": 3584, "transpose": True, "dtype": "f32"},
        # one generated token's bf16 activation through a down projection held in 4 bits
        {"name": "bf16 rows 1 4096x14336", "op": "bf16rows", "T": 1, "N": 4096, "K": 14336, "transpose": False, "dtype": "bf16"},
        # a prompt's bf16 activations through a gate projection held in 4 bits
        {"name": "bf16 rows 2048 14336x4096", "op": "bf16rows", "T": 2048, "N": 14336, "K": 4096, "transpose": False, "dtype": "bf16"},
        # the weight gradient of the training micro-batch
        {"name": "wgrad 8192 14336x4096", "op": "wgrad", "T": 8192, "N": 14336, "K": 4096, "add": False, "dtype": "bf16"},
        # odd sizes everywhere, added to an earlier micro-batch's gradient
        {"name": "wgrad 333 1001x513 f32 add", "op": "wgrad", "T": 333, "N": 1001, "K": 513, "add": True, "dtype": "f32"},
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(lo * (hi / lo) ** rng.random()))
        kind = rng.randrange(3)  # any size, a multiple of 8, a multiple of 128
        return max(1, v if kind == 0 else (v + 7) // 8 * 8 if kind == 1 else (v + 127) // 128 * 128)

    op = rng.choice(["quantise", "weights", "product", "product", "bf16rows", "bf16rows", "wgrad", "wgrad"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "quantise":
        k = size(16, 16384)
        return {"op": op, "T": max(1, min(size(1, 16384), 8192 * 4096 // (k * (2 if dtype == "f32" else 1)))), "K": k,
                "dtype": dtype, "transposed": rng.random() < 0.6, "random": rng.random() < 0.4}
    if op == "weights":
        return {"op": op, "shapes": ",".join("%dx%d" % (size(1, 8192), size(1, 8192)) for _ in range(rng.randrange(1, 4))), "dtype": dtype}
    n, k = size(32, 16384), size(32, 16384)
    t = max(1, min(size(1, 16384), 8192 * 14336 * 4096 // (2 * n * k)))
    if op == "wgrad":
        return {"op": op, "T": t, "N": n, "K": k, "add": rng.random() < 0.5, "dtype": dtype}
    return {"op": op, "T": t, "N": n, "K": k, "transpose": rng.random() < 0.5, "dtype": dtype}


# ---------------------------------------------------------------- inputs --

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _up(n, a):
    return (n + a - 1) // a * a


def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


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


def _operands(case, seed):
    """The values that a product's operands are quantised from."""
    gen = _generator(seed)
    t, n, k = case["T"], case["N"], case["K"]
    if case["op"] == "wgrad":
        dy = _tokens(gen, t, n, 1e-3, torch.bfloat16)
        x = _tokens(gen, t, k, 1.0, torch.bfloat16)
        return dy, x, (0.05 * _normal(gen, n, k)).to(_type(case["dtype"])) if case["add"] else None
    a = _tokens(gen, t, n if case["transpose"] else k, 1e-3 if case["transpose"] else 1.0, torch.bfloat16)
    return a, (0.02 * _normal(gen, n, k)).to(torch.bfloat16)


def prepare(case, seed):
    op, dtype = case["op"], _type(case["dtype"])
    state = {"case": case, "dtype": dtype}
    if op == "quantise":
        gen = _generator(seed)
        state["x"] = _tokens(gen, case["T"], case["K"], 1.0, dtype)
        state["random"] = torch.randint(0, 256, (case["T"], case["K"]), generator=gen, device="cuda", dtype=torch.uint8) if case["random"] else None
    elif op == "weights":
        gen = _generator(seed)
        state["w"] = [(0.02 * _normal(gen, r, c)).to(dtype) for r, c in _shapes(case)]
    elif op == "wgrad":
        dy, x, state["base"] = _operands(case, seed)
        state["dy"], state["x"] = _packed(dy.t()), _packed(x.t())
    else:
        a, w = _operands(case, seed)
        state["a"] = a if op == "bf16rows" else _packed(a)
        state["w"] = _packed(w.t() if case["transpose"] else w)
    return state


# ------------------------------------------------------------ plain forms --

def _power(e):
    """2^e as fp32, for e in the format's range."""
    return ((e + 127) << 23).view(torch.float32)


def _blocks(x):
    """x in fp32 as [R, blocks, 32], zeros behind its columns, and each block's e."""
    r, c = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _up(c, PAD) - c)).view(r, -1, BLOCK)
    bits = v.abs().amax(2).view(torch.int32)
    e = (bits >> 23) - 129 + ((bits & 0x7FFFFF) > 0x400000).to(torch.int32)
    return v, e.clamp(LO, HI)


def _rounded(v, e, random=None):
    """v * 2^-e rounded to E2M1, as fp32."""
    q = v * _power(-e)[:, :, None]
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    n = a / step
    if random is None:
        n = torch.round(n)
    else:
        f = torch.floor(n)
        n = f + (n - f >= (255.5 - random) / 256).float()
    return torch.copysign(n * step, q)


def _values(x, random=None):
    """What x's codes along its rows stand for."""
    r, c = x.shape
    v, e = _blocks(x)
    if random is not None:
        random = torch.nn.functional.pad(random.float(), (0, v.shape[1] * BLOCK - c)).view(v.shape)
    return (_rounded(v, e, random) * _power(e)[:, :, None]).view(r, -1)[:, :c]


def _packed(x):
    """x's codes along its rows, two to a byte, and scales."""
    r, c = x.shape
    v, e = _blocks(x)
    q = _rounded(v, e).view(r, -1)
    a = 2 * q.abs()  # 0 1 2 3 4 6 8 12
    code = torch.where(a < 4, a, torch.where(a < 8, a / 2 + 2, a / 4 + 4)).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    scales = torch.nn.functional.pad((e + 127).to(torch.uint8).t(), (0, _up(r, 16) - r), value=LO + 127).contiguous()
    return {"codes": code[:, 0::2] | (code[:, 1::2] << 4), "scales": scales, "rows": r, "cols": c}


def _unpacked(q):
    """The values of packed codes, with those behind the columns."""
    code = torch.stack((q["codes"] & 15, q["codes"] >> 4), 2).view(q["rows"], -1)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    v = table[(code & 7).int()] * (1 - 2 * (code >> 3).float())
    s = _power(q["scales"][:, :q["rows"]].t().to(torch.int32) - 127)
    return (v.view(q["rows"], -1, BLOCK) * s[:, :, None]).view(q["rows"], -1)


def _plain(s):
    case = s["case"]
    if case["op"] == "quantise":
        x, random = s["x"], s["random"]
        out = {"values": _values(x, random).to(torch.bfloat16)}
        if case["transposed"]:
            out["values_t"] = _values(x.t(), None if random is None else random.t()).to(torch.bfloat16)
        return out
    if case["op"] == "weights":
        return [{"values": _values(w).to(torch.bfloat16), "values_t": _values(w.t()).to(torch.bfloat16)} for w in s["w"]]
    if case["op"] == "wgrad":
        out = _unpacked(s["dy"]) @ _unpacked(s["x"]).t()
        return (out if s["base"] is None else s["base"].float() + out).to(s["dtype"])
    if case["op"] == "bf16rows":
        return (s["a"].float() @ _unpacked(s["w"])[:, :s["w"]["cols"]].t()).to(s["dtype"])
    return (_unpacked(s["a"]) @ _unpacked(s["w"]).t()).to(s["dtype"])


# ---------------------------------------------------- the framework's calls --

def _q4(nsd, q, transposed=False):
    if transposed:
        return nsd.Q4Matrix(codes_t=q["codes"], scales_t=q["scales"], rows=q["cols"], cols=q["rows"])
    return nsd.Q4Matrix(codes=q["codes"], scales=q["scales"], rows=q["rows"], cols=q["cols"])


def _own(s):
    import newton_schulz_dmuon_amd as nsd
    case = s["case"]
    if case["op"] == "quantise":
        q = nsd.q4_quantize(s["x"], transposed=case["transposed"], random=s["random"])
        out = {"values": nsd.q4_dequantize(q)}
        if case["transposed"]:
            out["values_t"] = nsd.q4_dequantize(q, transpose=True)
        return out
    if case["op"] == "weights":
        return [{"values": nsd.q4_dequantize(q), "values_t": nsd.q4_dequantize(q, transpose=True)}
                for q in nsd.q4_quantize_weights(s["w"])]
    if case["op"] == "wgrad":
        return nsd.q4_weight_grad(_q4(nsd, s["dy"], True), _q4(nsd, s["x"], True), dtype=s["dtype"], base=s["base"])
    a = s["a"] if case["op"] == "bf16rows" else _q4(nsd, s["a"])
    return nsd.q4_matmul(a, _q4(nsd, s["w"], case["transpose"]), transpose=case["transpose"], dtype=s["dtype"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work --

def work(case):
    item = 2 if case["dtype"] == "bf16" else 4
    packed = 0.5 + 1 / BLOCK  # bytes an element: half a byte and its share of a scale
    if case["op"] == "quantise":
        forms = 2 if case["transposed"] else 1
        # x read; the codes written, then read back; the values written
        return {"bytes": case["T"] * case["K"] * (item + case["random"] + forms * (2 * packed + 2)), "flops": 4 * forms * case["T"] * case["K"]}
    if case["op"] == "weights":
        elems = sum(r * c for r, c in _shapes(case))
        return {"bytes": elems * (item + 2 * (2 * packed + 2)), "flops": 8 * elems}
    t, n, k = case["T"], case["N"], case["K"]
    if case["op"] == "wgrad":
        return {"bytes": packed * t * (n + k) + item * n * k * (2 if case["add"] else 1), "flops": 2 * t * n * k}
    inner, outer = (n, k) if case["transpose"] else (k, n)
    return {"bytes": t * inner * (2 if case["op"] == "bf16rows" else packed) + packed * n * k + item * t * outer, "flops": 2 * t * n * k}


# --------------------------------------------- the definition in 64 bits --

def _exact_power(e):
    """2^e as fp64 (pow is not exact on the device)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(x, random=None):
    """What x's codes along its rows stand for: of each element's two
    neighbours among the codes, the one that the format takes."""
    r, c = x.shape
    v = torch.zeros(r, _up(c, BLOCK), dtype=torch.float64, device=x.device)
    v[:, :c] = x
    v = v.view(r, -1, BLOCK)
    amax = v.abs().amax(2, keepdim=True)
    _, p = torch.frexp(amax)
    e = p - 3
    e = e + (amax > 6 * _exact_power(e)).to(e.dtype)
    scale = _exact_power(torch.where(amax > 0, e, LO).clamp(LO, HI))
    a = v.abs() / scale
    codes = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    low = torch.bucketize(a, codes[1:], right=True).clamp(max=6)  # codes[low] <= a <= codes[low + 1]
    part = (a - codes[low]) / (codes[low + 1] - codes[low])
    if random is None:
        up = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
    else:
        n = torch.zeros(r, v.shape[1] * BLOCK, dtype=torch.float64, device=x.device)
        n[:, :c] = random
        up = 256 * part + n.view(v.shape) >= 255.5
    q = codes[low + up.to(low.dtype)] * scale
    return torch.where(v < 0, -q, q).view(r, -1)[:, :c]


def exact(case, seed):
    if case["op"] == "quantise":
        s = prepare(case, seed)
        out = {"values": _exact_values(s["x"], s["random"])}
        if case["transposed"]:
            out["values_t"] = _exact_values(s["x"].t(), None if s["random"] is None else s["random"].t())
        return out
    if case["op"] == "weights":
        return [{"values": _exact_values(w), "values_t": _exact_values(w.t())} for w in prepare(case, seed)["w"]]
    if case["op"] == "wgrad":
        dy, x, base = _operands(case, seed)
        out = _exact_values(dy.t()) @ _exact_values(x.t()).t()
        return out if base is None else base.double() + out
    a, w = _operands(case, seed)
    a = a.double() if case["op"] == "bf16rows" else _exact_values(a)
    return a @ _exact_values(w.t() if case["transpose"] else w).t()
