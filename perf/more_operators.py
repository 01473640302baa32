"""Cases, plain forms and work of the products in 8-bit floating point that stand beside
the W4A16 products:

  quantize        bf16 rows or weights in e4m3, a scale for 128 elements of a row or for
                  a block of 128 x 128
  gemm            the product of both, and with ``grad`` the gradient of its rows (the
                  same weights, summed over their rows)
  grouped         the same by expert, groups of ragged sizes on the device
  wgrad           the gradient of the experts' weights from bf16 rows

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits; with
``own`` true it calls the library.  A block's scale is max |x| / 448 and its codes are
448 x / max |x| rounded to the nearest e4m3, ties to even; a block of zeros has scale 0.
Row scales stand as [columns / 128, rows], weight scales as [rows / 128, columns / 128].
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the activations of a decode batch before a product: latency alone
        dict(name="quantize_decode", op="quantize", rows=16, width=8192, blocks=False, experts=0),
        # the rows of a long prefill, in expert order
        dict(name="quantize_prefill", op="quantize", rows=65536, width=4096, blocks=False, experts=0),
        # a layer's experts after a step of the optimiser
        dict(name="quantize_weights", op="quantize", rows=2048, width=4096, blocks=True, experts=8),
        # one token
        dict(name="gemm_decode", op="gemm", tokens=1, rows=8192, width=8192, grad=False),
        # a decode batch of odd size
        dict(name="gemm_decode_batch", op="gemm", tokens=61, rows=17408, width=5120, grad=False),
        # prefills of several requests, of ragged length together
        dict(name="gemm_prefill", op="gemm", tokens=2858, rows=19456, width=2560, grad=False),
        # the gradient that passes through a projection in a training step
        dict(name="gemm_grad", op="gemm", tokens=4096, rows=8192, width=8192, grad=True),
        # a decode batch of 16 tokens, 8 of 128 experts each
        dict(name="grouped_decode", op="grouped", tokens=128, experts=128, rows=2048, width=4096, skew=0.0,
             grad=False),
        # a long prefill over the same experts
        dict(name="grouped_prefill", op="grouped", tokens=65536, experts=128, rows=2048, width=4096, skew=0.3,
             grad=False),
        # its gradient in a training step, a row count that ends inside a block
        dict(name="grouped_grad", op="grouped", tokens=16384, experts=64, rows=1000, width=5120, skew=0.5,
             grad=True),
        # the weights' gradients of eight experts
        dict(name="wgrad_experts", op="wgrad", tokens=4096, experts=8, rows=2048, width=4096, skew=0.5,
             dtype="float32"),
        # a projection's weight gradient, in the weights' type
        dict(name="wgrad_projection", op="wgrad", tokens=4096, experts=1, rows=8192, width=8192, skew=0.0,
             dtype="bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "grouped", "grouped", "wgrad"])
    width = 128 * _log(rng, 4, 76)
    rows = _log(rng, 500, 19456)
    if rng.random() < 0.7:
        rows = rows // 8 * 8
    if op == "quantize":
        if rng.random() < 0.3:
            return dict(op=op, rows=rows, width=width, blocks=True, experts=rng.choice([0, 1, 3, 8]))
        if rng.random() < 0.3:
            width = _log(rng, 500, 9728)              # a gradient's width need not be a multiple of 128
        tokens = min(_log(rng, 1, 65536), 65536 * 4096 // width)
        return dict(op=op, rows=tokens, width=width, blocks=False, experts=0)
    if op == "gemm":
        tokens = min(_log(rng, 1, 8192), 4096 * 8192 * 8192 // (rows * width))
        return dict(op=op, tokens=max(1, tokens), rows=rows, width=width, grad=rng.random() < 0.4)
    width, rows = 128 * _log(rng, 4, 40), _log(rng, 500, 5120) // 8 * 8
    experts = _log(rng, 1, 128)
    experts = max(1, min(experts, 128 * 2048 * 4096 // (rows * width)))
    tokens = min(_log(rng, 16, 65536), 65536 * 2048 * 4096 // (rows * width) // (4 if op == "wgrad" else 1))
    case = dict(op=op, tokens=tokens, experts=experts, rows=rows, width=width, skew=rng.choice([0.0, 0.5, 1.5]))
    if op == "wgrad":
        case["dtype"] = rng.choice(["float32", "bfloat16"])
    else:
        case["grad"] = rng.random() < 0.4
    return case


# ------------------------------------------------------------------ inputs
def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + sum(map(ord, case["op"])))
    return g


def _normal(g, shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _activations(g, rows, width):
    """Rows with a few strong channels."""
    x = _normal(g, (rows, width))
    spread = torch.exp(0.5 * torch.randn(width, device="cuda", generator=g))
    return x.mul_(spread.to(torch.bfloat16))


def _weights(g, shape):
    """Codes and block scales of normal weights, an expert at a time."""
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(shape[:-2] + (-(-shape[-2] // 128), shape[-1] // 128), device="cuda")
    for c, s in zip(codes.view((-1,) + shape[-2:]), scales.view((-1,) + scales.shape[-2:])):
        code, scale = _plain_quantize(_normal(g, shape[-2:], shape[-1] ** -0.5), True)
        c.copy_(code)
        s.copy_(scale)
    return codes, scales


def _sizes(case, g):
    """Rows of each expert: a multinomial draw of popularities."""
    E, T = case["experts"], case["tokens"]
    liked = torch.softmax(case["skew"] * torch.randn(E, device="cuda", generator=g), 0)
    ids = torch.multinomial(liked, T, replacement=True, generator=g)
    return (ids[:, None] == torch.arange(E, device="cuda")).sum(0, dtype=torch.int32)


def prepare(case, seed):
    g = _generator(case, seed)
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        shape = (case["rows"], case["width"])
        if case["blocks"]:
            s["x"] = _normal(g, ((case["experts"],) if case["experts"] else ()) + shape, case["width"] ** -0.5)
        else:
            s["x"] = _activations(g, *shape)
        return s
    T, N, K = case["tokens"], case["rows"], case["width"]
    if op != "gemm":
        s["sizes"] = _sizes(case, g)
        s["counts"] = s["sizes"].tolist()
    if op == "wgrad":
        s["dy"], s["x"] = _normal(g, (T, N)), _activations(g, T, K)
        return s
    s["w"], s["ws"] = _weights(g, (case["experts"], N, K) if op == "grouped" else (N, K))
    s["x"], s["xs"] = _plain_quantize(_activations(g, T, N if case["grad"] else K), False)
    return s


# ------------------------------------------------------------- plain forms
def _plain_quantize(x, blocks):
    x = x.float()
    if not blocks:
        rows, width = x.shape
        x = torch.nn.functional.pad(x, (0, -width % 128)).view(rows, -1, 128)
        most = x.abs().amax(2)
        # 448 x has 11 significant bits: the quotient rounded to 32 bits rounds on as the exact one
        codes = torch.where(most[..., None] > 0, x * 448.0 / most[..., None], x)
        return codes.view(rows, -1).to(torch.float8_e4m3fn), (most / 448.0).t().contiguous()
    *lead, rows, width = x.shape
    x = torch.nn.functional.pad(x, (0, 0, 0, -rows % 128)).view(*lead, -(-rows // 128), 128, width // 128, 128)
    most = x.abs().amax((-3, -1))
    codes = torch.where(most[..., None, :, None] > 0, x * 448.0 / most[..., None, :, None], x)
    codes = codes.reshape(*lead, -1, width)[..., :rows, :]
    return codes.to(torch.float8_e4m3fn), most / 448.0


def _rows(s):
    return s["x"].float() * s["xs"].t().repeat_interleave(128, 1)


def _dense(codes, scales):
    spread = scales.repeat_interleave(128, 0)[:codes.shape[0]].repeat_interleave(128, 1)
    return codes.float() * spread


def _plain_product(x, w, grad):
    return x[:, :w.shape[0]] @ w if grad else x @ w.t()


def _plain_wgrad(s):
    dtype = getattr(torch, s["dtype"])
    dw = torch.zeros((s["experts"], s["rows"], s["width"]), dtype=dtype, device="cuda")
    row = 0
    for e, n in enumerate(s["counts"]):
        if n:
            dw[e] = (s["dy"][row:row + n].float().t() @ s["x"][row:row + n].float()).to(dtype)
        row += n
    return dw


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _plain_quantize(s["x"], s["blocks"])
    if op == "wgrad":
        return _plain_wgrad(s)
    x = _rows(s)
    if op == "gemm":
        return _plain_product(x, _dense(s["w"], s["ws"]), s["grad"]).to(torch.bfloat16)
    y = torch.empty((s["tokens"], s["width"] if s["grad"] else s["rows"]), dtype=torch.bfloat16, device="cuda")
    row = 0
    for e, n in enumerate(s["counts"]):
        if n:
            y[row:row + n] = _plain_product(x[row:row + n], _dense(s["w"][e], s["ws"][e]), s["grad"]).to(torch.bfloat16)
        row += n
    return y


def run(s):
    if not own:
        return _plain(s)
    import bf16_activation_quantized_gb300 as w4
    op = s["op"]
    if op == "quantize":
        return w4.quantize_fp8(s["x"], blocks=s["blocks"])
    if op == "gemm":
        return w4.gemm_fp8(s["x"], s["xs"], s["w"], s["ws"], transposed=s["grad"])
    if op == "grouped":
        return w4.gemm_fp8_grouped(s["x"], s["xs"], s["w"], s["ws"], s["sizes"], transposed=s["grad"])[0]
    return w4.gemm_grouped_wgrad(s["dy"], s["x"], s["sizes"], dtype=getattr(torch, s["dtype"]))[0]


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    N, K = case["rows"], case["width"]
    if op == "quantize":
        count = max(1, case["experts"]) * N * K
        scales = count / (128 * 128 if case["blocks"] else 128)
        return {"bytes": 3.0 * count + 4.0 * scales, "flops": 2.0 * count}
    T = case["tokens"]
    weights = N * K + 4.0 * -(-N // 128) * (K // 128)
    if op == "wgrad":
        each = 4 if case["dtype"] == "float32" else 2
        return {"bytes": 2.0 * T * (N + K) + each * case["experts"] * N * K, "flops": 2.0 * T * N * K}
    summed, out = (N, K) if case["grad"] else (K, N)
    summed = -(-summed // 128) * 128
    used = 1.0
    if op == "grouped":
        E = case["experts"]
        used = E * (1.0 - (1.0 - 1.0 / E) ** T) if E > 1 else 1.0
    return {"bytes": T * summed * (1 + 4 / 128) + used * weights + 2.0 * T * out, "flops": 2.0 * T * N * K}


# ------------------------------------------------------- from the definition
def _exact_codes(x, most):
    """448 x / most at the nearest multiple of the step of its binade, in 64 bits."""
    q = torch.where(most > 0, 448.0 * x / most, 0.0)
    exponent = torch.frexp(q).exponent - 1
    step = torch.exp2((exponent.clamp(min=-6) - 3).double())
    return torch.round(q / step) * step


def _exact_quantize(s):
    x = s["x"].double()
    if not s["blocks"]:
        parts = x.split(128, 1)
        most = [p.abs().max(1).values for p in parts]
        codes = [torch.nn.functional.pad(_exact_codes(p, m[:, None]), (0, 128 - p.shape[1]))
                 for p, m in zip(parts, most)]
        return torch.cat(codes, 1), torch.stack(most) / 448.0
    shape = x.shape
    codes, scales = [], []
    for w in x.reshape((-1,) + shape[-2:]):
        for band in w.split(128, 0):
            parts = band.split(128, 1)
            most = [p.abs().max() for p in parts]
            codes.append(torch.cat([_exact_codes(p, m) for p, m in zip(parts, most)], 1))
            scales.append(torch.stack(most))
    lead = tuple(shape[:-2])
    return (torch.cat(codes).reshape(shape),
            torch.stack(scales).reshape(lead + (-(-shape[-2] // 128), shape[-1] // 128)) / 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(s)
    if op == "wgrad":
        dw = []
        for dy, x in zip(s["dy"].split(s["counts"]), s["x"].split(s["counts"])):
            dw.append(torch.einsum("tn,tk->nk", dy.double(), x.double()))
        return torch.stack(dw)
    groups = [(s["x"], s["xs"], s["w"], s["ws"])]
    if op == "grouped":
        groups = list(zip(s["x"].split(s["counts"]), s["xs"].split(s["counts"], 1), s["w"], s["ws"]))
    out = []
    for x, xs, w, ws in groups:
        # block by block of the summed side: codes first, then both scales
        x, w, xs, ws = x.double(), w.double(), xs.double(), ws.double()
        if case["grad"]:
            y = torch.zeros((x.shape[0], w.shape[1] // 128, 128), dtype=torch.float64, device="cuda")
            for b in range(ws.shape[0]):
                part = w[128 * b:128 * b + 128]
                p = torch.einsum("tn,nk->tk", x[:, 128 * b:128 * b + part.shape[0]], part)
                y += xs[b][:, None, None] * ws[b][:, None] * p.view(y.shape)
            out.append(y.flatten(1))
        else:
            y = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device="cuda")
            each = ws.repeat_interleave(128, 0)[:w.shape[0]]
            for b in range(ws.shape[1]):
                p = torch.einsum("tk,nk->tn", x[:, 128 * b:128 * b + 128], w[:, 128 * b:128 * b + 128])
                y += xs[b][:, None] * each[:, b] * p
            out.append(y)
    return torch.cat(out)
