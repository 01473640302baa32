"""Cases, plain forms and work of the operators that stand beside the W4A16 products:

  dispatch / combine   rows sorted by expert for the grouped product and back with the
                       router's weights, each with its gradient
  lora                 low-rank adapters of many requests beside a shared projection,
                       served (forward) and trained (forward and backward)

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits; with
``own`` true it calls the library.  Conventions: an expert id outside [0, experts) drops its
slot, an adapter id outside [0, adapters) leaves its token without one.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a decode step picks 8 of 128 experts: latency alone
        dict(name="dispatch_decode", op="dispatch", tokens=1, top_k=8, experts=128, width=8192,
             ids64=False, drop=0.0, skew=0.0),
        # a prefill of ragged length over few experts, one of them popular
        dict(name="dispatch_ragged", op="dispatch", tokens=1322, top_k=2, experts=8, width=2560,
             ids64=False, drop=0.02, skew=1.0),
        # a long prefill, ids as torch.topk gives them
        dict(name="dispatch_prefill", op="dispatch", tokens=8192, top_k=8, experts=128, width=4096,
             ids64=True, drop=0.0, skew=0.3),
        # its gradient in a training step
        dict(name="dispatch_grad", op="dispatch_grad", tokens=4096, top_k=4, experts=64, width=5120,
             drop=0.01, skew=0.3),
        # a decode batch comes back from its experts
        dict(name="combine_decode", op="combine", tokens=16, top_k=8, experts=128, width=4096,
             drop=0.0, skew=0.0, weights="float32"),
        # a long prefill comes back
        dict(name="combine_prefill", op="combine", tokens=8192, top_k=8, experts=128, width=4096,
             drop=0.0, skew=0.3, weights="float32"),
        # a training step: gradients of the experts' rows and of the router's weights
        dict(name="combine_grad", op="combine_grad", tokens=4096, top_k=4, experts=64, width=5120,
             drop=0.01, skew=0.3, weights="bfloat16"),
        # one request decodes with its adapter
        dict(name="lora_decode", op="lora", tokens=1, adapters=8, rank=16, rows=8192, width=8192,
             segment=1, none=0.0),
        # a full decode batch, nearly every request with an adapter of its own, some with none
        dict(name="lora_decode_batch", op="lora", tokens=61, adapters=64, rank=32, rows=19456,
             width=2560, segment=1, none=0.1),
        # prefills of several requests in one batch, of ragged lengths
        dict(name="lora_prefill", op="lora", tokens=2858, adapters=12, rank=16, rows=17408,
             width=5120, segment=400, none=0.1),
        # training one adapter on frozen weights
        dict(name="lora_train", op="lora_train", tokens=4096, adapters=1, rank=64, rows=8192,
             width=8192, segment=4096, none=0.0),
        # training many small adapters in one batch, token by token mixed
        dict(name="lora_train_many", op="lora_train", tokens=2051, adapters=16, rank=8, rows=2560,
             width=9728, segment=1, none=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST = {"dispatch": 8192 * 8 * 4096, "combine": 8192 * 8 * 4096, "dispatch_grad": 4096 * 4 * 5120,
         "combine_grad": 4096 * 4 * 5120}


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "lora", "lora", "lora_train",
                     "lora_train"])
    if not op.startswith("lora"):
        top_k = rng.randint(1, 10)
        # the dispatched rows feed a product whose K is a multiple of 128; what comes back is any N
        width = 128 * _log(rng, 4, 76) if op.startswith("dispatch") else _log(rng, 500, 9728)
        if op.startswith("combine") and rng.random() < 0.6:
            width = max(8, width // 8 * 8)
        tokens = min(_log(rng, 1, 16384), _MOST[op] // (top_k * width))
        case = dict(op=op, tokens=tokens, top_k=top_k, experts=_log(rng, 2, 256), width=width,
                    drop=rng.choice([0.0, 0.02, 0.2]), skew=rng.choice([0.0, 0.5, 1.5]))
        if op == "dispatch":
            case["ids64"] = rng.random() < 0.5
        if op.startswith("combine"):
            case["weights"] = rng.choice(["float32", "bfloat16"])
        return case
    rank = rng.choice([8, 16, 16, 24, 32, 48, 64])
    width = 128 * _log(rng, 8, 76)
    rows = _log(rng, 1000, 19456)
    if rng.random() < 0.8:
        rows = rows // 8 * 8
    tokens = _log(rng, 1, 4096) if op == "lora" else _log(rng, 64, 4096)
    tokens = min(tokens, 4096 * 16384 // (rows + width))
    adapters = min(_log(rng, 1, 128), 2048 // rank)
    segment = rng.choice([1, 1, 37, 400])
    return dict(op=op, tokens=tokens, adapters=adapters, rank=rank, rows=rows, width=width,
                segment=segment, none=rng.choice([0.0, 0.1]))


# ------------------------------------------------------------------ inputs
def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + sum(map(ord, case["op"])))
    return g


def _normal(g, shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _uniform(g, shape):
    return torch.rand(shape, device="cuda", generator=g)


def _expert_ids(case, g):
    """Distinct experts per token as a router picks them (the largest of noisy, skewed logits);
    more slots than experts wrap around."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    liked = case["skew"] * torch.randn(E, device="cuda", generator=g)
    gumbel = -torch.log(-torch.log(_uniform(g, (T, E)).clamp(1e-6, 1 - 1e-6)))
    ids = torch.argsort(liked + gumbel, dim=1, descending=True)[:, torch.arange(k, device="cuda") % E]
    return torch.where(_uniform(g, (T, k)) < case["drop"], -1, ids).to(torch.int32)


def _adapter_ids(case, g):
    T, L, seg = case["tokens"], case["adapters"], case["segment"]
    n = -(-T // seg) + 1
    ids = torch.randint(0, L, (n,), device="cuda", generator=g)
    ids = torch.where(_uniform(g, (n,)) < case["none"], -1, ids)
    return ids.repeat_interleave(seg)[seg // 3:seg // 3 + T].to(torch.int32).contiguous()


def prepare(case, seed):
    g = _generator(case, seed)
    s = dict(case)
    if not case["op"].startswith("lora"):
        T, k, W = case["tokens"], case["top_k"], case["width"]
        ids = _expert_ids(case, g)
        if case["op"] == "dispatch":
            s["x"] = _normal(g, (T, W))
            s["ids"] = ids.long() if case["ids64"] else ids
            return s
        s["slots"] = _slots(ids, case["experts"])[0].to(torch.int32)
        if case["op"] != "combine_grad":
            s["ys"] = _normal(g, (T * k, W))
        else:
            s["ys"], s["dy"] = _normal(g, (T * k, W)), _normal(g, (T, W))
        if case["op"].startswith("combine"):
            w = _uniform(g, (T, k)) + 0.05
            s["w"] = (w / w.sum(1, keepdim=True)).to(getattr(torch, case["weights"]))
        return s
    T, L, r, N, K = (case[c] for c in ("tokens", "adapters", "rank", "rows", "width"))
    s["x"], s["base"] = _normal(g, (T, K)), _normal(g, (T, N))
    s["a"] = _normal(g, (L, r, K), K ** -0.5)
    s["b"] = _normal(g, (L, N, r), 0.2 * r ** -0.5)
    s["ids"] = _adapter_ids(case, g)
    s["scale"] = 0.5 + 1.5 * _uniform(g, (L,))
    if case["op"] == "lora_train":
        s["dy"] = _normal(g, (T, N))
    return s


# ------------------------------------------------------------- plain forms
def _slots(ids, experts):
    """Stable place of every slot in expert order, dropped ones last and marked ~place; the sizes."""
    key = ids.reshape(-1).long()
    key = torch.where((key >= 0) & (key < experts), key, experts)
    hot = (torch.arange(experts + 1, device=key.device)[:, None] == key).to(torch.int32)
    before = torch.cumsum(hot, 1, dtype=torch.int32)
    sizes = before[:, -1]
    start = torch.cumsum(sizes, 0) - sizes
    place = start[key] + before.gather(0, key[None])[0] - 1
    return torch.where(key < experts, place, ~place).reshape(ids.shape), sizes[:experts]


def _rows_of(slots):
    """The places with dropped ones mapped to their own row, and which are kept."""
    slots = slots.long()
    return torch.where(slots >= 0, slots, ~slots), slots >= 0


def _plain_dispatch(s):
    T, k = s["ids"].shape
    slots, sizes = _slots(s["ids"], s["experts"])
    place, kept = _rows_of(slots)
    xs = torch.empty((T * k, s["width"]), dtype=torch.bfloat16, device="cuda")
    rows = torch.where(kept[..., None], s["x"][:, None, :], torch.zeros((), dtype=torch.bfloat16, device="cuda"))
    xs[place.reshape(-1)] = rows.reshape(T * k, -1)
    return xs, sizes.to(torch.int32), slots.to(torch.int32)


def _plain_combine(ys, slots, w=None):
    place, kept = _rows_of(slots)
    rows = torch.where(kept[..., None], ys[place].float(), 0.0)
    if w is not None:
        rows = rows * w.float()[..., None]
    return rows.sum(1).to(torch.bfloat16)


def _plain_combine_grad(s):
    place, kept = _rows_of(s["slots"])
    dy = s["dy"].float()[:, None, :]
    dys = torch.empty_like(s["ys"])
    grad = torch.where(kept[..., None], dy * s["w"].float()[..., None], 0.0).to(torch.bfloat16)
    dys[place.reshape(-1)] = grad.reshape(dys.shape)
    dw = (torch.where(kept[..., None], s["ys"][place].float(), 0.0) * dy).sum(2)
    return dys, dw.to(s["w"].dtype)


def _plain_lora_few(s):
    """Few tokens: every token's own adapter gathered."""
    ids = s["ids"].long()
    has = (ids >= 0) & (ids < s["adapters"])
    at = torch.where(has, ids, 0)
    h = (s["a"][at].float() @ s["x"].float()[:, :, None])
    delta = (s["b"][at].float() @ h)[:, :, 0] * s["scale"][at][:, None]
    y = s["base"].float() + torch.where(has[:, None], delta, 0.0)
    return y.to(torch.bfloat16)


def _plain_lora(s, grad):
    """Many tokens: products with every adapter, all but the token's own masked out."""
    T, L, r, N, K = (s[c] for c in ("tokens", "adapters", "rank", "rows", "width"))
    mine = (s["ids"].long()[:, None] == torch.arange(L, device="cuda"))
    a = s["a"].float().reshape(L * r, K)
    b = s["b"].float().transpose(1, 2).reshape(L * r, N)
    scaled = torch.where(mine, s["scale"], 0.0)[..., None]
    has = mine.any(1, keepdim=True)
    x = torch.where(has, s["x"].float(), 0.0)
    h = torch.where(mine[..., None], (x @ a.t()).view(T, L, r), 0.0)
    y = (s["base"].float() + (h * scaled).view(T, L * r) @ b).to(torch.bfloat16)
    if not grad:
        return y
    dy = torch.where(has, s["dy"].float(), 0.0)
    g = (dy @ b.t()).view(T, L, r) * scaled
    g = torch.where(mine[..., None], g, 0.0).view(T, L * r)
    dx = (g @ a).to(torch.bfloat16)
    da = (g.t() @ x).view(L, r, K).to(torch.bfloat16)
    db = ((h * scaled).view(T, L * r).t() @ dy).view(L, r, N).transpose(1, 2)
    return y, dx, da, db.to(torch.bfloat16).contiguous()


def _plain(s):
    op = s["op"]
    if op == "dispatch":
        return _plain_dispatch(s)
    if op == "dispatch_grad":
        return _plain_combine(s["ys"], s["slots"])
    if op == "combine":
        return _plain_combine(s["ys"], s["slots"], s["w"])
    if op == "combine_grad":
        return _plain_combine_grad(s)
    if op == "lora" and s["tokens"] <= 64:
        return _plain_lora_few(s)
    return _plain_lora(s, op == "lora_train")


def run(s):
    if not own:
        return _plain(s)
    import bf16_activation_quantized_gb300 as w4
    op = s["op"]
    if op == "dispatch":
        return w4.dispatch(s["x"], s["ids"], s["experts"])
    if op == "dispatch_grad":
        return w4.dispatch_backward(s["ys"], s["slots"])
    if op == "combine":
        return w4.combine(s["ys"], s["slots"], s["w"])
    if op == "combine_grad":
        return w4.combine_backward(s["dy"], s["ys"], s["slots"], s["w"])
    if op == "lora":
        return w4.lora_add(s["x"], s["a"], s["b"], s["ids"], s["scale"], s["base"])
    y, hidden = w4.lora_add(s["x"], s["a"], s["b"], s["ids"], s["scale"], s["base"], return_hidden=True)
    return (y,) + w4.lora_add_backward(s["dy"], s["x"], hidden, s["a"], s["b"], s["ids"], s["scale"])


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if not op.startswith("lora"):
        T, k, W = case["tokens"], case["top_k"], case["width"]
        kept = T * k * (1.0 - case["drop"])
        if op == "dispatch":
            return {"bytes": T * k * (8 if case["ids64"] else 4) + 2.0 * T * W + 2.0 * T * k * W
                    + 4.0 * (T * k + case["experts"]), "flops": 0}
        if op == "dispatch_grad":
            return {"bytes": 2.0 * kept * W + 4.0 * T * k + 2.0 * T * W, "flops": kept * W}
        each = 4 if case["weights"] == "float32" else 2
        if op == "combine":
            return {"bytes": 2.0 * kept * W + (4 + each) * T * k + 2.0 * T * W, "flops": 2.0 * kept * W}
        return {"bytes": 2.0 * (kept + T * k + T) * W + (4 + 2 * each) * T * k, "flops": 3.0 * kept * W}
    T, L, r, N, K = (case[c] for c in ("tokens", "adapters", "rank", "rows", "width"))
    served = T * (1.0 - case["none"])
    draws = max(1.0, served / case["segment"])
    used = L * (1.0 - (1.0 - 1.0 / L) ** draws) if L > 1 else 1.0
    if op == "lora":
        return {"bytes": 2.0 * (served * K + 2 * T * N) + 2.0 * used * r * (K + N) + 4.0 * (T + L),
                "flops": 2.0 * served * r * (K + N)}
    return {"bytes": 2.0 * (served * K + 2 * T * N + served * N + T * K) + 2.0 * (used + L) * r * (K + N)
            + 4.0 * (T + L), "flops": 6.0 * served * r * (K + N)}


# ------------------------------------------------------- from the definition
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        return None          # copies and whole numbers
    if not op.startswith("lora"):
        slots = s["slots"].cpu()
        T, k = slots.shape
        # token by token over the kept slots, in blocks of tokens
        ys, out, dys, dw = s["ys"], [], None, None
        if op == "combine_grad":
            dys = torch.zeros(ys.shape, dtype=torch.float64, device="cuda")
            dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        else:
            out = torch.zeros((T, case["width"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(slots[:, j] >= 0)[:, 0].cuda()
            row = slots[:, j].cuda().long()[t]
            if op == "combine_grad":
                dy = s["dy"][t].double()
                dys[row] = dy * s["w"][t, j].double()[:, None]
                dw[t, j] = torch.einsum("tn,tn->t", dy, ys[row].double())
            else:
                w = s["w"][t, j].double()[:, None] if op == "combine" else 1.0
                out[t] += w * ys[row].double()
        return (dys, dw) if op == "combine_grad" else out
    y = s["base"].double()
    train = op == "lora_train"
    if train:
        dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
        da = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
        db = torch.zeros(s["b"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["adapters"]):
        t = torch.nonzero(s["ids"] == i)[:, 0]
        if not t.numel():
            continue
        x, a, b, c = s["x"][t].double(), s["a"][i].double(), s["b"][i].double(), s["scale"][i].double()
        h = torch.einsum("tk,rk->tr", x, a)
        y[t] += c * torch.einsum("tr,nr->tn", h, b)
        if train:
            dy = s["dy"][t].double()
            g = c * torch.einsum("tn,nr->tr", dy, b)
            dx[t] = torch.einsum("tr,rk->tk", g, a)
            da[i] = torch.einsum("tr,tk->rk", g, x)
            db[i] = c * torch.einsum("tn,tr->nr", dy, h)
    return (y, dx, da, db) if train else y
