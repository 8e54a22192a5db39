"""The cases that the two ends of a training step are measured on, in two forms.

Four operators, each reached through the package's tensor-level calls:

  embedding              out[t] = scale * table[tokens[t]], the rows of a table that a model's tokens
                         look up, in the table's type or another: embedding
  embedding gradient     dw[v] = scale * sum of dy[t] over the t whose token is v (+ dw[v]): what the
                         lookup gives back, written or added to the gradient that is there (the
                         output projection's, where a model ties the two): embedding_backward
  gradient norm          |scale| * sqrt(sum of squares) over all of a model's gradients, and over each
                         of them, as a training log shows them: grad_norm
  clipping               the gradients times scale * min(1, max_norm / norm), in place or into the
                         gradients of the weights' own type: clip_grad_norm

With own = False a pass computes the operators' plain form (elementary torch operations in 32 bits,
rounded once at the end); with own = True it makes the package's calls.
"""
import math

import torch

own = False

IGNORE = -100   # the token of a place that takes no part
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LOSS_SCALE = 16384.0  # of fp16 gradients


def listed():
    return [
        # the next token of one sequence: latency alone
        {"name": "embed 1 bf16", "op": "embed", "dtype": "bf16", "to": "bf16", "T": 1, "V": 32768, "D": 4096, "scale": 1.0, "keep": 1.0},
        # fp32 weights looked up for a 16-bit model that scales its embeddings; odd rows, some places padding
        {"name": "embed 2047 f32 to bf16", "op": "embed", "dtype": "f32", "to": "bf16", "T": 2047, "V": 50021, "D": 1001, "scale": 31.6, "keep": 0.9},
        # a batch of long sequences over a large vocabulary
        {"name": "embed 65536 bf16", "op": "embed", "dtype": "bf16", "to": "bf16", "T": 65536, "V": 131072, "D": 4096, "scale": 1.0, "keep": 1.0},
        # a small model's step in fp32, its rows of odd length, added to the tied projection's gradient
        {"name": "embed grad 61 f32 added", "op": "embed grad", "dtype": "f32", "to": "f32", "T": 61, "V": 8191, "D": 769, "scale": 1.0, "keep": 1.0, "add": True},
        # one sequence's step: nearly all rows of the gradient are zero, all are written
        {"name": "embed grad 4096 bf16", "op": "embed grad", "dtype": "bf16", "to": "bf16", "T": 4096, "V": 65536, "D": 4096, "scale": 1.0, "keep": 1.0, "add": False},
        # fp16 under a loss scale, ragged in every size, some places padding
        {"name": "embed grad 16383 f16", "op": "embed grad", "dtype": "f16", "to": "f16", "T": 16383, "V": 50021, "D": 1000, "scale": 31.6, "keep": 0.8, "add": False},
        # a batch of long sequences, added to the fp32 gradient of the steps before it
        {"name": "embed grad 65536 bf16 to f32 added", "op": "embed grad", "dtype": "bf16", "to": "f32", "T": 65536, "V": 131072, "D": 2048, "scale": 1.0, "keep": 1.0, "add": True},
        # a model of 110 tensors in fp16 under a loss scale, packed without gaps, of odd sizes
        {"name": "norm 12 x 1001 f16", "op": "norm", "dtype": "f16", "layers": 12, "hidden": 1001, "ffn": 2731, "vocab": 50021, "packed": True},
        # 4 layers of a large model with its embedding
        {"name": "norm 4 x 4096 bf16", "op": "norm", "dtype": "bf16", "layers": 4, "hidden": 4096, "ffn": 11008, "vocab": 65536, "packed": False},
        # a small model's gradients within the limit, in place: the norm, and nothing to write
        {"name": "clip 1 x 256 f32", "op": "clip", "dtype": "f32", "to": None, "layers": 1, "hidden": 256, "ffn": 704, "vocab": 5000, "packed": False, "over": 0.4},
        # the fp16 model's gradients taken out of the loss scale and clipped, as fp32
        {"name": "clip 12 x 1001 f16 to f32", "op": "clip", "dtype": "f16", "to": "f32", "layers": 12, "hidden": 1001, "ffn": 2731, "vocab": 50021, "packed": True, "over": 5.0},
        # the large model's, clipped into buffers of their own type
        {"name": "clip 4 x 4096 bf16", "op": "clip", "dtype": "bf16", "to": "bf16", "layers": 4, "hidden": 4096, "ffn": 11008, "vocab": 65536, "packed": False, "over": 2.5},
    ]


def _size(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["embed", "embed grad", "embed grad", "norm", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("embed", "embed grad"):
        T, V, D = _size(rng, 1, 65536), _size(rng, 256, 131072), _size(rng, 64, 4096)
        if rng.random() < 0.5:  # rows that begin on 16 bytes, as most models' do
            D = (D + 7) // 8 * 8
        while op == "embed grad" and max(2 * T, V) * D > 131072 * 2048:
            T, V = max(1, T // 2), max(256, V // 2)
        case = {"op": op, "dtype": dtype, "T": T, "V": V, "D": D, "scale": rng.choice([1.0, math.sqrt(D)]), "keep": rng.choice([1.0, 1.0, 0.9, 0.3])}
        if op == "embed":
            return dict(case, to=rng.choice([dtype, "bf16"]))
        return dict(case, to=rng.choice([dtype, "f32"]), add=rng.random() < 0.5)
    hidden = _size(rng, 64, 4096)
    if rng.random() < 0.6:
        hidden = (hidden + 7) // 8 * 8
    ffn, vocab, layers = int(hidden * rng.uniform(2.0, 4.0)), _size(rng, 256, 65536), _size(rng, 1, 24)
    while layers > 1 and layers * (4 * hidden * hidden + 3 * hidden * ffn) > 8e8:
        layers //= 2
    case = {"op": op, "dtype": dtype, "layers": layers, "hidden": hidden, "ffn": ffn, "vocab": vocab, "packed": rng.random() < 0.5}
    if op == "norm":
        return case
    # in place only within the limit and with no loss scale: what is scaled in place is another input for the next pass
    to = rng.choice([None if dtype != "f16" else "f32", dtype, "f32"])
    return dict(case, to=to, over=0.4 if to is None else rng.choice([0.4, 2.5, 20.0]))


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tokens(g, T, V, keep):
    """Tokens as text has them: the r-th most frequent one appears in proportion to 1 / r."""
    u = torch.rand(T, device="cuda", generator=g, dtype=torch.float64)
    ids = (torch.exp(u * math.log(V)).long() - 1).clamp(0, V - 1)
    return torch.where(torch.rand(T, device="cuda", generator=g) < keep, ids, IGNORE)


def _shapes(case):
    """A model's gradients: the embedding's, and four square, three wide matrices and two vectors a layer."""
    h, f = case["hidden"], case["ffn"]
    return [(case["vocab"], h)] + case["layers"] * [(h,), (h, h), (h, h), (h, h), (h, h), (h,), (f, h), (f, h), (h, f)]


def _elements(case):
    return sum(math.prod(s) for s in _shapes(case))


def _views(buffers, case, matrices):
    """The tensors of the model in flat buffers, one of `matrices`' type and one, in fp32, for the vectors; packed without
    gaps, or each from a multiple of 64 elements on."""
    at, out = {}, []
    for shape in _shapes(case):
        kind = "f32" if len(shape) == 1 else matrices
        n, start = math.prod(shape), at.get(kind, 0)
        at[kind] = start + (n if case["packed"] else -(-n // 64) * 64)
        if buffers is not None:
            out.append(buffers[kind][start:start + n].view(shape))
    return out, at


def _buffers(case, matrices, fill):
    _, sizes = _views(None, case, matrices)
    buffers = {kind: torch.full((n,), fill, dtype=DTYPES[kind], device="cuda") for kind, n in sizes.items()}
    return buffers, _views(buffers, case, matrices)[0]


def _loss_scale(case):
    return 1.0 / LOSS_SCALE if case["dtype"] == "f16" else 1.0


def _gradients(g, case):
    """Gradients of a size of their own for each tensor and row, the embedding's zero but for the tokens of a batch;
    together `over` long out of the loss scale."""
    buffers, views = _buffers(case, case["dtype"], 0.0)
    sizes = torch.exp(torch.randn(len(views), generator=torch.Generator().manual_seed(g.initial_seed())))
    sizes[0] = 1.0
    used = torch.rand(case["vocab"], device="cuda", generator=g) < 0.2
    share = [0.2] + [1.0] * (len(views) - 1)
    spread = math.exp(0.25)  # of the rows' sizes, exp(normal / 2): the mean of their squares is e^(1/2)
    length = math.sqrt(sum(x.numel() * float(s) ** 2 * p for x, s, p in zip(views, sizes, share))) * spread
    for i, (x, s) in enumerate(zip(views, sizes)):
        x.normal_(0.0, float(s) * case.get("over", 1.0) / (length * _loss_scale(case)), generator=g)
        if x.dim() == 2:
            x *= torch.exp(0.5 * torch.randn(x.size(0), 1, device="cuda", generator=g)).to(x.dtype)
    views[0].mul_(used.unsqueeze(1).to(views[0].dtype))
    return buffers, views


def prepare(case, seed):
    g, dtype = _generator(seed), DTYPES.get(case["dtype"])
    if case["op"] in ("embed", "embed grad"):
        T, V, D = case["T"], case["V"], case["D"]
        tokens = _tokens(g, T, V, case["keep"])
        if case["op"] == "embed":
            w = (torch.randn(V, D, device="cuda", generator=g) / math.sqrt(D)).to(dtype)
            return {"case": case, "w": w, "tokens": tokens}
        dy = torch.randn(T, D, device="cuda", generator=g) / math.sqrt(T)
        dw = torch.randn(V, D, device="cuda", generator=g).to(DTYPES[case["to"]]) if case["add"] else None
        return {"case": case, "dy": dy.to(dtype), "tokens": tokens, "dw": dw}
    buffers, views = _gradients(g, case)
    state = {"case": case, "buffers": buffers, "grads": views}
    if case["op"] == "clip":
        # where they go: other gradients of the same shapes, or the same ones
        state["out_buffers"], state["outs"] = (buffers, views) if case["to"] is None else _buffers(case, case["to"], float("nan") if case["packed"] else 0.0)
    if own:  # a program keeps its lists of gradients as it keeps the gradients
        import dense_gemm_14_gb300 as g14
        state["list"] = g14.GradList(views)
        if case["op"] == "clip" and case["to"] is not None:
            state["out_list"] = g14.GradList(state["outs"])
    return state


# ---- plain forms


def _plain_embed(s):
    case, w, tokens = s["case"], s["w"], s["tokens"]
    rows = w[tokens.clamp(min=0)].float() * case["scale"]
    return torch.where((tokens >= 0).unsqueeze(1), rows, 0.0).to(DTYPES[case["to"]])


def _plain_embed_grad(s):
    case, tokens = s["case"], s["tokens"]
    add = torch.where((tokens >= 0).unsqueeze(1), s["dy"].float() * case["scale"], 0.0)
    dw = s["dw"].float() if case["add"] else torch.zeros(case["V"], case["D"], device="cuda")
    dw.index_add_(0, tokens.clamp(min=0), add)
    if not case["add"]:
        return dw.to(DTYPES[case["to"]])
    if dw is not s["dw"]:
        s["dw"].copy_(dw)  # in place, as a step that adds its gradient does
    return s["dw"]


def _plain_norms(grads, scale):
    squares = torch.stack([x.float().square().sum() for x in grads]).double()
    return squares.sum().sqrt().mul(abs(scale)).float(), squares.sqrt().mul(abs(scale)).float()


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "embed":
            return {"out": _plain_embed(s)}
        if case["op"] == "embed grad":
            return {"dw": _plain_embed_grad(s)}
        norm, each = _plain_norms(s["grads"], _loss_scale(case))
        if case["op"] == "norm":
            return {"norm": norm, "each": each}
        factor = (1.0 / norm).clamp(max=1.0) * _loss_scale(case)
        for x, y in zip(s["grads"], s["outs"]):
            y.copy_(x.float() * factor)
        return {"norm": norm, "grads": s["out_buffers"]}
    import dense_gemm_14_gb300 as g14
    if case["op"] == "embed":
        return {"out": g14.embedding(s["w"], s["tokens"], scale=case["scale"], ignore_index=IGNORE, dtype=DTYPES[case["to"]])}
    if case["op"] == "embed grad":
        if case["add"]:
            return {"dw": g14.embedding_backward(s["dy"], s["tokens"], out=s["dw"], scale=case["scale"], beta=1.0, ignore_index=IGNORE)}
        return {"dw": g14.embedding_backward(s["dy"], s["tokens"], rows=case["V"], scale=case["scale"], ignore_index=IGNORE, dtype=DTYPES[case["to"]])}
    if case["op"] == "norm":
        norm, each = g14.grad_norm(s["list"], scale=_loss_scale(case), each=True)
        return {"norm": norm, "each": each}
    norm = g14.clip_grad_norm(s["list"], 1.0, scale=_loss_scale(case), out=s.get("out_list"))
    return {"norm": norm, "grads": s["out_buffers"]}


def _distinct(case):
    """How many rows of the table the tokens stand for, on average."""
    V, n = case["V"], max(1.0, case["T"] * case["keep"])
    top = min(V, 4096)
    each = [1.0 - (1.0 - math.log((r + 1) / r) / math.log(V)) ** n for r in range(1, top)]
    blocks, low = 0.0, top
    while low < V:  # the rest by blocks of near ranks
        high = min(V, low * 1.1 + 1)
        mid = 0.5 * (low + high)
        blocks += (high - low) * (1.0 - (1.0 - min(1.0, math.log1p(1.0 / mid) / math.log(V))) ** n)
        low = high
    return min(n, sum(each) + blocks)


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] in ("embed", "embed grad"):
        T, V, D, b, to = case["T"], case["V"], case["D"], size[case["dtype"]], size[case["to"]]
        n, rows = case["T"] * case["keep"], _distinct(case)
        if case["op"] == "embed":
            return {"bytes": 8 * T + rows * D * b + T * D * to, "flops": T * D}
        return {"bytes": 8 * T + n * D * b + (2 * rows if case["add"] else V) * D * to, "flops": 2 * n * D}
    n = _elements(case)
    vectors = case["layers"] * 2 * case["hidden"]
    read = (n - vectors) * size[case["dtype"]] + 4 * vectors
    if case["op"] == "norm" or case["to"] is None:
        return {"bytes": read + 4 * len(_shapes(case)), "flops": 2 * n}
    return {"bytes": read + (n - vectors) * size[case["to"]] + 4 * vectors, "flops": 3 * n}


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = torch.zeros(case["T"], case["D"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["tokens"] != IGNORE).squeeze(1)
        out[at] = torch.index_select(s["w"], 0, s["tokens"][at]).double() * case["scale"]
        return {"out": out}
    if case["op"] == "embed grad":
        at = torch.nonzero(s["tokens"] != IGNORE).squeeze(1)
        ids, order = torch.sort(s["tokens"][at], stable=True)
        rows, counts = torch.unique_consecutive(ids, return_counts=True)
        ends = torch.cumsum(counts, 0).tolist()
        dw = s["dw"].double() if case["add"] else torch.zeros(case["V"], case["D"], dtype=torch.float64, device="cuda")
        at = at[order]
        many = torch.nonzero(counts > 64).squeeze(1).tolist()
        for i in many:  # long sums one by one, the others together
            places = at[ends[i] - int(counts[i]):ends[i]]
            dw[rows[i]] += case["scale"] * s["dy"][places].double().sum(dim=0)
        start = torch.tensor([0] + ends[:-1], device="cuda")
        for k in range(64):
            has = torch.nonzero((counts > k) & (counts <= 64)).squeeze(1)
            if not has.numel():
                break
            dw[rows[has]] += case["scale"] * s["dy"][at[start[has] + k]].double()
        return {"dw": dw}
    squares = [float(x.double().square().sum()) for x in s["grads"]]
    norm = math.sqrt(math.fsum(squares)) * _loss_scale(case)
    out = {"norm": torch.tensor(norm, dtype=torch.float64)}
    if case["op"] == "norm":
        out["each"] = torch.tensor([math.sqrt(x) * _loss_scale(case) for x in squares], dtype=torch.float64)
        return out
    factor = min(1.0, 1.0 / norm) * _loss_scale(case)
    out["grads"] = {}
    for kind, buffer in s["out_buffers"].items():
        out["grads"][kind] = buffer.double()  # what lies between the tensors stays as it is
    into, _ = _views(out["grads"], case, case["to"] or case["dtype"])
    for x, y in zip(s["grads"], into):
        y.copy_(x.double() * factor)
    return out
