"""The cases that the training products are measured on, in two forms.

Two operators, each reached through the package's tensor-level calls:

  linear cross entropy   loss[t] = log sum_v exp(h_t . w_v) - h_t . w_y(t), the loss of an output
                         projection H W^T over a vocabulary, and its gradients in H and W:
                         linear_cross_entropy, linear_cross_entropy_backward
  8-bit checkpoints      activations kept as 8-bit integers with a power-of-two scale for each 32 of
                         a row, put back, or multiplied as they are into a weight gradient:
                         ckpt8_save, ckpt8_restore, ckpt8_weight_grad

With own = False a pass computes the operators' plain form (elementary torch operations in 32 bits,
rounded once at the end); with own = True it makes the package's calls.
"""
import math

import torch

own = False

IGNORE = -100   # the target of a row that takes no part
BLOCK = 32      # columns of a row that share a scale
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # how likely the model finds one given token: a single row against the whole projection,
        # a call whose time is one read of the weights
        {"name": "ce score 1 bf16", "op": "ce", "train": False, "dtype": "bf16", "T": 1, "V": 32768, "D": 4096, "keep": 1.0},
        # the same for the tokens of a short answer, with padding and sizes that no tile divides
        {"name": "ce score 61 f16", "op": "ce", "train": False, "dtype": "f16", "T": 61, "V": 50021, "D": 2056, "keep": 0.9},
        # a small model's step in fp32, its rows of odd length
        {"name": "ce train 515 f32", "op": "ce", "train": True, "dtype": "f32", "T": 515, "V": 8191, "D": 769, "keep": 1.0},
        # an ordinary step on one sequence: the loss and both gradients
        {"name": "ce train 4096 bf16", "op": "ce", "train": True, "dtype": "bf16", "T": 4096, "V": 65536, "D": 4096, "keep": 1.0},
        # the same in fp16 under a loss scale, ragged in every size, some rows padding
        {"name": "ce train 2047 f16", "op": "ce", "train": True, "dtype": "f16", "T": 2047, "V": 50021, "D": 1000, "keep": 0.8},
        # training on answers alone: most rows are prompt and take no part; a large vocabulary
        {"name": "ce train 8192 masked bf16", "op": "ce", "train": True, "dtype": "bf16", "T": 8192, "V": 131072, "D": 2048, "keep": 0.3},
        # one token's activations kept and put back: latency alone
        {"name": "ckpt8 keep 1 bf16", "op": "keep", "dtype": "bf16", "T": 1, "K": 4096},
        # odd rows, the last block of each a short one
        {"name": "ckpt8 keep 2049 f16", "op": "keep", "dtype": "f16", "T": 2049, "K": 1001},
        # the hidden activations of a transformer's MLP over one long batch
        {"name": "ckpt8 keep 16384 bf16", "op": "keep", "dtype": "bf16", "T": 16384, "K": 11008},
        # the weight gradient of that MLP's down projection from its kept input
        {"name": "ckpt8 wgrad 8192 bf16", "op": "wgrad", "dtype": "bf16", "T": 8192, "N": 4096, "K": 11008, "beta": 0.0},
        # a small model's in fp32, odd sizes, added to the gradient that is there
        {"name": "ckpt8 wgrad 777 f32", "op": "wgrad", "dtype": "f32", "T": 777, "N": 1001, "K": 515, "beta": 1.0},
        # few tokens, added: one read and one write of the gradient
        {"name": "ckpt8 wgrad 16 f16", "op": "wgrad", "dtype": "f16", "T": 16, "N": 4096, "K": 4096, "beta": 1.0},
    ]


def _size(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["ce", "ce", "keep", "wgrad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "ce":
        train = rng.random() < 0.6
        T, V, D = _size(rng, 1, 8192), _size(rng, 1000, 131072), _size(rng, 128, 4096)
        while T * V * D > 8192 * 131072 * 2048:
            T = max(1, T // 2)
        if rng.random() < 0.5:  # rows that begin on 16 bytes, as most models' do
            D = (D + 7) // 8 * 8
        return {"op": "ce", "train": train, "dtype": dtype, "T": T, "V": V, "D": D, "keep": rng.choice([1.0, 0.9, 0.5, 0.2])}
    K = _size(rng, 33, 11008)
    if rng.random() < 0.5:
        K = (K + 31) // 32 * 32
    if op == "keep":
        return {"op": "keep", "dtype": dtype, "T": _size(rng, 1, 16384), "K": K}
    N = _size(rng, 64, 8192)
    if rng.random() < 0.5:
        N = (N + 7) // 8 * 8
    return {"op": "wgrad", "dtype": dtype, "T": _size(rng, 1, 8192), "N": N, "K": K, "beta": rng.choice([0.0, 1.0])}


def _kept_rows(case):
    """Rows that take part: the share of them, one at least."""
    return max(1, round(case["T"] * case["keep"]))


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, T, K):
    """Rows as a block's output has them: each of its own scale, a few columns far larger than the rest, some entries zero."""
    x = torch.randn(T, K, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(T, 1, device="cuda", generator=g))
    x *= torch.where(torch.rand(K, device="cuda", generator=g) < 0.01, 20.0, 1.0)
    return x * (torch.rand(T, K, device="cuda", generator=g) > 0.02)


def _padded(x, multiple):
    """x as a view of rows whose pitch is a multiple of `multiple` elements."""
    out = torch.zeros(x.size(0), -(-x.size(1) // multiple) * multiple, dtype=x.dtype, device=x.device)
    view = out[:, :x.size(1)]
    view.copy_(x)
    return view


def prepare(case, seed):
    g, dtype = _generator(seed), DTYPES[case["dtype"]]
    if case["op"] == "ce":
        T, V, D = case["T"], case["V"], case["D"]
        w = (0.02 * torch.randn(V, D, device="cuda", generator=g)).to(dtype)
        y = torch.randint(0, V, (T,), device="cuda", generator=g)
        # a model that has learnt some of its targets: their rows lean towards them
        lean = 8.0 * torch.rand(T, 1, device="cuda", generator=g) / (0.02 * math.sqrt(D))
        wy = w[y].float()
        h = (torch.randn(T, D, device="cuda", generator=g) + lean * wy / wy.norm(dim=1, keepdim=True)).to(dtype)
        at = torch.randperm(T, device="cuda", generator=g)[_kept_rows(case):]
        y[at] = IGNORE
        # the mean over the rows that take part, weighted by row; fp16 under a loss scale
        up = (0.5 + torch.rand(T, device="cuda", generator=g)) / _kept_rows(case)
        if case["dtype"] == "f16":
            up *= 16384.0
        return {"case": case, "h": h, "w": w, "y": y, "up": up}
    if case["op"] == "keep":
        return {"case": case, "x": _activations(g, case["T"], case["K"]).to(dtype)}
    q, s = _keep(_activations(g, case["T"], case["K"]).to(dtype))
    dy = (torch.randn(case["T"], case["N"], device="cuda", generator=g) / math.sqrt(case["T"])).to(dtype)
    dw = torch.randn(case["N"], case["K"], device="cuda", generator=g)
    return {"case": case, "q": _padded(q, 16), "s": _padded(s, 16), "dy": dy, "dw": dw}


# ---- plain forms


def _keep(x):
    """The 8-bit form of x: whole numbers q in [-127, 127] and a byte s for each 32 columns; a value stands for q 2^(s - 133)."""
    T, K = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).view(T, -1, BLOCK)
    _, e = torch.frexp(x.abs().amax(dim=2))             # largest = m 2^e, 1/2 <= m < 1
    s = (e + 126).clamp(7, 254)
    q = torch.ldexp(x, (133 - s).unsqueeze(2)).round().clamp(-127, 127)
    return q.view(T, -1)[:, :K].to(torch.int8), s.to(torch.uint8)


def _put_back(q, s):
    """The values that q and s stand for, in 32 bits."""
    T, K = q.shape
    scale = torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.int() - 133)
    return q.float() * scale.repeat_interleave(BLOCK, dim=1)[:, :K]


def _plain_ce(s):
    case, h, w, y = s["case"], s["h"].float(), s["w"].float(), s["y"]
    valid = y != IGNORE
    at = torch.where(valid, y, 0).unsqueeze(1)
    logits = h @ w.t()
    top = logits.amax(dim=1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(dim=1, keepdim=True))
    loss = torch.where(valid, (lse - logits.gather(1, at)).squeeze(1), 0.0)
    out = {"loss": loss, "lse": torch.where(valid, lse.squeeze(1), 0.0)}
    if case["train"]:
        p = logits.sub_(lse).exp_()
        p.scatter_add_(1, at, torch.full_like(lse, -1.0))
        p *= torch.where(valid, s["up"], 0.0).unsqueeze(1)
        out["dh"] = (p @ w).to(s["h"].dtype)
        out["dw"] = (p.t() @ h).to(s["h"].dtype)
    return out


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "ce":
            return _plain_ce(s)
        if case["op"] == "keep":
            return {"x": _put_back(*_keep(s["x"])).to(s["x"].dtype)}
        new = s["dy"].float().t() @ _put_back(s["q"], s["s"])
        if case["beta"]:
            s["dw"] += new  # in place, as a step that adds its gradient does
        else:
            s["dw"] = new
        return {"dw": s["dw"]}
    import dense_gemm_14_gb300 as g14
    mode = "3xtf32" if case["dtype"] == "f32" else None
    if case["op"] == "ce":
        loss, lse = g14.linear_cross_entropy(s["h"], s["w"], s["y"], ignore_index=IGNORE, fp32_mode=mode)
        out = {"loss": loss, "lse": lse}
        if case["train"]:
            out["dh"], out["dw"] = g14.linear_cross_entropy_backward(s["h"], s["w"], s["y"], lse, s["up"], ignore_index=IGNORE, fp32_mode=mode)
        return out
    if case["op"] == "keep":
        return {"x": g14.ckpt8_restore(g14.ckpt8_save(s["x"]), s["x"].dtype)}
    g14.ckpt8_weight_grad(s["dy"], g14.Ckpt8(s["q"], s["s"]), out=s["dw"], beta=case["beta"], fp32_mode=mode)
    return {"dw": s["dw"]}


def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ce":
        n, T, V, D = _kept_rows(case), case["T"], case["V"], case["D"]
        read, written = (n + V) * D * b + 8 * T, 8 * T
        if case["train"]:  # three products: logits, dH, dW
            return {"bytes": read + 4 * T + written + (T + V) * D * b, "flops": 6 * n * V * D}
        return {"bytes": read + written, "flops": 2 * n * V * D}
    kept = case["T"] * (case["K"] + -(-case["K"] // BLOCK))
    if case["op"] == "keep":  # the values in, the 8-bit form out and in again, the values out
        return {"bytes": 2 * (case["T"] * case["K"] * b + kept), "flops": 4 * case["T"] * case["K"]}
    T, N, K = case["T"], case["N"], case["K"]
    return {"bytes": T * N * b + kept + N * K * 4 * (2 if case["beta"] else 1), "flops": 2 * T * N * K}


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ce":
        if (6 if case["train"] else 2) * _kept_rows(case) * case["V"] * case["D"] > 1e13:
            return None
        rows = torch.nonzero(s["y"] != IGNORE).squeeze(1)
        h, w, y = s["h"][rows].double(), s["w"].double(), s["y"][rows]
        z = torch.einsum("td,vd->tv", h, w)
        lse = torch.logsumexp(z, dim=1)
        out = {}
        for name, v in (("loss", lse - z[torch.arange(len(y), device=z.device), y]), ("lse", lse)):
            out[name] = torch.zeros(case["T"], dtype=torch.float64, device=z.device).index_copy_(0, rows, v)
        if case["train"]:
            p = torch.softmax(z, dim=1)
            del z
            p[torch.arange(len(y), device=p.device), y] -= 1.0
            p *= s["up"][rows].double().unsqueeze(1)
            out["dh"] = torch.zeros(case["T"], case["D"], dtype=torch.float64, device=p.device).index_copy_(0, rows, torch.einsum("tv,vd->td", p, w))
            out["dw"] = torch.einsum("tv,td->vd", p, h)
        return out
    if case["op"] == "keep":
        x = s["x"].double()
        out = torch.empty_like(x)
        for c in range(0, case["K"], BLOCK):
            part = x[:, c:c + BLOCK]
            top = part.abs().amax(dim=1, keepdim=True)
            top = top.clamp_min(2.0 ** -120)
            power = torch.floor(torch.log2(top))  # may be one short at a power of two
            power = torch.where(torch.exp2(power + 1) <= top, power + 1, power)
            step = torch.exp2(power - 6)
            out[:, c:c + BLOCK] = torch.clamp(torch.round(part / step), -127, 127) * step
        return {"x": out}
    if 2 * case["T"] * case["N"] * case["K"] > 1e13:
        return None
    back = torch.empty(case["T"], case["K"], dtype=torch.float64, device="cuda")
    for c in range(0, case["K"], BLOCK):
        back[:, c:c + BLOCK] = s["q"][:, c:c + BLOCK].double() * torch.exp2(s["s"][:, c // BLOCK].double() - 133).unsqueeze(1)
    dw = torch.einsum("tn,tk->nk", s["dy"].double(), back)
    return {"dw": dw + s["dw"].double() if case["beta"] else dw}
