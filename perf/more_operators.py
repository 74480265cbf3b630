"""What stands around and inside a transformer's feed-forward block, as cases to measure.

    residual_norm            S = R + scale * gate * norm(X), H = norm(S), and their gradients
    moe_sort, moe_dispatch,  rows sorted by expert for the experts' products, and back to their
    moe_combine              tokens with the routing weights applied, and its gradient
    quantize_mxfp4,          a linear layer in microscaled 4-bit floating point: the activations
    gemm_mxfp4               quantised in the call, the weights quantised beforehand

`run` computes them in a plain form (32-bit torch operations, rounded once at the end) or, where
`own` is true, by the calls of mbarrier_gemm_pipelines_gb300.  `exact` gives the same outputs from
the definitions in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-6


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # One token of a serving loop between two blocks: norm of the block's output, residual,
        # norm of the next block's input.
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "post": True,
         "gates": 0, "pre": True, "scale": 1.0},
        # A ragged small batch of 7 samples of 43 positions, each with its own gate, in 32 bits.
        {"name": "norm_ragged", "op": "norm", "rows": 301, "cols": 1001, "dtype": "fp32", "post": True,
         "gates": 7, "pre": True, "scale": 0.25},
        # The largest activation of a training step: residual scale and the next block's norm.
        {"name": "norm_large", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "post": True,
         "gates": 1, "pre": True, "scale": 0.25},
        # Gradients of the ragged batch.
        {"name": "norm_backward_ragged", "op": "norm_backward", "rows": 301, "cols": 1000, "dtype": "bf16",
         "post": True, "gates": 7, "pre": True, "scale": 0.25},
        # Gradients of a training step of 4096 tokens, one gate per channel.
        {"name": "norm_backward_4096", "op": "norm_backward", "rows": 4096, "cols": 4096, "dtype": "bf16",
         "post": True, "gates": 1, "pre": True, "scale": 0.25},
        # A decode batch that moe_layer no longer takes, over many small experts: sort and dispatch.
        {"name": "route_batch_100", "op": "route", "T": 100, "D": 2048, "E": 64, "top_k": 6, "dtype": "bf16",
         "masked": 0.0},
        # The mixture-of-experts workload: 4096 tokens, 2 of 8 experts.
        {"name": "route_4096", "op": "route", "T": 4096, "D": 4096, "E": 8, "top_k": 2, "dtype": "bf16",
         "masked": 0.0},
        # Back to the tokens, with the residual.
        {"name": "return_4096", "op": "return", "T": 4096, "D": 4096, "E": 8, "top_k": 2, "dtype": "bf16",
         "masked": 0.0, "residual": True},
        # Gradients of a ragged padded batch: a quarter of the choices dropped.
        {"name": "return_backward_ragged", "op": "return_backward", "T": 301, "D": 1000, "E": 64, "top_k": 6,
         "dtype": "bf16", "masked": 0.25},
        # One token through a 4096 -> 4096 projection with its residual.
        {"name": "mxfp4_one_token", "op": "mxfp4", "M": 1, "K": 4096, "N": 4096, "act": "none", "residual": True},
        # A decode batch through the up-projection; an odd row count.
        {"name": "mxfp4_batch_37", "op": "mxfp4", "M": 37, "K": 4096, "N": 14336, "act": "silu",
         "residual": False},
        # A prefill of 4096 tokens through the up-projection.
        {"name": "mxfp4_4096", "op": "mxfp4", "M": 4096, "K": 4096, "N": 14336, "act": "gelu", "residual": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm_backward", "route", "return", "return_backward", "mxfp4", "mxfp4"])
        if op in ("norm", "norm_backward"):
            case = {"op": op, "rows": _log_int(rng, 1, 16384), "cols": _log_int(rng, 32, 16384),
                    "dtype": rng.choice(["bf16", "bf16", "fp32"]), "post": rng.random() < 0.7, "pre": rng.random() < 0.8,
                    "scale": rng.choice([1.0, 0.25])}
            if rng.random() < 0.75:
                case["cols"] = -(-case["cols"] // 8) * 8
            # No gate, one for all rows, one for each sample, one for each row.
            kind, n = rng.randrange(4), _log_int(rng, 1, 64)
            if kind == 2:
                case["rows"] = -(-case["rows"] // n) * n
            case["gates"] = [0, 1, case["rows"] // n, case["rows"]][kind]
            if case["rows"] * case["cols"] > 16384 * 4096 // (1 if op == "norm" else 4):
                continue
        elif op == "mxfp4":
            case = {"op": op, "M": _log_int(rng, 1, 8192), "K": _log_int(rng, 64, 14336),
                    "N": _log_int(rng, 64, 14336), "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    "residual": rng.random() < 0.5}
            if rng.random() < 0.75:
                case["K"], case["N"] = -(-case["K"] // 32) * 32, -(-case["N"] // 8) * 8
            if case["M"] * case["K"] * case["N"] > 4096 * 4096 * 14336:
                continue
        else:
            E = rng.choice([4, 8, 16, 64, 256])
            case = {"op": op, "T": _log_int(rng, 1, 16384), "D": _log_int(rng, 64, 8192), "E": E,
                    "top_k": rng.randint(1, min(E, 8)), "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                    "masked": rng.choice([0.0, 0.0, 0.25, 0.75])}
            if case["T"] * case["top_k"] < 64:
                case["masked"] = 0.0
            if rng.random() < 0.75:
                case["D"] = -(-case["D"] // 8) * 8
            if op == "return":
                case["residual"] = rng.random() < 0.5
            if case["T"] * case["top_k"] * case["D"] > 4096 * 2 * 4096:
                continue
        return case


# ----------------------------------------------------------------------------- inputs

def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _choices(g, case):
    """Distinct experts for each token, some of them struck out (-1), as a router gives them."""
    T, E, k = case["T"], case["E"], case["top_k"]
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k).indices
    if case["masked"]:
        ids[torch.rand((T, k), generator=g, device="cuda") < case["masked"]] = -1
    return ids.contiguous()


def _two_to(exponent):
    """2^exponent in 32 bits, exactly (exponents of normal numbers)."""
    return ((exponent.int() + 127) << 23).view(torch.float32)


def _weights_mxfp4(g, rows, cols, std):
    """Weights as a program that serves them in 4 bits keeps them: two values a byte, blocks of 32
    along the columns, and the blocks' exponents in tiles of 128 rows x 4 blocks."""
    blocks = -(-cols // 32)
    w = torch.zeros((rows, blocks * 32), device="cuda")
    w[:, :cols] = torch.randn((rows, cols), generator=g, device="cuda").mul_(std)
    w = w.view(rows, blocks, 32)
    exponent = (torch.frexp(w.abs().amax(2)).exponent - 3).clamp_(-126, 126)
    w = w * _two_to(-exponent)[:, :, None]
    size = w.abs()
    code = sum((size > edge).to(torch.uint8) for edge in (0.25, 1.25, 2.5, 5.0))
    code += sum((size >= edge).to(torch.uint8) for edge in (0.75, 1.75, 3.5))
    code |= (w < 0).to(torch.uint8) << 3
    code = code.view(rows, blocks * 16, 2)
    data = code[:, :, 0] | code[:, :, 1] << 4
    tiles = torch.zeros((-(-rows // 128) * 128, -(-blocks // 4) * 4), device="cuda", dtype=torch.uint8)
    tiles[:rows, :blocks] = (exponent + 127).to(torch.uint8)
    tiles = tiles.view(tiles.shape[0] // 128, 4, 32, tiles.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return data.contiguous(), tiles.reshape(tiles.shape[0], tiles.shape[1], 512).contiguous()


def prepare(case, seed):
    g = _rng(seed)
    s = dict(case)
    bf = torch.bfloat16
    if case["op"] in ("norm", "norm_backward"):
        T, D, dt = case["rows"], case["cols"], _DTYPES[case["dtype"]]
        s["X"] = _normal(g, (T, D), 1.0, dt)
        s["w_post"] = 1.0 + _normal(g, (D,), 0.1) if case["post"] else None
        s["w_pre"] = 1.0 + _normal(g, (D,), 0.1) if case["pre"] else None
        s["gate"] = _normal(g, (case["gates"], D), 1.0, dt) if case["gates"] else None
        if case["op"] == "norm":
            s["R"] = _normal(g, (T, D), 2.0, dt)
        else:
            s["S"] = _normal(g, (T, D), 2.0, dt)
            s["dS"] = _normal(g, (T, D), 1.0, dt)
            s["dH"] = _normal(g, (T, D), 1.0, dt) if case["pre"] else None
    elif case["op"] == "mxfp4":
        M, K, N = case["M"], case["K"], case["N"]
        s["A"] = _normal(g, (M, K), 1.0, bf)
        s["W"], s["W_scales"] = _weights_mxfp4(g, N, K, 1.0 / math.sqrt(K))
        s["bias"] = _normal(g, (N,), 0.1)
        s["R"] = _normal(g, (M, N), 1.0, bf) if case["residual"] else None
    else:
        T, D, k, dt = case["T"], case["D"], case["top_k"], _DTYPES[case["dtype"]]
        s["ids"] = _choices(g, case)
        if case["op"] == "route":
            s["X"] = _normal(g, (T, D), 1.0, dt)
        else:
            s["positions"], s["offsets"] = _plain_sort(s["ids"], case["E"])
            s["Ys"] = _normal(g, (T * k, D), 1.0, dt)
            w = torch.rand((T, k), generator=g, device="cuda") + 0.1
            s["weights"] = w / w.sum(1, keepdim=True)
            s["R"] = _normal(g, (T, D), 1.0, dt) if case.get("residual") else None
            if case["op"] == "return_backward":
                s["dY"] = _normal(g, (T, D), 1.0, dt)
    return s


# ----------------------------------------------------------------------------- plain form

def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _root(x):
    return 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + _EPS)


def _spread(gate, rows):
    """One gate a row."""
    return gate.float().repeat_interleave(rows // gate.shape[0], 0)


def _plain_norm(s):
    x = s["X"].float()
    y = x if s["w_post"] is None else x * _root(x) * s["w_post"]
    if s["gate"] is not None:
        y = y * _spread(s["gate"], s["rows"])
    total = s["R"].float() + s["scale"] * y
    out = [total.to(s["X"].dtype)]
    if s["w_pre"] is not None:
        out.append((total * _root(total) * s["w_pre"]).to(s["X"].dtype))
    return out


def _norm_gradient(x, weight, dy):
    """(dx, dweight) of x * root(x) * weight."""
    r, u = _root(x), dy * weight
    return r * u - x * r * r * r * (u * x).mean(1, keepdim=True), (dy * x * r).sum(0)


def _plain_norm_backward(s):
    x, total, ds, dt = s["X"].float(), s["S"].float(), s["dS"].float(), s["X"].dtype
    dpost = dgate = dpre = None
    if s["w_pre"] is not None:
        d, dpre = _norm_gradient(total, s["w_pre"], s["dH"].float())
        ds = ds + d
    dy = s["scale"] * ds
    if s["gate"] is not None:
        y = x if s["w_post"] is None else x * _root(x) * s["w_post"]
        dgate = (dy * y).view(s["gates"], -1, s["cols"]).sum(1).to(dt)
        dy = dy * _spread(s["gate"], s["rows"])
    dx = dy
    if s["w_post"] is not None:
        dx, dpost = _norm_gradient(x, s["w_post"], dy)
    return [t for t in (dx.to(dt), ds.to(dt), dpost, dgate, dpre) if t is not None]


def _plain_sort(ids, experts):
    """(positions, offsets): counting, expert by expert in the order of the choices."""
    flat = ids.reshape(-1)
    chosen = (flat[:, None] == torch.arange(experts, device=ids.device)).long()
    ends = chosen.sum(0).cumsum(0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    place = (chosen.cumsum(0) - 1 + offsets[:-1]).gather(1, flat.clamp(min=0)[:, None])[:, 0]
    place = torch.where(flat >= 0, place, torch.full_like(place, -1))
    return place.view_as(ids).int(), offsets.int()


def _scatter(rows, positions):
    """`rows` [T, k, D] in the experts' order; places that nobody has are zero."""
    flat = positions.reshape(-1).long()
    out = torch.zeros((flat.shape[0] + 1, rows.shape[-1]), device=rows.device)
    out[torch.where(flat >= 0, flat, torch.full_like(flat, flat.shape[0]))] = rows.reshape(flat.shape[0], -1)
    return out[:-1]


def _plain_route(s):
    positions, offsets = _plain_sort(s["ids"], s["E"])
    x = s["X"].float()[:, None].expand(-1, s["top_k"], -1)
    return [positions, offsets, _scatter(x, positions).to(s["X"].dtype)]


def _picked(s):
    """(the experts' rows of each token [T, k, D], the weights [T, k]), zero where a choice is struck out."""
    taken = s["positions"] >= 0
    rows = s["Ys"].float()[s["positions"].clamp(min=0).long()]
    return torch.where(taken[..., None], rows, torch.zeros_like(rows)), torch.where(taken, s["weights"], 0.0)


def _plain_return(s):
    rows, weights = _picked(s)
    y = (rows * weights[..., None]).sum(1)
    if s["R"] is not None:
        y = y + s["R"].float()
    return [y.to(s["Ys"].dtype)]


def _plain_return_backward(s):
    rows, weights = _picked(s)
    dy = s["dY"].float()[:, None]
    return [_scatter(weights[..., None] * dy, s["positions"]).to(s["Ys"].dtype), (rows * dy).sum(2)]


def _plain_mxfp4(s):
    M, K = s["A"].shape
    blocks = s["W"].shape[1] // 16
    # The activations, to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times their block's power of two.
    a = torch.zeros((M, blocks * 32), device=s["A"].device)
    a[:, :K] = s["A"].float()
    a = a.view(M, blocks, 32)
    exponent = (torch.frexp(a.abs().amax(2, keepdim=True)).exponent - 3).clamp(-126, 126)
    v = (a * _two_to(-exponent)).clamp(-6.0, 6.0)
    step = torch.where(v.abs() < 2.0, 0.5, torch.where(v.abs() < 4.0, 1.0, 2.0))
    a = (torch.round(v / step) * step * _two_to(exponent)).view(M, -1)
    # The weights' values.
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=a.device)
    table = torch.cat([table, -table])
    w = torch.stack([table[(s["W"] & 15).long()], table[(s["W"] >> 4).long()]], 2)
    t = s["W_scales"].view(*s["W_scales"].shape[:2], 32, 4, 4).permute(0, 3, 2, 1, 4)
    t = t.reshape(t.shape[0] * 128, -1)[:w.shape[0], :blocks].int() - 127
    w = (w.view(w.shape[0], blocks, 32) * _two_to(t)[..., None]).view(w.shape[0], -1)
    c = _act(a @ w.t() + s["bias"], s["act"])
    if s["R"] is not None:
        c = c + s["R"].float()
    return [c.bfloat16()]


# ----------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "route": _plain_route,
                "return": _plain_return, "return_backward": _plain_return_backward, "mxfp4": _plain_mxfp4}[s["op"]](s)
    import mbarrier_gemm_pipelines_gb300 as gbr
    if s["op"] == "norm":
        out = gbr.residual_norm(s["X"], s["R"], post=s["w_post"], gate=s["gate"], scale=s["scale"], pre=s["w_pre"],
                                eps=_EPS)
        return [t for t in out if t is not None]
    if s["op"] == "norm_backward":
        out = gbr.residual_norm_backward(s["dS"], s["dH"], s["X"], s["S"], post=s["w_post"], gate=s["gate"],
                                         scale=s["scale"], pre=s["w_pre"], eps=_EPS)
        return [t for t in out if t is not None]
    if s["op"] == "route":
        positions, offsets = gbr.moe_sort(s["ids"], s["E"])
        return [positions, offsets, gbr.moe_dispatch(s["X"], positions, offsets)]
    if s["op"] == "return":
        return [gbr.moe_combine(s["Ys"], s["positions"], s["weights"], residual=s["R"])]
    if s["op"] == "return_backward":
        return list(gbr.moe_combine_backward(s["dY"], s["Ys"], s["positions"], s["offsets"], s["weights"]))
    weights = gbr.Mxfp4(s["W"], s["W_scales"], s["K"])
    return [gbr.gemm_mxfp4(gbr.quantize_mxfp4(s["A"]), weights, s["bias"], residual=s["R"], act=s["act"])]


# ----------------------------------------------------------------------------- what a pass needs

def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        n, e = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        small = case["cols"] * 4 * (int(case["post"]) + int(case["pre"])) + case["gates"] * case["cols"] * e
        if op == "norm":
            return {"bytes": n * e * (3 + int(case["pre"])) + small, "flops": 10 * n}
        # S is needed by its norm alone, X by the post-norm or the gate's gradient; without them
        # the gradient of X is the sum's, scaled.
        reads = 1 + 2 * int(case["pre"]) + int(case["post"] or case["gates"] > 0)
        return {"bytes": n * e * (reads + 2) + 2 * small, "flops": 20 * n}
    if op == "mxfp4":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + 17 * N * (-(-K // 32)) + 4 * N + 2 * M * N * (2 if case["residual"] else 1),
                "flops": 2 * M * N * K}
    T, D, E, k, e = case["T"], case["D"], case["E"], case["top_k"], 2 if case["dtype"] == "bf16" else 4
    live = 1.0 - case["masked"]                  # of the choices
    tokens = 1.0 - case["masked"] ** k           # with a choice left
    if op == "route":
        return {"bytes": int((tokens + k) * T * D * e) + 12 * T * k + 4 * E, "flops": T * k}
    if op == "return":
        return {"bytes": int((live * k + 1 + int(case["residual"])) * T * D * e) + 8 * T * k,
                "flops": int(2 * live * T * k * D)}
    return {"bytes": int(((1 + live) * k + tokens) * T * D * e) + 12 * T * k, "flops": int(3 * live * T * k * D)}


# ----------------------------------------------------------------------------- 64 bits

def _exact_rms(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * weight.double()


def _exact_sum(case, R, X, post, gate):
    y = X if post is None else _exact_rms(X, post)
    if gate is not None:
        y = (y.unflatten(0, (case["gates"], -1)) * gate[:, None]).flatten(0, 1)
    return R + case["scale"] * y


def _exact_act(z, name):
    f = torch.nn.functional
    if name == "relu":
        return torch.relu(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return f.gelu(z, approximate="tanh")
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def _exact_sorted(case, ids):
    """(positions, offsets) by a stable sort of the live choices."""
    flat = ids.flatten()
    live = torch.nonzero(flat >= 0).flatten()
    order = live[torch.argsort(flat[live], stable=True)]
    positions = torch.full_like(flat, -1, dtype=torch.int32)
    positions[order] = torch.arange(order.numel(), device=ids.device, dtype=torch.int32)
    counts = torch.bincount(flat[live], minlength=case["E"])
    offsets = torch.zeros(case["E"] + 1, device=ids.device, dtype=torch.int32)
    offsets[1:] = torch.cumsum(counts, 0)
    return positions.view_as(ids), offsets, order


def _exact_mxfp4_values(x):
    """64-bit values of x after rounding in blocks of 32: the nearest representable value, the one
    with the even code where two are as near."""
    M, K = x.shape
    pad = -K % 32
    b = torch.nn.functional.pad(x.double(), (0, pad)).unflatten(1, (-1, 32))
    top = b.abs().amax(2, keepdim=True)
    # The largest value's exponent, from the bits of the double.
    scale = ((((top.view(torch.int64) >> 52) & 0x7FF) - 2).clamp(min=1) << 52).view(torch.float64)
    size = b.abs() / scale
    best, dist = torch.zeros_like(size), size.clone()
    for code, value in enumerate((0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), 1):
        d = (size - value).abs()
        nearer = (d < dist) if code % 2 else (d <= dist)
        best, dist = torch.where(nearer, value, best), torch.where(nearer, d, dist)
    return (best * torch.sign(b) * scale).flatten(1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total = _exact_sum(case, *(None if s[n] is None else s[n].double() for n in ("R", "X", "w_post", "gate")))
        return [total] if s["w_pre"] is None else [total, _exact_rms(total, s["w_pre"])]
    if op == "norm_backward":
        def leaf(t):
            return None if t is None else t.double().requires_grad_(True)
        ds, dpre = s["dS"].double(), None
        if case["pre"]:
            total, pre = leaf(s["S"]), leaf(s["w_pre"])
            d, dpre = torch.autograd.grad(_exact_rms(total, pre), (total, pre), s["dH"].double())
            ds = ds + d
        X, post, gate = leaf(s["X"]), leaf(s["w_post"]), leaf(s["gate"])
        leaves = [t for t in (X, post, gate) if t is not None]
        grads = list(torch.autograd.grad(_exact_sum(case, 0.0, X, post, gate), leaves, ds))
        return [grads[0], ds] + grads[1:] + ([dpre] if case["pre"] else [])
    if op == "route":
        positions, offsets, order = _exact_sorted(case, s["ids"])
        Xs = torch.zeros((s["ids"].numel(), case["D"]), device=s["X"].device, dtype=torch.float64)
        Xs[:order.numel()] = s["X"].double()[order // case["top_k"]]
        return [positions, offsets, Xs]
    if op in ("return", "return_backward"):
        order = _exact_sorted(case, s["ids"])[2]
        token, w = order // case["top_k"], s["weights"].double().flatten()[order]
        rows = s["Ys"].double()[:order.numel()]
        if op == "return":
            y = torch.zeros((case["T"], case["D"]), device=rows.device, dtype=torch.float64)
            y.index_add_(0, token, w[:, None] * rows)
            return [y if s["R"] is None else y + s["R"].double()]
        dy = s["dY"].double()[token]
        dYs = torch.zeros(s["Ys"].shape, device=rows.device, dtype=torch.float64)
        dYs[:order.numel()] = w[:, None] * dy
        dw = torch.zeros(s["ids"].numel(), device=rows.device, dtype=torch.float64)
        dw[order] = torch.einsum("rd,rd->r", dy, rows)
        return [dYs, dw.view_as(s["weights"])]
    # The stored weights, nibble by nibble, and the exponent of (row, block) from its place in the tiles.
    N, blocks = s["W"].shape[0], s["W"].shape[1] // 16
    code = torch.stack([s["W"] % 16, s["W"] // 16], -1).flatten(1).long()
    n, b = torch.arange(N, device=code.device)[:, None], torch.arange(blocks, device=code.device)[None]
    exponent = s["W_scales"][n // 128, b // 4, n % 32 * 16 + n % 128 // 32 * 4 + b % 4].double() - 127.0
    mantissa, power = code % 2, code % 8 // 2
    size = torch.where(power == 0, 0.5 * mantissa.double(), (1.0 + 0.5 * mantissa) * torch.exp2(power.double() - 1.0))
    w = torch.where(code >= 8, -size, size) * torch.exp2(exponent).repeat_interleave(32, 1)
    z = torch.addmm(s["bias"].double(), _exact_mxfp4_values(s["A"]), w[:, :case["K"]].t())
    c = _exact_act(z, case["act"])
    return [c if s["R"] is None else c + s["R"].double()]
