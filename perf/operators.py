"""The feed-forward operators of a transformer block, as cases to measure.

    gemm_bias_act            C = residual + dropout(act(A B + bias)), and its gradients
    dropout_add              Y = residual + dropout(X), the mask from a counter-based generator
    moe_layer                a whole mixture-of-experts layer for a few tokens

`run` computes them in a plain form (32-bit torch operations, rounded once at the end) or, where
`own` is true, by the calls of mbarrier_gemm_pipelines_gb300.  `exact` gives the same outputs from
the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # One token of a serving loop through a 4096 -> 4096 output projection with its residual.
        {"name": "forward_one_token", "op": "forward", "M": 1, "K": 4096, "N": 4096, "act": "none",
         "p": 0.0, "residual": True, "z": False},
        # A decode batch through the up-projection; an odd row count.
        {"name": "forward_batch_37", "op": "forward", "M": 37, "K": 4096, "N": 14336, "act": "silu",
         "p": 0.0, "residual": False, "z": False},
        # A ragged small training batch: nothing is a multiple of a tile.
        {"name": "forward_ragged", "op": "forward", "M": 301, "K": 520, "N": 1000, "act": "gelu",
         "p": 0.1, "residual": True, "z": True},
        # Training, up-projection of 4096 tokens: GELU, pre-activation kept for the backward pass.
        {"name": "forward_up_4096", "op": "forward", "M": 4096, "K": 4096, "N": 14336, "act": "gelu",
         "p": 0.0, "residual": False, "z": True},
        # Training, down-projection: dropout and the residual stream in the epilogue.
        {"name": "forward_down_4096", "op": "forward", "M": 4096, "K": 14336, "N": 4096,
         "act": "none", "p": 0.1, "residual": True, "z": False},
        # Gradients of a small ragged batch.
        {"name": "backward_ragged", "op": "backward", "M": 301, "K": 520, "N": 1000, "act": "gelu",
         "p": 0.1},
        # Training, gradients of the up-projection of 4096 tokens.
        {"name": "backward_up_4096", "op": "backward", "M": 4096, "K": 4096, "N": 14336,
         "act": "gelu", "p": 0.0},
        # Dropout and residual of one decoder row, where the launch is what counts.
        {"name": "dropout_add_small", "op": "dropout", "rows": 33, "cols": 4095, "dtype": "bf16",
         "p": 0.1, "residual": True},
        # The largest activation of the copy workload, 32-bit.
        {"name": "dropout_add_large", "op": "dropout", "rows": 16384, "cols": 4096, "dtype": "fp32",
         "p": 0.1, "residual": True},
        # One token through 2 of 8 experts of the mixture-of-experts workload's sizes.
        {"name": "moe_one_token", "op": "moe", "T": 1, "D": 4096, "F": 14336, "E": 8, "top_k": 2,
         "act": "relu", "gated": False},
        # A few tokens over many small gated experts.
        {"name": "moe_small_experts", "op": "moe", "T": 19, "D": 2048, "F": 1000, "E": 64, "top_k": 6,
         "act": "silu", "gated": True},
        # A full decode batch: every expert has work.
        {"name": "moe_batch_64", "op": "moe", "T": 64, "D": 4096, "F": 14336, "E": 8, "top_k": 2,
         "act": "relu", "gated": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["forward", "forward", "backward", "dropout", "moe"])
        if op in ("forward", "backward"):
            case = {"op": op, "M": _log_int(rng, 1, 8192), "K": _log_int(rng, 64, 14336),
                    "N": _log_int(rng, 64, 14336), "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    "p": rng.choice([0.0, 0.0, 0.1, 0.5])}
            # Most models keep their widths at multiples of 8; some do not.
            if rng.random() < 0.75:
                case["K"], case["N"] = -(-case["K"] // 8) * 8, -(-case["N"] // 8) * 8
            if op == "forward":
                case["residual"] = rng.random() < 0.5
                case["z"] = rng.random() < 0.5
            if case["M"] * case["K"] * case["N"] > (4096 * 4096 * 14336) // (1 if op == "forward" else 2):
                continue
        elif op == "dropout":
            case = {"op": op, "rows": _log_int(rng, 1, 16384), "cols": _log_int(rng, 32, 16384),
                    "dtype": rng.choice(["bf16", "fp32"]), "p": rng.choice([0.1, 0.25, 0.5]),
                    "residual": rng.random() < 0.5}
            if case["rows"] * case["cols"] > 16384 * 4096:
                continue
        else:
            E = rng.choice([4, 8, 16, 32, 64])
            case = {"op": op, "T": _log_int(rng, 1, 64), "D": 8 * _log_int(rng, 32, 512),
                    "F": 8 * _log_int(rng, 32, 1792), "E": E, "top_k": rng.randint(1, min(E, 8)),
                    "act": rng.choice(["relu", "gelu", "gelu_tanh", "silu"]), "gated": rng.random() < 0.5}
            if case["E"] * case["D"] * case["F"] * (2 if case["gated"] else 1) > 8 * 4096 * 14336:
                continue
        return case


# ----------------------------------------------------------------------------- inputs

def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _normal_weights(g, shape, std):
    """Large weights, drawn in bf16 slab by slab."""
    w = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    for part in w:
        part.copy_(torch.randn(part.shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std))
    return w


def prepare(case, seed):
    g = _rng(seed)
    s = dict(case)
    # The generator's seed and position, as a training loop counts them.
    s["seed"] = 0x9E3779B97F4A7C15 ^ int(seed)
    s["offset"] = 5 * 2 ** 32 + int(seed)
    bf = torch.bfloat16
    if case["op"] in ("forward", "backward"):
        M, K, N = case["M"], case["K"], case["N"]
        s["A"] = _normal(g, (M, K), 1.0, bf)
        s["B"] = _normal(g, (K, N), 1.0 / math.sqrt(K), bf)
        if case["op"] == "forward":
            s["bias"] = _normal(g, (N,), 0.1)
            s["R"] = _normal(g, (M, N), 1.0, bf) if case["residual"] else None
        else:
            s["Z"] = _normal(g, (M, N), 1.0, bf) if case["act"] != "none" else None
            s["dC"] = _normal(g, (M, N), 1.0 / math.sqrt(M), bf)
    elif case["op"] == "dropout":
        dt = _DTYPES[case["dtype"]]
        s["X"] = _normal(g, (case["rows"], case["cols"]), 1.0, dt)
        s["R"] = _normal(g, (case["rows"], case["cols"]), 1.0, dt) if case["residual"] else None
    else:
        T, D, F, E = case["T"], case["D"], case["F"], case["E"]
        F1 = 2 * F if case["gated"] else F
        s["X"] = _normal(g, (T, D), 1.0, bf)
        s["Wr"] = _normal(g, (D, E), 1.0 / math.sqrt(D))
        s["W1"] = _normal_weights(g, (E, D, F1), 1.0 / math.sqrt(D))
        s["b1"] = _normal(g, (E, F1), 0.1)
        s["W2"] = _normal_weights(g, (E, F, D), 1.0 / math.sqrt(F))
        s["b2"] = _normal(g, (E, D), 0.1)
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


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).float()
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        q = 1.0 / (1.0 + torch.exp(-z))
        return q * (1.0 + z * (1.0 - q))
    return torch.ones_like(z)


_LOW = 0xFFFFFFFF


def _dropped(rows, cols, p, seed, offset, device):
    """(keep, scale).  Philox-4x32 with 10 rounds; the counter of columns 8 j .. 8 j + 7 of row r is
    (j, r, offset low, offset high), the key is the seed, and each column takes 16 of the 128 bits."""
    threshold = int(round(p * 65536))
    j = torch.arange((cols + 7) // 8, device=device).expand(rows, -1)
    c0, c1 = j, torch.arange(rows, device=device)[:, None].expand(-1, j.shape[1])
    c2, c3 = torch.full_like(j, offset & _LOW), torch.full_like(j, offset >> 32)
    k0, k1 = seed & _LOW, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW)
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    words = torch.stack([c0, c1, c2, c3], -1)
    halves = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(rows, -1)[:, :cols]
    return halves >= threshold, 65536.0 / (65536 - threshold)


def _drop(x, s):
    if s["p"] == 0.0:
        return x
    keep, scale = _dropped(x.shape[0], x.shape[1], s["p"], s["seed"], s["offset"], x.device)
    return torch.where(keep, x * scale, torch.zeros_like(x))


def _plain_forward(s):
    z = s["A"].float() @ s["B"].float() + s["bias"]
    c = _drop(_act(z, s["act"]), s)
    if s["R"] is not None:
        c = c + s["R"].float()
    return [c.bfloat16(), z.bfloat16()] if s["z"] else [c.bfloat16()]


def _plain_backward(s):
    dz = _drop(s["dC"].float(), s)
    if s["Z"] is not None:
        dz = dz * _act_grad(s["Z"].float(), s["act"])
    return [(dz @ s["B"].float().t()).bfloat16(), (s["A"].float().t() @ dz).bfloat16(), dz.sum(0)]


def _plain_dropout(s):
    y = _drop(s["X"].float(), s)
    if s["R"] is not None:
        y = y + s["R"].float()
    return [y.to(s["X"].dtype)]


def _plain_moe(s):
    X, E, F, k = s["X"].float(), s["E"], s["F"], s["top_k"]
    logits = X @ s["Wr"]
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    e = torch.exp(best - best[:, :1])
    weights = e / e.sum(1, keepdim=True)
    spread = ((ids[:, :, None] == torch.arange(E, device=X.device)) * weights[:, :, None]).sum(1)   # [T, E]
    h = torch.matmul(X, s["W1"].float()) + s["b1"][:, None]                                         # [E, T, F]
    h = _act(h[..., :F], s["act"]) * h[..., F:] if s["gated"] else _act(h, s["act"])
    y = torch.matmul(h, s["W2"].float()) + s["b2"][:, None]                                         # [E, T, D]
    return [(y * spread.t()[:, :, None]).sum(0).bfloat16(), ids, weights]


# ----------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if not own:
        return {"forward": _plain_forward, "backward": _plain_backward, "dropout": _plain_dropout,
                "moe": _plain_moe}[s["op"]](s)
    import mbarrier_gemm_pipelines_gb300 as gbr
    if s["op"] == "forward":
        out = gbr.gemm_bias_act(s["A"], s["B"], s["bias"], residual=s["R"], act=s["act"], p=s["p"],
                                seed=s["seed"], offset=s["offset"], return_z=s["z"])
        return list(out) if s["z"] else [out]
    if s["op"] == "backward":
        return list(gbr.gemm_bias_act_backward(s["dC"], s["A"], s["B"], s["Z"], act=s["act"], p=s["p"],
                                               seed=s["seed"], offset=s["offset"]))
    if s["op"] == "dropout":
        return [gbr.dropout_add(s["X"], s["R"], p=s["p"], seed=s["seed"], offset=s["offset"])]
    return list(gbr.moe_layer(s["X"], s["Wr"], s["W1"], s["b1"], s["W2"], s["b2"], top_k=s["top_k"],
                              act=s["act"], gated=s["gated"], return_routing=True))


# ----------------------------------------------------------------------------- what a pass needs

def work(case):
    if case["op"] in ("forward", "backward"):
        M, K, N = case["M"], case["K"], case["N"]
        if case["op"] == "forward":
            wide = 1 + int(case["residual"]) + int(case["z"])
            return {"bytes": 2 * (M * K + K * N + wide * M * N) + 4 * N, "flops": 2 * M * N * K}
        wide = 2 if case["act"] != "none" else 1
        return {"bytes": 2 * (2 * M * K + 2 * K * N + wide * M * N) + 4 * N, "flops": 4 * M * N * K}
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) * (3 if case["residual"] else 2), "flops": 2 * n}
    T, D, F, E, k = (case[x] for x in ("T", "D", "F", "E", "top_k"))
    F1 = 2 * F if case["gated"] else F
    used = E * (1.0 - (1.0 - k / E) ** T)        # experts that some token picks, on average
    return {"bytes": int(used * (2 * D * (F1 + F) + 4 * (F1 + D))) + 4 * D * E + 4 * T * D,
            "flops": 2 * T * k * D * (F1 + F) + 2 * T * D * E}


# ----------------------------------------------------------------------------- 64 bits

def _exact_keep(rows, cols, p, seed, offset):
    """The mask, counter by counter in unsigned 64-bit host arithmetic."""
    u = np.uint64
    groups = (cols + 7) // 8
    n = np.arange(rows * groups, dtype=u)
    ctr = [n % u(groups), n // u(groups), np.full_like(n, offset % 2 ** 32), np.full_like(n, offset // 2 ** 32)]
    low, shift = u(2 ** 32 - 1), u(32)
    for r in range(10):
        key = [u((seed + r * 0x9E3779B9) % 2 ** 32), u((seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32)]
        left, right = u(0xD2511F53) * ctr[0], u(0xCD9E8D57) * ctr[2]
        ctr = [(right >> shift) ^ ctr[1] ^ key[0], right & low, (left >> shift) ^ ctr[3] ^ key[1], left & low]
    bits = np.empty((rows * groups, 8), dtype=np.uint16)
    for w in range(4):
        bits[:, 2 * w] = ctr[w] & u(0xFFFF)
        bits[:, 2 * w + 1] = ctr[w] >> u(16)
    return torch.from_numpy((bits.reshape(rows, groups * 8)[:, :cols] >= int(round(p * 65536)))).cuda()


def _exact_factor(shape, s):
    """What dropout multiplies each element by."""
    if s["p"] == 0.0:
        return 1.0
    t = int(round(s["p"] * 65536))
    return _exact_keep(shape[0], shape[1], s["p"], s["seed"], s["offset"]).double() * (65536.0 / (65536.0 - t))


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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "forward":
        z = torch.addmm(s["bias"].double(), s["A"].double(), s["B"].double())
        c = _exact_act(z, case["act"]) * _exact_factor(z.shape, s)
        c = c if s["R"] is None else c + s["R"].double()
        return [c, z] if case["z"] else [c]
    if case["op"] == "backward":
        dz = s["dC"].double() * _exact_factor(s["dC"].shape, s)
        if s["Z"] is not None:
            z = s["Z"].double().requires_grad_(True)
            dz, = torch.autograd.grad(_exact_act(z, case["act"]), z, dz)
        A, B = s["A"].double(), s["B"].double()
        return [torch.einsum("mn,kn->mk", dz, B), torch.einsum("mk,mn->kn", A, dz), torch.einsum("mn->n", dz)]
    if case["op"] == "dropout":
        y = s["X"].double() * _exact_factor(s["X"].shape, s)
        return [y if s["R"] is None else y + s["R"].double()]
    X, F, k = s["X"].double(), case["F"], case["top_k"]
    logits = X @ s["Wr"].double()
    ids = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
    weights = torch.softmax(torch.gather(logits, 1, ids), 1)
    y = torch.zeros(case["T"], case["D"], device=X.device, dtype=torch.float64)
    for e in range(case["E"]):
        token, place = torch.nonzero(ids == e, as_tuple=True)
        if token.numel() == 0:
            continue
        h = X[token] @ s["W1"][e].double() + s["b1"][e].double()
        h = _exact_act(h[:, :F], case["act"]) * h[:, F:] if case["gated"] else _exact_act(h, case["act"])
        y.index_add_(0, token, weights[token, place][:, None] * (h @ s["W2"][e].double() + s["b2"][e].double()))
    return [y, ids, weights]
