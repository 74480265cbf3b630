"""The feed-forward operators from their definitions, in 64 bits (test
infrastructure; shares no code with the library).  Torch tensors on any
device; bf16 and fp32 inputs are taken as the exact values they hold."""
import math

import torch

LOW = 0xFFFFFFFF


def philox4x32_10(counter, key):
    """Philox-4x32-10 on Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & LOW, (a >> 32) ^ c[3] ^ k[1], a & LOW]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    return c


def _mul_hi_lo(m, x):
    """High and low words of m * x for int64 tensors of 32-bit values, by 16-bit halves."""
    lo, hi = (m & 0xFFFF) * x, (m >> 16) * x          # both below 2^48
    low = (lo + ((hi & 0xFFFF) << 16))
    return (hi >> 16) + (low >> 32), low & LOW


def keep_mask(rows, cols, p, seed, offset, device="cpu"):
    """(keep, scale) of dropout."""
    threshold = round(p * 65536)
    groups = -(-cols // 8)
    j = torch.arange(groups, device=device, dtype=torch.int64)[None].expand(rows, groups)
    r = torch.arange(rows, device=device, dtype=torch.int64)[:, None].expand(rows, groups)
    c = [j, r, torch.full_like(j, offset & LOW), torch.full_like(j, offset >> 32)]
    k = [seed & LOW, seed >> 32]
    for _ in range(10):
        ah, al = _mul_hi_lo(0xD2511F53, c[0])
        bh, bl = _mul_hi_lo(0xCD9E8D57, c[2])
        c = [bh ^ c[1] ^ k[0], bl, ah ^ c[3] ^ k[1], al]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    bits = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], -1).reshape(rows, groups * 8)
    scale = 65536.0 / (65536 - threshold) if threshold < 65536 else 0.0
    return bits[:, :cols] >= threshold, scale


def drop(x, p, seed, offset):
    if round(p * 65536) == 0:
        return x
    keep, scale = keep_mask(x.shape[0], x.shape[1], p, seed, offset, x.device)
    return torch.where(keep, x * scale, torch.zeros_like(x))


def act(z, name):
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def linear(A, B, bias, residual, name, p=0.0, seed=0, offset=0):
    """(C, Z)."""
    z = A.double() @ B.double()
    if bias is not None:
        z = z + bias.double()
    c = drop(act(z, name), p, seed, offset)
    return (c if residual is None else c + residual.double()), z


def linear_grad(dC, A, B, Z, name, p=0.0, seed=0, offset=0):
    """(dA, dB, dbias, dZ)."""
    dz = drop(dC.double(), p, seed, offset)
    if name != "none":
        dz = dz * act_slope(Z.double(), name)
    return dz @ B.double().t(), A.double().t() @ dz, dz.sum(0), dz


def moe(X, Wr, W1, b1, W2, b2, top_k, name, gated):
    """(Y, ids, weights)."""
    T, D = X.shape
    E, F = W2.shape[:2]
    logits = X.double() @ Wr.double()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, weights = order.indices[:, :top_k], torch.softmax(order.values[:, :top_k], 1)
    Y = torch.zeros(T, D, dtype=torch.float64, device=X.device)
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        h = X[t].double() @ W1[e].double()
        if b1 is not None:
            h = h + b1[e].double()
        h = act(h[:, :F], name) * h[:, F:] if gated else act(h, name)
        y = h @ W2[e].double()
        if b2 is not None:
            y = y + b2[e].double()
        Y.index_add_(0, t, weights[t, k][:, None] * y)
    return Y, ids, weights
