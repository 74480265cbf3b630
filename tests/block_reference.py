"""The operators around a feed-forward block from their definitions, in 64 bits
(test infrastructure; shares no code with the library).  Torch tensors on any
device; inputs are taken as the exact values they hold."""
import torch

import ffn_reference as ffn


def root(x, eps):
    return 1 / torch.sqrt(x.square().mean(1, keepdim=True) + eps)


def spread(gate, rows):
    """One row of the gate for each of `rows` rows."""
    return gate.double()[torch.arange(rows, device=gate.device) * gate.shape[0] // max(rows, 1)]


def block_out(X, post, eps):
    x = X.double()
    return x if post is None else x * root(x, eps) * post.double()


def residual_norm(X, R, post, gate, scale, pre, eps):
    """(S, H, |R| + |scale gate y|)."""
    y = scale * block_out(X, post, eps)
    if gate is not None:
        y = y * spread(gate, len(X))
    r = torch.zeros_like(y) if R is None else R.double()
    s = r + y
    return s, None if pre is None else s * root(s, eps) * pre.double(), r.abs() + y.abs()


def residual_norm_backward(dS, dH, X, S, post, gate, scale, pre, eps):
    """Gradients {dX, dR, dpost, dgate, dpre} and, by the same names, the sums of the sizes of what they are made of."""
    rows, g, m = len(X if X is not None else dS if dS is not None else dH), {}, {}
    ds = ms = 0
    if dS is not None:
        ds, ms = dS.double(), dS.double().abs()
    if pre is not None:
        s, h = S.double(), dH.double()
        r, u = root(s, eps), h * pre.double()
        ds = ds + r * u - s * r ** 3 * (u * s).mean(1, keepdim=True)
        ms = ms + (r * u).abs() + s.abs() * r ** 3 * (u * s).abs().mean(1, keepdim=True)
        g["dpre"], m["dpre"] = (h * s * r).sum(0), (h * s * r).abs().sum(0)
    g["dR"], m["dR"] = ds, ms
    dy, my = scale * ds, abs(scale) * ms
    if gate is not None:
        y = block_out(X, post, eps)
        g["dgate"], m["dgate"] = ((t * y_).view(gate.shape[0], -1, dy.shape[1]).sum(1)
                                  for t, y_ in ((dy, y), (my, y.abs())))
        dy, my = dy * spread(gate, rows), my * spread(gate, rows).abs()
    if post is not None:
        x = X.double()
        q, p = root(x, eps), post.double()
        g["dpost"], m["dpost"] = (dy * x * q).sum(0), (my * (x * q).abs()).sum(0)
        g["dX"] = q * dy * p - x * q ** 3 * (dy * p * x).mean(1, keepdim=True)
        m["dX"] = q * my * p.abs() + x.abs() * q ** 3 * (my * (p * x).abs()).mean(1, keepdim=True)
    else:
        g["dX"], m["dX"] = dy, my
    return g, m


def moe_sort(ids, experts):
    """(positions, offsets), one choice at a time."""
    flat = ids.flatten().tolist()
    counts = [0] * experts
    for e in flat:
        if 0 <= e < experts:
            counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    place, positions = list(offsets), []
    for e in flat:
        positions.append(-1)
        if 0 <= e < experts:
            positions[-1] = place[e]
            place[e] += 1
    return torch.tensor(positions, dtype=torch.int32).view(ids.shape), torch.tensor(offsets, dtype=torch.int32)


def two_to(e):
    """2^e of whole numbers, from the bits of a double (pow and ldexp of floats round)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def quantize(X):
    """(values, exponents): the values after rounding and each block's exponent (a NaN block: 128)."""
    x = torch.nn.functional.pad(X.double(), (0, -X.shape[1] % 32)).unflatten(1, (-1, 32))
    bad = ~torch.isfinite(x).all(2, keepdim=True)
    x = torch.where(bad, torch.zeros_like(x), x)
    top = x.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    size = x.abs() * two_to(-e)
    code = torch.zeros_like(size, dtype=torch.long)
    for i in range(7):                      # past the middle; at the middle only from an odd code
        mid = (VALUES[i] + VALUES[i + 1]) / 2
        code += (size > mid) | ((size == mid) & (i % 2 == 1))
    v = torch.tensor(VALUES, dtype=torch.float64, device=X.device)[code] * torch.where(x < 0, -1.0, 1.0) * two_to(e)
    v = torch.where(bad, torch.full_like(v, float("nan")), v)
    return v.flatten(1)[:, :X.shape[1]], torch.where(bad, 128, e)[:, :, 0]


def scale_bytes(scales, rows, blocks):
    """[rows, blocks] of the tiled scales, place by place."""
    n, b = torch.arange(rows, device=scales.device)[:, None], torch.arange(blocks, device=scales.device)[None]
    return scales[n // 128, b // 4, n % 32 * 16 + n % 128 // 32 * 4 + b % 4]


def values(Q):
    """The 64-bit values of a 4-bit matrix from its bytes."""
    code = torch.stack([Q.data & 15, Q.data >> 4], 2).flatten(1).long()
    v = torch.tensor(VALUES, dtype=torch.float64, device=code.device)[code & 7] * torch.where(code > 7, -1.0, 1.0)
    s = scale_bytes(Q.scales, len(code), code.shape[1] // 32).long()
    p = torch.where(s == 255, torch.full_like(s, float("nan"), dtype=torch.float64), two_to(s - 127))
    return (v * p.repeat_interleave(32, 1))[:, :Q.columns]


def linear(a, b, bias, residual, act):
    """act(a b^T + bias) + residual of 64-bit values."""
    z = a @ b.t()
    if bias is not None:
        z = z + bias.double()
    c = ffn.act(z, act)
    return c if residual is None else c + residual.double()
