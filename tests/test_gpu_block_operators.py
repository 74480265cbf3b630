"""The operators around a feed-forward block (residual_norm, rows by expert, 4-bit
products) on the GPU against their definitions in 64 bits.

Bars, elementwise.  half: a rounding to the output's type, finfo.eps / 2 of the
value (bf16 2^-8, fp32 2^-24).  m: the sum of the sizes of what is added.
  residual_norm     S: five fp32 operations and a root whose sum of squares (all
      positive) adds at most 40 in a row: below 2^-20 m.  H multiplies that by root
      and weight and has a root of its own: 2^-19 (m root |pre| + |H|)
  its gradients     the same twice over, with a mean of signed products, whose error
      is relative to the mean of their sizes: 2^-18 m; sums over rows add rows 2^-24 m
  combine           a product and a sum each: (k + 2) 2^-23 m
  its gradients     dYs one product: 2^-23 |dYs|; dweights at most 128 terms a thread
      and 10 levels: 2^-17 m
  4-bit values      equal
  4-bit product     products are exact; each of the K / 64 steps and the split's sums add to
      fp32 with at most 2^-22 of m: (K / 64 + 16) 2^-22 m.  Activations: in the
      norm, one rounding as for gemm_bias_act
"""
import math

import pytest
import torch

import block_reference as ref
from gpu_helpers import load_library, require_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF, "fp32": F32}


@pytest.fixture(scope="module")
def gbr():
    require_gpu()
    return load_library()


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def odd(t):
    """The same values as a view with odd strides and an odd start."""
    if t is None:
        return None
    big = torch.full((t.shape[0], t.shape[1] + 8), float("nan"), device=t.device, dtype=t.dtype)
    big[:, 3:3 + t.shape[1]] = t
    return big[:, 3:3 + t.shape[1]]


def placed(t, start, ld, fill=5.0):
    """A copy of `t` that begins `start` elements after a 16-byte boundary, rows `ld` apart; and all that lies around it."""
    whole = torch.full((start + len(t) * ld + 8,), fill, dtype=t.dtype, device=t.device)
    view = whole.as_strided(t.shape, (ld, 1), start)
    view.copy_(t)
    return view, whole


def others(view, whole):
    """What lies around a placed matrix."""
    rest = whole.clone()
    rest.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(5.0)
    return rest


def within(got, want, slack, name=""):
    assert got.shape == want.shape, name
    bar = torch.finfo(got.dtype).eps / 2 * want.abs() + slack
    err = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), name
    worst = (err - bar).max().item() if err.numel() else 0.0
    assert worst <= 0, "%s: %g over its bar" % (name, worst)


# ------------------------------------------------------------ residual_norm
NORM = [
    # rows, cols, type, post, gates, pre, residual, scale
    (1, 1, "bf16", True, 0, True, True, 1.0),
    (1, 4096, "bf16", True, 1, True, True, 1.0),
    (3, 31, "fp32", True, 3, True, True, 0.5),
    (7, 256, "bf16", False, 0, True, False, 1.0),
    (12, 257, "bf16", True, 4, False, True, -2.0),
    (30, 1000, "fp32", False, 5, True, True, 0.25),
    (301, 1000, "bf16", True, 7, True, True, 0.25),
    (64, 2048, "bf16", True, 64, True, True, 1.0),
    (65, 4095, "fp32", True, 1, True, True, 0.25),
    (9, 4104, "fp32", True, 9, True, True, 1.0),
    (1000, 96, "bf16", True, 250, True, True, 1.0),
    (513, 4096, "bf16", True, 1, True, True, 0.25),
    (40, 8192, "bf16", True, 2, True, True, 1.0),
    (6, 8191, "fp32", True, 1, True, True, 1.0),
    (5, 8200, "bf16", True, 5, True, True, 1.0),
    (11, 16384, "fp32", True, 1, True, True, 1.0),
    (4, 32768, "bf16", True, 0, True, True, 1.0),
    (3, 32769, "bf16", True, 1, True, True, 0.5),
    (2, 70000, "fp32", False, 2, True, True, 1.0),
    (700, 8, "fp32", True, 1, True, True, 1.0),
    # Enough rows for CTAs that stay, one or several rows a turn.
    (1300, 4096, "bf16", True, 1, True, True, 0.25),
    (1301, 2048, "fp32", True, 1301, True, True, 1.0),
    (1290, 8192, "bf16", True, 3, False, True, 1.0),
    (1217, 8184, "fp32", False, 1, True, False, 0.5),
    (5004, 1000, "bf16", True, 36, True, True, 0.25),
    (2500, 2048, "bf16", True, 0, True, True, 1.0),
    (5000, 1024, "bf16", True, 5000, True, False, 1.0),
    (40003, 128, "bf16", True, 1, True, True, 1.0),
    (80001, 40, "fp32", False, 3, True, True, 1.0),
    (160001, 24, "bf16", True, 0, False, True, 1.0),
]
NORM_IDS = ["-".join(map(str, c)) for c in NORM]
EPS = 1e-6


def norm_inputs(case, seed=1):
    rows, cols, dt, post, gates, pre, residual, scale = case
    g, t = rng(seed), TYPES[dt]
    return dict(X=normal(g, (rows, cols), 1.5, t), R=normal(g, (rows, cols), 2.0, t) if residual else None,
                post=1 + normal(g, (cols,), 0.2, F32) if post else None,
                gate=normal(g, (gates, cols), 1.0, t) if gates else None, scale=scale,
                pre=1 + normal(g, (cols,), 0.2, F32) if pre else None, eps=EPS)


def check_norm(a, S, H):
    s, h, m = ref.residual_norm(**a)
    within(S, s, 2.0 ** -20 * m, "S")
    assert (H is None) == (h is None)
    if h is not None:
        within(H, h, 2.0 ** -19 * (m * ref.root(s, a["eps"]) * a["pre"].double().abs() + h.abs()), "H")


@pytest.mark.parametrize("case", NORM, ids=NORM_IDS)
def test_residual_norm(gbr, case):
    a = norm_inputs(case)
    check_norm(a, *gbr.residual_norm(**a))
    b = dict(a, X=odd(a["X"]), R=odd(a["R"]), gate=odd(a["gate"]))
    check_norm(a, *gbr.residual_norm(**b))
    gbr.check_device()


def norm_grad_inputs(case, seed=2):
    a = norm_inputs(case, seed)
    g = rng(seed + 100)
    R = a.pop("R")
    a["S"] = normal(g, a["X"].shape, 2.0, a["X"].dtype)
    a["dS"] = normal(g, a["X"].shape, 1.0, a["X"].dtype)
    a["dH"] = normal(g, a["X"].shape, 1.0, a["X"].dtype) if a["pre"] is not None else None
    return a


NAMES = ("dX", "dR", "dpost", "dgate", "dpre")


def check_norm_grads(a, grads, names=NAMES):
    g, m = ref.residual_norm_backward(**a)
    rows = len(a["dS"] if a["dS"] is not None else a["dH"])
    for name, got in zip(NAMES, grads):
        if name not in g or name not in names:
            assert got is None, name
            continue
        sums = rows * 2.0 ** -24 if name in ("dpost", "dgate", "dpre") else 0.0
        within(got, g[name], (2.0 ** -18 + sums) * m[name], name)


@pytest.mark.parametrize("case", NORM, ids=NORM_IDS)
def test_residual_norm_backward(gbr, case):
    a = norm_grad_inputs(case)
    grads = gbr.residual_norm_backward(**a)
    check_norm_grads(a, grads)
    b = dict(a, **{n: odd(a[n]) for n in ("dS", "dH", "X", "S", "gate")})
    check_norm_grads(a, gbr.residual_norm_backward(**b))
    # The same call gives the same bits.
    for x, y in zip(grads, gbr.residual_norm_backward(**a)):
        assert (x is None and y is None) or torch.equal(x, y)
    gbr.check_device()


@pytest.mark.parametrize("needs", [(True, False, False, False, False), (False, True, False, False, False),
                                   (False, False, True, False, True), (False, False, False, True, False)])
@pytest.mark.parametrize("case", [(33, 1000, "bf16", True, 11, True, True, 0.5), (20, 9000, "fp32", True, 1, True, True, 1.0)])
def test_residual_norm_backward_needs(gbr, case, needs):
    a = norm_grad_inputs(case)
    grads = gbr.residual_norm_backward(**a, needs=needs)
    check_norm_grads(a, grads, [n for n, w in zip(NAMES, needs) if w])
    a["dS"] = None
    check_norm_grads(a, gbr.residual_norm_backward(**a, needs=needs), [n for n, w in zip(NAMES, needs) if w])


@pytest.mark.parametrize("gates", [0, 1, 5, 10])
@pytest.mark.parametrize("post", [False, True])
def test_residual_norm_backward_against_differences(gbr, gates, post):
    """<gradient, direction> against central differences of the 64-bit forward pass, whose error in h = 1e-5 is far
    below the gradients' 2^-18."""
    a = norm_inputs((10, 72, "fp32", post, gates, True, True, 0.5), 5)
    g = rng(6)
    s, _, _ = ref.residual_norm(**a)
    dS, dH = normal(g, s.shape, 1.0, F32), normal(g, s.shape, 1.0, F32)
    grads = dict(zip(NAMES, gbr.residual_norm_backward(dS, dH, a["X"], s.float(), post=a["post"], gate=a["gate"],
                                                       scale=a["scale"], pre=a["pre"], eps=EPS)))
    for name in ("X", "R", "post", "gate", "pre"):
        if a[name] is None:
            continue
        v, h = normal(g, a[name].shape, 1.0, F32).double(), 1e-5
        loss = []
        for sign in (1, -1):
            S, H, _ = ref.residual_norm(**dict(a, **{name: a[name].double() + sign * h * v}))
            loss.append((S * dS.double()).sum() + (H * dH.double()).sum())
        want = (loss[0] - loss[1]).item() / (2 * h)
        got = (grads["d" + name].double() * v).sum().item()
        # S is rounded to 24 bits between the passes: another 2^-22 of every term.
        size = (grads["d" + name].double() * v).abs().sum().item()
        assert abs(got - want) <= 2.0 ** -16 * size + 1e-7 * size, name


def test_residual_norm_plain_sum_and_norm_alone(gbr):
    g = rng(3)
    X, w = normal(g, (37, 520)), 1 + normal(g, (520,), 0.1, F32)
    S, H = gbr.residual_norm(X, pre=w)
    assert S is X
    assert torch.equal(gbr.residual_norm(X, pre=w, S=torch.empty_like(X))[0], X)
    check_norm(dict(X=X, R=None, post=None, gate=None, scale=1.0, pre=w, eps=1e-6), S, H)
    S, H = gbr.residual_norm(X, X, scale=-1.0)
    assert H is None and not S.any()


def test_residual_norm_in_place(gbr):
    for cols in (1000, 4096, 40000):
        a = norm_inputs((9, cols, "bf16", True, 3, True, True, 0.5))
        want = gbr.residual_norm(**a)
        for S, H in (("R", "X"), ("X", "R"), ("R", None)):
            b = dict(a, X=a["X"].clone(), R=a["R"].clone())
            out = gbr.residual_norm(**b, S=b[S], H=b[H] if H else None)
            assert out[0] is b[S] and torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_residual_norm_over_its_input(gbr):
    """H written over X leaves the sum in a tensor of its own."""
    g = rng(7)
    X, w = normal(g, (9, 512)), 1 + normal(g, (512,), 0.1, F32)
    want, copy = gbr.residual_norm(X, pre=w)[1], X.clone()
    S, H = gbr.residual_norm(copy, pre=w, H=copy)
    assert H is copy and torch.equal(H, want) and torch.equal(S, X)


@pytest.mark.parametrize("rows", [40, 2000])
def test_residual_norm_weights_and_outputs_anywhere(gbr, rows):
    """Weights that start between 16 bytes, outputs given with strides of their own."""
    case = (rows, 1024, "bf16", True, 4, True, True, 0.5)
    a, d = norm_inputs(case), norm_grad_inputs(case)
    want, grads = gbr.residual_norm(**a), gbr.residual_norm_backward(**d)

    def shifted(v):
        big = torch.empty(v.numel() + 1, device="cuda")
        big[1:] = v
        return big[1:]
    S, H = (odd(torch.empty_like(t)) for t in want)
    out = gbr.residual_norm(**dict(a, post=shifted(a["post"]), pre=shifted(a["pre"])), S=S, H=H)
    assert out[0] is S and out[1] is H
    check_norm(a, S, H)
    given = dict(dX=odd(torch.empty_like(grads[0])), dR=odd(torch.empty_like(grads[1])), dpost=shifted(grads[2]),
                 dgate=odd(torch.empty_like(grads[3])), dpre=shifted(grads[4]))
    for t in given.values():
        t.fill_(7)
    out = gbr.residual_norm_backward(**dict(d, post=shifted(d["post"])), **given)
    assert all(x is y for x, y in zip(out, given.values()))
    check_norm_grads(d, out)
    wide = gbr.residual_norm_backward(**d, dX=torch.empty(rows, 2048, device="cuda", dtype=BF)[:, 1024:])
    check_norm_grads(d, wide)


# Rows on numbers of warps that are no powers of two, several groups and one.
WARPS = [
    (2600, 1536, "bf16", True, 1, True, True, 0.25),
    (2601, 1440, "fp32", True, 3, True, True, 1.0),
    (1300, 2560, "bf16", True, 1, True, True, 0.25),
    (1300, 2568, "fp32", True, 13, True, True, 1.0),
    (1290, 5120, "bf16", True, 0, True, True, 1.0),
    (1290, 4104, "bf16", True, 5, True, True, 1.0),
    (1290, 5128, "bf16", True, 1290, True, True, 1.0),
    (1230, 5120, "fp32", True, 1, True, False, 1.0),
    (1230, 7000, "bf16", False, 1, True, True, 1.0),
    (37, 2560, "bf16", True, 1, True, True, 1.0),
    (37, 5000, "fp32", True, 37, True, True, 1.0),
]


@pytest.mark.parametrize("case", WARPS, ids=["-".join(map(str, c)) for c in WARPS])
def test_residual_norm_on_any_number_of_warps(gbr, case):
    a = norm_inputs(case)
    check_norm(a, *gbr.residual_norm(**a))
    d = norm_grad_inputs(case)
    check_norm_grads(d, gbr.residual_norm_backward(**d))
    check_norm_grads(d, gbr.residual_norm_backward(**d, needs=(True, False, False, True, False)), ("dX", "dgate"))


# Rows whose gradients two or four CTAs share.
LONG = [
    (650, 16384, "bf16", True, 1, True, True, 0.25),
    (650, 8200, "fp32", True, 13, True, True, 1.0),
    (640, 12288, "bf16", False, 640, True, True, 1.0),
    (640, 9008, "bf16", True, 0, False, True, 1.0),
    (309, 32768, "bf16", True, 1, True, False, 1.0),
    (310, 17000, "fp32", True, 5, True, True, 0.5),
    (100, 16384, "bf16", True, 10, True, True, 1.0),
    (80, 8192, "fp32", True, 1, True, True, 1.0),
    (78, 6000, "fp32", True, 3, True, True, 1.0),
    (41, 20008, "bf16", True, 41, True, True, 1.0),
    (1, 8208, "bf16", True, 0, True, True, 1.0),
]


@pytest.mark.parametrize("case", LONG, ids=["-".join(map(str, c)) for c in LONG])
def test_residual_norm_of_rows_cut_over_ctas(gbr, case):
    a = norm_inputs(case)
    out = gbr.residual_norm(**a)
    check_norm(a, *out)
    d = norm_grad_inputs(case)
    grads = gbr.residual_norm_backward(**d)
    check_norm_grads(d, grads)
    for _ in range(3):
        for x, y in zip(out + grads, gbr.residual_norm(**a) + gbr.residual_norm_backward(**d)):
            assert (x is None and y is None) or torch.equal(x, y)
    gbr.check_device()


@pytest.mark.parametrize("rows,cols,dt", [(1, 2048, "bf16"), (2, 2048, "fp32"), (3, 2048, "bf16"), (1, 2047, "bf16"),
                                          (2, 33, "fp32"), (8, 256, "bf16"), (17, 256, "bf16"), (2, 8192, "bf16"),
                                          (2, 16384, "bf16"), (3, 16384, "bf16")])
@pytest.mark.parametrize("gates", ["none", "one", "row"])
def test_residual_norm_backward_of_few_rows(gbr, rows, cols, dt, gates):
    """One CTA's sums, and those of several."""
    a = norm_grad_inputs((rows, cols, dt, True, {"none": 0, "one": 1, "row": rows}[gates], True, True, 0.5))
    check_norm_grads(a, gbr.residual_norm_backward(**a))
    if gates == "one":
        check_norm_grads(a, gbr.residual_norm_backward(**a, needs=(True, False, True, False, False)), ("dX", "dpost"))
        check_norm_grads(a, gbr.residual_norm_backward(**a, needs=(False, False, False, True, True)), ("dgate", "dpre"))
    if rows % 2 == 0:
        a = norm_grad_inputs((rows, cols, dt, True, 2, True, True, 0.5))
        check_norm_grads(a, gbr.residual_norm_backward(**a))


# Enough rows for CTAs that stay, starting anywhere: rows, cols, type, ..., distance of the rows.
ANYWHERE = [
    (1300, 4095, "bf16", True, 1, True, True, 0.25, 4095),
    (1301, 4089, "bf16", True, 1301, True, True, 1.0, 4091),
    (1250, 8185, "bf16", True, 0, True, True, 1.0, 8185),
    (1220, 4097, "fp32", True, 1, True, True, 0.5, 4098),
    (2500, 2047, "bf16", False, 2500, True, False, 1.0, 2047),
    (2500, 2045, "fp32", True, 1, False, True, 1.0, 2045),
    (5003, 1001, "fp32", True, 1, True, True, 0.25, 1001),
    (5003, 1000, "bf16", True, 0, True, True, 1.0, 1004),
    (10001, 500, "bf16", True, 1, True, True, 1.0, 504),
    (80001, 33, "bf16", True, 1, True, True, 1.0, 33),
    (160003, 7, "fp32", True, 0, True, True, 1.0, 7),
    (160003, 1, "bf16", True, 1, True, True, 1.0, 1),
]


@pytest.mark.parametrize("case", ANYWHERE, ids=["-".join(map(str, c)) for c in ANYWHERE])
def test_residual_norm_many_rows_start_anywhere(gbr, case):
    case, ld = case[:-1], case[-1]
    a = norm_inputs(case)
    rows = case[0]

    def apart(t):
        return placed(t, 0, ld)[0]
    b = dict(a, X=apart(a["X"]), R=None if a["R"] is None else apart(a["R"]),
             gate=apart(a["gate"]) if case[4] > 1 else a["gate"])
    S, around_s = placed(torch.zeros_like(a["X"]), 0, ld)
    H, around_h = placed(torch.zeros_like(a["X"]), 0, ld) if case[5] else (None, None)
    want = gbr.residual_norm(**b, S=S, H=H)
    check_norm(a, *want)
    assert bool((others(S, around_s) == 5).all()) and (H is None or bool((others(H, around_h) == 5).all()))
    # Over their inputs, the same.
    if H is not None and a["R"] is not None:
        c = dict(b, X=apart(a["X"]), R=apart(a["R"]))
        out = gbr.residual_norm(**c, S=c["R"], H=c["X"])
        assert out[0] is c["R"] and torch.equal(out[0], S) and torch.equal(out[1], H)
    # A row that is not a number spoils itself alone.
    if rows < 3000:
        c = dict(b, X=apart(a["X"]))
        c["X"][rows // 2] = float("nan")
        keep = torch.arange(rows, device="cuda") != rows // 2
        # (New outputs lie closer than these: another order of the sums may be taken, the same for both calls.)
        for given, want in ((None, gbr.residual_norm(**b)[0]), (placed(S, 0, ld)[0], S)):
            out = gbr.residual_norm(**c, S=given, H=None if H is None or given is None else placed(H, 0, ld)[0])[0]
            assert torch.equal(out[keep], want[keep]) and bool(out[rows // 2].isnan().all())


@pytest.mark.parametrize("case", ANYWHERE + [
    (301, 1001, "bf16", True, 1, True, True, 0.25, 1001),
    (300, 1001, "fp32", True, 300, True, True, 0.25, 1003),
    (9, 2047, "fp32", True, 1, True, True, 0.25, 2047),
    (13, 33, "bf16", True, 0, True, True, 0.25, 34),
    (13, 8191, "bf16", False, 0, True, True, 0.25, 8192),
    (7, 5, "fp32", True, 1, False, True, 1.0, 5),
], ids=lambda c: "-".join(map(str, c)))
def test_residual_norm_backward_rows_start_anywhere(gbr, case):
    case, ld = case[:-1], case[-1]
    a = norm_grad_inputs(case)
    b = dict(a, **{n: None if a[n] is None else placed(a[n], 0, ld)[0] for n in ("dS", "dH", "X", "S")})
    out = {}
    if case[4] > 1:
        b["gate"] = placed(a["gate"], 0, ld)[0]
        out["dgate"] = placed(torch.zeros_like(a["gate"]), 0, ld)
    for name in ("dX", "dR"):
        out[name] = placed(torch.zeros_like(a["X"]), 0, ld)
    grads = gbr.residual_norm_backward(**b, **{n: t[0] for n, t in out.items()})
    check_norm_grads(a, grads)
    for view, whole in out.values():
        assert bool((others(view, whole) == 5).all())
    for x, y in zip(grads, gbr.residual_norm_backward(**b, **{n: placed(torch.zeros_like(t[0]), 0, ld)[0]
                                                              for n, t in out.items()})):
        assert (x is None and y is None) or torch.equal(x, y)
    # Only some of them.
    some = gbr.residual_norm_backward(**b, dX=out["dX"][0], needs=(True, False, False, True, True))
    check_norm_grads(a, some, ("dX", "dgate", "dpre"))


def test_residual_norm_special_values(gbr):
    """A row of zeros stays zero; Inf and NaN spoil their own row alone."""
    g = rng(4)
    X, R, w = normal(g, (6, 300)), normal(g, (6, 300)), torch.ones(300, device="cuda")
    X[1], R[1] = 0, 0
    X[2, 7], X[4, 299] = float("inf"), float("nan")
    S, H = gbr.residual_norm(X, R, post=w, pre=w)
    assert not S[1].any() and not H[1].any()
    good = [0, 3, 5]
    check_norm(dict(X=X[good], R=R[good], post=w, gate=None, scale=1.0, pre=w, eps=1e-6), S[good], H[good])
    assert torch.isnan(H[2]).any() and torch.isnan(S[4]).all()
    dX = gbr.residual_norm_backward(R, R, X, R, post=w, pre=w)[0]
    assert torch.isfinite(dX[good].float()).all() and torch.isnan(dX[4].float()).all()


def test_residual_norm_empty(gbr):
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda", dtype=BF)
    S, H = gbr.residual_norm(e, e, post=w, pre=w)
    assert S.shape == H.shape == (0, 64)
    gate = torch.ones(1, 64, device="cuda", dtype=BF)
    dX, dR, dpost, dgate, dpre = gbr.residual_norm_backward(e, e, e, e, post=w, gate=gate, pre=w)
    assert dX.shape == dR.shape == (0, 64)
    for t in (dpost, dgate, dpre):
        assert t.numel() == 64 and not t.any()
    n = torch.empty(5, 0, device="cuda", dtype=BF)
    S, H = gbr.residual_norm(n, n, pre=w[:0])
    assert S.shape == H.shape == (5, 0)


# ------------------------------------------------------------ rows by expert
SORT = [(0, 2, 4), (1, 1, 1), (1, 8, 8), (5, 3, 7), (100, 6, 64), (301, 6, 64), (1000, 8, 1024), (4096, 2, 8), (4097, 2, 8),
        (9000, 1, 3), (16384, 8, 256), (70000, 4, 1000)]


def choices(T, k, E, seed=1, masked=0.0):
    g = rng(seed)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
    if masked:
        ids[torch.rand((T, k), generator=g, device="cuda") < masked] = -1
    return ids


@pytest.mark.parametrize("T,k,E", SORT)
@pytest.mark.parametrize("how", ["all", "some", "none", "one", "wild"])
def test_moe_sort(gbr, T, k, E, how):
    ids = choices(T, k, E, masked={"some": 0.3, "none": 1.1}.get(how, 0.0))
    if how == "one":
        ids.fill_(E - 1)
    if how == "wild":
        ids = ids * 3 - E
        if T:
            ids[0, 0], ids[-1, -1] = 2 ** 40, -2 ** 63
    positions, offsets = gbr.moe_sort(ids, E)
    p, o = ref.moe_sort(ids.cpu(), E)
    assert torch.equal(positions.cpu(), p) and torch.equal(offsets.cpu(), o)
    assert positions.dtype == offsets.dtype == torch.int32


ROWS = [
    # T, k, D, E, type, masked
    (1, 1, 1, 1, "bf16", 0.0), (1, 2, 4096, 8, "bf16", 0.0), (5, 3, 7, 4, "fp32", 0.5), (100, 6, 2048, 64, "bf16", 0.0),
    (301, 6, 1000, 64, "bf16", 0.25), (300, 2, 1001, 8, "bf16", 0.0), (64, 8, 260, 16, "fp32", 0.25), (33, 9, 64, 16, "bf16", 0.0),
    (17, 4, 8200, 4, "bf16", 0.5), (700, 1, 36, 3, "fp32", 0.9), (19, 2, 4100, 5, "fp32", 1.1), (3000, 2, 512, 8, "bf16", 0.1),
]


def row_inputs(case, seed=3):
    T, k, D, E, dt, masked = case
    g, t = rng(seed), TYPES[dt]
    ids = choices(T, k, E, seed, masked)
    p, o = ref.moe_sort(ids.cpu(), E)
    return dict(X=normal(g, (T, D), 1.0, t), Ys=normal(g, (T * k, D), 1.0, t), dY=normal(g, (T, D), 1.0, t),
                R=normal(g, (T, D), 1.0, t), w=torch.rand((T, k), generator=g, device="cuda"), p=p.cuda(), o=o.cuda())


def picked(a):
    """The choices' rows [T, k, D] and weights, zero where struck out."""
    on = a["p"] >= 0
    return a["Ys"].double()[a["p"].clamp(min=0).long()] * on[..., None], a["w"].double() * on


@pytest.mark.parametrize("case", ROWS, ids=["-".join(map(str, c)) for c in ROWS])
def test_moe_rows(gbr, case):
    a = row_inputs(case)
    T, k, D = case[:3]
    on = a["p"].flatten() >= 0
    at, token = a["p"].flatten()[on].long(), torch.arange(T, device="cuda").repeat_interleave(k)[on]
    for f in (lambda t: t, odd):
        Xs = gbr.moe_dispatch(f(a["X"]), a["p"], a["o"])
        want = torch.zeros_like(a["Ys"])
        want[at] = a["X"][token]
        assert torch.equal(Xs, want)
        rows, w = picked(a)
        for weights, residual in ((a["w"], a["R"]), (a["w"], None), (None, None)):
            y = gbr.moe_combine(f(a["Ys"]), a["p"], weights, residual=f(residual) if residual is not None else None)
            ww = w if weights is not None else (a["p"] >= 0).double()
            r = residual.double() if residual is not None else torch.zeros(T, D, device="cuda", dtype=torch.float64)
            m = (ww[..., None] * rows).abs().sum(1) + r.abs()
            within(y, (ww[..., None] * rows).sum(1) + r, (k + 2) * 2.0 ** -23 * m, "Y")
        dYs, dw = gbr.moe_combine_backward(f(a["dY"]), f(a["Ys"]), a["p"], a["o"], a["w"])
        want = torch.zeros(T * k, D, device="cuda", dtype=torch.float64)
        want[at] = (a["w"].double()[..., None] * a["dY"].double()[:, None]).flatten(0, 1)[on]
        within(dYs, want, 2.0 ** -23 * want.abs(), "dYs")
        prod = rows * a["dY"].double()[:, None]
        within(dw, prod.sum(2), 2.0 ** -17 * prod.abs().sum(2), "dweights")
    gbr.check_device()


@pytest.mark.parametrize("dt", [BF, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", [1, 7, 8, 9, 15, 17, 248, 257, 2047])
def test_moe_rows_and_quantize_start_anywhere(gbr, D, dt):
    T, k, E = 11, 2, 3
    ids = choices(T, k, E)
    positions, offsets = gbr.moe_sort(ids, E)
    g = rng(D)
    X, Ys, ones = normal(g, (T, D), dtype=dt), normal(g, (T * k, D), dtype=dt), torch.ones(T, k, device="cuda")
    at = positions.long()
    rows = torch.empty_like(Ys)
    for j in range(k):
        rows[at[:, j]] = X
    # two terms, weights of one: exact in fp32, rounded once
    total = (Ys.float()[at[:, 0]] + Ys.float()[at[:, 1]]).to(dt)
    want = gbr.quantize_mxfp4(X)
    for start in range(8):
        for ld in (D + (-D % 8), D + (-D % 8) + 3):
            x, _ = placed(X, start, ld)
            y, _ = placed(Ys, 7 - start, ld)
            out, around = placed(torch.zeros_like(Ys), start, ld)
            gbr.moe_dispatch(x, positions, offsets, Xs=out)
            assert torch.equal(out, rows) and bool((others(out, around) == 5).all())
            out, around = placed(torch.zeros_like(X), start, ld)
            gbr.moe_combine(y, positions, Y=out)
            assert torch.equal(out, total) and bool((others(out, around) == 5).all())
            out, around = placed(torch.zeros_like(Ys), start, ld)
            gbr.moe_combine_backward(x, y, positions, offsets, ones, dYs=out, needs=(True, False))
            assert torch.equal(out, rows) and bool((others(out, around) == 5).all())
            got = gbr.quantize_mxfp4(x)
            assert torch.equal(got.data, want.data) and torch.equal(got.scales, want.scales)


@pytest.mark.parametrize("dt", [BF, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", [9, 333, 2047])
def test_moe_rows_that_start_anywhere_in_place(gbr, D, dt):
    T, k, E = 300, 3, 5
    ids = choices(T, k, E)
    positions, offsets = gbr.moe_sort(ids, E)
    g = rng(D)
    Ys, R, w = normal(g, (T * k, D), dtype=dt), normal(g, (T, D), dtype=dt), normal(g, (T, k), 1.0, F32)
    want = gbr.moe_combine(Ys, positions, w, R)
    for _ in range(5):
        Y = R.clone()
        assert gbr.moe_combine(Ys, positions, w, Y, Y=Y) is Y and torch.equal(Y, want)


def test_moe_rows_needs_and_in_place(gbr):
    a = row_inputs((50, 3, 520, 8, "bf16", 0.2))
    dYs, dw = gbr.moe_combine_backward(a["dY"], a["Ys"], a["p"], a["o"], a["w"])
    x, none = gbr.moe_combine_backward(a["dY"], None, a["p"], a["o"], a["w"], needs=(True, False))
    assert none is None and torch.equal(x, dYs)
    none, y = gbr.moe_combine_backward(a["dY"], a["Ys"], a["p"], a["o"], a["w"], needs=(False, True))
    assert none is None and torch.equal(y, dw)
    want = gbr.moe_combine(a["Ys"], a["p"], a["w"], residual=a["R"])
    R = a["R"].clone()
    assert gbr.moe_combine(a["Ys"], a["p"], a["w"], residual=R, Y=R) is R and torch.equal(R, want)


def test_moe_struck_out_choices_count_nothing(gbr):
    """Not even with Inf or NaN as weight, and rows that nobody has are not read."""
    a = row_inputs((40, 4, 264, 8, "fp32", 0.4))
    off = a["p"] < 0
    want = gbr.moe_combine(a["Ys"], a["p"], a["w"])
    grads = gbr.moe_combine_backward(a["dY"], a["Ys"], a["p"], a["o"], a["w"])
    a["w"][off] = float("nan")
    a["Ys"][int(a["o"][-1]):] = float("inf")
    assert torch.equal(gbr.moe_combine(a["Ys"], a["p"], a["w"]), want)
    for x, y in zip(gbr.moe_combine_backward(a["dY"], a["Ys"], a["p"], a["o"], a["w"]), grads):
        assert torch.equal(x, y)
    assert not grads[1][off].any()


def test_moe_positions_outside_are_struck_out(gbr):
    """As with a shortened Ys: nothing out of range is read or written."""
    a = row_inputs((20, 3, 72, 4, "bf16", 0.0))
    short = a["Ys"][:25]
    p = torch.where(a["p"] < 25, a["p"], torch.full_like(a["p"], -1))
    assert torch.equal(gbr.moe_combine(short, a["p"], a["w"]), gbr.moe_combine(short, p, a["w"]))
    wild = a["p"].clone()
    wild[3, 1], wild[4, 2] = 60, 2 ** 31 - 1
    Xs = gbr.moe_dispatch(a["X"], wild, a["o"], Xs=torch.zeros_like(a["Ys"]))
    kept = (wild >= 0) & (wild < 60)
    want = torch.zeros_like(a["Ys"])
    want[wild[kept].long()] = a["X"][torch.arange(20, device="cuda")[:, None].expand(20, 3)[kept]]
    assert torch.equal(Xs, want)


def test_moe_rows_empty(gbr):
    p, o = gbr.moe_sort(torch.empty(0, 3, device="cuda", dtype=torch.long), 5)
    assert p.shape == (0, 3) and not o.any()
    e = torch.empty(0, 16, device="cuda")
    assert gbr.moe_dispatch(e, p, o).shape == (0, 16)
    assert gbr.moe_combine(e, p, torch.empty(0, 3, device="cuda")).shape == (0, 16)
    R = torch.randn(4, 16, device="cuda")
    p = torch.empty(4, 0, device="cuda", dtype=torch.int32)
    assert torch.equal(gbr.moe_combine(e, p, residual=R), R)
    p = torch.full((4, 2), -1, device="cuda", dtype=torch.int32)
    assert torch.equal(gbr.moe_combine(e, p, residual=R), R)


# ------------------------------------------------------------ 4 bits
def check_quantized(Q, X):
    rows, cols = X.shape
    want, e = ref.quantize(X)
    blocks = -(-cols // 32)
    assert Q.data.shape == (rows, blocks * 16) and Q.columns == cols
    assert Q.scales.shape == (-(-rows // 128), -(-cols // 128), 512)
    assert torch.equal(ref.scale_bytes(Q.scales, rows, blocks).long(), e + 127)
    got = ref.values(Q)
    assert torch.equal(torch.nan_to_num(got, 1e300), torch.nan_to_num(want, 1e300))
    # Padding: zeros in the last block's rest and in the tiles' unused places.
    if cols % 32 and torch.isfinite(X.double()).all():
        rest = ref.values(Q._replace(columns=blocks * 32))[:, cols:]
        assert not rest.any()
    used = torch.zeros_like(Q.scales)
    n, b = torch.arange(rows, device="cuda")[:, None], torch.arange(blocks, device="cuda")[None]
    used[n // 128, b // 4, n % 32 * 16 + n % 128 // 32 * 4 + b % 4] = 1
    assert not Q.scales[used == 0].any()


QUANT = [(1, 1), (1, 32), (3, 33), (5, 64), (37, 4096), (128, 128), (129, 160), (130, 1000), (257, 2056), (300, 97)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", QUANT)
def test_quantize(gbr, rows, cols, dt):
    g = rng(rows + cols)
    X = normal(g, (rows, cols), 1.0, F32) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g, device="cuda").float())
    X = X.to(TYPES[dt])
    for f in (lambda t: t, odd):
        Q = gbr.quantize_mxfp4(f(X))
        check_quantized(Q, X)
        back = gbr.dequantize_mxfp4(Q, dtype=TYPES[dt])
        assert torch.equal(back.double(), ref.values(Q))
        out = f(torch.empty_like(X))
        assert gbr.dequantize_mxfp4(Q, X=out) is out and torch.equal(out, back)
        T = gbr.quantize_mxfp4(f(X.t().contiguous()), transposed=True)
        assert torch.equal(T.data & 0x77, Q.data & 0x77) and torch.equal(T.scales, Q.scales)
        check_quantized(T, X)
    again = gbr.quantize_mxfp4(X, out=gbr.Mxfp4(torch.full_like(Q.data, 255), torch.full_like(Q.scales, 255), cols))
    assert torch.equal(again.data, gbr.quantize_mxfp4(X).data) and torch.equal(again.scales, Q.scales)


def test_quantize_every_bf16_and_ties(gbr):
    """All bf16 values in blocks with others of their size, ties, blocks of zeros, the ends of the range."""
    bits = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(BF)
    order = torch.argsort(torch.where(torch.isfinite(bits.float()), bits.float().abs(), torch.full_like(bits, 3e38).float()))
    X = bits[order][torch.isfinite(bits[order].float())]
    X = X[:len(X) // 32 * 32].view(-1, 32).contiguous()
    check_quantized(gbr.quantize_mxfp4(X), X)
    ties = torch.tensor([0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.9, 7.96, 0.2, 0.3, -0.25, -5.0, -0.0],
                        device="cuda").repeat(2)
    X = torch.stack([ties * 2.0 ** e for e in (-130, -126, -125, -100, -1, 0, 1, 60, 124)])
    X[:, 16] = 4.0 * torch.tensor([2.0 ** e for e in (-130, -126, -125, -100, -1, 0, 1, 60, 124)], device="cuda")
    check_quantized(gbr.quantize_mxfp4(X), X)
    X = torch.zeros(4, 64, device="cuda")
    X[1, 3], X[2, 40], X[3, 5] = float("inf"), float("nan"), 3e38
    Q = gbr.quantize_mxfp4(X)
    check_quantized(Q, X)
    assert torch.isnan(gbr.dequantize_mxfp4(Q)[1, :32].float()).all()


GEMM = [
    # M, N, K, bias, residual
    (1, 1, 1, True, True), (1, 4096, 4096, True, True), (2, 130, 33, False, False), (16, 128, 256, True, False),
    (17, 200, 320, True, True), (37, 1000, 1000, True, False), (48, 264, 544, False, True), (64, 4095, 512, True, True),
    (128, 512, 4096, False, False), (130, 384, 96, True, False), (200, 256, 2080, True, True), (257, 300, 288, True, True),
    (300, 1024, 14336, True, False), (500, 40, 64, True, True), (1024, 1024, 1024, True, True), (1000, 2000, 3000, True, True),
    (2049, 2056, 1056, False, True), (2048, 4096, 64, True, False), (2500, 2501, 500, True, True), (4096, 2048, 4128, False, False),
]


def gemm_inputs(gbr, M, N, K, seed=1):
    g = rng(seed)
    A = normal(g, (M, K), 1.0, F32) * torch.exp2(torch.randint(-6, 6, (M, 1), generator=g, device="cuda").float())
    B = normal(g, (N, K), max(K, 1) ** -0.5, F32) * torch.exp2(torch.randint(-3, 3, (N, 1), generator=g, device="cuda").float())
    # Blocks of different sizes along K.
    A *= torch.exp2((torch.arange(K, device="cuda") // 32 % 5 - 2).float())
    B *= torch.exp2((torch.arange(K, device="cuda") // 32 % 7 - 3).float())
    return gbr.quantize_mxfp4(A), gbr.quantize_mxfp4(B), normal(g, (N,), 1.0, F32), normal(g, (M, N))


def gemm_bar(a, b, K):
    return (K / 64 + 16) * 2.0 ** -22 * (a.abs() @ b.abs().t())


@pytest.mark.parametrize("M,N,K,bias,residual", GEMM)
def test_gemm(gbr, M, N, K, bias, residual):
    A, B, b, R = gemm_inputs(gbr, M, N, K)
    b, R = b if bias else None, R if residual else None
    C = gbr.gemm_mxfp4(A, B, b, residual=R)
    gbr.check_device()
    x, y = ref.values(A), ref.values(B)
    want, bar = ref.linear(x, y, b, R, "none"), gemm_bar(x, y, K)
    m = (b.double().abs() if bias else 0) + (R.double().abs() if residual else 0)
    within(C, want, bar + 2.0 ** -22 * (m + want.abs()), "C")
    # Any stride, and the residual itself as the output.
    out = odd(torch.empty_like(C))
    assert torch.equal(gbr.gemm_mxfp4(A, B, b, residual=odd(R), C=out), C)
    if residual:
        R2 = R.clone()
        assert gbr.gemm_mxfp4(A, B, b, residual=R2, C=R2) is R2 and torch.equal(R2, C)
    gbr.check_device()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N,K", [(5, 300, 200), (1500, 1600, 320)])
def test_gemm_activations(gbr, M, N, K, act):
    A, B, b, R = gemm_inputs(gbr, M, N, K)
    C = gbr.gemm_mxfp4(A, B, b, residual=R, act=act)
    want = ref.linear(ref.values(A), ref.values(B), b, R, act)
    assert (C.double() - want).norm() <= 1.0625 * 2.0 ** -9 * want.norm()


def test_gemm_no_contraction_and_empty(gbr):
    A, B, b, R = gemm_inputs(gbr, 5, 40, 0)
    assert torch.equal(gbr.gemm_mxfp4(A, B, b, residual=None), b.to(BF).expand(5, 40))
    A, B, b, R = gemm_inputs(gbr, 0, 40, 64)
    assert gbr.gemm_mxfp4(A, B, b).shape == (0, 40)
    A, B, b, R = gemm_inputs(gbr, 5, 0, 64)
    assert gbr.gemm_mxfp4(A, B, b).shape == (5, 0)


@pytest.mark.parametrize("M,N,K", [(20, 200, 512), (1500, 1600, 512)])
def test_gemm_nan_blocks_stay_in_their_rows(gbr, M, N, K):
    g = rng(7)
    X, W = normal(g, (M, K)), normal(g, (N, K))
    X[3, 40], W[130, 500] = float("nan"), float("inf")
    C = gbr.gemm_mxfp4(gbr.quantize_mxfp4(X), gbr.quantize_mxfp4(W))
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[3], bad[:, 130] = True, True
    assert torch.equal(torch.isnan(C), bad)


# ------------------------------------------------------------ all of them
def calls(gbr):
    """Every operator, as functions of the stream that return their outputs."""
    g = rng(9)
    a = norm_inputs((64, 1000, "bf16", True, 8, True, True, 0.5))
    d = norm_grad_inputs((64, 1000, "bf16", True, 8, True, True, 0.5))
    long = norm_grad_inputs((8, 9000, "bf16", True, 1, True, True, 0.5))
    r = row_inputs((64, 3, 520, 8, "bf16", 0.2))
    ids, X = choices(9000, 2, 16), normal(g, (300, 1000), 1.0, F32)
    small, large = gemm_inputs(gbr, 20, 300, 1000), gemm_inputs(gbr, 1500, 1600, 320)
    return [
        lambda s: list(gbr.residual_norm(**a, stream=s)),
        lambda s: list(gbr.residual_norm_backward(**d, stream=s)),
        lambda s: list(gbr.residual_norm_backward(**long, stream=s))[:3],
        lambda s: list(gbr.moe_sort(ids, 16, stream=s)),
        lambda s: [gbr.moe_dispatch(r["X"], r["p"], r["o"], stream=s)],
        lambda s: [gbr.moe_combine(r["Ys"], r["p"], r["w"], residual=r["R"], stream=s)],
        lambda s: list(gbr.moe_combine_backward(r["dY"], r["Ys"], r["p"], r["o"], r["w"], stream=s)),
        lambda s: list(gbr.quantize_mxfp4(X, stream=s))[:2],
        lambda s: [gbr.dequantize_mxfp4(small[0], stream=s)],
        lambda s: [gbr.gemm_mxfp4(*small[:3], residual=small[3], stream=s)],
        lambda s: [gbr.gemm_mxfp4(*large[:3], residual=large[3], act="gelu", stream=s)],
    ]


def test_streams(gbr):
    from test_gpu_operator_streams import owner
    side = torch.cuda.Stream()
    for call in calls(gbr):
        want = call(None)
        torch.cuda.synchronize()
        got = call(side)
        side.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
            assert owner(x) == side.cuda_stream and owner(y) == torch.cuda.current_stream().cuda_stream
    gbr.check_device()


def test_captured_together_and_replayed(gbr):
    """Two graphs of all operators, replayed on two streams at once."""
    every = calls(gbr)
    want = [f(None) for f in every]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append([f(None) for f in every])
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for out in outs:
            for call in out:
                for t in call:
                    t.fill_(1)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            for call, expected in zip(out, want):
                for x, y in zip(call, expected):
                    assert torch.equal(x, y)
    gbr.check_device()


def test_two_streams_at_once(gbr):
    every = calls(gbr)
    want = [f(None) for f in every]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(9):
        for j, f in enumerate(every):
            got.append((j, f(streams[(i + j) % 3])))
    torch.cuda.synchronize()
    for j, out in got:
        for x, y in zip(out, want[j]):
            assert torch.equal(x, y)
    gbr.check_device()


def test_threads_at_once(gbr):
    """Calls from several host threads, each on a stream of its own."""
    import threading
    every = calls(gbr)
    want = [f(None) for f in every]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        try:
            for n in range(10):
                j = (i + n) % len(every)
                got = every[j](stream)
                stream.synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, want[j])):
                    bad.append(j)
        except Exception as e:                              # noqa: BLE001 (reported below)
            bad.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    gbr.check_device()


def test_outputs_that_are_given(gbr):
    r = row_inputs((50, 3, 520, 8, "bf16", 0.2))
    ids = choices(50, 3, 8, 3, 0.2)
    p, o = torch.full_like(r["p"], 9), torch.full_like(r["o"], 9)
    assert gbr.moe_sort(ids, 8, positions=p, offsets=o)[0] is p and torch.equal(p, r["p"]) and torch.equal(o, r["o"])
    for out in (torch.full_like(r["Ys"], 9), odd(torch.empty_like(r["Ys"]))):
        assert gbr.moe_dispatch(r["X"], p, o, Xs=out) is out and torch.equal(out, gbr.moe_dispatch(r["X"], p, o))
        w = torch.full_like(r["w"], 9)
        x, y = gbr.moe_combine_backward(r["dY"], r["Ys"], p, o, r["w"], dYs=out, dweights=w)
        want = gbr.moe_combine_backward(r["dY"], r["Ys"], p, o, r["w"])
        assert x is out and y is w and torch.equal(x, want[0])
        within(y, want[1].double(), 2.0 ** -17 * want[1].double().abs().max(), "dweights")


def test_written_tensors_move_their_version(gbr):
    r = row_inputs((8, 2, 64, 4, "bf16", 0.0))
    Y = torch.empty_like(r["X"])
    v = Y._version
    gbr.moe_combine(r["Ys"], r["p"], r["w"], Y=Y)
    assert Y._version > v
    S = torch.empty_like(r["X"])
    gbr.residual_norm(r["X"], r["R"], S=S)
    assert S._version > 0


def test_a_stage_that_is_never_filled(gbr):
    for M, N, K in ((20, 300, 4096), (1500, 1600, 4096)):
        A, B, _, _ = gemm_inputs(gbr, M, N, K)
        want = gbr.gemm_mxfp4(A, B)
        gbr.selftest_mxfp4_skip_load(A, B, 0, 1, 20_000_000)
        with pytest.raises(gbr.GbrError):
            gbr.check_device()
        assert torch.equal(gbr.gemm_mxfp4(A, B), want)
        gbr.check_device()


# ------------------------------------------------------------ refusals that need tensors of the GPU
def test_shapes_are_refused(gbr):
    g = rng(20)
    X, w = normal(g, (12, 64)), torch.ones(64, device="cuda")
    ids = torch.zeros(12, 2, device="cuda", dtype=torch.long)
    p, o = gbr.moe_sort(ids, 4)
    Q, W = gbr.quantize_mxfp4(X), gbr.quantize_mxfp4(normal(g, (40, 96)))
    R = normal(g, (12, 63))
    bad = [
        lambda: gbr.residual_norm(X, R), lambda: gbr.residual_norm(X, post=w[:63]), lambda: gbr.residual_norm(X, gate=X[:5]),
        lambda: gbr.residual_norm(X, H=X), lambda: gbr.residual_norm(X, X, pre=w, S=X[:11]), lambda: gbr.residual_norm(X[0]),
        lambda: gbr.residual_norm(X.t()), lambda: gbr.residual_norm_backward(X, None, None, None, pre=w),
        lambda: gbr.residual_norm_backward(X, None, None, None, post=w), lambda: gbr.residual_norm_backward(X, X, X, X, needs=(1, 1)),
        lambda: gbr.moe_sort(ids[0], 4), lambda: gbr.moe_sort(ids, 0), lambda: gbr.moe_sort(ids.t(), 4),
        lambda: gbr.moe_dispatch(X[:11], p, o), lambda: gbr.moe_dispatch(X, p, o[:1]), lambda: gbr.moe_dispatch(X, p[0], o),
        lambda: gbr.moe_combine(X, p, w), lambda: gbr.moe_combine(X, p, residual=R),
        lambda: gbr.moe_combine_backward(X, X, p, o, torch.ones(12, 2, device="cuda")),
        lambda: gbr.gemm_mxfp4(Q, W), lambda: gbr.gemm_mxfp4(Q, Q, w), lambda: gbr.gemm_mxfp4(Q, Q, act="tanh"),
        lambda: gbr.gemm_mxfp4(Q._replace(columns=200), Q), lambda: gbr.gemm_mxfp4(Q, Q, C=X),
        lambda: gbr.dequantize_mxfp4(Q, X=X[:5]), lambda: gbr.quantize_mxfp4(X, out=W),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)
    for call in (lambda: gbr.residual_norm(X, X.float()), lambda: gbr.moe_sort(ids.int(), 4), lambda: gbr.moe_dispatch(X, p.long(), o),
                 lambda: gbr.moe_combine(X, p, torch.ones(12, 2, device="cuda", dtype=BF)),
                 lambda: gbr.dequantize_mxfp4(Q, dtype=torch.float16), lambda: gbr.gemm_mxfp4(Q, Q, residual=X.float())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: gbr.moe_sort(ids, 1025), lambda: gbr.residual_norm(X, eps=-1.0, pre=w),
                 lambda: gbr.residual_norm(X, X, S=X[:, :64], scale=float("nan"))):
        with pytest.raises(gbr.GbrError):
            call()


# ------------------------------------------------------------ as they are used
def relative(got, want):
    return (got.double() - want).norm().item() / max(want.norm().item(), 1e-300)


ROUNDED = 2.0 ** -9                 # one rounding to bf16, in the norm (see test_gpu_operators.py)


def test_normed_feed_forward(gbr):
    """Outputs and gradients against 64-bit autograd over the same parameters.  Four roundings lie between x and the
    sum (h, u, y, S) and up to eight on the way back."""
    import ffn_reference as ffn
    from mbarrier_gemm_pipelines_gb300 import feed_forward
    g, T, D, F = rng(30), 300, 264, 520
    net = feed_forward.NormedFeedForward(D, F, act="gelu_tanh", scale=0.5, seed=3)
    for t in (net.pre, net.post, net.next):
        t.copy_(1 + normal(g, (D,), 0.2, F32))
    net.gate.copy_(normal(g, (1, D)))
    net.block.b1.copy_(normal(g, (F,), 0.1, F32))
    x, ds, dn = normal(g, (T, D)), normal(g, (T, D)), normal(g, (T, D))
    s, n = net.forward(x)
    grads = net.backward(ds, dn)
    leaf = {k: v.double().requires_grad_(True) for k, v in dict(x=x, pre=net.pre, post=net.post, gate=net.gate, next=net.next,
                                                                W1=net.block.W1, b1=net.block.b1, W2=net.block.W2,
                                                                b2=net.block.b2).items()}

    def rms(t, w):
        return t / torch.sqrt(t.square().mean(1, keepdim=True) + net.eps) * w
    h = rms(leaf["x"], leaf["pre"])
    y = ffn.act(h @ leaf["W1"] + leaf["b1"], "gelu_tanh") @ leaf["W2"] + leaf["b2"]
    want_s = leaf["x"] + net.scale * leaf["gate"] * rms(y, leaf["post"])
    want_n = rms(want_s, leaf["next"])
    want = dict(zip(leaf, torch.autograd.grad((want_s * ds.double()).sum() + (want_n * dn.double()).sum(), list(leaf.values()))))
    assert relative(s, want_s) <= 4 * ROUNDED and relative(n, want_n) <= 5 * ROUNDED
    for k, v in want.items():
        assert relative(grads[k], v) <= 8 * ROUNDED, k
    gbr.check_device()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("padded", [False, True])
def test_sorted_experts(gbr, gated, padded):
    """More tokens than moe_layer takes, against the definition over the routing that was made; a padded batch."""
    import ffn_reference as ffn
    from mbarrier_gemm_pipelines_gb300 import feed_forward
    g, T, D, F, E, k = rng(31), 200, 136, 264, 6, 2
    net = feed_forward.ExpertFeedForward(D, F, experts=E, top_k=k, act="silu", gated=gated, seed=4)
    net.b1.copy_(normal(g, net.b1.shape, 0.1, F32)), net.b2.copy_(normal(g, net.b2.shape, 0.1, F32))
    x, dy = normal(g, (T, D)), normal(g, (T, D))
    live = torch.arange(T, device="cuda") < (150 if padded else T)
    y = net.forward_sorted(x, live if padded else None)
    _, ids, weights, positions, offsets = net._saved[:5]
    assert int(offsets[-1]) == int(live.sum()) * k
    leaf = {n: getattr(net, n).double().requires_grad_(True) for n in ("Wr", "W1", "b1", "W2", "b2")}
    leaf["x"] = x.double().requires_grad_(True)
    w = torch.softmax((leaf["x"] @ leaf["Wr"]).gather(1, ids.clamp(min=0)), 1)
    assert (w - weights)[live].abs().max() <= 1e-5
    want = torch.zeros(T, D, device="cuda", dtype=torch.float64)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        z = leaf["x"][t] @ leaf["W1"][e] + leaf["b1"][e]
        h = ffn.act(z[:, :F], "silu") * z[:, F:] if gated else ffn.act(z, "silu")
        want = want.index_add(0, t, w[t, j][:, None] * (h @ leaf["W2"][e] + leaf["b2"][e]))
    assert relative(y, want) <= 4 * ROUNDED
    assert not y[~live].any()
    if gated:
        with pytest.raises(NotImplementedError):
            net.backward(dy)
        return
    grads = net.backward(dy)
    exact = dict(zip(leaf, torch.autograd.grad((want * dy.double()).sum(), list(leaf.values()))))
    for n, v in exact.items():
        assert relative(grads[n], v) <= 8 * ROUNDED, n
    assert not grads["x"][~live].any()
    gbr.check_device()


def test_sorted_experts_agree_with_the_layer_for_few_tokens(gbr):
    from mbarrier_gemm_pipelines_gb300 import feed_forward
    net = feed_forward.ExpertFeedForward(264, 520, experts=8, top_k=2, act="gelu", seed=5)
    x = normal(rng(32), (60, 264))
    few, many = net.forward(x), net.forward_sorted(x)
    assert relative(many, few.double()) <= 4 * ROUNDED
    assert net.forward(torch.cat([x, x])).shape == (120, 264)


def test_feed_forward_in_4_bits(gbr):
    """Against the definition with the same roundings: the hidden values, rounded to bf16, may fall to the other side of
    a 4-bit border (half a step of up to 1/4 of a value, in about one value of 64), so the second product is compared on
    the hidden values that were served."""
    from mbarrier_gemm_pipelines_gb300 import feed_forward
    block = feed_forward.FeedForward(512, 1056, act="silu", seed=6)
    x = normal(rng(33), (70, 512))
    net = feed_forward.FeedForward4Bit(block)
    y = net.forward(x)
    xq, W1, W2 = ref.quantize(x)[0], ref.quantize(block.W1.t())[0], ref.quantize(block.W2.t())[0]
    h = gbr.gemm_mxfp4(gbr.quantize_mxfp4(x), net.W1, net.b1, act="silu")
    assert relative(h, ref.linear(xq, W1, net.b1, None, "silu")) <= 1.0625 * ROUNDED
    assert relative(y, ref.linear(ref.quantize(h)[0], W2, net.b2, x, "none")) <= 1.0625 * ROUNDED


def test_example_runs(gbr):
    from mbarrier_gemm_pipelines_gb300 import feed_forward
    for name, t in feed_forward.example_forms(T=130, D=256, F=512).items():
        assert t.shape == (130, 256) and torch.isfinite(t.float()).all(), name


# ------------------------------------------------------------ past 32-bit offsets
def test_offsets_past_32_bits(gbr):
    """Row strides and matrices that leave 2^31 elements behind them: the last rows against the definition."""
    free = torch.cuda.mem_get_info()[0]
    if free < 60 << 30:
        pytest.skip("needs 60 GB")
    g = rng(40)
    pitch = 1 << 28
    wide = torch.zeros(16, pitch, device="cuda", dtype=BF)      # 2^32 elements
    X = wide[:, 8:1032]
    X.copy_(normal(g, (16, 1024)))
    w = 1 + normal(g, (1024,), 0.1, F32)
    S, H = gbr.residual_norm(X, X, post=w, pre=w)
    check_norm(dict(X=X.contiguous(), R=X.contiguous(), post=w, gate=None, scale=1.0, pre=w, eps=1e-6), S, H)
    a = dict(dS=X, dH=X, X=X, S=X, post=w, gate=None, scale=1.0, pre=w, eps=1e-6)
    check_norm_grads({k: v.contiguous() if torch.is_tensor(v) else v for k, v in a.items()}, gbr.residual_norm_backward(**a))
    ids = torch.arange(16, device="cuda").flip(0)[:, None].contiguous()
    p, o = gbr.moe_sort(ids, 16)
    Xs = gbr.moe_dispatch(X, p, o)
    assert torch.equal(Xs, X.flip(0))
    assert torch.equal(gbr.moe_combine(X, p), X.flip(0))
    dYs, dw = gbr.moe_combine_backward(X, X, p, o, torch.ones(16, 1, device="cuda"))
    assert torch.equal(dYs, X.flip(0))
    Q = gbr.quantize_mxfp4(X)
    check_quantized(Q, X.contiguous())
    back = gbr.dequantize_mxfp4(Q, X=wide[:, 4096:5120])
    assert torch.equal(back.double(), ref.values(Q))
    C = gbr.gemm_mxfp4(Q, Q, C=wide[:, 8192:8208])
    x = ref.values(Q)
    within(C, x @ x.t(), gemm_bar(x, x, 1024) + 2.0 ** -22 * (x @ x.t()).abs(), "C")
    del wide, X, back, C
    # Data of more than 2^31 bytes: 70000 rows of 65536 values.
    rows, cols = 70000, 65536
    X = torch.empty(rows, cols, device="cuda", dtype=BF)
    X.copy_(normal(g, (1, cols)).expand(rows, cols))
    X[-1] = normal(g, (cols,), 3.0)
    Q = gbr.quantize_mxfp4(X)
    tail = gbr.quantize_mxfp4(X[-1:].contiguous())
    assert torch.equal(Q.data[-1], tail.data[0])
    assert torch.equal(ref.scale_bytes(Q.scales, rows, cols // 32)[-1], ref.scale_bytes(tail.scales, 1, cols // 32)[0])
    back = gbr.dequantize_mxfp4(Q)
    assert torch.equal(back[-1], gbr.dequantize_mxfp4(tail)[0]) and torch.equal(back[0], back[rows - 2])
    gbr.check_device()
