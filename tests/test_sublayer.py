"""The operators around the block against the float64 oracle: norms fused with
the combine, gate and residual, their backward pass, gradient clipping, their
refusals, and a whole sub-layer (serving and training step).

Tolerances, from the arithmetic (u = 2^-24, a float32 rounding; a stored bf16
value adds half a step, 2^-8 of itself):
  - a row sum is a tree of at most 64 values per thread and ten levels over the
    threads, a combine at most 24 additions, and N(v) a handful of products: in
    all under 128 roundings of magnitudes that M (the same expression with
    every term's magnitude) bounds, so float32 work is off by at most 128 u M;
  - xn adds the error of h, passed on by at most r |w| (its part through the
    row statistics is no larger): another 256 u r |w| max M;
  - column sums are at most T terms in one thread's chain and the partial sums
    of the CTAs: (T + 128) u times the sum of the magnitudes.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import oracle.sublayer as ref
import sparse_mixture_experts_07_b200 as moe
from parity_util import BF16_TOL, rel_l2, to_device
from sparse_mixture_experts_07_b200.inputs import MoEConfig, make_inputs
from sparse_mixture_experts_07_b200.moe import MoEShape
from sparse_mixture_experts_07_b200.sublayer import MoENormSpec

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _shape(T, H, k=2, S=0, dtype=torch.bfloat16):
    return moe.Shape(T=T, H=H, I=8, E=16, k=k, n_shared=S, I_shared=8 if S else 0,
                     dtype=moe.MOE_BF16 if dtype == torch.bfloat16 else moe.MOE_F32)


def _params(g, kind, H, eps=1e-5):
    """(Norm on the device, oracle keyword arguments)."""
    if kind == "none":
        return moe.Norm("none"), dict(kind="none")
    w = 1.0 + 0.2 * torch.randn(H, generator=g)
    b = 0.3 * torch.randn(H, generator=g) if kind == "layer" else None
    spec = moe.Norm(kind, eps, w.cuda(), None if b is None else b.cuda())
    return spec, dict(kind=kind, eps=spec.c().eps, weight=_np(w), bias=_np(b))


def _gate(g, kind, T, H):
    if kind is None:
        return None
    return torch.rand(*((T, 1) if kind == "token" else (H,)), generator=g) * 2 - 0.5


def _close(name, got, want, tol):
    got = np.asarray(got, dtype=np.float64)
    bad = np.abs(got - want) > tol
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, worst "
                           f"{(np.abs(got - want) / tol).max():.2f} of the tolerance")


def _norm_mag(y, kind, eps=0.0, weight=None, bias=None):
    """(magnitude of N(y)'s terms, r |w| per element)."""
    if kind == "none":
        return np.abs(y), np.ones_like(y)
    m = y.mean(axis=1, keepdims=True) if kind == "layer" else np.zeros((y.shape[0], 1))
    r = 1.0 / np.sqrt(((y - m) ** 2).mean(axis=1, keepdims=True) + eps)
    w = np.ones(y.shape[1]) if weight is None else np.abs(weight)
    mean_abs = np.abs(y).mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    return (np.abs(y) + mean_abs) * r * w + (0 if bias is None else np.abs(bias)), r * w


# ------------------------------------------------------------------ the oracle itself
@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate", [None, "token", "channel"])
def test_oracle_gradients_match_differences(kind, gate):
    rng = np.random.default_rng(3)
    T, H, scale, step = 3, 7, 0.6, 2.0 ** -14
    x, R = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    p = dict(kind=kind) if kind == "none" else dict(
        kind=kind, eps=1e-3, weight=rng.standard_normal(H), bias=rng.standard_normal(H))
    g = {None: None, "token": rng.random((T, 1)), "channel": rng.random(H)}[gate]
    got = ref.norm_backward(x, R, gate=g, scale=scale, **p)

    def loss(x, p, g):
        return (ref.residual_norm(x, None, p, g, scale, None)[0] * R).sum()

    def differences(a, f):
        d = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            hi, lo = a.copy(), a.copy()
            hi[i] += step
            lo[i] -= step
            d[i] = (f(hi) - f(lo)) / (2 * step)
        return d
    # third derivatives of order 10 times step^2 / 6, and 2^-52 / step of the loss
    want = {"x": differences(x, lambda a: loss(a, p, g))}
    if kind != "none":
        want["weight"] = differences(p["weight"], lambda a: loss(x, {**p, "weight": a}, g))
        want["bias"] = differences(p["bias"], lambda a: loss(x, {**p, "bias": a}, g))
    if g is not None:
        want["gate"] = differences(g, lambda a: loss(x, p, a))
    for n, w in want.items():
        assert np.abs(got[n] - w).max() < 1e-6, n


def test_oracle_closed_forms():
    x = np.array([[3.0, 4.0]])
    assert np.allclose(ref.norm(x, "rms"), x / np.sqrt(12.5))
    assert np.allclose(ref.norm(x, "layer"), [[-1.0, 1.0]])
    n, (g,) = ref.clip([x], 1.0)
    assert n == 5.0 and np.allclose(g, x / (5.0 + 1e-6))
    assert np.array_equal(ref.clip([x], 6.0)[1][0], x)


# -------------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from sparse_mixture_experts_07_b200 import build as moe_build
    moe_build.build()
    return moe.load_library()


def _c(**kw):
    base = dict(T=4, H=128, I=8, E=16, k=2, n_shared=0, I_shared=0, routed_scale=1.0,
                dtype=moe.MOE_BF16)
    base.update(kw)
    return ctypes.byref(MoEShape(**base))


def test_norm_refusals(lib):
    ok, odd = 4096, 4096 + 2
    spec = ctypes.byref(MoENormSpec(1, 1e-5, ok, None))
    f = lib.moe_norm_forward
    assert f(None, spec, ok, ok, None) == 1
    assert f(_c(), None, ok, ok, None) == 1
    for bad in (MoENormSpec(3, 1e-5, ok, None), MoENormSpec(-1, 1e-5, ok, None),
                MoENormSpec(1, -1.0, ok, None), MoENormSpec(1, float("nan"), ok, None),
                MoENormSpec(0, 0.0, ok, None)):
        assert f(_c(), ctypes.byref(bad), ok, ok, None) == 1
    assert f(_c(), spec, None, ok, None) == 1
    assert f(_c(), spec, ok, None, None) == 1
    assert f(_c(), spec, odd, ok, None) == 2
    assert f(_c(), ctypes.byref(MoENormSpec(1, 1e-5, odd, None)), ok, ok, None) == 2
    assert f(_c(H=32776), spec, ok, ok, None) == 2
    assert f(_c(H=100), spec, ok, ok, None) == 2
    assert f(_c(T=0), spec, None, None, None) == 0


def test_combine_norm_refusals(lib):
    ok = 4096
    spec = ctypes.byref(MoENormSpec(2, 1e-5, ok, ok))

    def f(shape=None, slots=ok, inv=ok, res=ok, post=spec, kind=0, gate=None, nxt=None, y=None,
          h=ok, xn=None):
        return lib.moe_combine_norm(shape or _c(), slots, inv, res, post, kind, gate, 1.0, nxt, y,
                                    h, xn, None)
    assert f(slots=None) == 1 and f(inv=None) == 1 and f(h=None) == 1
    assert f(kind=1) == 1 and f(kind=0, gate=ok) == 1 and f(kind=3, gate=ok) == 1
    assert f(nxt=spec) == 1 and f(xn=ok) == 1
    assert f(nxt=ctypes.byref(MoENormSpec(9, 0, None, None)), xn=ok) == 1
    assert f(res=ok + 8) == 2 and f(y=ok + 8) == 2
    assert f(kind=2, gate=ok + 4) == 2
    assert f(shape=_c(H=40000)) == 2
    assert f(shape=_c(T=0), slots=None, inv=None, res=None, h=None) == 0


def test_norm_backward_refusals(lib):
    ok = 4096
    spec = ctypes.byref(MoENormSpec(1, 1e-5, ok, None))
    n = ctypes.c_size_t(0)
    assert lib.moe_norm_backward_workspace_size(_c(), None) == 1
    assert lib.moe_norm_backward_workspace_size(_c(H=32776), ctypes.byref(n)) == 2
    assert lib.moe_norm_backward_workspace_size(_c(), ctypes.byref(n)) == 0
    need = n.value
    assert need >= 4 * 2 * 128 * 4                  # four rows: a part each at most

    def f(shape=None, norm=spec, x=ok, dout=ok, kind=0, gate=None, dadd=None, dx=ok, dw=ok,
          db=None, dg=None, ws=ok, size=need):
        return lib.moe_norm_backward(shape or _c(), norm, x, dout, kind, gate, 1.0, dadd, dx, dw,
                                     db, dg, ws, size, None)
    assert f(norm=None) == 1 and f(x=None) == 1 and f(dout=None) == 1 and f(dx=None) == 1
    assert f(dg=ok) == 1 and f(kind=1) == 1
    assert f(norm=ctypes.byref(MoENormSpec(0, 0, None, None))) == 1
    assert f(ws=None) == 3 and f(size=need - 1) == 3
    assert f(dx=ok + 8) == 2 and f(dadd=ok + 2) == 2 and f(ws=ok + 8) == 2
    assert f(shape=_c(T=0), dw=None, ws=None, size=0) == 0


def test_clip_refusals(lib):
    n = ctypes.c_size_t(0)
    assert lib.moe_grad_norm_workspace_size(None) == 1
    assert lib.moe_grad_norm_workspace_size(ctypes.byref(n)) == 0
    ok = 4096

    def f(ptrs=(4096, 65536), sizes=(16, 16), types=(0, 1), max_norm=1.0, norm=ok, ws=ok,
          size=n.value, count=None):
        k = len(ptrs)
        return lib.moe_clip_grad_norm(
            k if count is None else count, (ctypes.c_void_p * k)(*ptrs),
            (ctypes.c_int64 * k)(*sizes), (ctypes.c_int32 * k)(*types), max_norm, norm, ws, size,
            None)
    assert f(ptrs=(4096, 4096)) == 1                       # the same tensor twice
    assert f(ptrs=(65536, 65536 - 28)) == 1                # the second runs into the first
    assert f(ptrs=(4096, None)) == 1 and f(sizes=(16, -1)) == 1 and f(types=(0, 5)) == 1
    assert f(max_norm=-1.0) == 1 and f(max_norm=float("nan")) == 1 and f(count=-1) == 1
    assert f(ptrs=(4098, 65536)) == 2 and f(ws=ok + 8) == 2
    assert f(ws=None) == 3 and f(size=n.value - 1) == 3
    arrays = ((ctypes.c_void_p * 1)(4096), (ctypes.c_int64 * 1)(4), (ctypes.c_int32 * 1)(0))
    assert lib.moe_clip_grads(1, *arrays, None, 1.0, None, None) == 1
    assert lib.moe_clip_grads(1, *arrays, 4100, 1.0, None, None) == 2
    assert lib.moe_grad_square_sum(1, *arrays, None, ok, n.value, None) == 1


def test_binding_refusals(lib):
    """Shapes, types, layouts and devices are checked before the library is called."""
    s = _shape(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.norm(s, moe.Norm(), torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        moe.clip_grad_norm([torch.zeros(3)], 1.0)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        moe.clip_grad_norm([torch.zeros(3, dtype=torch.float16)], 1.0)
    with pytest.raises(ValueError, match="no gradients"):
        moe.clip_grad_norm([None], 1.0)
    with pytest.raises(ValueError, match="kind"):
        moe.Norm("batch")
    with pytest.raises(ValueError, match="weight"):
        moe.Norm("none", weight=torch.ones(4))


@pytest.mark.gpu
def test_binding_refusals_on_device(cuda_ok):
    s = _shape(4, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (x[:3], x.float(), torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda").t()):
        with pytest.raises(ValueError):
            moe.norm(s, moe.Norm(), bad)
    with pytest.raises(ValueError):
        moe.norm(s, moe.Norm(weight=torch.ones(64)), x)
    with pytest.raises(ValueError):
        moe.norm(s, moe.Norm(weight=torch.ones(63, device="cuda")), x)
    slots = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    inv = torch.arange(8, dtype=torch.int32, device="cuda")
    for kw in (dict(gate=torch.ones(4, device="cuda")), dict(residual=x[:2]),
               dict(gate=torch.ones(64, dtype=torch.float64, device="cuda")),
               dict(out={"h": x[:, :32]})):
        with pytest.raises(ValueError):
            moe.combine_norm(s, slots, inv, **kw)
    with pytest.raises(ValueError):
        moe.combine_norm(s, slots, inv.long())
    with pytest.raises(ValueError):
        moe.combine_norm(s, slots[:7], inv)
    with pytest.raises(ValueError, match="contiguous"):
        moe.clip_grad_norm([torch.zeros(4, 6, device="cuda").t()], 1.0)
    g = torch.ones(8, device="cuda")
    with pytest.raises(moe.MoEError, match="INVALID"):
        moe.clip_grad_norm([g, g], 1.0)
    with pytest.raises(moe.MoEError, match="INVALID"):
        moe.clip_grad_norm([g[:6], g[4:]], 1.0)


# ------------------------------------------------------------------- forward, on the GPU
FORWARD = [
    # T, H, k, S, dtype, post, gate, next
    (1, 64, 2, 0, torch.bfloat16, "rms", None, "rms"),
    (1, 4096, 2, 0, torch.bfloat16, "rms", None, "rms"),
    (3, 8, 1, 0, torch.bfloat16, "layer", "channel", "rms"),
    (130, 2880, 4, 0, torch.bfloat16, "rms", "token", "layer"),
    (257, 2048, 6, 2, torch.bfloat16, "none", "token", "rms"),
    (2500, 264, 16, 8, torch.bfloat16, "layer", None, "none"),
    (5, 8200, 3, 1, torch.bfloat16, "layer", "channel", "layer"),
    (2, 32768, 1, 0, torch.bfloat16, "rms", "channel", "rms"),
    (1, 1, 1, 0, torch.float32, "rms", "token", "layer"),
    (33, 129, 2, 1, torch.float32, "layer", "token", "layer"),
    (64, 1024, 4, 0, torch.float32, "rms", "channel", "rms"),
    (3, 4100, 2, 1, torch.float32, "layer", None, "layer"),
    (3, 5001, 2, 0, torch.float32, "rms", "token", "rms"),
    (2, 32767, 1, 1, torch.float32, "layer", "channel", "rms"),
    (2, 32768, 1, 1, torch.float32, "layer", "channel", "rms"),
]


def _forward_inputs(T, H, k, S, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    inv = torch.randperm(T * k, generator=g).to(torch.int32)
    slots = (torch.randn(T * (k + S), H, generator=g) + 0.25).to(dtype)
    res = (torch.randn(T, H, generator=g) * 2).to(dtype)
    return g, slots, inv, res


def _check_forward(got, slots, inv, res, T, k, S, po, no, gate, scale, dtype):
    h, xn, y = got
    yr = ref.combine(_np(slots), _np(inv), T, k, S)
    hr, xr = ref.residual_norm(yr, _np(res), po, gate, scale, no)
    mag = ref.combine(np.abs(_np(slots)), _np(inv), T, k, S)
    half = HALF[dtype]
    if y is not None:
        _close("y", _np(y), yr, half * np.abs(yr) + 32 * U * mag + 1e-40)
    M, rw = _norm_mag(yr, **po)
    M = M + mag * rw
    M = M * np.abs(scale if gate is None else scale * gate) + np.abs(_np(res))
    _close("h", _np(h), hr, half * np.abs(hr) + 128 * U * M + 1e-40)
    if no is not None:
        M2, rw2 = _norm_mag(hr, **no)
        top = M.max(axis=1, keepdims=True)
        _close("xn", _np(xn), xr, half * np.abs(xr) + U * (128 * M2 + 256 * rw2 * top) + 1e-40)


@pytest.mark.gpu
@pytest.mark.parametrize("case", FORWARD, ids=lambda c: "-".join(str(v) for v in c))
def test_combine_norm_matches_oracle(cuda_ok, case):
    T, H, k, S, dtype, post, gate, nxt = case
    g, slots, inv, res = _forward_inputs(T, H, k, S, dtype)
    post, po = _params(g, post, H)
    nx, no = _params(g, nxt, H)
    gt = _gate(g, gate, T, H)
    s = _shape(T, H, k, S, dtype)
    got = moe.combine_norm(s, slots.cuda(), inv.cuda(), res.cuda(), post=post,
                           gate=None if gt is None else gt.cuda(), scale=0.7,
                           next_norm=nx, keep_y=True)
    _check_forward(got, slots, inv, res, T, k, S, po, no, _np(gt), np.float64(np.float32(0.7)),
                   dtype)
    # the same call twice gives the same bits; in place over the residual too
    r2 = res.cuda()
    again = moe.combine_norm(s, slots.cuda(), inv.cuda(), r2, post=post,
                             gate=None if gt is None else gt.cuda(), scale=0.7, next_norm=nx,
                             out={"h": r2})
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1]) and again[2] is None
    assert again[0] is r2


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,kind,dtype", [
    (1, 4096, "rms", torch.bfloat16), (700, 136, "layer", torch.bfloat16),
    (9, 77, "layer", torch.float32), (300, 512, "rms", torch.float32),
    (4, 16, "none", torch.float32)])
def test_norm_matches_oracle(cuda_ok, T, H, kind, dtype):
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(T, H, generator=g) * 3 + 20).to(dtype)     # a mean far from zero
    spec, po = _params(g, kind, H)
    got = _np(moe.norm(_shape(T, H, dtype=dtype), spec, x.cuda()))
    want = ref.norm(_np(x), **po)
    M, rw = _norm_mag(_np(x), **po)
    _close("xn", got, want, HALF[dtype] * np.abs(want) + 128 * U * M + 1e-40)


@pytest.mark.gpu
def test_norm_without_weight_zero_rows_and_views(cuda_ok):
    """No weight; a row of zeros (eps alone under the root); float32 rows that
    start off a 16-byte boundary; a NaN and an infinity stay in their rows."""
    T, H = 6, 64
    g = torch.Generator().manual_seed(2)
    buf = torch.randn(T * H + 1, generator=g).cuda()
    x = buf[1:].view(T, H)
    x[2] = 0
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    s = _shape(T, H, dtype=torch.float32)
    y = moe.norm(s, moe.Norm("rms", 1e-6), x)
    assert torch.equal(y[2], torch.zeros(H, device="cuda"))
    assert y[4].isnan().all() and y[3, 5].isnan() and torch.equal(y[3, :5], torch.zeros(5).cuda())
    for t in (0, 1, 5):
        want = ref.norm(_np(x[t:t + 1]), "rms", 1e-6)
        _close("row", _np(y[t:t + 1]), want, 130 * U * np.abs(want))


@pytest.mark.gpu
def test_combine_norm_skips_holes_and_stops_at_the_last_row(cuda_ok):
    """Slots that a plan left unset add nothing; nothing is written past row T."""
    T, H, k = 5, 64, 2
    _, slots, inv, res = _forward_inputs(T, H, k, 0, torch.bfloat16)
    inv[3], inv[6] = -1, T * k
    h = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    xn = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    got = moe.combine_norm(_shape(T, H, k), slots.cuda(), inv.cuda(), res.cuda(),
                           next_norm=moe.Norm("rms", 1e-5), out={"h": h[:T], "xn": xn[:T]})
    assert got[0].data_ptr() == h.data_ptr()
    _check_forward((h[:T], xn[:T], None), slots, inv, res, T, k, 0, dict(kind="none"),
                   dict(kind="rms", eps=np.float64(np.float32(1e-5))), None, 1.0, torch.bfloat16)
    assert (h[T:] == 7).all() and (xn[T:] == 7).all()


@pytest.mark.gpu
def test_zero_tokens(cuda_ok):
    s = _shape(0, 64)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    assert moe.norm(s, moe.Norm(weight=w), e).shape == (0, 64)
    h, xn, y = moe.combine_norm(s, e, torch.empty(0, dtype=torch.int32, device="cuda"), e,
                                next_norm=moe.Norm(weight=w), keep_y=True)
    assert h.shape == xn.shape == y.shape == (0, 64)
    gate = torch.ones(64, device="cuda")
    g = moe.norm_backward(s, moe.Norm(weight=w), e, e, gate=gate)
    assert not g["weight"].any() and not g["gate"].any()


# ------------------------------------------------------------------ backward, on the GPU
BACKWARD = [
    # T, H, dtype, kind, gate, add
    (1, 4096, torch.bfloat16, "rms", None, False),
    (1, 8, torch.bfloat16, "layer", "token", True),
    (300, 2880, torch.bfloat16, "rms", "channel", True),
    (777, 264, torch.bfloat16, "layer", "channel", False),
    (1500, 64, torch.bfloat16, "rms", "token", True),
    (65, 8192, torch.bfloat16, "layer", None, True),
    (3, 16392, torch.bfloat16, "layer", "channel", True),
    (2, 32768, torch.bfloat16, "rms", "token", False),
    (40, 512, torch.bfloat16, "none", "channel", True),
    (40, 512, torch.bfloat16, "none", None, False),
    (1, 1, torch.float32, "rms", "token", True),
    (129, 129, torch.float32, "layer", "token", False),
    (300, 1024, torch.float32, "rms", "channel", True),
    (3, 4100, torch.float32, "layer", "token", True),
    (3, 5001, torch.float32, "rms", "channel", False),
    (2, 32768, torch.float32, "layer", None, True),
    (2, 32767, torch.float32, "layer", "token", True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "-".join(str(v) for v in c))
def test_norm_backward_matches_oracle(cuda_ok, case):
    T, H, dtype, kind, gate, add = case
    g = torch.Generator().manual_seed(4)
    x = (torch.randn(T, H, generator=g) + 0.5).to(dtype)
    dout = torch.randn(T, H, generator=g).to(dtype)
    dadd = torch.randn(T, H, generator=g).to(dtype) if add else None
    spec, po = _params(g, kind, H, eps=1e-2)
    gt = _gate(g, gate, T, H)
    scale = np.float64(np.float32(0.3))
    s = _shape(T, H, dtype=dtype)

    def run(dx=None):
        d = dout.cuda() if dx is None else dx
        return moe.norm_backward(s, spec, x.cuda(), d, gate=None if gt is None else gt.cuda(),
                                 scale=0.3, dadd=None if dadd is None else dadd.cuda(), dx=dx)
    got = run()
    want = ref.norm_backward(_np(x), _np(dout), gate=_np(gt), scale=scale, dadd=_np(dadd), **po)
    # magnitudes of the terms
    xd, dd = _np(x), np.abs(_np(dout))
    w = np.ones(H) if po.get("weight") is None else np.abs(po["weight"])
    b = np.zeros(H) if po.get("bias") is None else np.abs(po["bias"])
    gm = 1.0 if gt is None else np.abs(_np(gt))
    m = xd.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    r = 1.0 / np.sqrt(((xd - m) ** 2).mean(axis=1, keepdims=True) + po["eps"]) \
        if kind != "none" else 1.0
    mean_abs = np.abs(xd).mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    xh = (np.abs(xd) + mean_abs) * r
    wD = scale * gm * w * dd
    M = wD
    if kind != "none":
        M = r * (wD + wD.mean(axis=1, keepdims=True)
                 + xh * (wD * xh).mean(axis=1, keepdims=True))
    if dadd is not None:
        M = M + np.abs(_np(dadd))
    _close("dx", _np(got["x"]), want["x"],
           HALF[dtype] * np.abs(want["x"]) + 160 * U * M + 1e-40)
    cols = (T + 128) * U
    if spec.weight is not None:
        _close("dweight", _np(got["weight"]), want["weight"],
               cols * (scale * gm * dd * xh).sum(axis=0) + 1e-40)
    else:
        assert got["weight"] is None
    if spec.bias is not None:
        _close("dbias", _np(got["bias"]), want["bias"],
               cols * (scale * gm * dd).sum(axis=0) + 1e-40)
    if gt is not None:
        terms = scale * dd * (xh * w + b)
        axis = 1 if gate == "token" else 0
        tol = terms.sum(axis=axis) * (160 * U if gate == "token" else cols)
        _close("dgate", _np(got["gate"]).reshape(-1), want["gate"].reshape(-1), tol + 1e-40)
    # deterministic, and in place over dout
    again = run(dx=dout.cuda())
    for n in got:
        assert (got[n] is None and again[n] is None) or torch.equal(got[n], again[n]), n


@pytest.mark.gpu
def test_norm_backward_matches_differences_of_the_kernel(cuda_ok):
    """A directional derivative of the forward kernel itself (float32): the
    central difference over step e is off by e^2 / 6 of a third derivative
    (order 10 |v|^3 sum|R|/H here, |v| about 1 per element) and by 2^-23 / e of
    the outputs' magnitudes: with e = 2^-7 both stay under 1e-3 of sum|R|."""
    T, H, e = 16, 96, 2.0 ** -7
    g = torch.Generator().manual_seed(5)
    x, v, R = (torch.randn(T, H, generator=g).cuda() for _ in range(3))
    s = _shape(T, H, dtype=torch.float32)
    for kind in ("rms", "layer"):
        spec, _ = _params(g, kind, H)
        d = moe.norm_backward(s, spec, x, R)["x"]
        hi, lo = (moe.norm(s, spec, x + sign * e * v).double() for sign in (1, -1))
        want = float(((hi - lo) / (2 * e) * R.double()).sum())
        got = float((d.double() * v.double()).sum())
        assert abs(got - want) <= 1e-3 * float(R.abs().sum()), kind


# -------------------------------------------------------------------- clipping, on the GPU
def _grads(sizes, seed=0, scale=1e-2):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(*size, generator=g) * scale).to(dt).cuda() for size, dt in sizes]


CLIP = {
    "one": [((1,), torch.float32)],
    "empty": [((0, 3), torch.float32), ((5,), torch.bfloat16)],
    "odd": [((3, 5, 7), torch.float32), ((1,), torch.bfloat16), ((4097,), torch.float32),
            ((1023, 9), torch.bfloat16)],
    "chunks": [((4096,), torch.float32), ((8192,), torch.bfloat16), ((4095,), torch.float32)],
    "many": [((n % 37 + 1, 3), torch.float32 if n % 3 else torch.bfloat16) for n in range(150)],
    "large": [((1 << 26,), torch.float32), ((123457,), torch.bfloat16)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CLIP)
@pytest.mark.parametrize("max_norm", [1e-3, 1e9])
def test_clip_matches_oracle(cuda_ok, name, max_norm):
    grads = _grads(CLIP[name])
    before = [g.clone() for g in grads]
    n, want = ref.clip([_np(g) for g in grads], float(np.float32(max_norm)))
    got = moe.clip_grad_norm(grads + [None], max_norm)
    # float64 sums, one rounding to float32
    assert abs(float(got) - n) <= 2.0 ** -23 * n
    for g, b, w in zip(grads, before, want):
        if max_norm > n:
            assert torch.equal(g, b)
        else:       # the factor and the product are rounded, and a bf16 result once more
            _close("g", _np(g), w, (HALF[g.dtype] + 4 * U) * np.abs(w) + 1e-40)
    # the two-call form does the same
    two = [b.clone() for b in before]
    total = moe.grad_square_sum(two)
    assert abs(float(total) - n * n) <= 1e-12 * n * n
    norm2 = moe.clip_grads(two, max_norm, total)
    assert torch.equal(norm2, got) and all(torch.equal(a, b) for a, b in zip(two, grads))


@pytest.mark.gpu
def test_clip_range_views_and_nonfinite(cuda_ok):
    """Squares outside float32's range; views off the vector boundary, whose
    neighbours stay; infinity and NaN as the formula has them."""
    big = torch.full((1000,), 1e30, device="cuda")
    tiny = torch.full((1000,), 1e-30, device="cuda")
    n = moe.clip_grad_norm([big], 1.0)
    assert abs(float(n) / (1e30 * 1000 ** 0.5) - 1) < 1e-6
    assert torch.allclose(big, torch.full_like(big, 1000 ** -0.5), rtol=1e-6)
    assert abs(float(moe.clip_grad_norm([tiny], 1.0)) / (1e-30 * 1000 ** 0.5) - 1) < 1e-6
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.ones(103, device="cuda", dtype=dt)
        moe.clip_grad_norm([buf[1:102]], 0.5)
        assert buf[0] == 1 and buf[102] == 1 and (buf[1:102] < 0.06).all()
    g = torch.ones(10, device="cuda")
    g[3] = float("inf")
    assert float(moe.clip_grad_norm([g], 1.0)) == float("inf")
    assert g[3].isnan() and not g[:3].any()
    g = torch.ones(10, device="cuda")
    g[3] = float("nan")
    assert moe.clip_grad_norm([g], 1.0).isnan() and g.isnan().all()
    g = torch.ones(10, device="cuda")
    moe.clip_grad_norm([g], 0.0)
    assert not g.any()
    g = torch.ones(10, device="cuda")
    moe.clip_grad_norm([g], float("inf"))
    assert (g == 1).all()


@pytest.mark.gpu
def test_other_stream_and_graph(cuda_ok):
    """The calls on a given stream, and captured twice into graphs with a
    workspace of their own, give what they give eagerly."""
    T, H = 37, 264
    g, slots, inv, res = _forward_inputs(T, H, 2, 0, torch.bfloat16)
    slots, inv, res = slots.cuda(), inv.cuda(), res.cuda()
    spec, _ = _params(g, "layer", H)
    s = _shape(T, H)
    gate = _gate(g, "channel", T, H).cuda()
    dout = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    grads = _grads(CLIP["odd"])

    def step(stream=None, ws=None, wsn=None, grads=grads):
        h, xn, y = moe.combine_norm(s, slots, inv, res, post=spec, gate=gate, scale=0.5,
                                    next_norm=spec, keep_y=True, stream=stream)
        b = moe.norm_backward(s, spec, y, dout, gate=gate, scale=0.5, dadd=dout, workspace=ws,
                              stream=stream)
        n = moe.clip_grad_norm(grads, 0.1, workspace=wsn, stream=stream)
        return [h, xn, y, b["x"], b["weight"], b["bias"], b["gate"], n] + list(grads)
    mine = [[g.clone() for g in grads] for _ in range(4)]
    want = step(grads=mine[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side, grads=mine[1])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for m in mine[2:]:
        ws, wsn = moe.alloc_norm_backward_workspace(s), moe.alloc_grad_norm_workspace()
        first = [g.clone() for g in m]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(ws=ws, wsn=wsn, grads=m)
        graphs.append((graph, out, m, first, ws, wsn))     # a graph's workspaces live with it
    for _ in range(2):
        for graph, out, m, first, _, _ in graphs:
            for a, b in zip(m, first):
                a.copy_(b)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


# -------------------------------------------------------------- the whole sub-layer
SUB = MoEConfig("sublayer", T=200, H=128, I=96, E=4, k=2, n_shared=1, I_shared=64,
                routed_scale=2.5)


def _sublayer(cfg, gate=None, nxt=True):
    inp = make_inputs(cfg, seed=0)
    d = to_device(inp)
    g = torch.Generator().manual_seed(8)
    pre, po = _params(g, "rms", cfg.H)
    post, pp = _params(g, "layer", cfg.H)
    nx, pn = _params(g, "rms", cfg.H)
    layer = moe.MoELayer(moe.Shape.from_config(cfg), d["w_router"], d["router_bias"],
                         d["gate_up"], d["down"], d["sh_gate_up"], d["sh_down"],
                         merge_shared=False)
    gt = _gate(g, gate, cfg.T, cfg.H)
    sub = moe.MoESublayer(layer, pre, post, None if gt is None else gt.cuda(), 0.22,
                          nx if nxt else None)
    h = (torch.randn(cfg.T, cfg.H, generator=g) * 1.5).to(torch.bfloat16)
    return inp, sub, h, (po, pp, pn), _np(gt)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8, 200])
def test_sublayer_serving(cuda_ok, T):
    """norm, block, combine + norm + gate + residual + next norm in a run.  The
    block's routing is taken from the device, on the same bf16 rows the kernel
    normed, so that no near tie decides; the outputs are held to the block's
    bf16 bound relative to what the block adds."""
    cfg = MoEConfig("s", T=T, H=128, I=96, E=4, k=2, n_shared=1, I_shared=64, routed_scale=2.5)
    inp, sub, h, (po, pp, pn), gate = _sublayer(cfg, "channel")
    h2, xn2 = sub(h.cuda())
    torch.cuda.synchronize()
    assert sub.layer.device_error() == 0
    xn = sub.xn.cpu()
    _close("xn", _np(xn), ref.norm(_np(h), **po),
           2.0 ** -8 * np.abs(ref.norm(_np(h), **po)) + 1e-5)
    idx, w = (sub.layer.last[n].cpu().numpy() for n in ("topk_idx", "topk_w"))
    y = oracle.moe_block_routed({**inp, "x": xn}, idx, w.astype(np.float64), cfg.routed_scale)
    hr, xr = ref.residual_norm(y, _np(h), pp, gate, np.float64(np.float32(0.22)), pn)
    assert rel_l2(_np(h2) - _np(h), hr - _np(h)) < 2 * BF16_TOL + 2.0 ** -8 * np.linalg.norm(
        hr) / np.linalg.norm(hr - _np(h))
    assert rel_l2(_np(xn2), xr) < BF16_TOL
    # the next layer's norm handed over: the first norm is left out
    again = sub(h.cuda(), xn=xn.cuda())
    assert torch.equal(again[0], h2) and torch.equal(again[1], xn2)


@pytest.mark.gpu
def test_sublayer_training_step(cuda_ok):
    """forward_train, backward and clip in a run, against the chain of oracles.
    Each bf16 link (xn, y, dy, dxn) is off by at most 2^-8 relative, the
    block's gradients by their own 1e-2."""
    inp, sub, h, (po, pp, _), gate = _sublayer(SUB, "token", nxt=False)
    g = torch.Generator().manual_seed(9)
    dh = torch.randn(SUB.T, SUB.H, generator=g).to(torch.bfloat16)
    h2, saved = sub.forward_train(h.cuda())
    got = sub.backward(saved, dh.cuda())
    torch.cuda.synchronize()
    assert sub.layer.device_error() == 0
    scale = np.float64(np.float32(0.22))
    y = _np(saved["y"])
    hr, _ = ref.residual_norm(y, _np(h), pp, gate, scale, None)
    assert rel_l2(_np(h2), hr) < BF16_TOL
    gp = ref.norm_backward(y, _np(dh), gate=gate, scale=scale, **pp)
    gb = oracle.moe_backward({**inp, "x": saved["xn"].cpu()}, SUB.k, gp["x"],
                             routed_scale=SUB.routed_scale)
    gn = ref.norm_backward(_np(h), gb["x"], dadd=_np(dh), **po)
    want = {"post_weight": gp["weight"], "post_bias": gp["bias"], "gate": gp["gate"],
            "pre_weight": gn["weight"], "h": gn["x"]}
    want.update({n: gb[n] for n in ("gate_up", "down", "w_router", "router_bias", "sh_gate_up",
                                    "sh_down")})
    assert set(got) == set(want)
    for n, v in want.items():
        assert rel_l2(_np(got[n]), v) < 2 * BF16_TOL, n
    params = [got[n] for n in sorted(got) if n != "h"]
    before = [p.clone() for p in params]
    n, clipped = ref.clip([_np(p) for p in before], 0.5)
    norm = moe.clip_grad_norm(params, 0.5)
    assert abs(float(norm) - n) <= 2.0 ** -23 * n
    for p, w in zip(params, clipped):
        _close("clipped", _np(p), w, 5 * U * np.abs(w) + 1e-40)


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_ok):
    """Slot rows, norm rows and a gradient tensor of more than 2^32 bytes and
    2^31 values: rows at both ends against the oracle, and sums in closed form."""
    T, H, k = 132000, 2048, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    s = _shape(T, H, k)
    assert T * k * H > 1 << 31
    slots = torch.randn(T * k, H, generator=g, device="cuda", dtype=torch.bfloat16)
    inv = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    h, xn, _ = moe.combine_norm(s, slots, inv, post=moe.Norm("rms", 1e-5),
                                next_norm=moe.Norm("layer", 1e-5))
    for t in (0, 1, T // 2, T - 1):
        y = sum(_np(slots[int(inv[t * k + j])]) for j in range(k))[None]
        hr, xr = ref.residual_norm(y, None, dict(kind="rms", eps=1e-5), None, 1.0,
                                   dict(kind="layer", eps=1e-5))
        _close("h", _np(h[t:t + 1]), hr, 2.0 ** -8 * np.abs(hr) + 1e-5)
        _close("xn", _np(xn[t:t + 1]), xr, 2.0 ** -8 * np.abs(xr) + 2e-5)
    del slots, h, xn
    T = 1050000
    s = _shape(T, H)
    assert T * H > 1 << 31
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    dout = torch.ones(T, H, device="cuda", dtype=torch.bfloat16)
    got = moe.norm_backward(s, moe.Norm("layer", 1e-5, torch.ones(H, device="cuda"),
                                        torch.zeros(H, device="cuda")), x, dout)
    assert (got["bias"] == float(T)).all()          # sums of ones: exact in float32
    for t in (0, T // 2, T - 1):
        # a constant gradient of a layer norm with equal weights vanishes
        assert got["x"][t].float().abs().max() <= 1e-5
    del x, dout, got
    n = (1 << 31) + 12345
    grad = torch.full((n,), 2.0, device="cuda")
    assert abs(float(moe.clip_grad_norm([grad], 1.0)) / (2 * n ** 0.5) - 1) <= 2.0 ** -23
    want = 1.0 / n ** 0.5
    assert abs(float(grad[0]) / want - 1) < 1e-6 and abs(float(grad[-1]) / want - 1) < 1e-6


@pytest.mark.gpu
def test_large_values_and_small_variance(cuda_ok):
    """Rows whose mean is 1000 times their spread: the variance is taken about
    the mean.  The input's own rounding is none (float32); x - m is off by about
    70 roundings of |m|, so relative to the spread by 70 u 1000."""
    T, H = 64, 1000
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(T, H, generator=g) + 1000.0).cuda()
    got = _np(moe.norm(_shape(T, H, dtype=torch.float32), moe.Norm("layer", 0.0), x))
    want = ref.norm(_np(x), "layer", 0.0)
    _close("xn", got, want, 128 * U * (np.abs(want) + 1000.0))
    d = torch.randn(T, H, generator=g).cuda()
    got = moe.norm_backward(_shape(T, H, dtype=torch.float32), moe.Norm("layer", 0.0), x, d)["x"]
    want = ref.norm_backward(_np(x), _np(d), "layer", 0.0)["x"]
    assert rel_l2(_np(got), want) < 1000 * 256 * U


@pytest.mark.gpu
@pytest.mark.parametrize("gate", [None, "channel"])
def test_sublayer_without_a_norm_after(cuda_ok, gate):
    """No norm after the block: the gate and the scale alone, forward and backward."""
    inp, sub, h, (po, _, _), gt = _sublayer(SUB, gate, nxt=False)
    sub.post = None
    dh = torch.randn(SUB.T, SUB.H, generator=torch.Generator().manual_seed(10)).to(torch.bfloat16)
    h2, saved = sub.forward_train(h.cuda())
    got = sub.backward(saved, dh.cuda())
    scale, y = np.float64(np.float32(0.22)), _np(saved["y"])
    none = dict(kind="none")
    assert rel_l2(_np(h2), ref.residual_norm(y, _np(h), none, gt, scale, None)[0]) < BF16_TOL
    gp = ref.norm_backward(y, _np(dh), gate=gt, scale=scale, **none)
    gb = oracle.moe_backward({**inp, "x": saved["xn"].cpu()}, SUB.k, gp["x"],
                             routed_scale=SUB.routed_scale)
    want = ref.norm_backward(_np(h), gb["x"], dadd=_np(dh), **po)
    assert rel_l2(_np(got["h"]), want["x"]) < 2 * BF16_TOL
    assert rel_l2(_np(got["pre_weight"]), want["weight"]) < 2 * BF16_TOL
    assert "post_weight" not in got and ("gate" in got) == (gate is not None)
    if gate:
        assert rel_l2(_np(got["gate"]), gp["gate"]) < 1e-5
    # serving gives the same h'
    assert rel_l2(_np(sub(h.cuda())[0]), _np(h2)) < BF16_TOL


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_clip_without_a_limit_only_measures(cuda_ok, bad):
    """max_norm = infinity returns the norm, infinite or NaN as it may be, and
    changes no gradient, in one call and in two; a finite one as the formula says."""
    def grads():
        g = torch.Generator().manual_seed(3)
        out = [torch.randn(n, generator=g).to(t).cuda()
               for n, t in ((5000, torch.float32), (77, torch.bfloat16), (1, torch.float32))]
        out[0][4321] = bad
        return out
    inf, first = float("inf"), grads()
    for two in (False, True):
        got = grads()
        n = moe.clip_grads(got, inf, moe.grad_square_sum(got)) if two else \
            moe.clip_grad_norm(got, inf)
        assert n.isnan() if bad != bad else n == inf
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(got, first))
        got = grads()
        n = moe.clip_grads(got, 1.0, moe.grad_square_sum(got)) if two else \
            moe.clip_grad_norm(got, 1.0)
        if bad != bad:
            assert all(t.isnan().all() for t in got)
        else:
            assert got[0][4321].isnan() and not got[1].any() and not got[2].any()
            assert not got[0][:4321].any() and not got[0][4322:].any()


def test_overlapping_buffers_are_refused(lib):
    """Outputs that share memory with one another or with the slots, or with an
    input's rows at another offset, are refused before any launch."""
    spec = ctypes.byref(MoENormSpec(1, 1e-5, None, None))
    row, size = 128 * 2, 4 * 128 * 2                 # bytes of a row, of T = 4 rows
    slots, inv, res, h, xn, y = (1 << 20, 1 << 24, 2 << 20, 3 << 20, 4 << 20, 5 << 20)

    def f(h=h, xn=xn, y=y):
        return lib.moe_combine_norm(_c(), slots, inv, res, spec, 0, None, 1.0, spec, y, h, xn,
                                    None)
    assert f(xn=h) == 1 and f(y=h) == 1 and f(y=xn) == 1
    assert f(xn=h + size - row) == 1 and f(y=h - row) == 1
    assert f(h=slots) == 1 and f(xn=slots + 7 * row) == 1 and f(y=slots - size + row) == 1
    assert f(h=res + row) == 1 and f(xn=res - row) == 1 and f(y=res + size - 16) == 1
    assert f(h=res, y=res) == 1

    assert lib.moe_norm_forward(_c(), spec, res, res + row, None) == 1
    assert lib.moe_norm_forward(_c(), spec, res, res - size + 16, None) == 1
    n = ctypes.c_size_t(0)
    assert lib.moe_norm_backward_workspace_size(_c(), ctypes.byref(n)) == 0

    def b(x=res, dout=h, dadd=y, dx=xn):
        return lib.moe_norm_backward(_c(), spec, x, dout, 0, None, 1.0, dadd, dx, None, None,
                                     None, inv, n.value, None)
    assert b(dx=res + row) == 1 and b(dx=h - row) == 1 and b(dx=y + size - row) == 1


def test_unknown_output_names_are_refused(lib):
    class Device(torch.Tensor):
        is_cuda = True
    t = torch.zeros(8, 128, dtype=torch.bfloat16).as_subclass(Device)
    with pytest.raises(ValueError, match="h, xn and y"):
        moe.combine_norm(_shape(4, 128), t, torch.zeros(8, dtype=torch.int32), out={"hn": t[:4]})


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H", [(torch.bfloat16, 264), (torch.float32, 131)])
def test_outputs_in_place_of_inputs(cuda_ok, dtype, H):
    """Each output in the residual's place, N(x) in x's and dx in any input's:
    the values of separate buffers."""
    T = 300
    g, slots, inv, res = _forward_inputs(T, H, 2, 0, dtype)
    s = _shape(T, H, dtype=dtype)
    spec, _ = _params(g, "layer", H)
    slots, inv, res = slots.cuda(), inv.cuda(), res.cuda()
    want = moe.combine_norm(s, slots, inv, res, post=spec, next_norm=spec, keep_y=True)
    for i, name in enumerate(("h", "xn", "y")):
        place = res.clone()
        got = moe.combine_norm(s, slots, inv, place, post=spec, next_norm=spec, keep_y=True,
                               out={name: place})
        assert got[i].data_ptr() == place.data_ptr()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    place = res.clone()
    assert torch.equal(moe.norm(s, spec, place, out=place), moe.norm(s, spec, res))
    ins = dict(x=res, dout=want[0], dadd=want[1])
    dx = moe.norm_backward(s, spec, **ins)["x"]
    for name in ins:
        place = ins[name].clone()
        assert torch.equal(moe.norm_backward(s, spec, **{**ins, name: place}, dx=place)["x"], dx)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [100, 300])
def test_training_steps_route_by_the_weight_they_find(cuda_ok, T):
    """The router's weight changes in place between steps, as an optimiser leaves
    it: each step's selection and outputs are a fresh layer's, and after
    refresh_router the serving form's and a captured graph's are too."""
    cfg = MoEConfig("steps", T=T, H=128, I=96, E=4, k=2, n_shared=1, I_shared=64)
    _, sub, h, _, _ = _sublayer(cfg)
    layer, h = sub.layer, h.cuda()
    graph = layer.capture(moe.norm(layer.shape, sub.pre, h))
    for step in range(3):
        layer.w_router.copy_(layer.w_router.roll(1, 0) * 1.25)
        fresh = moe.MoELayer(layer.shape, layer.w_router.clone(), layer.router_bias,
                             layer.gate_up, layer.down, layer.sh_gate_up, layer.sh_down,
                             merge_shared=False)
        again = moe.MoESublayer(fresh, sub.pre, sub.post, None, sub.scale, sub.next_norm)
        h2, saved = sub.forward_train(h)
        want, w_saved = again.forward_train(h)
        assert torch.equal(saved["topk_idx"], w_saved["topk_idx"])
        assert torch.equal(saved["logits"], w_saved["logits"]) and torch.equal(h2, want)
        layer.w_router.copy_(layer.w_router.flip(0))
        fresh.w_router.copy_(layer.w_router)
        fresh = moe.MoELayer(layer.shape, fresh.w_router, layer.router_bias, layer.gate_up,
                             layer.down, layer.sh_gate_up, layer.sh_down, merge_shared=False)
        layer.refresh_router()
        want = fresh(graph.x).clone()
        assert torch.equal(layer(graph.x), want)
        layer.buf["y"].zero_()
        assert torch.equal(graph.replay(), want)


@pytest.mark.gpu
def test_two_steps_with_gates_of_their_own(cuda_ok):
    """A gate per token comes with each call; two training steps whose backward
    passes run after both, as with accumulated micro-batches, and after the
    sub-layer's own attributes changed, give what each alone gives."""
    _, sub, h, _, _ = _sublayer(SUB, nxt=False)
    g = torch.Generator().manual_seed(12)
    hs = [h.cuda(), (h + 1).cuda()]
    gates = [torch.rand(SUB.T, 1, generator=g).cuda() for _ in hs]
    dh = torch.randn(SUB.T, SUB.H, generator=g).to(torch.bfloat16).cuda()
    alone = []
    for x, gate in zip(hs, gates):
        one = moe.MoESublayer(sub.layer, sub.pre, sub.post, gate, sub.scale)
        h2, saved = one.forward_train(x)
        alone.append((h2, one.backward(saved, dh), one(x)[0].clone()))
    steps = [sub.forward_train(x, gate=gate) for x, gate in zip(hs, gates)]
    served = [sub(x, gate=gate)[0] for x, gate in zip(hs, gates)]
    sub.gate, sub.scale, sub.post = gates[0].clone().fill_(9.0), 3.0, None
    for (h2, saved), y, (want, grads, serving) in zip(steps, served, alone):
        assert torch.equal(h2, want) and torch.equal(y, serving)
        got = sub.backward(saved, dh)
        assert set(got) == set(grads) and "gate" in got
        assert all(torch.equal(got[n], grads[n]) for n in grads)


def test_workspaces_are_sized_on_their_device(lib, monkeypatch):
    """The sizes go by the SMs of the current device: the one asked for is current
    while they are taken."""
    seen = []

    class Current:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(self.device)

        def __exit__(self, *exc):
            seen.append(None)
    monkeypatch.setattr(torch.cuda, "device", Current)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: (n, device))
    for module, size, alloc in (
            (moe.sublayer, "norm_backward_workspace_size", moe.alloc_norm_backward_workspace),
            (moe.fp8, "fp8_workspace_size", moe.alloc_fp8_workspace)):
        seen.clear()
        monkeypatch.setattr(module, size, lambda shape: seen.append("sized") or 7)
        assert alloc(_shape(4, 128), "cuda:1") == (7, "cuda:1")
        assert seen == [torch.device("cuda:1"), "sized", None]


def test_workspaces_are_one_run_of_bytes():
    """A strided view spans memory that is not its own."""
    check, cpu = moe.sublayer._check_workspace, torch.device("cpu")
    check(None, cpu)
    check(torch.zeros(64, dtype=torch.uint8), cpu)
    with pytest.raises(ValueError, match="contiguous"):
        check(torch.zeros(64, dtype=torch.uint8)[::2], cpu)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        check(torch.zeros(64, dtype=torch.uint8), torch.device("cuda:0"))


@pytest.mark.gpu
def test_workspaces_of_any_type(cuda_ok):
    """Bytes count, whatever the element; one too short, or strided, is refused."""
    T, H = 40, 264
    s, g = _shape(T, H), torch.Generator().manual_seed(2)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    spec, _ = _params(g, "rms", H)
    want = moe.norm_backward(s, spec, x, x)
    n = moe.norm_backward_workspace_size(s)
    got = moe.norm_backward(s, spec, x, x, workspace=torch.empty(n // 4, device="cuda"))
    assert torch.equal(got["weight"], want["weight"])
    grads = [x.clone()]
    for m in (moe.alloc_grad_norm_workspace().numel(),):
        ws = torch.empty(m // 8, dtype=torch.float64, device="cuda")
        assert torch.equal(moe.clip_grad_norm(grads, 1e9, workspace=ws),
                           moe.clip_grad_norm(grads, 1e9))
        assert torch.equal(moe.grad_square_sum(grads, workspace=ws), moe.grad_square_sum(grads))
        with pytest.raises(moe.MoEError, match="WORKSPACE"):
            moe.clip_grad_norm(grads, 1.0, workspace=ws[1:])
        with pytest.raises(ValueError, match="contiguous"):
            moe.clip_grad_norm(grads, 1.0, workspace=torch.empty(2 * m, dtype=torch.uint8,
                                                                 device="cuda")[::2])


def test_sublayer_runs_on_its_layers_device(monkeypatch):
    """Each form makes the layer's device (and the stream given) current around
    the block's calls, which go by what is current."""
    from types import SimpleNamespace
    from sparse_mixture_experts_07_b200 import sublayer
    seen, inside = [], []

    class Launch:
        def __init__(self, device, stream):
            self.args = (device, stream)

        def __enter__(self):
            inside.append(self.args)

        def __exit__(self, *exc):
            inside.pop()

    def call(name, result):
        def f(*args, **kw):
            seen.append((name, inside[-1] if inside else None))
            return result
        return f
    t = torch.zeros(1, dtype=torch.int32)
    block = SimpleNamespace(
        route=call("route", (t, t, t)), permute=call("permute", (t, t, t, t)),
        train_state_size=lambda s: 1, forward_train=call("forward_train", t),
        backward_workspace_size=lambda s: 1, backward=call("backward", {"x": t}))
    monkeypatch.setattr(sublayer, "_launch", Launch)
    monkeypatch.setattr(sublayer, "_moe", block)
    monkeypatch.setattr(sublayer, "norm", call("norm", t))
    monkeypatch.setattr(sublayer, "combine_norm", call("combine_norm", (t, t, t)))
    monkeypatch.setattr(sublayer, "norm_backward", call(
        "norm_backward", dict(x=t, weight=None, bias=None, gate=None)))
    layer = SimpleNamespace(shape=_shape(1, 8), err_flag=t, slots=call("slots", (t, t)),
                            refresh_router=call("refresh_router", None), gate_up=t, down=t,
                            routing=None, w_router=t, router_bias=t, w_split=None, workspace=t,
                            sh_gate_up=None, sh_down=None)
    sub = moe.MoESublayer(layer, moe.Norm())
    h = torch.zeros(1, 8, dtype=torch.bfloat16)
    sub(h, stream="a stream")
    assert seen == [(n, (t.device, "a stream")) for n in ("norm", "slots", "combine_norm")]
    seen.clear()
    sub.backward(sub.forward_train(h)[1], h)
    assert len(seen) == 9 and all(at == (t.device, None) for _, at in seen)


def test_sublayer_checks_what_the_block_reads():
    """`xn` goes to the block as a bare pointer."""
    from types import SimpleNamespace
    t = torch.zeros(1, dtype=torch.int32)
    sub = moe.MoESublayer(SimpleNamespace(shape=_shape(4, 64), err_flag=t), moe.Norm())
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for bad in (x[:3], x.float(), torch.zeros(64, 4, dtype=torch.bfloat16).t(), x[:, :32]):
        with pytest.raises(ValueError, match="xn must be"):
            sub(x, xn=bad)
        with pytest.raises(ValueError, match="h must be"):
            sub(bad)
