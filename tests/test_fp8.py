"""Experts on E4M3 codes with block scales, against the float64 oracle.

Tolerance of the slot outputs (relative L2): an output is rounded to bf16 once,
at most 2^-8 of itself.  h is rounded to E4M3 from float32 sums that are off by
about 64 roundings (64 2^-24); where that crosses a rounding border (borders
are 2^-4 of the value apart at least: a share of 64 2^-24 / 2^-4 = 2^-14 of
all h) one h moves by at most 2^-3 of itself, in the L2 norm over all h
sqrt(2^-14) 2^-3 = 2^-10.  Together less than 2^-8 + 2^-10.  Weight codes and
scales are bit exact.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle.fp8 as ref
import oracle.sublayer as ref_sub
import sparse_mixture_experts_07_b200 as moe
from parity_util import rel_l2
from sparse_mixture_experts_07_b200.moe import MoEShape

TOL = 2.0 ** -8 + 2.0 ** -10


# ------------------------------------------------------------------------ the oracle
def test_oracle_e4m3_values_and_rounding():
    assert ref.e4m3(0x7E) == 448 and np.isnan(ref.e4m3(0x7F)) and ref.e4m3(1) == 2.0 ** -9
    assert ref.e4m3(0x08) == 2.0 ** -6 and ref.e4m3(0xB8) == -1.0
    finite = [c for c in range(256) if c & 0x7F != 0x7F]
    assert np.array_equal(ref.encode(ref.VALUES[finite]), np.array(finite, dtype=np.uint8))
    # halfway cases go to the even code; just beside them to the nearer one
    for c in range(0, 126):
        mid = (ref.VALUES[c] + ref.VALUES[c + 1]) / 2
        assert ref.encode(mid) == (c if c % 2 == 0 else c + 1)
        assert ref.encode(mid * (1 - 2.0 ** -40)) == c
        assert ref.encode(-mid * (1 + 2.0 ** -40)) == (c + 1) | 0x80
    assert ref.encode(1e9) == 0x7E and ref.encode(np.inf) == 0x7F and ref.encode(np.nan) == 0x7F


def test_oracle_agrees_with_torch_rounding():
    v = torch.randn(4000, generator=torch.Generator().manual_seed(0)) * 100
    v = v.clamp(-448, 448)
    want = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(v.double().numpy()), want)


def test_oracle_block_scales():
    v = np.zeros((4, 256))
    v[0, :] = 448.0 * 8
    v[1, 3], v[1, 130] = 449.0, -1.0
    v[2, 0] = 2.0 ** -140
    r = ref.round_rows(v)
    assert np.array_equal(r[0], v[0])
    assert r[1, 3] == 448.0 and r[1, 130] == -1.0     # 449 / 2 = 224.5 -> 224, ties apart
    assert r[2, 0] == 0.0
    q, s = ref.quantize_weights(np.full((130, 16), -3.0))
    assert s.shape == (2, 1) and (s == np.float32(3) / np.float32(448)).all() and (q == 0xFE).all()
    assert np.allclose(ref.dequantize(q, s), -3.0, rtol=1e-6)
    assert (ref.quantize_weights(np.zeros((4, 16)))[1] == 1).all()


# -------------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from sparse_mixture_experts_07_b200 import build as moe_build
    moe_build.build()
    return moe.load_library()


def _c(**kw):
    base = dict(T=4, H=128, I=64, E=4, k=2, n_shared=0, I_shared=0, routed_scale=1.0,
                dtype=moe.MOE_BF16)
    base.update(kw)
    return ctypes.byref(MoEShape(**base))


def test_quantize_refusals(lib):
    ok = 4096
    f = lib.moe_fp8_quantize
    assert f(-1, 128, 128, ok, 1, ok, ok, None) == 1
    assert f(1, 128, 128, ok, 2, ok, ok, None) == 1
    for i in range(3):
        p = [ok, ok, ok]
        p[i] = None
        assert f(1, 128, 128, p[0], 1, p[1], p[2], None) == 1
    assert f(1, 128, 24, ok, 1, ok, ok, None) == 2
    assert f(1, 128, 128, ok + 8, 1, ok, ok, None) == 2
    assert f(1, 128, 128, ok, 1, ok + 4, ok, None) == 2
    assert f(1 << 40, 128, 128, ok, 1, ok, ok, None) == 2
    assert f(0, 128, 128, None, 1, None, None, None) == 0


def test_forward_refusals(lib):
    n = ctypes.c_size_t(0)
    f = lib.moe_fp8_workspace_size
    assert f(_c(), None) == 1
    for kw in (dict(H=136), dict(I=24), dict(dtype=moe.MOE_F32), dict(n_shared=1, I_shared=24),
               dict(E=256, I=1 << 23)):
        assert f(_c(**kw), ctypes.byref(n)) == 2, kw
    assert f(_c(k=5), ctypes.byref(n)) == 1
    assert f(_c(), ctypes.byref(n)) == 0
    need, ok = n.value, 4096
    # x, offsets, perm, topk_w, gate_up_q, gate_up_s, down_q, down_s, 4 shared, y_slots
    args = [ok] * 8 + [None] * 4 + [ok, None, ok, need, None]
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 12):
        a = list(args)
        a[i] = None
        assert lib.moe_forward_fp8(_c(), *a) == 1, i
    for i in (0, 4, 6, 12, 14):
        a = list(args)
        a[i] = ok + 8
        assert lib.moe_forward_fp8(_c(), *a) == 2, i
    for i, v in ((14, None), (15, need - 1)):
        a = list(args)
        a[i] = v
        assert lib.moe_forward_fp8(_c(), *a) == 3
    assert lib.moe_forward_fp8(_c(n_shared=1, I_shared=64), *args) == 1
    assert lib.moe_forward_fp8(_c(H=136), *args) == 2
    assert lib.moe_forward_fp8(_c(T=0), *([None] * 14), None, 0, None) == 0


def test_binding_refusals(lib):
    with pytest.raises(ValueError, match="CUDA"):
        moe.fp8_quantize(torch.zeros(128, 128))
    s = moe.Shape(T=4, H=128, I=64, E=4, k=2)
    good = dict(gate_up_q=torch.zeros(4, 128, 128, dtype=torch.uint8),
                gate_up_s=torch.ones(4, 2, 1, 1),
                down_q=torch.zeros(4, 128, 64, dtype=torch.float8_e4m3fn),
                down_s=torch.ones(4, 1, 1))
    cpu = torch.device("cpu")
    moe.fp8.check_fp8_experts(s, good, cpu)
    for name, bad in (("gate_up_q", good["gate_up_q"].float()), ("gate_up_q", good["down_q"]),
                      ("gate_up_s", torch.ones(4, 1, 1)), ("down_s", torch.ones(4, 1, 1).double()),
                      ("down_q", None), ("down_q", good["down_q"].transpose(1, 2))):
        with pytest.raises(ValueError, match=name):
            moe.fp8.check_fp8_experts(s, {**good, name: bad}, cpu)
    with pytest.raises(ValueError, match="sh_gate_up_q"):
        moe.fp8.check_fp8_experts(moe.Shape(T=4, H=128, I=64, E=4, k=2, n_shared=1, I_shared=64),
                                  good, cpu)


# ------------------------------------------------------------------ weights, on the GPU
@pytest.mark.gpu
@pytest.mark.parametrize("n,R,C,dtype", [
    (1, 1, 16, torch.float32), (2, 128, 128, torch.bfloat16), (3, 130, 144, torch.float32),
    (2, 257, 400, torch.bfloat16), (1, 127, 1024, torch.float32)])
def test_quantize_matches_oracle(cuda_ok, n, R, C, dtype):
    g = torch.Generator().manual_seed(R)
    w = (torch.randn(n, R, C, generator=g) * torch.exp2(torch.randint(-20, 20, (n, R, 1),
                                                                      generator=g))).to(dtype)
    w[0, 0, :4] = torch.tensor([0.0, -0.0, 3e38, 1e-40])
    if n > 1:
        w[1, :128, :128] = 0                       # a block of zeros
    q, s = moe.fp8_quantize(w.cuda())
    assert q.dtype == torch.float8_e4m3fn and q.shape == w.shape
    for i in range(n):
        qr, sr = ref.quantize_weights(w[i].float().numpy())
        assert np.array_equal(s[i].cpu().numpy(), sr)
        assert np.array_equal(q[i].view(torch.uint8).cpu().numpy(), qr)


@pytest.mark.gpu
def test_quantize_tiny_and_not_finite(cuda_ok):
    w = torch.full((1, 128, 256), 1e-42)
    w[0, :, 128:] = 2.0
    w[0, 5, 130], w[0, 6, 131], w[0, 7, 132] = float("inf"), -float("inf"), float("nan")
    q, s = moe.fp8_quantize(w.cuda())
    qr, sr = ref.quantize_weights(w[0].numpy())
    assert np.array_equal(s[0].cpu().numpy(), sr) and s[0, 0, 0] == 2.0 ** -126
    assert np.array_equal(q[0].view(torch.uint8).cpu().numpy(), qr)
    assert q[0].float().isnan().sum() == 3


# ------------------------------------------------------------------ experts, on the GPU
CASES = [
    # T, H, I, E, k, S, Is
    (1, 16, 16, 1, 1, 0, 0),
    (1, 128, 128, 4, 2, 0, 0),
    (1, 512, 384, 8, 2, 1, 256),
    (3, 720, 208, 5, 3, 0, 0),
    (8, 1040, 656, 4, 2, 2, 144),
    (9, 256, 256, 16, 4, 0, 0),
    (64, 384, 640, 16, 2, 0, 0),
    (33, 144, 112, 256, 8, 0, 0),
    (200, 272, 400, 4, 2, 1, 80),
    (129, 512, 256, 1, 1, 0, 0),
    (520, 400, 272, 2, 1, 0, 0),
    (600, 272, 400, 4, 2, 2, 240),
    (1000, 1152, 128, 3, 2, 0, 0),
]


def _plan(g, T, E, k, skip=()):
    logits = torch.randn(T, E, generator=g)
    for e in skip:                        # experts that no token takes
        logits[:, e] = -100.0
    top = torch.topk(logits, k, dim=1)
    idx = top.indices.to(torch.int32)
    perm = torch.sort(idx.reshape(-1), stable=True).indices.to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(idx.reshape(-1).long(), minlength=E).cumsum(0)
    return perm, offsets, torch.softmax(top.values, dim=1)


def _experts(g, H, E, I, pre=""):
    out = {}
    for name, n, R, C in (("gate_up", 2 * E, I, H), ("down", E, H, I)):
        q = (torch.randn(n, R, C, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        # scales as a checkpoint has them: no powers of two, some blocks far apart
        s = torch.exp(torch.randn(n, -(-R // 128), -(-C // 128), generator=g)) * 0.01 / C ** 0.5
        if name == "gate_up":
            q, s = q.view(E, 2 * I, C), s.view(E, 2, *s.shape[1:])
        out[f"{pre}{name}_q"], out[f"{pre}{name}_s"] = q, s
    return out


def _setup(T, H, I, E, k, S, Is, seed=0, skip=()):
    g = torch.Generator().manual_seed(seed)
    fp8 = _experts(g, H, E, I)
    if S:
        fp8.update(_experts(g, H, S, Is, "sh_"))
    x = (torch.randn(T, H, generator=g) * torch.exp2(torch.randint(-6, 6, (T, 1), generator=g))
         ).to(torch.bfloat16)
    perm, offsets, w = _plan(g, T, E, k, skip)
    shape = moe.Shape(T=T, H=H, I=I, E=E, k=k, n_shared=S, I_shared=Is, routed_scale=2.5)
    return shape, x, perm, offsets, w, fp8


def _oracle(shape, x, perm, offsets, w, fp8):
    arrays = {n: (t.view(torch.uint8) if n.endswith("_q") else t).numpy() for n, t in fp8.items()}
    return ref.slots(x.double().numpy(), perm.numpy(), offsets.numpy(), w.numpy(), arrays,
                     shape.k, shape.routed_scale)


def _run(shape, x, perm, offsets, w, fp8, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.forward_fp8(shape, x.cuda(), offsets.cuda(), perm.cuda(), w.cuda(),
                        {n: t.cuda() for n, t in fp8.items()}, err_flag=err, **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_matches_oracle(cuda_ok, case):
    T, H, I, E, k, S, Is = case
    args = _setup(*case, skip=range(1, E, 3) if E - (E - 2) // 3 - 1 >= k and E > 2 else ())
    y = _run(*args)
    want = _oracle(*args)
    got = y.double().cpu().numpy()
    assert got.shape == want.shape
    err = rel_l2(got, want)
    print(f"  relative L2 {err:.2e} of {TOL:.2e}")
    assert err <= TOL
    # row by row too: small groups and their last rows weigh as much as large ones
    rows = np.linalg.norm(got - want, axis=1) / np.maximum(np.linalg.norm(want, axis=1), 1e-300)
    # one row has few h: a border crossed there weighs 2^-3 of one of I values
    assert rows.max() <= TOL + 2.0 ** -3 * 2 / np.sqrt(min(I, Is or I)), rows.argmax()
    # bit for bit the same again, codes given as bytes
    as_bytes = {n: t.view(torch.uint8) if n.endswith("_q") else t for n, t in args[5].items()}
    assert torch.equal(_run(*args[:5], as_bytes), y)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(1, 128, 128, 4, 2, 0, 0), (8, 256, 144, 4, 2, 1, 64),
                                  (200, 256, 144, 4, 2, 1, 64), (600, 256, 144, 4, 2, 1, 64)])
def test_rows_are_independent_and_bounded(cuda_ok, case):
    """A NaN and an infinity reach their own tokens' rows alone; a zero token
    gives zero rows; nothing is written past the last row."""
    shape, x, perm, offsets, w, fp8 = _setup(*case, seed=3)
    T, k = shape.T, shape.k
    y = _run(shape, x, perm, offsets, w, fp8)
    bad = x.clone()
    special = {0: float("nan")}
    if T > 4:
        special.update({3: float("inf"), T - 1: 0.0})
    for t, v in special.items():
        bad[t, 5] = v
        if v == 0:
            bad[t] = 0
    buf = torch.full((shape.slot_rows + 3, shape.H), 7.0, dtype=torch.bfloat16, device="cuda")
    _run(shape, bad, perm, offsets, w, fp8, y_slots=buf[:shape.slot_rows])
    assert (buf[shape.slot_rows:] == 7).all()
    token = torch.cat([perm.long() // k, torch.arange(T).repeat(shape.n_shared)]).cuda()
    clean = torch.ones(shape.slot_rows, dtype=torch.bool, device="cuda")
    for t, v in special.items():
        rows = token == t
        clean &= ~rows
        assert buf[:shape.slot_rows][rows].isnan().all() if v != 0 else \
            not buf[:shape.slot_rows][rows].any()
    assert torch.equal(buf[:shape.slot_rows][clean], y[clean])


@pytest.mark.gpu
def test_zero_tokens_and_zero_blocks(cuda_ok):
    shape, x, perm, offsets, w, fp8 = _setup(4, 256, 128, 2, 1, 0, 0)
    empty = moe.forward_fp8(moe.Shape(T=0, H=256, I=128, E=2, k=1), x[:0].cuda(),
                            torch.zeros(3, dtype=torch.int32, device="cuda"),
                            perm[:0].cuda(), w[:0].cuda(), {n: t.cuda() for n, t in fp8.items()})
    assert empty.shape == (0, 256)
    fp8["gate_up_s"][:, :, :, 0] = 0.0                 # a scale of zero drops its block
    x2 = x.clone()
    x2[:, :128] = 1.0
    assert torch.equal(_run(shape, x2, perm, offsets, w, fp8)[:, :1].isnan(),
                       torch.zeros(4, 1, dtype=torch.bool, device="cuda"))
    x3 = x.clone()
    x3[:, :128] = -5.0
    assert torch.equal(_run(shape, x2, perm, offsets, w, fp8),
                       _run(shape, x3, perm, offsets, w, fp8))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 64, 600])
def test_layer_graph_stream_and_sublayer(cuda_ok, T):
    """MoELayer on quantised weights: routing, plan, experts and combine; then
    captured, on another stream, and inside a MoESublayer."""
    H, I, E, k, S, Is = 256, 144, 4, 2, 1, 80
    g = torch.Generator().manual_seed(11)
    gu, dn = torch.randn(E, 2 * I, H, generator=g) * 0.05, torch.randn(E, H, I, generator=g) * 0.05
    sgu = torch.randn(S, 2 * Is, H, generator=g) * 0.05
    sdn = torch.randn(S, H, Is, generator=g) * 0.05
    fp8 = moe.fp8_experts(*(t.to(torch.bfloat16).cuda() for t in (gu, dn, sgu, sdn)))
    shape = moe.Shape(T=T, H=H, I=I, E=E, k=k, n_shared=S, I_shared=Is, routed_scale=2.5)
    wr = (torch.randn(E, H, generator=g) * 0.05).cuda()
    layer = moe.MoELayer(shape, wr, None, fp8=fp8)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    y = layer(x).clone()
    torch.cuda.synchronize()
    assert layer.device_error() == 0
    b = layer.last
    arrays = {n: (t.view(torch.uint8) if n.endswith("_q") else t).cpu().numpy()
              for n, t in fp8.items()}
    want = ref.slots(x.double().cpu().numpy(), b["perm"].cpu().numpy(), b["offsets"].cpu().numpy(),
                     b["topk_w"].cpu().numpy(), arrays, k, 2.5)
    want = ref_sub.combine(want, b["inv"].cpu().numpy(), T, k, S)
    assert rel_l2(y.double().cpu().numpy(), want) <= 2 * TOL     # slots, then y, rounded
    graph = layer.capture(x)
    for _ in range(3):
        layer.buf["y"].zero_()
        assert torch.equal(graph.replay(), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = layer(x, stream=side, y=torch.empty_like(y))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, y)
    sub = moe.MoESublayer(layer, moe.Norm("rms", 1e-5), moe.Norm("rms", 1e-5), scale=0.5,
                          next_norm=moe.Norm("rms", 1e-5))
    h2, xn2 = sub(x)
    y_slots = layer.last["y_slots"].double().cpu().numpy()
    hr, xr = ref_sub.residual_norm(
        ref_sub.combine(y_slots, layer.last["inv"].cpu().numpy(), T, k, S),
        x.double().cpu().numpy(), dict(kind="rms", eps=1e-5), None, 0.5,
        dict(kind="rms", eps=1e-5))
    assert rel_l2(h2.double().cpu().numpy(), hr) <= 2.0 ** -8
    assert rel_l2(xn2.double().cpu().numpy(), xr) <= 2.0 ** -8
    with pytest.raises(ValueError):
        moe.MoELayer(shape, wr, None, gu.cuda(), dn.cuda(), fp8=fp8)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 16, 31, 32, 33, 64, 128])
def test_batch_sizes_around_the_split(cuda_ok, T):
    """Up to 32 tokens share K-blocks out over the SMs, tiles then being summed
    from parts; a tile may also lie whole in one share."""
    for H, I, E, k, S, Is in ((1280, 640, 6, 2, 1, 384), (256, 4096, 64, 6, 0, 0)):
        args = _setup(T, H, I, E, k, S, Is, seed=T)
        y = _run(*args)
        assert rel_l2(y.double().cpu().numpy(), _oracle(*args)) <= TOL
        assert torch.equal(_run(*args), y)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [8, 32, 64, 300])
def test_every_slot_on_one_expert(cuda_ok, T):
    """A plan may name one expert in all of a token's slots: more rows in a
    group than tokens."""
    k, E = 8, 16
    shape, x, _, _, w, fp8 = _setup(T, 144, 272, E, k, 0, 0, seed=4)
    perm = torch.arange(T * k, dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[6:] = T * k
    args = (shape, x, perm, offsets, w, fp8)
    assert rel_l2(_run(*args).double().cpu().numpy(), _oracle(*args)) <= TOL


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 100])
def test_holes_in_the_plan(cuda_ok, T):
    """Entries of perm outside the slots (a plan with a bad expert index) are
    not followed; their rows get weight 0, the others are as without them."""
    shape, x, perm, offsets, w, fp8 = _setup(T, 144, 272, 4, 2, 1, 64, seed=5)
    y = _run(shape, x, perm, offsets, w, fp8)
    holed = perm.clone()
    holed[1], holed[3] = -7, T * 2
    # the rows that holes leave unset in the workspace are whatever was there
    ws = torch.zeros(moe.fp8_workspace_size(shape), dtype=torch.uint8, device="cuda")
    got = _run(shape, x, holed, offsets, w, fp8, workspace=ws)
    keep = torch.ones(shape.slot_rows, dtype=torch.bool, device="cuda")
    keep[[1, 3]] = False
    assert torch.equal(got[keep], y[keep]) and not got[~keep].any()


@pytest.mark.gpu
def test_two_streams_at_once(cuda_ok):
    """Two calls in flight, each with a workspace and outputs of its own."""
    cases = [_setup(48, 512, 384, 8, 2, 1, 256, seed=6), _setup(700, 512, 384, 4, 2, 0, 0, seed=7)]
    want = [_run(*c) for c in cases]
    dev = [[c[i].cuda() for i in (1, 3, 2, 4)] + [{n: t.cuda() for n, t in c[5].items()}]
           for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, (c, d, st) in enumerate(zip(cases, dev, streams)):
            outs[i].append(moe.forward_fp8(c[0], *d, stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_ok):
    """More than 2^32 values of x codes and of y_slots; rows at both ends and
    in the middle against the oracle."""
    T, H, I, E, k = 262200, 2048, 16, 8, 8
    g = torch.Generator(device="cuda").manual_seed(8)
    cpu = torch.Generator().manual_seed(8)
    shape = moe.Shape(T=T, H=H, I=I, E=E, k=k)
    assert T * k * H > 1 << 32
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    fp8 = _experts(cpu, H, E, I)
    # every token on every expert, in sorted order
    perm = (torch.arange(T, device="cuda")[None, :] * k +
            torch.arange(E, device="cuda")[:, None]).reshape(-1).to(torch.int32)
    offsets = torch.arange(E + 1, device="cuda", dtype=torch.int32) * T
    w = torch.rand(T, k, generator=g, device="cuda")
    y = moe.forward_fp8(shape, x, offsets, perm, w, {n: t.cuda() for n, t in fp8.items()})
    arrays = {n: (t.view(torch.uint8) if n.endswith("_q") else t).numpy() for n, t in fp8.items()}
    for e in (0, 3, E - 1):
        for t0 in (0, T // 2, T - 40):
            rows = slice(t0, t0 + 40)
            want = ref.expert(x[rows].double().cpu().numpy(), arrays["gate_up_q"][e],
                              arrays["gate_up_s"][e], arrays["down_q"][e], arrays["down_s"][e])
            want *= w[rows, e].double().cpu().numpy()[:, None]
            got = y[e * T + t0:e * T + t0 + 40].double().cpu().numpy()
            assert rel_l2(got, want) <= TOL + 2.0 ** -3 / np.sqrt(40 * I)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 90, 400])
def test_outputs_off_the_32_byte_boundary(cuda_ok, T):
    """y_slots and the workspace may start on any 16-byte boundary."""
    for I in (272, 288):
        shape, x, perm, offsets, w, fp8 = _setup(T, 144, I, 4, 2, 1, 96, seed=9)
        want = _run(shape, x, perm, offsets, w, fp8)
        y = torch.zeros(shape.slot_rows * shape.H + 8, dtype=torch.bfloat16, device="cuda")[8:]
        ws = torch.zeros(moe.fp8_workspace_size(shape) + 16, dtype=torch.uint8, device="cuda")[16:]
        got = _run(shape, x, perm, offsets, w, fp8, y_slots=y.view(shape.slot_rows, shape.H),
                   workspace=ws)
        assert got.data_ptr() % 32 == 16 and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 32, 200, 700])
def test_replays_follow_the_routing(cuda_ok, T):
    """A captured step whose tokens, and with them the plan, change from replay
    to replay, and eager steps back to back: as a fresh layer computes each."""
    H, I, E, k = 256, 272, 8, 2
    g = torch.Generator().manual_seed(12)
    fp8 = moe.fp8_experts((torch.randn(E, 2 * I, H, generator=g) * 0.05).cuda(),
                          (torch.randn(E, H, I, generator=g) * 0.05).cuda())
    wr = torch.randn(E, H, generator=g).cuda()
    shape = moe.Shape(T=T, H=H, I=I, E=E, k=k)
    xs = [torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(6)]
    want = []
    for x in xs:
        fresh = moe.MoELayer(shape, wr, None, fp8=fp8)
        torch.cuda.synchronize()
        want.append(fresh(x).clone())
        torch.cuda.synchronize()
    layer = moe.MoELayer(shape, wr, None, fp8=fp8)
    got = [layer(x, y=torch.empty_like(x)) for x in xs]          # nothing waits between
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    static = xs[0].clone()
    graph = layer.capture(static)
    for _ in range(3):
        for x, w in zip(xs, want):
            static.copy_(x)
            assert torch.equal(graph.replay(), w)
    assert layer.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,S", [(20, 0), (40, 1), (300, 2)])
def test_slots_that_the_plan_skipped(cuda_ok, T, S):
    """A plan that skipped slots defines perm[0 .. offsets[E]) only.  Whatever the
    rest of it holds, an earlier plan's slots here, each named by a placed row too,
    the placed rows are as with nothing there, and (whole tiles: no sums whose
    parts move with the rows) as in the plan without skips, bit for bit."""
    E, k = 6, 3
    shape, x, perm, offsets, w, fp8 = _setup(T, 272, 144, E, k, S, 80 if S else 0, seed=13)
    full = _run(shape, x, perm, offsets, w, fp8)
    expert = torch.bucketize(torch.arange(T * k), offsets[1:].long(), right=True)
    kept = torch.arange(T * k) % 7 != 2
    kept[offsets[3]:offsets[3] + 2] = False
    n = int(kept.sum())
    assert n < T * k - T // 4
    skipped = torch.cat([perm[kept], perm[kept].flip(0)[:T * k - n]])
    counts = torch.bincount(expert[kept], minlength=E)
    short = torch.zeros(E + 1, dtype=torch.int32)
    short[1:] = counts.cumsum(0)
    bare = torch.cat([perm[kept], torch.full((T * k - n,), -1, dtype=torch.int32)])
    want = _run(shape, x, bare, short, w, fp8)
    if T > 32:
        assert torch.equal(want[:n], full[:T * k][kept.cuda()])
        assert torch.equal(want[T * k:], full[T * k:])
    for fill in (0x00, 0xFF):
        ws = torch.full((moe.fp8_workspace_size(shape),), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            got = _run(shape, x, skipped, short, w, fp8, workspace=ws)
            assert torch.equal(got[:n], want[:n]) and torch.equal(got[T * k:], want[T * k:])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 32, 100])
def test_offsets_out_of_order(cuda_ok, T):
    """Offsets that no plan has (down as well as up, outside the slots): each
    counts as the smallest from it on, and nothing is written past the workspace
    or the slot rows."""
    E, k = 6, 2
    shape, x, perm, offsets, w, fp8 = _setup(T, 272, 144, E, k, 1, 80, seed=14)
    n, size = T * k, moe.fp8_workspace_size(shape)
    for odd in ([0, n, 0, n, 0, n, 0], [-5, 3, 2, 2 ** 31 - 1, 7, -2 ** 31, 1],
                [n, 1, 2, 3, 4, 5, 6], [0, 1, 1, n - 1, 2, n, n + 1]):
        got = []
        for o in (odd, np.minimum.accumulate(np.clip(odd, 0, n)[::-1])[::-1].tolist()):
            ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
            y = torch.full((shape.slot_rows + 2, shape.H), 7.0, dtype=torch.bfloat16,
                           device="cuda")
            _run(shape, x, perm, torch.tensor(o, dtype=torch.int32), w, fp8, workspace=ws[:size],
                 y_slots=y[1:-1])
            assert (ws[size:] == 0x5A).all() and (y[0] == 7).all() and (y[-1] == 7).all()
            got.append(y)
        assert torch.equal(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 32, 100])
@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFF])
def test_holes_are_zero_on_any_workspace(cuda_ok, T, fill):
    """Rows of holes in perm are zeros whatever the workspace held (0xFF, 0x7F:
    codes that are NaN, 0xFF a scale that is), the others as without the holes."""
    shape, x, perm, offsets, w, fp8 = _setup(T, 272, 144, 4, 2, 1, 64, seed=15)
    y = _run(shape, x, perm, offsets, w, fp8)
    holed = perm.clone()
    rows = [0] if T == 1 else [1, 4, 2 * T - 1]
    holed[rows] = torch.tensor([-1, 2 * T, 2 ** 31 - 1], dtype=torch.int32)[:len(rows)]
    ws = torch.full((moe.fp8_workspace_size(shape),), fill, dtype=torch.uint8, device="cuda")
    got = _run(shape, x, holed, offsets, w, fp8, workspace=ws)
    keep = torch.ones(shape.slot_rows, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(got[keep], y[keep]) and (got[~keep] == 0).all()


@pytest.mark.gpu
def test_workspace_and_error_word_refusals(cuda_ok):
    shape, x, perm, offsets, w, fp8 = _setup(5, 144, 272, 4, 2, 0, 0, seed=16)
    want = _run(shape, x, perm, offsets, w, fp8)
    n = moe.fp8_workspace_size(shape)
    got = _run(shape, x, perm, offsets, w, fp8,
               workspace=torch.empty(n // 4 + 1, dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want)
    dev = [t.cuda() for t in (x, offsets, perm, w)] + [{m: t.cuda() for m, t in fp8.items()}]
    for kw, match in (
            (dict(workspace=torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]),
             "contiguous"),
            (dict(workspace=torch.empty(n, dtype=torch.uint8)), "workspace is on cpu"),
            (dict(err_flag=torch.zeros(1, device="cuda")), "err_flag"),
            (dict(err_flag=torch.zeros(1, dtype=torch.int32)), "err_flag"),
            (dict(err_flag=torch.zeros(0, dtype=torch.int32, device="cuda")), "err_flag")):
        with pytest.raises(ValueError, match=match):
            moe.forward_fp8(shape, *dev, **kw)
    with pytest.raises(moe.MoEError, match="WORKSPACE"):
        moe.forward_fp8(shape, *dev, workspace=torch.empty(n - 1, dtype=torch.uint8,
                                                           device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 24, 96, 400])
def test_fine_grained_layer_with_noaux_routing(cuda_ok, T):
    """64 experts, top-6 by groups, two shared experts: the layer on E4M3 weights
    against the oracle on the device's plan; then a token of NaN, which stays in
    its row (up to 32 tokens the others' sums are cut at other places: TOL)."""
    H, I, E, k, S, Is = 256, 96, 64, 6, 2, 128
    g = torch.Generator().manual_seed(17)
    fp8 = _experts(g, H, E, I)
    fp8.update(_experts(g, H, S, Is, "sh_"))
    dev = {n: t.cuda() for n, t in fp8.items()}
    shape = moe.Shape(T=T, H=H, I=I, E=E, k=k, n_shared=S, I_shared=Is, routed_scale=2.5)
    layer = moe.MoELayer(shape, torch.randn(E, H, generator=g).cuda(),
                         (torch.randn(E, generator=g) * 0.1).cuda(), fp8=dev,
                         routing=("noaux_tc", 8, 4))
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    y = layer(x.cuda(), y=torch.empty(T, H, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert layer.device_error() == 0
    b = {n: layer.last[n].cpu() for n in ("perm", "offsets", "topk_w", "inv")}
    slots = _oracle(shape, x, b["perm"], b["offsets"], b["topk_w"], fp8)
    want = ref_sub.combine(slots, b["inv"].numpy(), T, k, S)
    assert rel_l2(y.double().cpu().numpy(), want) <= 2 * TOL       # slots, then y, rounded
    x[T // 2] = float("nan")
    got = layer(x.cuda(), y=torch.empty(T, H, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert layer.device_error() == 0 and got[T // 2].isnan().all()
    others = torch.arange(T, device="cuda") != T // 2
    if T > 32:
        assert torch.equal(got[others], y[others])
    elif T > 1:
        assert rel_l2(got[others].double().cpu().numpy(),
                      want[others.cpu().numpy()]) <= 2 * TOL
