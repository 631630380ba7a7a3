"""The RMS norm with the residual's addition, its 8-bit form and its backward pass against plain float64 forms.

Tolerances are bounds, not fits.  u is the rounding of a stored result (half a step: 2^-8 relative for bf16, 2^-24 for
fp32, 2^-4 for e4m3); every other term counts the fp32 roundings on the way (E = 2^-24).
"""
import math

import pytest
import torch

from transformer_depth_wise_gb300 import _lib, api
from transformer_depth_wise_gb300 import workloads as wk

gpu_only = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
E = 2.0 ** -24
EPS = 1e-6
LEAST = 2.0 ** -126
FAKE = 0x7F0000000000      # 16-byte aligned stand-in for a device pointer (never dereferenced)
OK, NULL, SHAPE, DTYPE, ALIGN, CAP, VALUE = 0, -1, -2, -3, -4, -7, -8


def cpu(t):
    return t.detach().cpu().double()


def within(got, want, tol, what=""):
    got, want = cpu(got), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert bool(torch.isfinite(got).all()), what
    d = (got - want).abs() - tol
    assert d.numel() == 0 or float(d.max()) <= 0.0, f"{what}: over the bound by {float(d.max()):.3e}"


def rand(g, *shape, dtype=BF, scale=1.0):
    return (torch.empty(shape, dtype=F32, device=g.device).normal_(generator=g) * scale).to(dtype)


def inputs(dev, dtype, rows, D, residual, seed):
    g = wk.generator(seed, dev)
    x, w = rand(g, rows, D, dtype=dtype), 1 + rand(g, D, dtype=F32, scale=0.2)
    r = rand(g, rows, D, dtype=dtype, scale=3.0) if residual else None
    if residual:
        r[:, ::37] *= 8
    return x, r, w


def forward_ref(x, r, w, eps=EPS):
    s = cpu(x) if r is None else cpu(x) + cpu(r)
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return (y if w is None else y * cpu(w)), s


# the sum 1 (relative to itself, and through the root), the sum of squares (16 terms per lane at most and a tree of 10
# levels, halved by the root) 13, mean, eps, root 3, the two products 2: less than 24 roundings
FORWARD = 24 * E

CASES = [  # dtype, rows, D, residual
    (BF, 1, 8, True), (BF, 33, 64, True), (BF, 257, 128, False), (BF, 5, 136, True), (BF, 64, 512, True),
    (BF, 7, 520, True), (BF, 1000, 2048, True), (BF, 256, 7168, True), (BF, 3, 8192, False), (BF, 2, 16384, True),
    (BF, 700, 4096, True), (F32, 333, 256, True), (F32, 1, 4, True), (F32, 9, 64, False), (F32, 50, 100, True),
    (F32, 31, 1028, True), (F32, 400, 4096, True), (F32, 5, 8192, True), (BF, 5000, 96, True),
]


@gpu_only
@pytest.mark.parametrize("dtype,rows,D,residual", CASES)
def test_forward(gpu, dtype, rows, D, residual):
    x, r, w = inputs(gpu, dtype, rows, D, residual, rows + D)
    y, total = api.add_rms_norm(x, r, w, EPS)
    want, s = forward_ref(x, r, w)
    within(y, want, (U[dtype] + FORWARD) * want.abs(), "y")
    if residual:
        within(total, s, (U[dtype] + E) * s.abs(), "sum")
        # a bf16 sum is the rounding of the fp32 one
        assert torch.equal(total, (x.float() + r.float()).to(dtype))
    else:
        assert total is None
        assert torch.equal(api.add_rms_norm(x, None, w, EPS, sum_out=torch.empty_like(x))[1], x)
    within(api.add_rms_norm(x, r, None, EPS)[0], forward_ref(x, r, None)[0],
           (U[dtype] + FORWARD) * forward_ref(x, r, None)[0].abs(), "no weight")
    # outputs on the inputs, each way round
    if residual:
        for swap in (False, True):
            a, b = x.clone(), r.clone()
            got = api.add_rms_norm(a, b, w, EPS, sum_out=a if swap else b, out=b if swap else a)
            assert torch.equal(got[0], y) and torch.equal(got[1], total)


def check_8bit(x, r, w, group, y8, scales, what=""):
    want, s = forward_ref(x, r, w)
    rows, D = want.shape
    z = want.view(rows, -1, group or D)
    top = z.abs().amax(-1)
    scale = (top / 448).clamp_min(LEAST)
    # the scale is the largest value's error, a division and nothing else (y near the smallest normal numbers: a step)
    within(scales.view(scale.shape), scale, (FORWARD + 2 * E) * scale, what + " scales")
    q, v = cpu(y8.float()).view(z.shape), z / scale[..., None]
    # half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6), and the quotient's own roundings
    within(q, v, 2.0 ** -4 * v.abs().clamp_min(2.0 ** -6) + (2 * FORWARD + 8 * E) * v.abs(), what + " y8")
    assert float(q.abs().max()) <= 448


@gpu_only
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype,rows,D,residual", CASES)
def test_8bit(gpu, dtype, rows, D, residual, group):
    if group and D % group:
        D = max(group, D // group * group)
    x, r, w = inputs(gpu, dtype, rows, D, residual, 3 * rows + D)
    y8, scales, total = api.add_rms_norm_8bit(x, r, w, EPS, group=group)
    assert y8.dtype is F8 and scales.shape == (rows, D // group if group else 1)
    check_8bit(x, r, w, group, y8, scales)
    y, want = api.add_rms_norm(x, r, w, EPS)
    assert total is None if not residual else torch.equal(total, want)
    if dtype is F32:
        # y in fp32 is the same number: its quotient by the scale rounds to y8, by torch's own cast
        q = (y.view(rows, -1, group or D) * (1.0 / scales.view(rows, -1, 1))).clamp(-448, 448).to(F8).view(rows, D)
        assert torch.equal(q.view(torch.uint8), y8.view(torch.uint8))
    if residual:                       # the sum on the residual
        again = api.add_rms_norm_8bit(x, r, w, EPS, group=group, sum_out=r)
        assert torch.equal(again[0].view(torch.uint8), y8.view(torch.uint8)) and torch.equal(r, want)


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
def test_8bit_zeros_tiny_and_huge_rows(gpu, dtype):
    D = 256
    x, _, w = inputs(gpu, dtype, 6, D, False, 4)
    x[0] = 0
    x[1, :128] = 0                                   # a group of zeros in a row that has others
    x[2] *= 1e-30
    x[3] *= 1e17
    x[4] = 2.0 ** -130                               # below the smallest normal number
    x[5, 7] = 2.0 ** 20                              # one value over all others
    for group in (0, 32, 128):
        y8, scales, _ = api.add_rms_norm_8bit(x, None, w, EPS, group=group)
        check_8bit(x, None, w, group, y8, scales)
        zero = scales.view(6, -1)
        assert float(zero[0].max()) == LEAST and not bool(y8[0].float().any())
    y, _ = api.add_rms_norm(x, None, w, 0.0)         # eps 0: a row of zeros has no norm
    assert bool(y[0].isnan().all()) and bool(y[[1, 3]].isfinite().all())


@gpu_only
@pytest.mark.parametrize("dtype,D", [(BF, 256), (F32, 256), (BF, 2048), (BF, 64)])
def test_what_is_no_number(gpu, dtype, D):
    x, r, w = inputs(gpu, dtype, 5, D, True, 9)
    x[1, 3] = math.nan
    x[2, 5] = math.inf
    r[3, D - 1] = -math.inf
    w[40] = math.nan
    y, total = api.add_rms_norm(x, r, w, EPS)
    assert bool(y[1].isnan().all()) and bool(total[1].isnan().sum() == 1)
    assert bool(y[2, 5].isnan()) and bool(y[3, D - 1].isnan()) and bool((y[2, 6:40] == 0).all())
    only = torch.zeros(D, dtype=torch.bool, device=gpu)
    only[40] = True
    assert torch.equal(y[0].isnan(), only) and torch.equal(y[4].isnan(), only)
    for group in (0, 32):
        y8, scales, _ = api.add_rms_norm_8bit(x, r, w, EPS, group=group)
        bad, q = scales.view(5, -1).isnan(), y8.float().view(5, -1, group or D)
        assert torch.equal(q.isnan().all(-1), bad) and torch.equal(q.isnan().any(-1), bad)
        assert bool(bad[1].all()) and bool(bad[:, 40 // group if group else 0].all())
        if group:
            assert bool(bad[2, 0]) and bool(bad[3, D // group - 1]) and int(bad[0].sum()) == 1


def backward_ref(s, w, gy, gs, eps=EPS):
    s, gy = cpu(s), cpu(gy)
    u = gy if w is None else gy * cpu(w)
    r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    c = (u * s).mean(-1, keepdim=True)
    dx = r * (u - s * r * r * c)
    dw = gy * s * r
    size = r * (u.abs() + s.abs() * r * r * (u * s).abs().mean(-1, keepdim=True))
    if gs is not None:
        dx, size = dx + cpu(gs), size + cpu(gs).abs()
    return dx, dw.sum(0), size, dw.abs().sum(0)


def test_backward_formula_against_differences():
    g = torch.Generator().manual_seed(2)
    s, gy, gs = (torch.randn(3, 12, dtype=torch.float64, generator=g) for _ in range(3))
    w = torch.randn(12, dtype=torch.float64, generator=g)
    dx, dw, _, _ = backward_ref(s, w, gy, gs, 1e-3)

    def loss(s, w):
        y, total = forward_ref(s, None, w, 1e-3)
        return float((y * gy).sum() + (total * gs).sum())

    h = 1e-5
    for t, d in ((s, dx), (w, dw)):
        for i in range(t.numel()):
            e = torch.zeros(t.numel(), dtype=torch.float64)
            e[i] = h
            e = e.view(t.shape)
            lo, hi = (loss(t - e, w), loss(t + e, w)) if t is s else (loss(s, t - e), loss(s, t + e))
            # central differences: h^2 of the third derivative (below 1000 here) and 2^-52 * |loss| / h
            assert abs((hi - lo) / (2 * h) - float(d.reshape(-1)[i])) < 1e-7


@gpu_only
@pytest.mark.parametrize("dtype,rows,D,residual", CASES)
def test_backward(gpu, dtype, rows, D, residual):
    s, gs, w = inputs(gpu, dtype, rows, D, residual, rows + 2 * D)
    gy = rand(wk.generator(5, gpu), rows, D, dtype=dtype)
    dx, dw = api.add_rms_norm_backward(s, w, EPS, gy, gs)
    want, rw, size, absw = backward_ref(s, w, gy, gs)
    # the terms' roundings, 13 + 13 of the two means' sums (relative to the sums of absolute values), root and products
    within(dx, want, U[dtype] * want.abs() + 48 * E * size, "dx")
    # every term is off by 24 E of itself; the sums have the CTA's rows, the teams, 76 CTAs a strand and 8 strands
    depth = 24 + rows / min(rows, 4 * 152) + 32 + 608 / 8 + 8
    within(dw, rw, depth * E * absw, "dw")
    again = api.add_rms_norm_backward(s, w, EPS, gy, gs)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])                  # a fixed order of sums
    only = api.add_rms_norm_backward(s, w, EPS, gy, gs, want_weight=False)
    assert torch.equal(only[0], dx) and only[1] is None
    one = api.add_rms_norm_backward(s, w, EPS, gy, gs, workspace=torch.full((1, D), math.nan, device=gpu))   # one CTA
    assert torch.equal(one[0], dx)
    within(one[1], rw, (24 + rows + 40) * E * absw, "dw of one CTA")
    for name in ("s", "gy", "gs"):                   # the gradient on each of the inputs
        if name == "gs" and gs is None:
            continue
        t = {"s": s.clone(), "gy": gy.clone(), "gs": None if gs is None else gs.clone()}
        got = api.add_rms_norm_backward(t["s"], w, EPS, t["gy"], t["gs"], dx=t[name])
        assert got[0] is t[name] and torch.equal(got[0], dx) and torch.equal(got[1], dw)


@gpu_only
def test_directional_differences(gpu):
    # the fp32 kernels against one another: (loss(s + h v) - loss(s - h v)) / 2h with the forward kernel
    rows, D, h = 40, 256, 2.0 ** -7
    s, gs, w = inputs(gpu, F32, rows, D, True, 6)
    g = wk.generator(8, gpu)
    gy, v, dwv = rand(g, rows, D, dtype=F32), rand(g, rows, D, dtype=F32), rand(g, D, dtype=F32)
    dx, dw = api.add_rms_norm_backward(s, w, EPS, gy, gs)

    def loss(s, w):
        y, total = api.add_rms_norm(s, None, w, EPS, sum_out=torch.empty_like(s))
        return (cpu(y) * cpu(gy)).sum() + (cpu(total) * cpu(gs)).sum()

    exact = float((cpu(dx) * cpu(v)).sum() + (cpu(dw) * cpu(dwv)).sum())
    got = float(loss(s + h * v, w + h * dwv) - loss(s - h * v, w - h * dwv)) / (2 * h)
    # y's fp32 roundings, 24 E of |y gy| each way, and those of the shifted inputs; the third derivative of a normed
    # row of scale 3 and more under steps of unit scale: h^2 of a few times the terms' sizes
    y, total = forward_ref(s, None, w)
    terms = float((y * cpu(gy)).abs().sum() + (total * cpu(gs)).abs().sum())
    assert abs(got - exact) <= 26 * E * terms / h + h * h * float((cpu(gy) * y).abs().sum())


@gpu_only
def test_empty_shapes_views_and_streams(gpu):
    w = torch.ones(64, device=gpu)
    for shape in ((0, 64), (2, 0, 64)):
        e = torch.empty(shape, device=gpu, dtype=BF)
        y, total = api.add_rms_norm(e, e.clone(), w)
        assert y.shape == shape and total.shape == shape
        assert api.add_rms_norm_8bit(e, None, w, group=32)[1].shape == (*shape[:-1], 2)
        dx, dw = api.add_rms_norm_backward(e, w, EPS, e.clone())
        assert dx.shape == shape and not bool(dw.any())
    x, r, w = inputs(gpu, BF, 12, 2048, True, 3)
    flat = api.add_rms_norm_8bit(x, r, w, EPS, group=64)
    cube = api.add_rms_norm_8bit(x.view(3, 4, 2048), r.view(3, 4, 2048), w, EPS, group=64)
    assert cube[1].shape == (3, 4, 32) and all(torch.equal(a.float().view(b.shape), b.float()) for a, b in zip(cube, flat))

    def step():
        y8, sc, total = api.add_rms_norm_8bit(x, r, w, EPS)
        y, _ = api.add_rms_norm(total, None, w, EPS)
        return (y8.view(torch.uint8), sc, total, y, *api.add_rms_norm_backward(total, w, EPS, y, x))

    side = torch.cuda.Stream(gpu)
    side.wait_stream(torch.cuda.current_stream(gpu))
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
        x.mul_(0.5).add_(0.25)
        graph.replay()
    torch.cuda.current_stream(gpu).wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


FIRST_CALLS = """
import threading, torch
from transformer_depth_wise_gb300 import api
dev = torch.device("cuda:0")
x = torch.linspace(-3, 3, 64 * 2048, device=dev).view(64, 2048)
w = torch.linspace(0.5, 1.5, 2048, device=dev)
cache = x.view(-1)[:32 * 2 * 16 * 64].view(32, 2, 16, 64).contiguous()
pages, table = torch.arange(20, device=dev).int(), torch.arange(20, 32, device=dev).view(4, 3).int()
length, own = torch.tensor([310], device=dev).int(), torch.tensor([40, 1, 0, 17], device=dev).int()
query = x.view(-1)[:4 * 8 * 64].view(4, 8, 64).contiguous()
torch.cuda.synchronize()
start, got = threading.Barrier(8), [None] * 8

def work(i):
    dtype = (torch.float32, torch.bfloat16)[i % 2]
    a, q, c = x.to(dtype), query.to(dtype), cache.to(dtype)
    with torch.cuda.stream(torch.cuda.Stream(dev)):
        torch.cuda.synchronize()
        start.wait()
        y, s = api.add_rms_norm(a, a, w)
        y8, sc, _ = api.add_rms_norm_8bit(a, None, w, group=64)
        dx, dw = api.add_rms_norm_backward(s, w, 1e-6, y)
        o, lse = api.shared_prefix_attention(q, c, c, pages, length, table, own, 0.125)
        n = api.rms_norm(a, w)
        h = api.depth_aggregate([a, y, s], w)
        grads, gq, gg = api.depth_aggregate_backward([a, y, s], w, w, 1e-6, h)
        p1, _, p1_lse = api.block_phase1([a, y, s], torch.stack((w, 2 * w)))
        torch.cuda.current_stream().synchronize()
    got[i] = (y, s, y8.float(), sc, dx, dw, o, lse, n, h, *grads, gq, gg, p1, p1_lse)

threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
for i in range(2, 8):
    assert all(torch.equal(p, q) for p, q in zip(got[i], got[i % 2])), i
"""


@gpu_only
def test_first_calls_from_several_threads(gpu):
    """What the library finds once and keeps (SMs, resident CTAs, shared-memory limits) may be found by threads at once."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, check=True, timeout=300)


# --------------------------------------------------------------------------
# refusals
# --------------------------------------------------------------------------
def norm(x=FAKE, r=FAKE + 64, B=1, T=2, D=256, dtype=1, w=None, eps=1e-6, total=None, y=FAKE + 128):
    return _lib.lib().attnres_add_rms_norm(x, r, B, T, D, dtype, w, eps, total, y, None)


def norm8(x=FAKE, r=FAKE + 64, B=1, T=2, D=256, dtype=1, w=None, eps=1e-6, total=None, y=FAKE + 128, group=64,
          sc=FAKE + 256):
    return _lib.lib().attnres_add_rms_norm_8bit(x, r, B, T, D, dtype, w, eps, group, total, y, sc, None)


def backward(s=FAKE, B=1, T=2, D=256, dtype=1, w=None, eps=1e-6, gy=FAKE, gs=None, dx=FAKE, gw=FAKE + 512, ws=FAKE,
             rows=1):
    return _lib.lib().attnres_add_rms_norm_backward(s, B, T, D, dtype, w, eps, gy, gs, dx, gw, ws, rows, None)


def test_refusals():
    for call in (norm, norm8, backward):
        assert call(dtype=2) == DTYPE and call(B=-1) == SHAPE and call(T=-1) == SHAPE and call(D=0) == SHAPE
        assert call(D=16384 + 128) == SHAPE and call(D=8192 + 128, dtype=0) == SHAPE
        assert call(eps=-1.0) == VALUE and call(eps=math.nan) == VALUE and call(w=FAKE + 4) == ALIGN
    for call in (norm, norm8):
        assert call(D=68) in (ALIGN, SHAPE) and call(D=66, dtype=0) in (ALIGN, SHAPE)
        assert call(x=None) == NULL and call(y=None) == NULL and call(r=FAKE + 8) == ALIGN and call(y=FAKE + 8) == ALIGN
        assert call(total=FAKE + 128) == VALUE and call(w=FAKE + 128) == VALUE and call(B=0, x=None, y=None) == OK
    assert norm8(group=16) == VALUE and norm8(group=256) == VALUE and norm8(group=-32) == VALUE
    assert norm8(D=96) == SHAPE and norm8(sc=None) == NULL and norm8(sc=FAKE + 258) == ALIGN
    assert norm8(y=FAKE) == VALUE and norm8(y=FAKE + 64) == VALUE and norm8(sc=FAKE + 128) == VALUE
    assert backward(D=68) == ALIGN and backward(s=None) == NULL and backward(gy=None) == NULL and backward(dx=None) == NULL
    assert backward(ws=None) == NULL and backward(rows=0) == CAP and backward(gw=FAKE + 4) == ALIGN
    assert backward(gs=FAKE + 8) == ALIGN and backward(gw=FAKE) == VALUE and backward(B=0, gw=None, s=None) == OK
    assert _lib.lib().attnres_add_rms_norm_backward_workspace_rows() >= 1


def test_refusal_of_partial_overlaps():
    """Outputs lie on an input row on row, or apart: anything between is a race of one row's reads with another's writes."""
    far, row, n = FAKE + (1 << 20), 512, 1024                        # two rows of 256 bf16
    apart = dict(x=FAKE, r=far, y=far + (1 << 20))
    for name in ("y", "total"):
        for at in (FAKE + row, FAKE - row, FAKE + n - 16, FAKE + 16 - n, far + row, far - 16):
            assert norm(**(apart | {name: at})) == VALUE, (name, at - FAKE)
        assert norm(**(apart | {name: FAKE, "r": FAKE + row})) == VALUE, name           # on x, and the residual half on it
        assert norm(**(apart | {name: far, "w": far + n - 64})) == VALUE, name          # the weight (1024 bytes) too
        assert norm(**(apart | {name: far + n, "w": far + n - 64})) == VALUE, name
    assert norm(**(apart | {"total": apart["y"] + row})) == VALUE and norm(**(apart | {"total": apart["y"] - row})) == VALUE
    eight = dict(x=FAKE, r=far, y=far + (1 << 20), sc=far + (1 << 21), total=far + (1 << 22))
    assert norm8(**(eight | {"total": FAKE + row})) == VALUE and norm8(**(eight | {"total": far - row})) == VALUE
    for base, size in ((FAKE, n), (far, n), (eight["total"], n)):
        for at in (base, base + row, base + size - 16, base - 256):  # y8 has 512 bytes
            assert norm8(**(eight | {"y": at})) == VALUE
        for at in (base, base + row, base + size - 4, base - 28):    # the scales 32
            assert norm8(**(eight | {"sc": at})) == VALUE
    assert norm8(**(eight | {"sc": eight["y"] + 508})) == VALUE and norm8(**(eight | {"sc": eight["y"] - 28})) == VALUE
    assert norm8(**(eight | {"w": eight["sc"] - 1008})) == VALUE and norm8(**(eight | {"w": eight["y"] + 496})) == VALUE
    back = dict(s=FAKE, gy=far, gs=far + (1 << 20), dx=far + (1 << 21), gw=far + (1 << 22), ws=far + (1 << 23))
    for base in (back["s"], back["gy"], back["gs"]):
        assert backward(**(back | {"dx": base + row})) == VALUE and backward(**(back | {"dx": base - row})) == VALUE
        for name in ("gw", "ws"):
            assert backward(**(back | {name: base})) == VALUE and backward(**(back | {name: base - row})) == VALUE
            assert backward(**(back | {name: base + n - 16})) == VALUE
    for at in (back["dx"] + row, back["gw"] + row, back["ws"] + row):
        assert backward(**(back | {"w": at})) == VALUE
    assert backward(**(back | {"gw": back["dx"] - 16})) == VALUE and backward(**(back | {"ws": back["gw"] - row})) == VALUE
    assert backward(**(back | {"ws": back["gw"] - 4096, "rows": 5})) == VALUE           # a later row of the workspace


@gpu_only
def test_neighbours_are_no_overlap(gpu):
    """Rows right behind one another in one buffer are apart."""
    g = wk.generator(14, gpu)
    for dtype in (BF, F32):
        buf = rand(g, 12, 256, dtype=dtype)
        x, r, w = buf[0:3].clone(), buf[3:6].clone(), 1 + rand(g, 256, dtype=F32, scale=0.1)
        want = api.add_rms_norm(x, r, w)
        got = api.add_rms_norm(buf[0:3], buf[3:6], w, sum_out=buf[6:9], out=buf[9:12])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        dx, dw = api.add_rms_norm_backward(want[1], w, EPS, x, r)
        buf[0:3], buf[3:6], buf[6:9] = want[1], x, r
        got = api.add_rms_norm_backward(buf[0:3], w, EPS, buf[3:6], buf[6:9], dx=buf[9:12])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
        with pytest.raises(_lib.AttnResError):
            api.add_rms_norm(buf[1:4], r, w, out=buf[0:3])


@gpu_only
def test_wrapper_refusals(gpu):
    x, r, w = inputs(gpu, BF, 4, 256, True, 1)
    for bad in (dict(x=x.cpu()), dict(x=x[:, ::2]), dict(r=r[:2].contiguous()), dict(w=w[:8].contiguous())):
        a = dict(x=x, r=r, w=w) | bad
        with pytest.raises(ValueError):
            api.add_rms_norm(a["x"], a["r"], a["w"])
    with pytest.raises(TypeError):
        api.add_rms_norm(x.half(), None, w)
    with pytest.raises(TypeError):
        api.add_rms_norm(x, r.float(), w)
    with pytest.raises(TypeError):
        api.add_rms_norm_8bit(x, r, w, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        api.add_rms_norm_8bit(x, r, w, group=96)
    with pytest.raises(_lib.AttnResError):
        api.add_rms_norm_8bit(x, r, w, group=16)
    with pytest.raises(_lib.AttnResError):
        api.add_rms_norm(x, r, w, sum_out=r, out=r)
    with pytest.raises(ValueError):
        api.add_rms_norm_backward(x, w, EPS, None)


@gpu_only
@pytest.mark.parametrize("group", [-32, -1])
def test_negative_group_is_refused_by_name(gpu, group):
    x, r, w = inputs(gpu, BF, 4, 256, True, 1)
    with pytest.raises(ValueError, match="group"):
        api.add_rms_norm_8bit(x, r, w, group=group)
