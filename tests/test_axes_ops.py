"""The head norm with positions of several axes against plain float64 forms of its definition: forward, into a paged
cache, backward, and the refusals.

Tolerances as in test_attention_ops.py, whose reference this one meets where all axes agree: u is the rounding of a
stored result (half a step), the other terms count the fp32 roundings on the way.
"""
import pytest
import torch

from transformer_depth_wise_gb300 import _lib, api
from transformer_depth_wise_gb300 import workloads as wk

gpu_only = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
E = 2.0 ** -24
EPS = 1e-6
FAKE = 0x7F0000000000      # 16-byte aligned stand-in for a device pointer (never dereferenced)
OK, NULL, SHAPE, DTYPE, ALIGN, CAP, VALUE = 0, -1, -2, -3, -4, -7, -8


def cpu(t):
    return t.detach().cpu().double()


def within(got, want, tol, what=""):
    got, want = cpu(got), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: finite in different places"
    d = torch.where(fine, (got - want).abs() - tol, torch.full_like(want, -1.0))
    assert d.numel() == 0 or float(d.max()) <= 0.0, f"{what}: over the bound by {float(d.max()):.3e}"


def rand(g, *shape, dtype=BF, scale=1.0):
    return (torch.empty(shape, dtype=F32, device=g.device).normal_(generator=g) * scale).to(dtype)


def angles(pos, axes, inv_freq):
    """[B,T,1,rot/2] in float64; a pair whose axis there is not keeps its place."""
    pos, inv_freq = cpu(pos), cpu(inv_freq)
    A = pos.shape[-1]
    cols = [pos[..., int(a)] * f if 0 <= int(a) < A else torch.zeros_like(pos[..., 0])
            for a, f in zip(axes.cpu(), inv_freq)]
    return torch.stack(cols, -1)[:, :, None]


def turn(z, a, inter, back=False):
    n = a.shape[-1]
    c, s = a.cos(), -a.sin() if back else a.sin()
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    y = z.clone()
    y[..., i] = z[..., i] * c - z[..., j] * s
    y[..., j] = z[..., j] * c + z[..., i] * s
    return y


def forward_ref(x, w, a, inter):
    x = cpu(x)
    z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * cpu(w)
    return turn(z, a, inter), z.abs().amax(-1, keepdim=True)


def backward_ref(x, w, a, inter, grad):
    x, w = cpu(x), cpu(w)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    dz = turn(cpu(grad), a, inter, back=True)
    u = dz * w
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdim=True))
    return dx, (dz * x * r).sum((0, 1, 2)), (dz * x * r).abs().sum((0, 1, 2)), r * u.abs().amax(-1, keepdim=True)


def inputs(dev, dtype, B, T, Hq, Hk, d, rot, A, seed):
    g = wk.generator(seed, dev)
    qkv = rand(g, B, T, (Hq + 2 * Hk) * d, dtype=dtype, scale=2.0)
    q, k, v = qkv.split([Hq * d, Hk * d, Hk * d], -1)
    q, k, v = q.unflatten(-1, (Hq, d)), k.unflatten(-1, (Hk, d)), v.unflatten(-1, (Hk, d))
    wq, wk_ = 1 + rand(g, d, dtype=F32, scale=0.1), 1 + rand(g, d, dtype=F32, scale=0.1)
    pos = torch.randint(-50, 5000, (B, T, A), generator=g, device=dev).int()
    axes = torch.randint(0, A, (rot // 2,), generator=g, device=dev).int()
    return q, k, v, wq, wk_, pos, axes, api.rotary_frequencies(rot, device=dev)


CASES = [  # dtype, B, T, Hq, Hk, d, rot, interleaved, axes
    (BF, 1, 1, 1, 1, 16, 16, False, 1), (BF, 3, 7, 5, 2, 64, 64, False, 2), (BF, 2, 33, 4, 4, 128, 64, True, 3),
    (BF, 1, 700, 8, 1, 128, 128, False, 3), (BF, 256, 1, 56, 8, 128, 128, False, 3), (BF, 2, 5, 3, 1, 80, 32, False, 4),
    (BF, 1, 9, 2, 2, 96, 96, True, 8), (BF, 1, 3, 2, 1, 512, 512, False, 5), (BF, 2, 70, 2, 1, 192, 96, False, 2),
    (F32, 3, 111, 4, 2, 64, 32, True, 3), (F32, 1, 2, 1, 1, 8, 8, False, 8), (F32, 2, 65, 7, 7, 128, 128, False, 2),
    (F32, 1, 40, 3, 1, 256, 256, True, 4), (F32, 1, 5, 40, 40, 72, 24, False, 3),
]


@gpu_only
@pytest.mark.parametrize("dtype,B,T,Hq,Hk,d,rot,inter,A", CASES)
def test_forward(gpu, dtype, B, T, Hq, Hk, d, rot, inter, A):
    q, k, _, wq, wk_, pos, axes, fr = inputs(gpu, dtype, B, T, Hq, Hk, d, rot, A, B * 7 + T * 3 + d)
    axes[-1] = A                       # no axis: not turned
    axes[0] = -1
    qo, ko = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS, interleaved=inter, axes=axes)
    a = angles(pos, axes, fr)
    for x, w, got in ((q, wq, qo), (k, wk_, ko)):
        y, zmax = forward_ref(x, w, a, inter)
        # sum of squares 12, root and products 4, cosine and sine 2 each, the angle's argument pi / 2, products and sum 5
        within(got, y, U[dtype] * y.abs() + 32 * E * 1.5 * zmax)
    qi, ki = q.clone(), k.clone()
    api.head_norm_rotate(qi, ki, wq, wk_, pos, fr, EPS, interleaved=inter, axes=axes, q_out=qi, k_out=ki)
    assert torch.equal(qi, qo) and torch.equal(ki, ko)


@gpu_only
@pytest.mark.parametrize("dtype,B,T,Hq,Hk,d,rot,inter,A", CASES)
def test_equal_axes_are_one_position(gpu, dtype, B, T, Hq, Hk, d, rot, inter, A):
    q, k, _, wq, wk_, pos, axes, fr = inputs(gpu, dtype, B, T, Hq, Hk, d, rot, A, 5 * B + d)
    one = pos[..., 0].contiguous()
    want = api.head_norm_rotate(q, k, wq, wk_, one, fr, EPS, interleaved=inter)
    same = one[..., None].expand(B, T, A).contiguous()
    got = api.head_norm_rotate(q, k, wq, wk_, same, fr, EPS, interleaved=inter, axes=axes)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    gq, gk = torch.ones_like(want[0]), want[1] * 0.5
    want = api.head_norm_rotate_backward(q, k, wq, wk_, one, fr, EPS, gq, gk, interleaved=inter)
    got = api.head_norm_rotate_backward(q, k, wq, wk_, same, fr, EPS, gq, gk, interleaved=inter, axes=axes)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@gpu_only
def test_far_positions_and_frequencies_that_are_no_number(gpu):
    q, k, _, wq, wk_, _, _, fr = inputs(gpu, F32, 1, 4, 2, 1, 64, 64, 3, 5)
    far = torch.tensor([0, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 123456789, -1, 5, 10 ** 6, 77, -10 ** 9, 1, 2])
    pos = far.view(1, 4, 3).int().to(gpu)
    axes = api.rotary_axes((8, 12, 12), device=gpu)
    qo, _ = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS, axes=axes)
    y, zmax = forward_ref(q, wq, angles(pos, axes, fr), False)
    # the reference's own angle is off by up to 2^31 * 2^-53 radians per unit of inv_freq, the kernel's by as much
    within(qo, y, U[F32] * y.abs() + 48 * E * zmax + 2.0 ** -20 * zmax)
    fr[3] = float("nan")
    fr[9] = float("inf")
    axes[9] = 7                        # no axis: not turned, whatever its frequency
    qn, _ = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS, axes=axes)
    bad = torch.zeros(64, dtype=torch.bool)
    bad[[3, 35]] = True
    assert torch.equal(qn.isnan().cpu(), bad.expand(1, 4, 2, 64))


def test_axes_table():
    t = lambda *a: api.rotary_axes(*a, device="cpu").tolist()  # noqa: E731
    assert t((2, 3, 1)) == [0, 0, 1, 1, 1, 2] and t((2, 3, 1), True) == [0, 1, 2, 0, 1, 1] and t((0, 2)) == [1, 1]
    for bad in ((), (1,) * 9, (2, -1)):
        with pytest.raises(ValueError):
            api.rotary_axes(bad, device="cpu")


@gpu_only
@pytest.mark.parametrize("dtype,B,T,Hq,Hk,d,page,A", [(BF, 4, 1, 8, 2, 128, 16, 3), (BF, 3, 70, 2, 2, 64, 32, 2),
                                                      (F32, 2, 9, 3, 1, 64, 7, 4), (BF, 300, 1, 7, 1, 80, 1, 3)])
def test_append(gpu, dtype, B, T, Hq, Hk, d, page, A):
    q, k, v, wq, wk_, pos, axes, fr = inputs(gpu, dtype, B, T, Hq, Hk, d, d, A, 3 * B + T)
    g = wk.generator(99, gpu)
    per = (T + 20) // page + 1
    table = torch.randperm(B * per, device=gpu, generator=g).view(B, per).int()
    places = (torch.randint(0, 20, (B, 1), device=gpu, generator=g) + torch.arange(T, device=gpu)).int()
    places[0, 0] = -3                  # padding, a place behind the table, pages outside the pool
    places[1, T - 1] = per * page
    lost = int(table[2 if B > 2 else 1, 0])
    table[table == lost] = B * per if B % 2 else -1
    kc, vc = rand(g, B * per, Hk, page, d, dtype=dtype), rand(g, B * per, Hk, page, d, dtype=dtype)
    k0, v0 = kc.clone(), vc.clone()
    qo = api.head_norm_rotate_append(q, k, v, wq, wk_, pos, fr, kc, vc, table, EPS, axes=axes, places=places)
    qw, kw = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS, axes=axes)
    assert torch.equal(qo, qw)
    for b in range(B):
        for t in range(T):
            p = int(places[b, t])
            if p < 0 or p >= per * page or not 0 <= int(table[b, p // page]) < B * per:
                continue
            k0[int(table[b, p // page]), :, p % page] = kw[b, t]
            v0[int(table[b, p // page]), :, p % page] = v[b, t]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)        # stored ones exactly, all others as they were
    # positions of one number with places of their own, and places that are the positions
    one = pos[..., 0].contiguous()
    qo = api.head_norm_rotate_append(q, k, v, wq, wk_, one, fr, kc, vc, table, EPS, places=places)
    assert torch.equal(qo, api.head_norm_rotate(q, k, wq, wk_, one, fr, EPS)[0])
    kc2, vc2 = kc.clone(), vc.clone()
    a = api.head_norm_rotate_append(q, k, v, wq, wk_, places, fr, kc, vc, table, EPS)
    b = api.head_norm_rotate_append(q, k, v, wq, wk_, places, fr, kc2, vc2, table, EPS, places=places)
    assert torch.equal(a, b) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


@gpu_only
@pytest.mark.parametrize("dtype,B,T,Hq,Hk,d,rot,inter,A", CASES)
def test_backward(gpu, dtype, B, T, Hq, Hk, d, rot, inter, A):
    q, k, _, wq, wk_, pos, axes, fr = inputs(gpu, dtype, B, T, Hq, Hk, d, rot, A, B + T + d)
    axes[0] = A
    g = wk.generator(17, gpu)
    gq, gk = rand(g, B, T, Hq, d, dtype=dtype), rand(g, B, T, Hk, d, dtype=dtype)
    args = (q, k, wq, wk_, pos, fr, EPS, gq, gk)
    dq, dk, dwq, dwk = api.head_norm_rotate_backward(*args, interleaved=inter, axes=axes)
    again = api.head_norm_rotate_backward(*args, interleaved=inter, axes=axes)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dwq, dwk), again))        # a fixed order of sums
    a = angles(pos, axes, fr)
    for x, w, gr, dx, dw in ((q, wq, gq, dq, dwq), (k, wk_, gk, dk, dwk)):
        rx, rw, absw, big = backward_ref(x, w, a, inter, gr)
        # as the forward, with a second mean whose terms cancel: its roundings are in units of |u|'s largest value
        within(dx, rx, U[dtype] * rx.abs() + 64 * E * big, "dx")
        # every term is off by 32 E of itself, and the sums have three levels of at most T Hq / 32 + 64 + 32 terms
        within(dw, rw, (32 + B * T * max(Hq, Hk) / 32 + 96) * E * absw, "dw")


def test_backward_formula_against_differences():
    g = torch.Generator().manual_seed(1)
    x, grad = (torch.randn(1, 2, 2, 16, dtype=torch.float64, generator=g) for _ in range(2))
    w = torch.randn(16, dtype=torch.float64, generator=g)
    a = angles(torch.tensor([[[3, 70], [9, -4]]]), torch.tensor([0, 1, 1, 0]), api.rotary_frequencies(8, device="cpu"))
    h = 1e-5
    for inter in (False, True):
        dx, dw, _, _ = backward_ref(x, w, a, inter, grad)
        loss = lambda x, w: float((forward_ref(x, w, a, inter)[0] * grad).sum())  # noqa: B023, E731
        for t, d in ((x, dx), (w, dw)):
            for i in range(0, t.numel(), 5):
                e = torch.zeros(t.numel(), dtype=torch.float64)
                e[i] = h
                e = e.view(t.shape)
                lo, hi = (loss(t - e, w), loss(t + e, w)) if t is x else (loss(x, t - e), loss(x, t + e))
                # central differences: h^2 of the third derivative (below 100 here) and 2^-52 * |loss| / h
                assert abs((hi - lo) / (2 * h) - float(d.reshape(-1)[i])) < 1e-7


@gpu_only
def test_captured_on_another_stream(gpu):
    q, k, v, wq, wk_, pos, axes, fr = inputs(gpu, BF, 3, 5, 4, 2, 64, 64, 3, 8)
    kc, vc = (torch.zeros(6, 2, 16, 64, device=gpu, dtype=BF) for _ in range(2))
    table = torch.arange(6, device=gpu).view(3, 2).int()
    places = torch.arange(5, device=gpu).expand(3, 5).int().contiguous()
    gq, gk = torch.ones_like(q).contiguous(), torch.ones_like(k).contiguous()

    def step():
        qo = api.head_norm_rotate_append(q, k, v, wq, wk_, pos, fr, kc, vc, table, EPS, axes=axes, places=places)
        return (qo, *api.head_norm_rotate_backward(q, k, wq, wk_, pos, fr, EPS, gq, gk, axes=axes))

    side = torch.cuda.Stream(gpu)
    side.wait_stream(torch.cuda.current_stream(gpu))
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
        q.mul_(0.5).add_(0.25)
        pos.add_(3)
        graph.replay()
    torch.cuda.current_stream(gpu).wait_stream(side)
    kc1 = kc.clone()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(kc1, kc)


# --------------------------------------------------------------------------
# refusals (CPU)
# --------------------------------------------------------------------------
def rotate(A=3, axes=FAKE, pos=FAKE, rot=64, fr=FAKE, B=1, T=2, q=FAKE, qo=FAKE, d=64):
    return _lib.lib().attnres_head_norm_rotate_axes(q, FAKE, B, T, 4, 2, d, 1, 256, 128, None, None, pos, A, axes, fr, rot,
                                                    0, 1e-6, qo, FAKE, 256, 128, None)


def append(A=3, axes=FAKE, places=FAKE, pos=FAKE, B=1, T=1, num=4, kc=FAKE, rot=64):
    return _lib.lib().attnres_head_norm_rotate_axes_append(FAKE, FAKE, FAKE, B, T, 4, 2, 64, 1, 256, 128, 128, None, None,
                                                           pos, A, axes, places, FAKE, rot, 0, 1e-6, FAKE, 256, kc, FAKE,
                                                           num, 16, FAKE, 2, None)


def backward(A=3, axes=FAKE, pos=FAKE, B=1, gw=FAKE, ws=FAKE, rows=2):
    return _lib.lib().attnres_head_norm_rotate_axes_backward(FAKE, FAKE, B, 1, 4, 2, 64, 1, 256, 128, None, None, pos, A,
                                                             axes, FAKE, 64, 0, 1e-6, FAKE, FAKE, 256, 128, FAKE,
                                                             FAKE, gw, None, ws, rows, None)


def test_refusals():
    for call in (rotate, append, backward):
        assert call(A=0) == SHAPE and call(A=9) == SHAPE and call(A=-1) == SHAPE
        assert call(axes=FAKE + 2) == ALIGN and call(pos=FAKE + 2) == ALIGN and call(pos=None) == NULL
    assert rotate(rot=8) == ALIGN and rotate(fr=None) == NULL and rotate(q=None) == NULL and rotate(qo=FAKE + 8) == ALIGN
    assert rotate(B=0, q=None, pos=None) == OK and rotate(d=0) == SHAPE
    assert append(places=None) == NULL and append(places=FAKE + 2) == ALIGN and append(num=-1) == SHAPE
    assert append(kc=None) == NULL and append(places=None, num=0) == NULL and append(B=0, places=None) == OK
    assert backward(ws=None) == NULL and backward(rows=1) == CAP and backward(B=0, gw=None, pos=None) == OK


@gpu_only
def test_wrapper_refusals(gpu):
    q, k, v, wq, wk_, pos, axes, fr = inputs(gpu, BF, 2, 3, 2, 1, 64, 64, 3, 1)
    call = lambda p=pos, a=axes, f=fr: api.head_norm_rotate(q, k, wq, wk_, p, f, EPS, axes=a)  # noqa: E731
    for bad in (dict(p=pos[..., 0].contiguous()), dict(p=None), dict(a=axes[:-1].contiguous()), dict(f=None),
                dict(p=pos[:1].contiguous()), dict(p=pos.expand(2, 3, 3).transpose(0, 1)),
                dict(p=torch.zeros(2, 3, 9, device=gpu).int()), dict(a=axes.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        call(a=axes.long())
    with pytest.raises(TypeError):
        call(p=pos.long())
    kc = torch.zeros(2, 1, 16, 64, device=gpu, dtype=BF)
    table = torch.zeros(2, 1, device=gpu).int()
    with pytest.raises(ValueError, match="places"):
        api.head_norm_rotate_append(q, k, v, wq, wk_, pos, fr, kc, kc.clone(), table, EPS, axes=axes)
