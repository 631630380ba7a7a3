"""The attention sublayer's operators against plain float64 forms of their definitions.

Head norm with rotation (forward, into a paged cache, backward), paged attention of one token, linear attention with a
decay per head (prompts, backward, single tokens).  The references work in float64 on the CPU from the same values.
Tolerances are bounds, not fits.  u is the rounding of a stored result (half a step: 2^-8 relative for bf16, 2^-24 for
fp32); every other term counts the fp32 roundings on the way, as the comment at each check says.
"""
import math

import pytest
import torch

from transformer_depth_wise_gb300 import api
from transformer_depth_wise_gb300 import workloads as wk

gpu_only = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
E = 2.0 ** -24
EPS = 1e-6


def cpu(t):
    return t.detach().cpu().double()


def within(got, want, tol, what=""):
    """|got - want| <= tol element by element; infinities and NaN where want has them."""
    got, want = cpu(got), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: finite in different places"
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), what
    d = (got - want).abs() - (tol if torch.is_tensor(tol) else torch.tensor(float(tol), dtype=torch.float64))
    d = torch.where(fine, d, torch.full_like(d, -1.0))
    assert d.numel() == 0 or float(d.max()) <= 0.0, f"{what}: over the bound by {float(d.max()):.3e}"


def rand(g, *shape, dtype=BF, scale=1.0):
    return (torch.empty(shape, dtype=F32, device=g.device).normal_(generator=g) * scale).to(dtype)


# --------------------------------------------------------------------------
# head norm and rotation
# --------------------------------------------------------------------------
def rotate_ref(x, w, pos, inv_freq, inter, eps=EPS):
    """(y, largest |z| of the head) in float64; x [B,T,H,d], pos [B,T], inv_freq [rot/2]."""
    x = cpu(x)
    z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        z = z * cpu(w)
    y = z.clone()
    if inv_freq is not None and inv_freq.numel():
        n = inv_freq.numel()
        a = (cpu(pos)[..., None] * cpu(inv_freq))[:, :, None]
        c, s = a.cos(), a.sin()
        i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
        y[..., i] = z[..., i] * c - z[..., j] * s
        y[..., j] = z[..., j] * c + z[..., i] * s
    return y, z.abs().amax(-1, keepdim=True)


def rotate_tol(y, zmax, dtype, d):
    # fp32 roundings, in units of E times the head's largest |z|: the sum of squares (at most 16 terms per lane and a
    # tree over the lanes, halved by the root) 12, root and products 4, cosine and sine 2 each, the angle's argument
    # (2^-25 of half a turn: pi E / 2) and the two products and their sum 5.
    return U[dtype] * y.abs() + 32 * E * 1.5 * zmax


def norm_inputs(gpu, dtype, B, T, Hq, Hk, d, rot, seed, packed=True):
    g = wk.generator(seed, gpu)
    qkv = rand(g, B, T, (Hq + 2 * Hk) * d, dtype=dtype, scale=2.0)
    q, k, v = qkv.split([Hq * d, Hk * d, Hk * d], -1)
    q, k, v = q.unflatten(-1, (Hq, d)), k.unflatten(-1, (Hk, d)), v.unflatten(-1, (Hk, d))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    wq, wk_ = 1 + rand(g, d, dtype=F32, scale=0.1), 1 + rand(g, d, dtype=F32, scale=0.1)
    pos = torch.randint(0, 5000, (B, T), generator=g, device=gpu).int()
    return q, k, v, wq, wk_, pos, api.rotary_frequencies(rot, device=gpu)


ROTATE = [  # dtype, B, T, Hq, Hk, d, rot, interleaved
    (BF, 1, 1, 1, 1, 16, 16, False), (BF, 3, 7, 5, 2, 64, 64, False), (BF, 2, 33, 4, 4, 128, 64, True),
    (BF, 1, 1000, 8, 1, 128, 128, False), (BF, 256, 1, 56, 8, 128, 128, False), (BF, 2, 5, 3, 1, 80, 32, False),
    (BF, 1, 9, 2, 2, 96, 96, True), (BF, 1, 3, 2, 1, 512, 512, False), (BF, 2, 70, 2, 1, 192, 0, False),
    (BF, 1, 17, 1, 3, 256, 16, True), (F32, 3, 111, 4, 2, 64, 32, True), (F32, 1, 2, 1, 1, 8, 8, False),
    (F32, 2, 65, 7, 7, 128, 128, False), (F32, 1, 40, 3, 1, 256, 256, True), (F32, 1, 5, 40, 40, 72, 24, False),
    (BF, 1, 5000, 2, 1, 32, 32, False),
]


@gpu_only
@pytest.mark.parametrize("dtype,B,T,Hq,Hk,d,rot,inter", ROTATE)
@pytest.mark.parametrize("packed", [True, False])
def test_rotate(gpu, dtype, B, T, Hq, Hk, d, rot, inter, packed):
    q, k, _, wq, wk_, pos, fr = norm_inputs(gpu, dtype, B, T, Hq, Hk, d, rot, B * 7 + T * 3 + d, packed)
    fr = fr if rot else None
    qo, ko = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS, interleaved=inter)
    for x, w, got in ((q, wq, qo), (k, wk_, ko)):
        y, zmax = rotate_ref(x, w, pos, fr, inter)
        within(got, y, rotate_tol(y, zmax, dtype, d))
    # the defaults: no weights, positions 0 .. T-1
    qo, ko = api.head_norm_rotate(q, k, None, None, None, fr, EPS, interleaved=inter)
    y, zmax = rotate_ref(k, None, torch.arange(T).expand(B, T), fr, inter)
    within(ko, y, rotate_tol(y, zmax, dtype, d), "default positions")


@gpu_only
def test_rotate_far_positions(gpu):
    q, k, _, wq, wk_, _, fr = norm_inputs(gpu, F32, 1, 8, 2, 1, 64, 64, 5)
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 10 ** 9 + 7, 123456789]], device=gpu).int()
    qo, _ = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS)
    y, zmax = rotate_ref(q, wq, pos, fr, False)
    # the reference's own angle is off by up to 2^31 * 2^-53 radians per unit of inv_freq, the kernel's by as much
    within(qo, y, rotate_tol(y, zmax, F32, 64) + 2.0 ** -20 * zmax)


@gpu_only
def test_rotate_in_place_leaves_the_rest(gpu):
    q, k, v, wq, wk_, pos, fr = norm_inputs(gpu, BF, 2, 37, 4, 2, 64, 64, 11)
    want = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS)
    v0 = v.clone()
    got = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, v0)


def cache_of(g, pages, Hk, page, d, dtype, fill=None):
    shape = (pages, Hk, page, d)
    return rand(g, *shape, dtype=dtype) if fill is None else torch.full(shape, fill, dtype=dtype, device=g.device)


@gpu_only
@pytest.mark.parametrize("dtype,B,T,Hq,Hk,d,page", [(BF, 4, 1, 8, 2, 128, 16), (BF, 3, 70, 2, 2, 64, 32),
                                                    (F32, 2, 9, 3, 1, 64, 7), (BF, 300, 1, 7, 1, 80, 1)])
def test_append(gpu, dtype, B, T, Hq, Hk, d, page):
    q, k, v, wq, wk_, _, fr = norm_inputs(gpu, dtype, B, T, Hq, Hk, d, d, 3 * B + T)
    g = wk.generator(99, gpu)
    per = (T + 20) // page + 1
    table = torch.randperm(B * per, device=gpu, generator=g).view(B, per).int()
    start = torch.randint(0, 20, (B, 1), device=gpu, generator=g)
    pos = (start + torch.arange(T, device=gpu)).int()
    # tokens without a place: a negative position, one behind the table, and pages outside the pool
    pos[0, 0] = -3
    pos[1, T - 1] = per * page
    lost = int(table[2 if B > 2 else 1, 0])
    table[table == lost] = B * per if B % 2 else -1
    kc, vc = cache_of(g, B * per, Hk, page, d, dtype), cache_of(g, B * per, Hk, page, d, dtype)
    k0, v0 = kc.clone(), vc.clone()
    qo = api.head_norm_rotate_append(q, k, v, wq, wk_, pos, fr, kc, vc, table, EPS)
    qw, kw = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS)
    assert torch.equal(qo, qw)
    for b in range(B):
        for t in range(T):
            p = int(pos[b, t])
            if p < 0 or p >= per * page or not 0 <= int(table[b, p // page]) < B * per:
                continue
            k0[int(table[b, p // page]), :, p % page] = kw[b, t]
            v0[int(table[b, p // page]), :, p % page] = v[b, t]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)        # stored ones exactly, all others as they were


def rotate_bwd_ref(x, w, pos, inv_freq, inter, grad, eps=EPS):
    x, grad = cpu(x), cpu(grad)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else cpu(w)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dz = grad.clone()
    if inv_freq is not None and inv_freq.numel():
        n = inv_freq.numel()
        a = (cpu(pos)[..., None] * cpu(inv_freq))[:, :, None]
        c, s = a.cos(), a.sin()
        i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
        dz[..., i] = grad[..., i] * c + grad[..., j] * s
        dz[..., j] = grad[..., j] * c - grad[..., i] * s
    u = dz * w
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdim=True))
    return dx, (dz * x * r).sum((0, 1, 2)), (dz * x * r).abs().sum((0, 1, 2)), r * u.abs().amax(-1, keepdim=True)


def test_rotate_backward_formula_against_differences():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, 2, 2, 16, dtype=torch.float64, generator=g)
    w = torch.randn(16, dtype=torch.float64, generator=g)
    grad = torch.randn(1, 2, 2, 16, dtype=torch.float64, generator=g)
    pos, fr = torch.tensor([[3, 70]]), api.rotary_frequencies(8, device="cpu")
    for inter in (False, True):
        dx, dw, _, _ = rotate_bwd_ref(x, w, pos, fr, inter, grad)
        loss = lambda x, w: float((rotate_ref(x, w, pos, fr, inter)[0] * grad).sum())  # noqa: B023, E731
        h = 1e-5
        for t, d in ((x, dx), (w, dw)):
            for i in range(0, t.numel(), 5):
                e = torch.zeros_like(t).view(-1)
                e[i] = h
                e = e.view(t.shape)
                lo, hi = (loss(t - e, w), loss(t + e, w)) if t is x else (loss(x, t - e), loss(x, t + e))
                # central differences: h^2 of the third derivative (below 100 here) and 2^-52 * |loss| / h
                assert abs((hi - lo) / (2 * h) - float(d.reshape(-1)[i])) < 1e-7


@gpu_only
@pytest.mark.parametrize("dtype,B,T,Hq,Hk,d,rot,inter", ROTATE)
def test_rotate_backward(gpu, dtype, B, T, Hq, Hk, d, rot, inter):
    q, k, _, wq, wk_, pos, fr = norm_inputs(gpu, dtype, B, T, Hq, Hk, d, rot, B + T + d)
    fr = fr if rot else None
    g = wk.generator(17, gpu)
    packed = rand(g, B, T, (Hq + Hk) * d, dtype=dtype)
    gq, gk = packed[..., :Hq * d].unflatten(-1, (Hq, d)), packed[..., Hq * d:].unflatten(-1, (Hk, d))
    dq, dk, dwq, dwk = api.head_norm_rotate_backward(q, k, wq, wk_, pos, fr, EPS, gq, gk, interleaved=inter)
    again = api.head_norm_rotate_backward(q, k, wq, wk_, pos, fr, EPS, gq, gk, interleaved=inter)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dwq, dwk), again))        # a fixed order of sums
    for x, w, gr, dx, dw in ((q, wq, gq, dq, dwq), (k, wk_, gk, dk, dwk)):
        rx, rw, absw, big = rotate_bwd_ref(x, w, pos, fr, inter, gr)
        # as the forward, with a second mean whose terms cancel: its roundings are in units of |u|'s largest value
        within(dx, rx, U[dtype] * rx.abs() + 64 * E * big, "dx")
        # every term is off by 32 E of itself, and the sums have three levels of at most T Hq / 32 + 64 + 32 terms
        within(dw, rw, (32 + B * T * max(Hq, Hk) / 32 + 96) * E * absw, "dw")
    only = api.head_norm_rotate_backward(q, k, wq, wk_, pos, fr, EPS, gq, gk, interleaved=inter, want_weights=False)
    assert torch.equal(only[0], dq) and torch.equal(only[1], dk) and only[2] is None and only[3] is None
    small = torch.full((2, d), float("nan"), device=gpu)                              # a single CTA
    one = api.head_norm_rotate_backward(q, k, wq, wk_, pos, fr, EPS, gq, gk, interleaved=inter, workspace=small)
    assert torch.equal(one[0], dq)
    _, rw, absw, _ = rotate_bwd_ref(q, wq, pos, fr, inter, gq)
    within(one[2], rw, (32 + B * T * Hq / 4 + 96) * E * absw, "dw of one CTA")


# --------------------------------------------------------------------------
# paged attention of one token
# --------------------------------------------------------------------------
def paged_ref(q, kc, vc, table, lengths, scale):
    """(out, lse, bound on out's error before its last rounding, the same of lse) in float64."""
    q, kc, vc = cpu(q), cpu(kc), cpu(vc)
    B, Hq, d = q.shape
    N, Hk, page, _ = kc.shape
    G = Hq // Hk
    out, lse = torch.zeros_like(q), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(q), torch.zeros(B, Hq, dtype=torch.float64)
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * page)
        j = torch.arange(n)
        pg = table[b].cpu().long()[j // page] if n else j
        ok = (pg >= 0) & (pg < N)
        pg, sl = pg[ok], (j % page)[ok]
        if not len(pg):
            continue
        for h in range(Hq):
            k, v = kc[pg, h // G, sl], vc[pg, h // G, sl]
            s = k @ q[b, h] * scale
            p = torch.softmax(s, 0)
            out[b, h] = p @ v
            lse[b, h] = torch.logsumexp(s, 0)
            # a score is a sum of d products: d roundings of its absolute sum; the exponential's argument and value
            # 16 E + |s - max| E; sums over n tokens in at least 16 strands; the weights enter the second product
            # with 16 bits or more (2^-17)
            ds = (d + 2) * E * float((k.abs() @ q[b, h].abs()).max() * abs(scale))
            ds += 2 * E * float(s.max() - s.min()) + (16 + n / 16) * E
            tol[b, h] = (2 * ds + 2.0 ** -17) * (p @ v.abs())
            ltol[b, h] = ds + E * abs(lse[b, h])
    return out, lse, tol, ltol


def paged_inputs(gpu, dtype, B, Hq, Hk, d, page, lengths, seed, spare=0):
    g = wk.generator(seed, gpu)
    per = max(1, -(-max(lengths) // page)) + spare
    q = rand(g, B, Hq, d, dtype=dtype, scale=1.5)
    kc, vc = cache_of(g, B * per + 1, Hk, page, d, dtype), cache_of(g, B * per + 1, Hk, page, d, dtype)
    table = torch.randperm(B * per, device=gpu, generator=g).view(B, per).int()
    return q, kc, vc, table, torch.tensor(lengths, device=gpu).int(), 1 / math.sqrt(d)


PAGED = [  # dtype, Hq, Hk, d, page, lengths
    (BF, 1, 1, 128, 16, [1]), (BF, 16, 16, 128, 16, [777]), (BF, 56, 8, 128, 64, [0, 1, 63, 64, 65, 500, 1300]),
    (BF, 8, 1, 64, 32, [5000, 3, 0, 31]), (BF, 16, 1, 128, 64, [1000, 17]), (BF, 32, 2, 64, 16, [129, 128, 127]),
    (BF, 6, 2, 96, 16, [100, 211]), (BF, 4, 4, 80, 8, [90, 1]), (BF, 8, 2, 256, 64, [70, 400]),
    (BF, 3, 1, 8, 1, [33]), (BF, 9, 1, 128, 128, [300]), (BF, 10, 2, 128, 7, [100, 50]), (BF, 2, 2, 192, 3, [65]),
    (F32, 4, 4, 64, 16, [70, 0, 300]), (F32, 6, 3, 128, 16, [65, 0, 333]), (F32, 3, 3, 256, 8, [77]),
    (F32, 4, 2, 48, 16, [300, 1]), (F32, 7, 1, 128, 32, [513]), (F32, 32, 2, 256, 64, [65, 130]),
    (F32, 2, 1, 4, 1, [9]), (F32, 12, 4, 100, 5, [64, 1]), (BF, 4, 2, 128, 64, [20000]),
]


@gpu_only
@pytest.mark.parametrize("dtype,Hq,Hk,d,page,lengths", PAGED)
def test_paged(gpu, dtype, Hq, Hk, d, page, lengths):
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, len(lengths), Hq, Hk, d, page, lengths, sum(lengths) + d)
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    want, wlse, tol, ltol = paged_ref(q, kc, vc, table, n, scale)
    within(out, want, U[dtype] * want.abs() + tol, "out")
    within(lse, wlse, ltol, "lse")
    again = api.paged_attention(q, kc, vc, table, n, scale)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@gpu_only
@pytest.mark.parametrize("dtype,B,Hq,Hk,d,page,longest,seed", [
    (BF, 400, 2, 1, 64, 16, 300, 1), (BF, 90, 4, 4, 128, 32, 900, 2), (F32, 200, 3, 1, 64, 16, 200, 3),
    (BF, 1000, 1, 1, 32, 1, 70, 4), (BF, 3, 16, 4, 256, 64, 9000, 5), (F32, 2, 5, 5, 96, 64, 4000, 6)])
def test_paged_ragged_batches(gpu, dtype, B, Hq, Hk, d, page, longest, seed):
    # pairs cut at any place, whole ones, empty sequences in a row, more CTAs than tiles and fewer
    rng = torch.Generator().manual_seed(seed)
    lengths = torch.randint(0, longest + 1, (B,), generator=rng)
    lengths[torch.rand(B, generator=rng) < 0.3] = 0
    lengths[-1] = longest
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, B, Hq, Hk, d, page, lengths.tolist(), seed)
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    want, wlse, tol, ltol = paged_ref(q, kc, vc, table, n, scale)
    within(out, want, U[dtype] * want.abs() + tol, "out")
    within(lse, wlse, ltol, "lse")


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
def test_paged_unused_cache_is_never_used(gpu, dtype):
    lengths = [0, 5, 64, 100, 129]
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, 5, 8, 2, 128, 16, lengths, 3, spare=4)
    want = api.paged_attention(q, kc, vc, table, n, scale)
    used = torch.zeros(kc.shape[0], 16, dtype=torch.bool, device=gpu)
    for b, m in enumerate(lengths):
        for j in range(m):
            used[int(table[b, j // 16]), j % 16] = True
    for bad in (float("nan"), float("inf")):
        k2 = torch.where(used[:, None, :, None], kc, torch.full_like(kc, bad))
        v2 = torch.where(used[:, None, :, None], vc, torch.full_like(vc, bad))
        got = api.paged_attention(q, k2, v2, table, n, scale)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
def test_paged_pages_outside_the_pool_and_lengths_outside_the_table(gpu, dtype):
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, 4, 4, 2, 64, 16, [100, 100, 100, 40], 8)
    table[0, 2], table[1, 0], table[2] = -1, kc.shape[0], 1 << 30
    n[0], n[3] = 1 << 30, -5
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    want, wlse, tol, ltol = paged_ref(q, kc, vc, table, n, scale)
    assert bool((want[2:] == 0).all()) and bool((wlse[2:] == -math.inf).all())
    within(out, want, U[dtype] * want.abs() + tol)
    within(lse, wlse, ltol)


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
def test_paged_large_scores_and_minus_infinity(gpu, dtype):
    # scores in the thousands (one token takes all the weight), and keys of -infinity, whose weight is zero
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, 2, 4, 2, 64, 16, [200, 77], 9)
    out, lse = api.paged_attention(q, kc, vc, table, n, 60.0)
    want, wlse, tol, ltol = paged_ref(q, kc, vc, table, n, 60.0)
    within(out, want, U[dtype] * want.abs() + tol)
    within(lse, wlse, ltol)
    q = q.abs() + 0.1
    kc[table[0, 1].long(), :, 3] = -math.inf
    kc[table[1].long()] = -math.inf                                     # nothing of sequence 1 has a weight
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    assert bool(torch.isfinite(out[0]).all()) and bool(torch.isfinite(lse[0]).all())
    assert bool((lse[1] == -math.inf).all()) and bool((out[1] == 0).all())


@gpu_only
def test_paged_lse_merges_with_another_state(gpu):
    # two halves of a cache merged by the depth aggregation's phase-2 rule give the whole
    q, kc, vc, table, n, scale = paged_inputs(gpu, F32, 1, 2, 2, 64, 16, [96], 10)
    whole, wl = api.paged_attention(q, kc, vc, table, n, scale)
    a, la = api.paged_attention(q, kc, vc, table[:, :3].contiguous(), n, scale)
    b, lb = api.paged_attention(q, kc, vc, table[:, 3:].contiguous(), n - 48, scale)
    m = torch.maximum(la, lb)
    ea, eb = torch.exp(la - m)[..., None], torch.exp(lb - m)[..., None]
    torch.testing.assert_close((ea * a + eb * b) / (ea + eb), whole, rtol=1e-5, atol=1e-5)


@gpu_only
def test_paged_graph_and_streams(gpu):
    lengths = [40, 300, 7]
    q, kc, vc, table, n, scale = paged_inputs(gpu, BF, 3, 8, 2, 128, 16, lengths, 12)
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = api.paged_attention(q, kc, vc, table, n, scale)
    graph.replay()
    assert torch.equal(go, out) and torch.equal(gl, lse)
    n.copy_(torch.tensor([1, 0, 290], device=gpu))                      # a replay follows the lengths it finds
    graph.replay()
    want = api.paged_attention(q, kc, vc, table, n, scale)
    assert torch.equal(go, want[0]) and torch.equal(gl, want[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(api.paged_attention(q, kc, vc, table, n, scale))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(x, want[1]) for o, x in got)


# --------------------------------------------------------------------------
# linear attention with a decay per head
# --------------------------------------------------------------------------
def linear_ref(q, k, v, g, scale, state=None, lengths=None):
    """Token by token in float64: (out, final state)."""
    q, k, v, g = cpu(q), cpu(k), cpu(v), cpu(g)
    B, T, H, dk = q.shape
    lam = torch.exp(g)[None, :, None, None]
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64) if state is None else cpu(state).clone()
    out = torch.zeros(B, T, H, v.shape[-1], dtype=torch.float64)
    n = torch.full((B,), T) if lengths is None else lengths.cpu().clamp(0, T)
    for t in range(T):
        on = (t < n).double()[:, None, None, None]
        S = S * (lam * on + (1 - on)) + on * k[:, t, :, :, None] * v[:, t, :, None, :]
        out[:, t] = scale * torch.einsum("bhk,bhkv->bhv", q[:, t], S) * on[..., 0]
    return out, S


def linear_inputs(gpu, dtype, B, T, H, dk, dv, seed, decay=None):
    g = wk.generator(seed, gpu)
    q, k, v = rand(g, B, T, H, dk, dtype=dtype), rand(g, B, T, H, dk, dtype=dtype), rand(g, B, T, H, dv, dtype=dtype)
    ld = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=gpu, dtype=F32) / H) if decay is None else \
        torch.full((H,), decay, device=gpu)
    return q, k, v, ld, 1 / math.sqrt(dk)


def linear_bounds(q, k, v, ld, scale, state, lengths, dtype, T, dk):
    """Bounds on out's and the state's errors from the same recurrence over absolute values.

    Every product and sum on the way is an fp32 rounding: a decay weight 4 E plus its exponent's rounding (at most
    88 E before it underflows), dk + 64 terms within a chunk, one addition per chunk.  bf16 inputs: the masked
    products and the state are rounded to bf16 (2^-8) before the product that forms out."""
    absn = lambda t: None if t is None else t.abs()  # noqa: E731
    ao, aS = linear_ref(q.abs(), k.abs(), v.abs(), ld, scale, absn(state), lengths)
    f = (dk + 64 + 100 + 2 * T / 64) * E
    return (f + (2.0 ** -8 if dtype is BF else 0.0)) * ao, f * aS


LINEAR = [  # dtype, B, T, H, dk, dv, ragged lengths or None, with a state
    (BF, 1, 1, 1, 128, 128, None, False), (BF, 2, 63, 3, 64, 64, None, True), (BF, 1, 64, 2, 128, 128, None, True),
    (BF, 1, 65, 1, 128, 64, None, False), (BF, 3, 200, 2, 64, 128, [200, 0, 77], True),
    (BF, 2, 129, 4, 96, 80, [64, 129], False), (BF, 1, 1500, 2, 128, 128, None, True),
    (BF, 2, 700, 1, 16, 24, [700, 300], True), (BF, 5, 130, 2, 8, 8, [1, 2, 128, 129, 130], True),
    # several segments of the time axis, cut sequences in some of them, an empty last segment
    (BF, 1, 2100, 2, 128, 128, None, True), (BF, 2, 1300, 3, 128, 96, [1300, 700], True),
    (BF, 2, 1000, 2, 72, 128, [100, 993], False), (BF, 40, 64, 5, 128, 128, None, False),
    # less than a chunk of 64 tokens, alone and in a batch
    (BF, 1, 2, 3, 128, 64, None, True), (BF, 7, 33, 2, 40, 128, [0, 1, 33, 32, 17, 5, 31], True),
    (BF, 1, 17, 1, 8, 16, None, False),
    # fp32 in as many segments as chunks, and in fewer
    (F32, 1, 257, 1, 128, 128, None, True), (F32, 2, 640, 2, 32, 64, [640, 65], True),
    (F32, 1, 100, 2, 128, 128, None, True), (F32, 2, 1100, 1, 64, 64, [1100, 513], True),
    (F32, 1, 70, 3, 100, 4, None, False), (F32, 3, 5, 1, 4, 12, [0, 5, 3], True),
]


@gpu_only
@pytest.mark.parametrize("dtype,B,T,H,dk,dv,lengths,with_state", LINEAR)
@pytest.mark.parametrize("decay", [None, 0.0, -3.0])
def test_linear(gpu, dtype, B, T, H, dk, dv, lengths, with_state, decay):
    q, k, v, ld, scale = linear_inputs(gpu, dtype, B, T, H, dk, dv, B + T + dk, decay)
    n = None if lengths is None else torch.tensor(lengths, device=gpu).int()
    state = rand(wk.generator(4, gpu), B, H, dk, dv, dtype=F32, scale=2.0) if with_state else None
    out, last = api.linear_attention(q, k, v, ld, scale, state=state, lengths=n)
    want, wS = linear_ref(q, k, v, ld, scale, state, n)
    to, ts = linear_bounds(q, k, v, ld, scale, state, n, dtype, T, dk)
    within(out, want, U[dtype] * want.abs() + to, "out")
    within(last, wS, ts + E * wS.abs(), "state")
    if dtype is BF and T >= 63:
        # independent roundings: the stored result, the masked products and the state, each at most 2^-8 / sqrt(3)
        # of its part in the root mean square
        rms = (cpu(out) - want).square().mean().sqrt() / want.square().mean().sqrt()
        assert float(rms) <= 2.0 ** -8, float(rms)
    alone, none = api.linear_attention(q, k, v, ld, scale, state=state, lengths=n, want_state=False)
    assert none is None and torch.equal(alone, out)
    if state is not None:                                               # the state updated in place
        _, same = api.linear_attention(q, k, v, ld, scale, state=state, lengths=n, state_out=state)
        assert same is state and torch.equal(state, last)


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay", [-100.0, -math.inf, -1e-30])
def test_linear_extreme_decays(gpu, dtype, decay):
    q, k, v, ld, scale = linear_inputs(gpu, dtype, 1, 150, 2, 64, 64, 21, decay)
    state = rand(wk.generator(4, gpu), 1, 2, 64, 64, dtype=F32)
    out, last = api.linear_attention(q, k, v, ld, scale, state=state)
    want, wS = linear_ref(q, k, v, ld, scale, state)
    to, ts = linear_bounds(q, k, v, ld, scale, state, None, dtype, 150, 64)
    within(out, want, U[dtype] * want.abs() + to)
    within(last, wS, ts + 1e-37)
    go = torch.randn_like(v)
    grads = api.linear_attention_backward(q, k, v, ld, scale, go, state=state, grad_state=torch.ones_like(state))
    assert all(bool(torch.isfinite(x).all()) for x in grads)


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,g,back", [(3000, -0.25, 5), (3000, -0.25, 400), (65536, -1.0, 150), (65536, -1.0, 165)])
def test_linear_old_large_tokens_are_not_forgotten(gpu, dtype, T, g, back):
    # one token of 1e18 among zeros: its trace in the final state, 1e36 e^{g back}, is small but no zero, also when
    # it comes from an earlier segment of the time axis, and when its weight alone is below fp32's smallest number
    q, k, v, _, scale = linear_inputs(gpu, dtype, 1, T, 1, 64, 64, 3)
    k.zero_(), v.zero_()
    k[0, T - 1 - back, 0, 3] = v[0, T - 1 - back, 0, 5] = 1e18
    ld = torch.full((1,), g, device=gpu)
    _, last = api.linear_attention(q, k, v, ld, scale)
    want = torch.zeros(1, 1, 64, 64, dtype=torch.float64)
    want[0, 0, 3, 5] = float(k[0, T - 1 - back, 0, 3].double()) * float(v[0, T - 1 - back, 0, 5].double()) * math.exp(g * back)
    # products of decays over chunks: each a rounding of its exponent (at most 64 |g| E) and of itself
    within(last, want, want.abs() * (back / 64 + 2) * (64 * abs(g) + 4) * E)


@gpu_only
def test_linear_nan_and_large_decays_stay_in_their_heads(gpu):
    q, k, v, ld, scale = linear_inputs(gpu, BF, 2, 700, 4, 64, 128, 5)
    want = api.linear_attention(q, k, v, ld, scale)
    ld[2] = float("nan")
    out, last = api.linear_attention(q, k, v, ld, scale)
    keep = [0, 1, 3]
    assert torch.equal(out[:, :, keep], want[0][:, :, keep]) and torch.equal(last[:, keep], want[1][:, keep])


@gpu_only
def test_linear_wait_that_runs_out_reports_timeout(gpu):
    """With a limit of one clock cycle the tensor-core kernels' waits give up: every role stops or runs to its end
    without waiting, the CTA drains what it has in flight, the error is reported, and the device stays usable."""
    from transformer_depth_wise_gb300 import _lib
    L = _lib.lib()
    q, k, v, ld, scale = linear_inputs(gpu, BF, 2, 2000, 4, 128, 128, 6)
    want = api.linear_attention(q, k, v, ld, scale)
    assert L.attnres_take_device_error() == 0
    assert L.attnres_set_wait_limit(1) == 0
    try:
        api.linear_attention(q, k, v, ld, scale)
        rc = L.attnres_take_device_error()
    finally:
        assert L.attnres_set_wait_limit(0) == 0
    assert rc == -9, _lib.STATUS.get(rc, rc)                              # ATTNRES_ERR_TIMEOUT
    got = api.linear_attention(q, k, v, ld, scale)
    assert L.attnres_take_device_error() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu_only
def test_linear_views_of_one_projection_and_split_prompts(gpu):
    B, T, H, d = 2, 300, 4, 64
    g = wk.generator(31, gpu)
    x = rand(g, B, T, 3 * H * d)
    q, k, v = (t.unflatten(-1, (H, d)) for t in x.split(H * d, -1))
    ld = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=gpu, dtype=F32) / H)
    out, last = api.linear_attention(q, k, v, ld, 0.125)
    o2, l2 = api.linear_attention(q.contiguous(), k.contiguous(), v.contiguous(), ld, 0.125)
    assert torch.equal(out, o2) and torch.equal(last, l2)
    # the prompt in two calls: at a chunk's border the same sums are formed in the same order but for the state's
    state, outs = None, []
    for a, b in ((0, 128), (128, 300)):
        o, state = api.linear_attention(q[:, a:b].contiguous(), k[:, a:b].contiguous(), v[:, a:b].contiguous(), ld,
                                        0.125, state=state)
        outs.append(o)
    want, wS = linear_ref(q, k, v, ld, 0.125)
    to, ts = linear_bounds(q, k, v, ld, 0.125, None, None, BF, T, d)
    within(torch.cat(outs, 1), want, U[BF] * want.abs() + to)
    within(state, wS, ts)


@gpu_only
@pytest.mark.parametrize("dtype,T", [(BF, 33), (BF, 100), (BF, 1500), (F32, 33), (F32, 300)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_linear_whatever_is_behind_the_sequences(gpu, dtype, T, bad):
    q, k, v, ld, scale = linear_inputs(gpu, dtype, 3, T, 2, 64, 72, T)
    go = rand(wk.generator(5, gpu), 3, T, 2, 72, dtype=dtype)
    state = rand(wk.generator(4, gpu), 3, 2, 64, 72, dtype=F32)
    n = torch.tensor([0, 17, T - 1], device=gpu).int()

    def run():
        out, last = api.linear_attention(q, k, v, ld, scale, state=state, lengths=n)
        return (out, last, *api.linear_attention_backward(q, k, v, ld, scale, go, state=state, lengths=n, grad_state=state))
    want = run()
    for b in range(3):
        for t in (q, k, v, go):
            t[b, int(n[b]):] = bad
    for x, y in zip(run(), want):
        assert bool(torch.isfinite(x).all()) and torch.equal(x, y)


@gpu_only
def test_linear_outputs_are_not_inputs(gpu):
    from transformer_depth_wise_gb300 import _lib
    q, k, v, ld, scale = linear_inputs(gpu, BF, 1, 70, 2, 64, 64, 1)
    state = torch.zeros(1, 2, 64, 64, device=gpu)
    for x in (q, k, v):
        with pytest.raises(_lib.AttnResError):
            api.linear_attention(q, k, v, ld, scale, out=x)
        one = x[:, 0].contiguous()
        with pytest.raises(_lib.AttnResError):
            api.linear_attention_step(one, one, one, ld, scale, state, out=one)
    assert bool((state == 0).all())


@gpu_only
def test_linear_empty(gpu):
    q, k, v, ld, scale = linear_inputs(gpu, BF, 2, 0, 3, 64, 64, 1)
    state = rand(wk.generator(4, gpu), 2, 3, 64, 64, dtype=F32)
    out, last = api.linear_attention(q, k, v, ld, scale, state=state)
    assert out.shape == (2, 0, 3, 64) and torch.equal(last, state)
    _, last = api.linear_attention(q, k, v, ld, scale)
    assert bool((last == 0).all())
    dq, dk, dv, ds = api.linear_attention_backward(q, k, v, ld, scale, v, state=state, grad_state=state)
    torch.testing.assert_close(ds, state)


def linear_grad_ref(q, k, v, ld, scale, go, state, lengths, gstate):
    """Gradients by float64 autograd through the token-by-token recurrence."""
    t = [cpu(x).requires_grad_() for x in (q, k, v)]
    s = None if state is None else cpu(state).requires_grad_()
    out, last = linear_ref_grad(*t, cpu(ld), scale, s, lengths)
    loss = (out * cpu(go)).sum()
    if gstate is not None:
        loss = loss + (last * cpu(gstate)).sum()
    wanted = t + ([s] if s is not None else [])
    return torch.autograd.grad(loss, wanted)


def linear_ref_grad(q, k, v, g, scale, state, lengths):
    B, T, H, dk = q.shape
    lam = torch.exp(g)[None, :, None, None]
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64) if state is None else state
    n = torch.full((B,), T) if lengths is None else lengths.cpu().clamp(0, T)
    rows = []
    for t in range(T):
        on = (t < n).double()[:, None, None, None]
        S = S * (lam * on + (1 - on)) + on * k[:, t, :, :, None] * v[:, t, :, None, :]
        rows.append(scale * torch.einsum("bhk,bhkv->bhv", q[:, t], S) * on[..., 0])
    return torch.stack(rows, 1), S


def test_linear_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    q, k, v, go = (torch.randn(1, 5, 2, 4, dtype=torch.float64, generator=g) for _ in range(4))
    state, gs = (torch.randn(1, 2, 4, 4, dtype=torch.float64, generator=g) for _ in range(2))
    ld, n = torch.tensor([-0.3, -0.01], dtype=torch.float64), torch.tensor([4])
    grads = linear_grad_ref(q, k, v, ld, 0.5, go, state, n, gs)
    loss = lambda *a: float((linear_ref(*a[:3], ld, 0.5, a[3], n)[0] * go).sum()  # noqa: E731
                            + (linear_ref(*a[:3], ld, 0.5, a[3], n)[1] * gs).sum())
    args = [q, k, v, state]
    for which in range(4):
        for i in range(0, args[which].numel(), 7):
            e = torch.zeros(args[which].numel(), dtype=torch.float64)
            e[i] = 1e-5
            e = e.view(args[which].shape)
            hi = loss(*[a + e if j == which else a for j, a in enumerate(args)])
            lo = loss(*[a - e if j == which else a for j, a in enumerate(args)])
            assert abs((hi - lo) / 2e-5 - float(grads[which].reshape(-1)[i])) < 1e-7


@gpu_only
@pytest.mark.parametrize("dtype,B,T,H,dk,dv,lengths,with_state", LINEAR)
def test_linear_backward(gpu, dtype, B, T, H, dk, dv, lengths, with_state):
    q, k, v, ld, scale = linear_inputs(gpu, dtype, B, T, H, dk, dv, B + T + dv)
    g = wk.generator(8, gpu)
    n = None if lengths is None else torch.tensor(lengths, device=gpu).int()
    state = rand(g, B, H, dk, dv, dtype=F32, scale=2.0) if with_state else None
    gs = rand(g, B, H, dk, dv, dtype=F32) if with_state else None
    go = rand(g, B, T, H, dv, dtype=dtype)
    got = api.linear_attention_backward(q, k, v, ld, scale, go, state=state, lengths=n, grad_state=gs)
    want = linear_grad_ref(q, k, v, ld, scale, go, state, n, gs)
    # the same recurrences over absolute values bound every term; the two roundings to bf16 as in the forward
    absn = lambda t: None if t is None else t.abs()  # noqa: E731
    mags = linear_grad_ref(q.abs(), k.abs(), v.abs(), ld, scale, go.abs(), absn(state), n, absn(gs))
    f = (max(dk, dv) + 64 + 100 + 2 * T / 64) * E
    for i, (a, b, m) in enumerate(zip(got, want, mags)):
        rounding = 2.0 ** -8 if dtype is BF and i < 3 else 0.0
        within(a, b, (U[dtype] if i < 3 else E) * b.abs() + (f + rounding) * m, "qkvs"[i])
        if dtype is BF and i < 3 and T >= 63:
            rms = (cpu(a) - b).square().mean().sqrt() / b.square().mean().sqrt()
            assert float(rms) <= 2.0 ** -8, ("qkv"[i], float(rms))
    again = api.linear_attention_backward(q, k, v, ld, scale, go, state=state, lengths=n, grad_state=gs)
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)
    if state is None:
        assert got[3] is None


@gpu_only
@pytest.mark.parametrize("dtype,B,H,dk,dv", [(BF, 4, 16, 128, 128), (BF, 1, 1, 64, 64), (BF, 300, 3, 96, 80),
                                             (F32, 5, 2, 100, 4), (BF, 2, 3, 8, 128), (F32, 400, 1, 128, 64)])
def test_linear_step(gpu, dtype, B, H, dk, dv):
    q, k, v, ld, scale = linear_inputs(gpu, dtype, B, 1, H, dk, dv, B + dk)
    state = rand(wk.generator(4, gpu), B, H, dk, dv, dtype=F32, scale=3.0)
    want, wS = linear_ref(q, k, v, ld, scale, state)
    ao, aS = linear_ref(q.abs(), k.abs(), v.abs(), ld, scale, state.abs())
    new = torch.empty_like(state)
    out = api.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], ld, scale, state, state_out=new)
    within(out, want[:, 0], U[dtype] * want[:, 0].abs() + (dk + 10) * E * ao[:, 0])
    within(new, wS, 5 * E * aS)
    again = api.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], ld, scale, state)
    assert torch.equal(again, out) and torch.equal(state, new)          # in place


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------
@gpu_only
def test_decode_layer(gpu):
    """Two sublayers of a hybrid layer between two fused merges, for several tokens: the pre-normed input of the
    fused step goes through a projection, norm and rotation into the cache, paged attention and an output
    projection, whose result is the next fused step's sublayer output; then the same with a linear attention."""
    B, Hq, Hk, d, D, page, steps = 5, 4, 2, 64, 256, 16, 19
    g = wk.generator(77, gpu)
    wqkv = rand(g, D, (Hq + 2 * Hk) * d, scale=D ** -0.5)
    wlin, wo = rand(g, D, 3 * Hq * d, scale=D ** -0.5), rand(g, Hq * d, D, scale=(Hq * d) ** -0.5)
    hq, hk = 1 + rand(g, d, dtype=F32, scale=0.1), 1 + rand(g, d, dtype=F32, scale=0.1)
    nw = 1 + rand(g, D, dtype=F32, scale=0.1)
    query, gain = wk.queries_and_gains(g, 1, D, gpu)
    fr = api.rotary_frequencies(d, device=gpu)
    per = 4
    table = torch.randperm(B * per, device=gpu, generator=g).view(B, per).int()
    kc, vc = (torch.full((B * per, Hk, page, d), float("nan"), dtype=BF, device=gpu) for _ in range(2))
    state = torch.zeros(B, Hq, d, d, dtype=F32, device=gpu)
    ld = -torch.exp2(-2.0 * torch.arange(1, Hq + 1, device=gpu, dtype=F32))
    keys, vals, S64 = [], [], torch.zeros(B, Hq, d, d, dtype=torch.float64)
    A64 = torch.zeros_like(S64)
    for t in range(steps):
        inter, lse = rand(g, B, 1, D), rand(g, B, 1, dtype=F32)
        sub = rand(g, B, 1, D)
        partial, h, y = api.block_merge_update(inter, lse, None, sub, None, query[0], gain[0], norm_weight=nw)
        qkv = (y.view(B, D) @ wqkv).view(B, 1, -1)
        q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hk * d, Hk * d], -1))
        pos = torch.full((B, 1), t, device=gpu).int()
        qr = api.head_norm_rotate_append(q, k, v, hq, hk, pos, fr, kc, vc, table, EPS)
        n = torch.full((B,), t + 1, device=gpu).int()
        att, _ = api.paged_attention(qr.view(B, Hq, d), kc, vc, table, n, d ** -0.5)
        sub2 = (att.view(B, -1) @ wo).view(B, 1, D)
        partial, h, y2 = api.block_merge_update(inter, lse, partial, sub2, None, query[0], gain[0], norm_weight=nw)
        ql, kl, vl = (x.view(B, Hq, d) for x in (y2.view(B, D) @ wlin).split(Hq * d, -1))
        lin = api.linear_attention_step(ql, kl, vl, ld, d ** -0.5, state)
        # float64 from the same projections
        keys.append(rotate_ref(k, hk, pos, fr, False)[0][:, 0])
        vals.append(cpu(v)[:, 0])
        q64 = rotate_ref(q, hq, pos, fr, False)[0][:, 0]
        K, V = torch.stack(keys, 2).repeat_interleave(Hq // Hk, 1), torch.stack(vals, 2).repeat_interleave(Hq // Hk, 1)
        p = torch.softmax(torch.einsum("bhd,bhtd->bht", q64, K) * d ** -0.5, -1)
        want = torch.einsum("bht,bhtd->bhd", p, V)
        # q and k stored in bf16 shift a score by at most 2 * 2^-8 of its absolute sum (below 2 sqrt(d) here by
        # Cauchy-Schwarz with head norms of at most 1.4 sqrt(d)), which moves a weight by twice that
        shift = 2 * 2 * 2.0 ** -8 * 2 * math.sqrt(d)
        within(att, want, 2.0 ** -8 * want.abs() + shift * torch.einsum("bht,bhtd->bhd", p, V.abs()))
        S64 = S64 * torch.exp(cpu(ld))[:, None, None] + cpu(kl)[..., None] * cpu(vl)[..., None, :]
        # the stored result is rounded by at most 2^-8 of itself whatever its size (a value of 16 by 2^-4, so a fixed
        # bound for values up to 8 does not hold); d products and t + 1 updates of fp32 in units of the absolute sum
        A64 = A64 * torch.exp(cpu(ld))[:, None, None] + cpu(kl).abs()[..., None] * cpu(vl).abs()[..., None, :]
        wl = torch.einsum("bhk,bhkv->bhv", cpu(ql), S64) * d ** -0.5
        al = torch.einsum("bhk,bhkv->bhv", cpu(ql).abs(), A64) * d ** -0.5
        within(lin, wl, 2.0 ** -8 * wl.abs() + (d + 10 + 4 * (t + 1)) * E * al)
    within(state, S64, 4 * steps * E * A64)


@gpu_only
def test_prompt_then_tokens(gpu):
    """A prompt through linear_attention and its last tokens through the step: the same as the whole prompt."""
    q, k, v, ld, scale = linear_inputs(gpu, BF, 2, 90, 3, 64, 128, 55)
    want, wS = linear_ref(q, k, v, ld, scale)
    to, ts = linear_bounds(q, k, v, ld, scale, None, None, BF, 90, 64)
    _, state = api.linear_attention(q[:, :80].contiguous(), k[:, :80].contiguous(), v[:, :80].contiguous(), ld, scale)
    for t in range(80, 90):
        out = api.linear_attention_step(q[:, t], k[:, t], v[:, t], ld, scale, state)
        within(out, want[:, t], U[BF] * want[:, t].abs() + to[:, t])
    within(state, wS, 2 * ts)


@gpu_only
def test_all_captured_and_on_another_stream(gpu):
    """Every operator in one captured graph, and on a side stream, gives the eager results bit for bit."""
    q, k, v, wq, wk_, pos, fr = norm_inputs(gpu, BF, 2, 70, 4, 4, 64, 64, 61)
    ld = torch.full((4,), -0.1, device=gpu)
    go = torch.randn(2, 70, 4, 64, device=gpu).to(BF)

    def everything():
        qr, kr = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS)
        o, s = api.linear_attention(qr, kr, v, ld, 0.125)
        dq, dk, dv, _ = api.linear_attention_backward(qr, kr, v, ld, 0.125, go)
        return (qr, kr, o, s, dq, dk, dv) + api.head_norm_rotate_backward(q, k, wq, wk_, pos, fr, EPS, dq, dk)

    want = everything()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = everything()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = everything()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
