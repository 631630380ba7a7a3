"""Attention of one new token per sequence behind a shared prefix, against a plain float64 form, and a serving layer's
operators in a row.

Tolerances are bounds, not fits.  u is the rounding of a stored result (half a step: 2^-8 relative for bf16, 2^-24 for
fp32); every other term counts the roundings on the way, as the comment at each check says (E = 2^-24).
"""
import math

import pytest
import torch

from transformer_depth_wise_gb300 import _lib, api
from transformer_depth_wise_gb300 import workloads as wk

gpu_only = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
E = 2.0 ** -24
FAKE = 0x7F0000000000      # 16-byte aligned stand-in for a device pointer (never dereferenced)
OK, NULL, SHAPE, DTYPE, ALIGN, CAP, VALUE = 0, -1, -2, -3, -4, -7, -8


def cpu(t):
    return t.detach().cpu().double()


def within(got, want, tol, what=""):
    got, want = cpu(got), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: finite in different places"
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), what
    d = torch.where(fine, (got - want).abs() - tol, torch.full_like(want, -1.0))
    assert d.numel() == 0 or float(d.max()) <= 0.0, f"{what}: over the bound by {float(d.max()):.3e}"


def rand(g, *shape, dtype=BF, scale=1.0):
    return (torch.empty(shape, dtype=F32, device=g.device).normal_(generator=g) * scale).to(dtype)


def tokens_of(table, n, page, pool):
    """Pages and slots of the first n tokens of a table's row, those on pages outside the pool left out."""
    j = torch.arange(min(max(int(n), 0), table.numel() * page))
    pg = table.cpu().long()[j // page] if len(j) else j
    ok = (pg >= 0) & (pg < pool)
    return pg[ok], (j % page)[ok]


def shared_ref(q, kc, vc, prefix_table, prefix, table, lengths, scale, coarse):
    """(out, lse, bound on out's error before its last rounding, the same of lse) in float64; `coarse`: the rounding of
    the prefix's weights on their way into the product with the values."""
    q, kc, vc = cpu(q), cpu(kc), cpu(vc)
    B, Hq, d = q.shape
    N, Hk, page, _ = kc.shape
    G = Hq // Hk
    out, lse = torch.zeros_like(q), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(q), torch.zeros(B, Hq, dtype=torch.float64)
    fp, fs = tokens_of(prefix_table, int(prefix), page, N)
    for hk in range(Hk):
        kp, vp = kc[fp, hk, fs], vc[fp, hk, fs]
        for b in range(B):
            op, os_ = tokens_of(table[b], int(lengths[b]), page, N)
            k, v = torch.cat((kp, kc[op, hk, os_])), torch.cat((vp, vc[op, hk, os_]))
            n, h = len(k), slice(hk * G, hk * G + G)
            if n == 0:
                continue
            qh = q[b, h]
            s = qh @ k.T * scale
            p = torch.softmax(s, -1)
            out[b, h], lse[b, h] = p @ v, torch.logsumexp(s, -1)
            # a score is a sum of d products: d roundings of its absolute sum; the exponential's argument and value
            # 16 E + |s - max| E, once more at the join; sums over n tokens in at least eight strands; the own tokens'
            # weights enter the second product with 16 bits or more (2^-17), the prefix's with `coarse`
            ds = (d + 2) * E * (qh.abs() @ k.abs().T).amax(-1) * abs(scale)
            ds = ds + 4 * E * (s.amax(-1) - s.amin(-1)) + (32 + n / 8) * E
            tol[b, h] = (2 * ds[:, None] + 2.0 ** -17) * (p @ v.abs()) + coarse * (p[:, :len(kp)] @ vp.abs())
            ltol[b, h] = ds + 2 * E * lse[b, h].abs()
    return out, lse, tol, ltol


def inputs(dev, dtype, Hq, Hk, d, page, prefix, lengths, seed, spare=0):
    g = wk.generator(seed, dev)
    B = len(lengths)
    first, per = -(-prefix // page) + spare, max(1, -(-max(lengths) // page)) + spare
    pool = first + B * per + 1
    pages = torch.randperm(first + B * per, device=dev, generator=g).int()
    q = rand(g, B, Hq, d, dtype=dtype, scale=1.5)
    kc, vc = rand(g, pool, Hk, page, d, dtype=dtype), rand(g, pool, Hk, page, d, dtype=dtype)
    return [q, kc, vc, pages[:first].contiguous(), torch.tensor([prefix], device=dev).int(),
            pages[first:].view(B, per).contiguous(), torch.tensor(lengths, device=dev).int(), 1 / math.sqrt(d)]


def coarse_of(dtype, d):
    return 2.0 ** -8 if dtype is BF else 0.0           # the prefix's weights in bf16 are off by half a step


def check(args, dtype, d, what=""):
    out, lse = api.shared_prefix_attention(*args)
    want, wlse, tol, ltol = shared_ref(*args, coarse_of(dtype, d))
    within(out, want, U[dtype] * want.abs() + tol, what + " out")
    within(lse, wlse, ltol, what + " lse")
    again = api.shared_prefix_attention(*args)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    return out, lse


CASES = [  # dtype, Hq, Hk, d, page, prefix, lengths
    (BF, 1, 1, 128, 16, 1, [1]), (BF, 16, 16, 128, 16, 1111, [0, 100, 37, 1]), (BF, 8, 2, 64, 32, 127, [5, 0, 31]),
    (BF, 56, 8, 128, 64, 1000, [0, 1, 63, 64, 65, 300]), (BF, 16, 1, 128, 64, 129, list(range(17))),
    (BF, 32, 2, 64, 16, 700, [i % 5 for i in range(40)]), (BF, 6, 2, 96, 16, 257, [3, 200]),
    (BF, 4, 4, 80, 8, 90, [9, 1]), (BF, 8, 2, 256, 64, 300, [70, 5]), (BF, 3, 1, 8, 1, 33, [2]),
    (BF, 9, 1, 128, 128, 384, [3, 0, 7]), (BF, 10, 2, 128, 7, 500, [10, 50]), (BF, 2, 2, 192, 3, 65, [3, 65]),
    (BF, 14, 2, 128, 16, 2049, [1] * 37), (BF, 2, 1, 40, 16, 1030, [4] * 130), (BF, 4, 2, 128, 64, 20000, [20, 1]),
    (BF, 7, 1, 128, 32, 128, [6] * 300), (F32, 4, 4, 64, 16, 70, [0, 300]), (F32, 6, 3, 128, 16, 333, [65, 0, 3]),
    (F32, 3, 3, 256, 8, 77, [5]), (F32, 8, 2, 64, 32, 1025, [7] * 33), (F32, 7, 1, 128, 32, 513, [1] * 19),
    (F32, 2, 1, 4, 1, 9, [1]), (F32, 12, 4, 100, 5, 64, [64, 1]), (F32, 16, 1, 192, 64, 200, [1] * 9),
]


@gpu_only
@pytest.mark.parametrize("dtype,Hq,Hk,d,page,prefix,lengths", CASES)
def test_shared(gpu, dtype, Hq, Hk, d, page, prefix, lengths):
    check(inputs(gpu, dtype, Hq, Hk, d, page, prefix, lengths, prefix + d), dtype, d)


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("prefix,lengths", [(0, [5, 0, 17]), (0, [0, 0]), (200, [0, 0, 0]), (1, [0]), (64, [64, 1])])
def test_empty_parts(gpu, dtype, prefix, lengths):
    # tables that cover more than the lengths say, a prefix of no tokens with a table and without one
    a = inputs(gpu, dtype, 8, 2, 64, 16, prefix, lengths, 3, spare=2)
    out, lse = check(a, dtype, 64)
    if prefix == 0:
        a[3] = a[3][:0].contiguous()
        none = api.shared_prefix_attention(*a)
        alone = api.paged_attention(a[0], a[1], a[2], a[5], a[6], a[7])
        assert torch.equal(none[0], out)
        within(none[0], cpu(alone[0]), 2 * U[dtype] * cpu(alone[0]).abs())
        within(none[1], cpu(alone[1]), 4 * E * cpu(alone[1]).abs().clamp_min(1))
    a[5] = a[5][:, :0].contiguous()                  # no own pages at all
    a[6] = a[6] * 0
    check(a, dtype, 64)
    a[4] = a[4] * 0 - 5                              # lengths below zero and behind the tables
    a[6] = a[6] - 1
    out, lse = check(a, dtype, 64)
    assert not bool(out.any()) and bool((lse == -math.inf).all())
    if a[3].numel():
        a[4] = a[4] * 0 + 10 ** 6
        check(a, dtype, 64)


@gpu_only
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 256), (F32, 64)])
def test_empty_pool_and_empty_batch(gpu, dtype, d):
    q, kc, vc, pt, n, t, lengths, scale = inputs(gpu, dtype, 4, 2, d, 16, 200, [20, 5], 2)
    out, lse = api.shared_prefix_attention(q, kc[:0], vc[:0], pt, n, t, lengths, scale)
    assert not bool(out.any()) and bool((lse == -math.inf).all())
    out, lse = api.shared_prefix_attention(q[:0], kc, vc, pt, n, t[:0], lengths[:0], scale)
    assert out.shape == (0, 4, d) and lse.shape == (0, 4)


@gpu_only
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 256), (F32, 64)])
def test_one_cache_or_two(gpu, dtype, d):
    # a prefix of whole pages in front of each sequence's own table is the same attention
    q, kc, vc, pt, n, t, lengths, scale = inputs(gpu, dtype, 8, 2, d, 16, 160, [0, 1, 16, 100, 33], 5)
    out, lse = api.shared_prefix_attention(q, kc, vc, pt, n, t, lengths, scale)
    whole = torch.cat((pt.expand(5, -1), t), 1).contiguous()
    want, wlse = api.paged_attention(q, kc, vc, whole, lengths + 160, scale)
    _, _, tol, ltol = shared_ref(q, kc, vc, pt, n, t, lengths, scale, coarse_of(dtype, d))
    within(out, cpu(want), 2 * U[dtype] * cpu(want).abs() + 2 * tol)
    within(lse, cpu(wlse), 2 * ltol)


@gpu_only
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 256), (F32, 64)])
def test_unused_cache_and_bad_pages(gpu, dtype, d):
    a = inputs(gpu, dtype, 6, 2, d, 16, 300, [33, 0, 5, 47], 7)
    q, kc, vc, pt, n, t, lengths, _ = a
    pt[3], pt[7], t[0, 1] = -1, kc.shape[0], kc.shape[0] + 5        # pages outside the pool are left out
    used = torch.zeros(kc.shape[0], 16, dtype=torch.bool)
    for table, count in ((pt, 300), *((t[b], int(lengths[b])) for b in range(4))):
        pg, sl = tokens_of(table, count, 16, kc.shape[0])
        used[pg, sl] = True
    want = api.shared_prefix_attention(*a)
    check(a, dtype, d)
    for fill in (math.nan, math.inf, -math.inf):
        mask = (~used).to(gpu)[:, None, :, None]
        kc.masked_fill_(mask, fill)
        vc.masked_fill_(mask, fill)
        got = api.shared_prefix_attention(*a)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    pt.fill_(-1)                                                     # nothing of the prefix is left
    kc, vc = kc.nan_to_num(0.5, 0.5, 0.5), vc.nan_to_num(0.5, 0.5, 0.5)
    check([q, kc, vc, *a[3:]], dtype, d)


@gpu_only
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 256), (F32, 64)])
def test_what_is_no_number(gpu, dtype, d):
    a = inputs(gpu, dtype, 8, 2, d, 16, 400, [20, 3, 0], 9)
    q, kc, vc, pt, _, t, _, _ = a
    k0, v0, want = kc.clone(), vc.clone(), api.shared_prefix_attention(*a)

    def reset():
        kc.copy_(k0)
        vc.copy_(v0)

    heads = torch.arange(8, device=gpu) // 4 == 1
    kc[pt[12], 1, 3, 2] = math.nan                                   # a key of the prefix: its key head's queries, all rows
    out, lse = api.shared_prefix_attention(*a)
    assert torch.equal(lse.isnan(), heads.expand(3, 8)) and torch.equal(out.isnan().all(-1), heads.expand(3, 8))
    assert torch.equal(out[:, :4], want[0][:, :4])
    reset()
    vc[pt[5], 0, 7, 9] = math.nan                                    # a value: one element of its head's queries
    out, lse = api.shared_prefix_attention(*a)
    bad = torch.zeros(3, 8, d, dtype=torch.bool, device=gpu)
    bad[:, :4, 9] = True
    assert torch.equal(out.isnan(), bad) and torch.equal(lse, want[1])
    reset()
    vc[pt[5], 0, 7, 9] = math.inf
    out, lse = api.shared_prefix_attention(*a)
    assert torch.equal(~out.isfinite(), bad) and torch.equal(lse, want[1])
    reset()
    q0 = q.clone()
    q[1, 3, 0] = math.nan                                            # a query: its row alone
    out, lse = api.shared_prefix_attention(*a)
    bad = torch.zeros(3, 8, dtype=torch.bool, device=gpu)
    bad[1, 3] = True
    assert torch.equal(lse.isnan(), bad) and torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad)
    q.copy_(q0)
    kc[t[0, 0], 0, 2, 1] = math.nan                                  # an own key: its sequence alone
    out, lse = api.shared_prefix_attention(*a)
    bad = torch.zeros(3, 8, dtype=torch.bool, device=gpu)
    bad[0, :4] = True
    assert torch.equal(lse.isnan(), bad) and torch.equal(out[1:], want[0][1:])
    reset()
    q[:, :, :] = q.abs() + 0.1                                       # keys at minus infinity take no part
    gone = torch.arange(0, 400, 3)
    kc[pt.cpu().long()[gone // 16], :, gone % 16] = -math.inf
    out, lse = api.shared_prefix_attention(*a)
    kept = torch.ones(400, dtype=torch.bool)
    kept[gone] = False
    reset()
    pages, slots = pt.cpu().long()[torch.arange(400) // 16][kept], (torch.arange(400) % 16)[kept]
    for b in range(3):
        op, os_ = tokens_of(t[b], int(a[6][b]), 16, kc.shape[0])
        for hk in range(2):
            k = cpu(torch.cat((kc[pages, hk, slots], kc[op, hk, os_])))
            s = cpu(q[b, hk * 4:hk * 4 + 4]) @ k.T * a[7]
            # as shared_ref's bound on lse, with scores below 64 in size
            within(lse[b, hk * 4:hk * 4 + 4], torch.logsumexp(s, -1), (d + 2) * E * 64 + 4 * E * 128 + 90 * E)


@gpu_only
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 256), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("prefix,own", [(100, 40), (4000, 40), (100, 3000), (20000, 5000)])
def test_infinity_behind_a_weight_that_is_too_small(gpu, dtype, d, prefix, own):
    """Values that are no numbers show however far their token's score lies below the others', in whichever part."""
    for far in ("prefix", "own"):
        a = inputs(gpu, dtype, 4, 2, d, 16, prefix, [own, own // 2, own], 70)
        q, kc, vc, pt, n, t, lengths, _ = a
        q.copy_(q.abs() + 0.5)                       # scores of some +-8 sqrt(d): more than e^-100 apart
        low, high = (pt, t.flatten()) if far == "prefix" else (t.flatten(), pt)
        kc[low.long()], kc[high.long()] = -8.0, 8.0
        if far == "prefix":
            vc[pt[3], 0, 5, 9], vc[pt[2], 1, 0, 4] = math.inf, math.nan
            rows = [0, 1, 2]
        else:
            vc[t[1, 0], 0, 5, 9], vc[t[1, 1], 1, 0, 4] = math.inf, math.nan
            rows = [1]
        out, lse = api.shared_prefix_attention(*a)
        bad = torch.zeros(3, 4, d, dtype=torch.bool, device=gpu)
        for b in rows:
            bad[b, :2, 9] = bad[b, 2:, 4] = True
        assert torch.equal(~out.isfinite(), bad), far
        assert bool(lse.isfinite().all())
        # the same of one cache
        whole = torch.cat((pt.expand(3, -1), t), 1).contiguous()
        if prefix % 16 == 0:
            out, _ = api.paged_attention(q, kc, vc, whole, lengths + prefix, a[7])
            assert torch.equal(~out.isfinite(), bad), far


@gpu_only
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 256), (F32, 64)])
def test_rising_and_large_scores(gpu, dtype, d):
    # the maximum rises from tile to tile, then falls; and scores far apart
    for seed, order in ((1, 1), (2, -1), (3, 0)):
        a = inputs(gpu, dtype, 4, 1, d, 16, 1500, [40] * 40, seed)
        q, kc, pt = a[0], a[1], a[3]
        q.copy_(q.abs())
        up = torch.linspace(-4, 4, 1500, device=gpu)
        up = up if order > 0 else up.flip(0) if order < 0 else torch.where(torch.arange(1500, device=gpu) % 500 == 77, 12.0, -3.0)
        j = torch.arange(1500, device=gpu)
        kc[pt.long()[j // 16], 0, j % 16] = (kc[pt.long()[j // 16], 0, j % 16].float() * 0.1 + up[:, None]).to(dtype)
        check(a, dtype, d, f"order {order}")


def ranges_of(dev, dtype, B, Hq, Hk, d, page, pages):
    """Ranges that a call without own pages cuts the prefix into: each adds its outputs and lse to the workspace."""
    size = lambda n: api._sized("attnres_shared_prefix_attention_workspace_bytes", dev, B, Hq, Hk, d,  # noqa: E731
                                api._CODES[dtype], page, n, 0)
    part, over = divmod(size(pages) - size(0), 4 * B * Hq * (d + 1))
    assert over == 0 and B * Hq % 4 == 0
    return part


def prefix_ref(q, kc, vc, fp, fs, scale, coarse):
    """shared_ref for a prefix alone, in float64 on the GPU; fp, fs: its tokens' pages and slots."""
    B, Hq, d = q.shape
    Hk, n = kc.shape[1], len(fp)
    parts = []
    for hk in range(Hk):
        k, v = kc[fp, hk, fs].double(), vc[fp, hk, fs].double()
        rows = q.unflatten(1, (Hk, -1))[:, hk].flatten(0, 1).double()
        x = rows @ k.T * scale
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[:, None])
        size = p @ v.abs()
        ds = (d + 2) * E * (rows.abs() @ k.abs().T).amax(-1) * abs(scale)
        ds = ds + 4 * E * (x.amax(-1) - x.amin(-1)) + (32 + n / 8) * E
        o = p @ v
        tol = (2 * ds[:, None] + 2.0 ** -17 + coarse) * size
        parts.append([t.unflatten(0, (B, -1)) for t in (o, lse, tol, ds + 2 * E * lse.abs())])
    return [torch.stack(t, 1).flatten(1, 2).cpu() for t in zip(*parts)]


@gpu_only
@pytest.mark.parametrize("pattern", ["random", "rising", "falling", "slowly rising", "spikes", "gaps"])
@pytest.mark.parametrize("dtype,d,B,G,tile", [(BF, 64, 3, 2, 128), (BF, 64, 150, 1, 128), (BF, 128, 4, 3, 128), (BF, 128, 50, 4, 128),
                                              (BF, 96, 41, 4, 128), (BF, 256, 2, 1, 64), (BF, 256, 33, 3, 64),
                                              (F32, 64, 3, 2, 64), (F32, 128, 20, 4, 64), (F32, 256, 2, 1, 64)])
def test_many_steps_in_one_range(gpu, dtype, d, B, G, tile, pattern):
    """So many key heads that a range has 20 steps and more: references, maxima and sums go on from step to step, and
    every ring's places are used again and again."""
    many_steps(gpu, dtype, d, B, G, tile, pattern, 16)


@gpu_only
@pytest.mark.parametrize("pattern", ["rising", "spikes", "gaps"])
@pytest.mark.parametrize("dtype,d,B,G,tile", [(BF, 64, 150, 1, 128), (BF, 128, 50, 4, 128), (BF, 72, 9, 2, 128), (BF, 256, 5, 4, 64),
                                              (F32, 64, 3, 2, 64)])
@pytest.mark.parametrize("page", [128, 64, 32, 12])
def test_many_steps_over_other_pages(gpu, dtype, d, B, G, tile, pattern, page):
    """Pages that hold a warp's tokens of a step side by side, and pages that end inside them."""
    many_steps(gpu, dtype, d, B, G, tile, pattern, page)


def many_steps(gpu, dtype, d, B, G, tile, pattern, page):
    Hk = 136
    steps = 45 if dtype is F32 and d == 64 else 23
    prefix = steps * tile - 37                                       # the last step is a partial one
    g = wk.generator(50, gpu)
    pages = -(-prefix // page)
    if torch.cuda.get_device_properties(gpu).multi_processor_count == 152:
        assert steps // ranges_of(gpu, dtype, B, G * Hk, Hk, d, page, pages) >= 20
    pt = torch.randperm(pages, device=gpu, generator=g).int()
    q = rand(g, B, G * Hk, d, dtype=dtype, scale=1.5).abs()
    kc, vc = rand(g, pages, Hk, page, d, dtype=dtype), rand(g, pages, Hk, page, d, dtype=dtype)
    j = torch.arange(pages * page, device=gpu)
    # a query's product with one key is some 1.2 sqrt(d) times what is added to the key's elements: 9 to 19 here
    if pattern == "random":
        up = None
    elif pattern in ("rising", "falling"):                           # by 70 to 150 in all, a few powers of two per step
        up = torch.linspace(-4, 4, pages * page, device=gpu) * (1 if pattern == "rising" else -1)
    elif pattern == "slowly rising":                                 # the weights pass the reference, mostly within 2^10
        up = torch.linspace(0, 0.8, pages * page, device=gpu)
    elif pattern == "spikes":                                        # alone by hundreds of powers of two, each above the last
        up = torch.full((pages * page,), -3.0, device=gpu)
        for i, at in enumerate((5 * tile + 3, 11 * tile + tile // 2, 11 * tile + tile // 2 + 1, prefix - 1)):
            up[at] = 6.0 + 6 * i
    else:                                                            # the first steps, one in the middle and parts of others on no page
        up = torch.linspace(-2, 2, pages * page, device=gpu)
        pt[:2 * tile // page + 1] = -1
        pt[9 * tile // page:10 * tile // page + 1] = pages
        pt[12 * tile // page + 1:max(14 * tile // page - 1, 12 * tile // page + 2)] = -7
    if up is not None:
        at = pt.long()[j // page]
        ok = at >= 0
        ok &= at < pages
        kc[at[ok], :, (j % page)[ok]] = (kc[at[ok], :, (j % page)[ok]].float() * 0.1 + up[ok, None, None]).to(dtype)
    a = [q, kc, vc, pt, torch.tensor([prefix], device=gpu).int(), torch.empty(B, 0, device=gpu, dtype=torch.int32),
         torch.zeros(B, device=gpu, dtype=torch.int32), d ** -0.5]
    out, lse = api.shared_prefix_attention(*a)
    want, wlse, tol, ltol = prefix_ref(q, kc, vc, *(t.to(gpu) for t in tokens_of(pt, prefix, page, pages)), a[7],
                                       coarse_of(dtype, d))
    within(out, want, U[dtype] * want.abs() + tol, "out")
    within(lse, wlse, ltol, "lse")
    again = api.shared_prefix_attention(*a)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@gpu_only
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 256), (F32, 64)])
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_scales_that_are_not_positive(gpu, dtype, d, scale):
    # the largest weight is the lowest product's; with none, every token weighs the same
    a = inputs(gpu, dtype, 12, 2, d, 16, 300, [0, 3, 70, 1] * 12, 23)
    a[7] = scale
    check(a, dtype, d)


@gpu_only
@pytest.mark.parametrize("seed", range(12))
def test_ragged_batches(gpu, seed):
    g = torch.Generator().manual_seed(100 + seed)
    pick = lambda *x: x[int(torch.randint(0, len(x), (1,), generator=g))]  # noqa: E731
    dtype, d, Hk, G, page = pick(BF, BF, F32), pick(64, 128, 128, 72, 16, 256), pick(1, 2, 5), pick(1, 2, 7, 16), pick(1, 16, 24, 64)
    B = int(torch.randint(1, 70, (1,), generator=g))
    prefix = int(torch.randint(1, 1800, (1,), generator=g))
    lengths = [int(x) for x in torch.randint(0, 90, (B,), generator=g)]
    check(inputs(gpu, dtype, G * Hk, Hk, d, page, prefix, lengths, seed), dtype, d)


@gpu_only
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B", [1, 31, 33, 63, 97, 127, 129, 161, 191, 255, 257])
def test_warps_partly_behind_the_batch(gpu, d, B):
    # B rows per key head: in one warp of a tile some lanes have a row and others none
    check(inputs(gpu, BF, 2, 2, d, 16, 150, [b % 3 for b in range(B)], 40 + B), BF, d)


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
def test_cache_offsets_past_32_bits(gpu, dtype):
    """Pages whose elements and bytes lie behind 2^31 and 2^32."""
    Hk, page, d, B = 2, 64, 128, 5
    pool = 2 ** 32 // (Hk * page * d) + 40
    q, kc, vc, pt, n, t, lengths, scale = inputs(gpu, dtype, 8, Hk, d, page, 700, [100, 0, 64, 1, 128], 90)
    size = pt.numel() + t.numel()
    far_k, far_v = (torch.empty(pool, Hk, page, d, device=gpu, dtype=dtype) for _ in range(2))
    # the same pages at the pool's end, and some about the borders
    at = torch.arange(pool - size, pool, device=gpu)
    at[:4] = torch.tensor([2 ** 31 // (Hk * page * d) - 1, 2 ** 31 // (Hk * page * d), 2 ** 32 // (Hk * page * d) - 1, 0], device=gpu)
    far_k[at], far_v[at] = kc[:size], vc[:size]
    got = api.shared_prefix_attention(q, far_k, far_v, at[pt.long()].int(), n, at[t.long()].int(), lengths, scale)
    want = api.shared_prefix_attention(q, kc, vc, pt, n, t, lengths, scale)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu_only
def test_strided_and_broadcast_queries(gpu):
    q, kc, vc, pt, n, t, lengths, scale = inputs(gpu, BF, 8, 2, 128, 16, 300, [5, 9, 0, 20], 4)
    wide = torch.zeros(4, 24 * 128, device=gpu, dtype=BF)
    wide[:, 8 * 128:16 * 128] = q.flatten(1)
    view = wide[:, 8 * 128:16 * 128].unflatten(1, (8, 128))
    want = api.shared_prefix_attention(q, kc, vc, pt, n, t, lengths, scale)
    got = api.shared_prefix_attention(view, kc, vc, pt, n, t, lengths, scale)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    same = q[:1].expand(4, 8, 128)                                   # one query for all
    got = api.shared_prefix_attention(same, kc, vc, pt, n, t, lengths, scale)
    want = api.shared_prefix_attention(same.contiguous(), kc, vc, pt, n, t, lengths, scale)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu_only
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_graph_with_growing_lengths_and_two_streams(gpu, dtype, d):
    a = inputs(gpu, dtype, 8, 2, d, 16, 500, [40, 3, 17], 6, spare=3)
    n, lengths = a[4], a[6]
    full = n.clone(), lengths.clone()
    need = api._sized("attnres_shared_prefix_attention_workspace_bytes", gpu, 3, 8, 2, d, api._CODES[dtype], 16,
                      a[3].numel(), a[5].shape[1])
    ws = [torch.full((need,), 255, device=gpu, dtype=torch.uint8) for _ in range(2)]
    sides = [torch.cuda.Stream(gpu) for _ in range(2)]
    graphs, outs = [], []
    for w, s in zip(ws, sides):
        s.wait_stream(torch.cuda.current_stream(gpu))
        with torch.cuda.stream(s):
            api.shared_prefix_attention(*a, workspace=w)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                outs.append(api.shared_prefix_attention(*a, workspace=w))
            graphs.append(graph)
    torch.cuda.synchronize()
    for step in range(3):                                            # the lengths on the device decide
        n.copy_(full[0] - 200 * step)
        lengths.copy_((full[1] + 5 * step) * (step != 1))
        torch.cuda.synchronize()
        for graph, s in zip(graphs, sides):                          # side by side, a workspace each
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        want = api.shared_prefix_attention(*a)
        for got in outs:
            assert all(torch.equal(x, y) for x, y in zip(got, want))


@gpu_only
@pytest.mark.parametrize("d", [64, 128, 256])
def test_wait_that_runs_out_reports_timeout(gpu, d):
    a = inputs(gpu, BF, 8, 2, d, 16, 3000, [20] * 40, 11)
    lib = _lib.lib()
    want = api.shared_prefix_attention(*a)
    assert lib.attnres_take_device_error() == 0
    try:
        assert lib.attnres_set_wait_limit(1) == 0
        api.shared_prefix_attention(*a)
        assert lib.attnres_take_device_error() == -9                 # and the flag is cleared
    finally:
        lib.attnres_set_wait_limit(0)
    got = api.shared_prefix_attention(*a)
    assert lib.attnres_take_device_error() == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@gpu_only
def test_two_calls_at_once_and_many_in_a_row(gpu):
    """Eager calls on two streams side by side, and calls whose kernels overlap the next call's."""
    cases = [inputs(gpu, BF, 16, 2, 128, 16, 2000 + 500 * k, [50 + k] * 30, 20 + k) for k in range(2)]
    want = [api.shared_prefix_attention(*a) for a in cases]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(gpu) for _ in range(2)]
    for _ in range(20):
        got = []
        for s, a in zip(sides, cases):
            with torch.cuda.stream(s):
                got.append(api.shared_prefix_attention(*a))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))
    ws = torch.empty(1 << 26, device=gpu, dtype=torch.uint8)         # one workspace, one call after the other
    out = [[torch.empty_like(t) for t in w] for w in want]
    for k in range(40):
        api.shared_prefix_attention(*cases[k % 2], out=out[k % 2][0], lse=out[k % 2][1], workspace=ws)
    for g, w in zip(out, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))


@gpu_only
def test_inputs_written_just_before_and_outputs_read_just_after(gpu):
    """The kernels of one call overlap, but not what comes before and after it on the stream."""
    a = inputs(gpu, BF, 16, 4, 128, 32, 4000, [200] * 16, 30)
    n = a[1].shape[0] * a[1].shape[1]
    k0, v0, q0 = (t.clone() for t in a[:3][1:] + a[:1])
    for step in range(10):
        f = 1.0 + 0.125 * step
        torch.mul(k0, f, out=a[1])
        torch.mul(v0, f, out=a[2])
        torch.mul(q0, 1.0 / f, out=a[0])
        out, lse = api.shared_prefix_attention(*a)
        got = out.clone(), lse.clone()
        a[1].zero_()
        torch.cuda.synchronize()
        torch.mul(k0, f, out=a[1])
        torch.cuda.synchronize()
        want = api.shared_prefix_attention(*a)
        assert all(torch.equal(x, y) for x, y in zip(got, want)), (step, n)


@gpu_only
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 256), (F32, 64)])
@pytest.mark.parametrize("per", [3, 40])
def test_every_input_written_just_before(gpu, dtype, d, per):
    """Caches, queries, tables, the prefix's length and the sequences' own, each from a kernel right before the call; with
    short tables, and with long ones, whose tokens are worked on beside the prefix."""
    B, Hk, page, first = 32, 4, 16, 250
    g = wk.generator(31, gpu)
    pool = first + B * per
    sets = []
    for k in range(2):
        pages = torch.randperm(pool, device=gpu, generator=g).int()
        sets.append([rand(g, B, 16, d, dtype=dtype), rand(g, pool, Hk, page, d, dtype=dtype),
                     rand(g, pool, Hk, page, d, dtype=dtype), pages[:first].contiguous(),
                     torch.tensor([4000 - 777 * k], device=gpu).int(), pages[first:].view(B, per).contiguous(),
                     torch.randint(0, per * page + 1, (B,), device=gpu, generator=g).int()])
    want = [api.shared_prefix_attention(*s, d ** -0.5) for s in sets]
    torch.cuda.synchronize()
    a = [torch.zeros_like(t) for t in sets[0]]
    ws = torch.full((1 << 28,), 1, device=gpu, dtype=torch.uint8)
    out, lse = (torch.empty_like(t) for t in want[0])
    for step in range(12):
        k = step % 2
        for to, t in zip(a, sets[k]):
            to.copy_(t)
        if step % 3 == 0:                                             # what a workspace held does not matter
            ws.view(torch.int32).fill_(1)
        api.shared_prefix_attention(*a, d ** -0.5, out=out, lse=lse, workspace=ws)
        got = out.clone(), lse.clone()
        for to in a:
            to.zero_()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want[k])), step


FIRST_CAPTURED = """
import torch
from transformer_depth_wise_gb300 import api
dev = torch.device("cuda:0")
g = torch.Generator(device=dev).manual_seed(5)
B, Hk, page, d, first, per = 32, 4, 16, 128, 200, 40
pool = first + B * per
def some():
    pages = torch.randperm(pool, device=dev, generator=g).int()
    r = lambda *s: torch.empty(s, device=dev).normal_(generator=g).bfloat16()
    return [r(B, 16, d), r(pool, Hk, page, d), r(pool, Hk, page, d), pages[:first].contiguous(),
            torch.randint(1, first * page, (1,), device=dev, generator=g).int(), pages[first:].view(B, per).contiguous(),
            torch.randint(0, per * page + 1, (B,), device=dev, generator=g).int()]
sets, a = [some() for _ in range(4)], some()
torch.cuda.synchronize()
graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(graph, stream=side):
    got = [api.shared_prefix_attention(*a, 0.09) for _ in range(3)]
for step in range(12):
    with torch.cuda.stream(side):
        for to, t in zip(a, sets[step % 4]):
            to.copy_(t)
        graph.replay()
        for to in a:
            to.zero_()
    torch.cuda.synchronize()
    want = api.shared_prefix_attention(*sets[step % 4], 0.09)
    for out in got:
        assert all(torch.equal(x, y) for x, y in zip(out, want)), step
"""


@gpu_only
def test_first_call_is_captured(gpu):
    """A process whose first call goes into a graph; replays read what was written right before them."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST_CAPTURED], cwd=root, check=True, timeout=300)


@gpu_only
def test_more_calls_than_marks(gpu):
    """Calls side by side on two streams, so many that they take the same places in the table of marks again."""
    cases = [inputs(gpu, dtype, 16, 4, 64, 16, 400, [200] * 8, 100 + k) for k, dtype in enumerate((BF, F32))]
    want = [api.shared_prefix_attention(*a) for a in cases]
    sides = [torch.cuda.Stream(gpu) for _ in range(2)]
    ws = [torch.full((1 << 26,), 255, device=gpu, dtype=torch.uint8) for _ in range(2)]
    got = [[torch.empty_like(t) for t in w] for w in want]
    torch.cuda.synchronize()
    for k in range(5000):
        for i in range(2):
            with torch.cuda.stream(sides[i]):
                api.shared_prefix_attention(*cases[i], out=got[i][0], lse=got[i][1], workspace=ws[i])
        if k % 1000 == 999:
            torch.cuda.synchronize()
            for x, y in zip(got, want):
                assert all(torch.equal(a, b) for a, b in zip(x, y))
            for x in got:
                for t in x:
                    t.zero_()
            torch.cuda.synchronize()


@gpu_only
def test_serving_layer(gpu):
    """One decoded token of a batch behind a shared image and text prefix: add + norm in 8 bits, the projection, head
    norm with three axes into the cache, attention behind the prefix."""
    g = wk.generator(12, gpu)
    B, D, Hq, Hk, d, page, prefix = 9, 512, 8, 2, 64, 16, 200
    proj = rand(g, D, (Hq + 2 * Hk) * d, dtype=F32, scale=D ** -0.5)
    wn, fr, axes = 1 + rand(g, D, dtype=F32, scale=0.1), api.rotary_frequencies(d, device=gpu), api.rotary_axes((8, 12, 12), device=gpu)
    pages = torch.randperm(13 + 2 * B, device=gpu, generator=g).int()
    pt, t = pages[:13].contiguous(), pages[13:].view(B, 2).contiguous()
    kc, vc = (torch.zeros(13 + 2 * B, Hk, page, d, device=gpu, dtype=BF) for _ in range(2))

    def layer(x, r, pos, places, table):
        y8, sc, total = api.add_rms_norm_8bit(x, r, wn, group=128)
        h = (y8.float().unflatten(-1, (-1, 128)) * sc[..., None]).flatten(-2) @ proj
        q, k, v = (u.unflatten(-1, (-1, d)) for u in h.bfloat16().split([Hq * d, Hk * d, Hk * d], -1))
        q = api.head_norm_rotate_append(q, k, v, None, None, pos, fr, kc, vc, table, axes=axes, places=places)
        return q, total

    # the prefix: an image of 14 x 14 patches and four text tokens, once for all
    i = torch.arange(prefix, device=gpu)
    img = i < 196
    pos = torch.stack((torch.where(img, 0, i - 182), torch.where(img, i // 14, i - 182), torch.where(img, i % 14, i - 182)), -1)
    x0, r0 = rand(g, 1, prefix, D), rand(g, 1, prefix, D, scale=3.0)
    layer(x0, r0, pos[None].int().contiguous(), i[None].int().contiguous(), pt[None].contiguous())
    # each sequence has 0 .. 8 tokens and appends one
    have = torch.arange(B, device=gpu)
    x1, r1 = rand(g, B, 9, D), rand(g, B, 9, D, scale=3.0)
    own = 18 + torch.arange(9, device=gpu)[None, :, None].expand(B, 9, 3)
    places = torch.where(torch.arange(9, device=gpu)[None] < have[:, None], torch.arange(9, device=gpu)[None], -1).int()
    layer(x1, r1, own.int().contiguous(), places.contiguous(), t)
    x2, r2 = rand(g, B, 1, D), rand(g, B, 1, D, scale=3.0)
    last = (18 + have)[:, None, None].expand(B, 1, 3).int().contiguous()
    q, total = layer(x2, r2, last, have[:, None].int().contiguous(), t)
    n, lengths = torch.tensor([prefix], device=gpu).int(), (have + 1).int()
    args = [q[:, 0], kc, vc, pt, n, t, lengths, d ** -0.5]
    check(args, BF, d)
    assert torch.equal(total, (x2.float() + r2.float()).bfloat16())
    # the cache holds what was normed, turned and appended
    y8, sc, _ = api.add_rms_norm_8bit(x2, r2, wn, group=128)
    h = (y8.float().unflatten(-1, (-1, 128)) * sc[..., None]).flatten(-2) @ proj
    q2, k2, v2 = (u.unflatten(-1, (-1, d)) for u in h.bfloat16().split([Hq * d, Hk * d, Hk * d], -1))
    qr, kr = api.head_norm_rotate(q2, k2, None, None, last, fr, axes=axes)
    for b in range(B):
        pg = int(t[b, b // page])
        assert torch.equal(kc[pg, :, b % page], kr[b, 0]) and torch.equal(vc[pg, :, b % page], v2[b, 0])
    assert torch.equal(qr, q)


# --------------------------------------------------------------------------
# refusals
# --------------------------------------------------------------------------
def shared(q=FAKE, qs=512, kc=FAKE + 64, vc=FAKE + 128, num=8, page=16, ptab=FAKE, pp=4, pl=FAKE, table=FAKE, maxp=4,
           n=FAKE, B=2, Hq=8, Hk=2, d=64, dtype=1, scale=0.1, out=FAKE + 192, lse=None, ws=FAKE + 256, bytes_=1 << 40):
    return _lib.lib().attnres_shared_prefix_attention(q, qs, kc, vc, num, page, ptab, pp, pl, table, maxp, n, B, Hq, Hk, d,
                                                      dtype, scale, out, lse, ws, bytes_, None)


def test_refusals():
    size = lambda B=2, Hq=8, Hk=2, d=64, dtype=1, page=16, pp=4, mp=4: \
        _lib.lib().attnres_shared_prefix_attention_workspace_bytes(B, Hq, Hk, d, dtype, page, pp, mp)  # noqa: E731
    need = size()
    assert need > 0 and size(pp=0) > 0 and size(B=0) > 0 and size(mp=0) > 0
    assert size(dtype=5) == DTYPE and size(Hk=3) == SHAPE and size(d=60) == ALIGN
    assert size(Hq=17, Hk=1) == SHAPE and size(d=264) == SHAPE and size(B=-1) == SHAPE
    assert size(page=0) == SHAPE and size(pp=-1) == SHAPE and size(mp=-1) == SHAPE
    assert size(page=1 << 20, pp=1 << 12) == SHAPE and size(page=1 << 20, mp=1 << 12) == SHAPE and size(B=1 << 30) == SHAPE
    assert shared(dtype=3) == DTYPE and shared(B=-1) == SHAPE and shared(page=0) == SHAPE and shared(maxp=-1) == SHAPE
    assert shared(pp=-1) == SHAPE and shared(num=-1) == SHAPE and shared(Hq=7) == SHAPE and shared(d=4) == ALIGN
    assert shared(scale=math.inf) == VALUE and shared(scale=math.nan) == VALUE
    for name in ("q", "kc", "vc", "ptab", "pl", "table", "n", "out", "ws"):
        assert shared(**{name: None}) == NULL, name
    assert shared(bytes_=need - 1) == CAP and shared(qs=516) == ALIGN
    for name in ("q", "kc", "vc", "out", "ws"):
        assert shared(**{name: FAKE + 8}) == ALIGN, name
    for name in ("ptab", "pl", "table", "n", "lse"):
        assert shared(**{name: FAKE + 2}) == ALIGN, name
    assert shared(out=FAKE + 64) == VALUE and shared(ws=FAKE + 128) == VALUE and shared(ws=FAKE) == VALUE
    assert shared(B=0, q=None, out=None, n=None) == OK


def test_refusal_of_partial_overlaps():
    M = 1 << 30
    apart = dict(q=FAKE, kc=FAKE + M, vc=FAKE + 2 * M, ptab=FAKE + 3 * M, pl=FAKE + 4 * M, table=FAKE + 5 * M, n=FAKE + 6 * M,
                 out=FAKE + 7 * M, lse=FAKE + 8 * M, ws=FAKE + 9 * M)
    need = _lib.lib().attnres_shared_prefix_attention_workspace_bytes(2, 8, 2, 64, 1, 16, 4, 4)
    size = dict(q=2 * 1024, kc=8 * 2 * 16 * 128, vc=8 * 2 * 16 * 128, ptab=16, pl=4, table=32, n=8, out=2048, lse=64, ws=need)
    assert need < M
    for name in ("out", "lse", "ws"):
        for other in apart:
            if other == name or (other == "q" and name != "ws"):
                continue
            for at in (apart[other], apart[other] + (size[other] - 1) // 16 * 16, apart[other] - size[name] // 16 * 16 + 16):
                assert shared(**(apart | {name: at})) == VALUE, (name, other, at - apart[other])


@gpu_only
def test_outputs_on_the_queries(gpu):
    for dtype, d in ((BF, 128), (F32, 64)):
        q, kc, vc, pt, n, t, lengths, scale = inputs(gpu, dtype, 8, 2, d, 16, 700, [20, 300, 0] * 9, 80)
        want = api.shared_prefix_attention(q, kc, vc, pt, n, t, lengths, scale)
        got = api.shared_prefix_attention(q, kc, vc, pt, n, t, lengths, scale, out=q)
        assert got[0] is q and all(torch.equal(x, y) for x, y in zip(got, want))


@gpu_only
def test_wrapper_refusals(gpu):
    a = inputs(gpu, BF, 4, 2, 64, 16, 40, [3, 5], 1)
    for at, bad in ((0, a[0].cpu()), (0, a[0][0]), (1, a[1][:, :1].contiguous()), (2, a[2][:1]), (3, a[3][None]), (4, None),
                    (4, a[4].repeat(2)), (5, a[5][:1]), (6, a[6][:1]), (6, None)):
        b = list(a)
        b[at] = bad
        with pytest.raises(ValueError):
            api.shared_prefix_attention(*b)
    for at in (3, 4, 5, 6):
        b = list(a)
        b[at] = a[at].long()
        with pytest.raises(TypeError):
            api.shared_prefix_attention(*b)
    with pytest.raises(_lib.AttnResError):
        api.shared_prefix_attention(*a, workspace=torch.empty(64, device=gpu, dtype=torch.uint8))
