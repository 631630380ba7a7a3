"""The attention sublayer's operators at the edges of what they take."""
import math

import pytest
import torch

from test_attention_ops import (BF, E, EPS, F32, U, linear_grad_ref, linear_inputs, norm_inputs, paged_inputs,
                                rand, within)
from transformer_depth_wise_gb300 import _lib, api
from transformer_depth_wise_gb300 import workloads as wk

gpu_only = pytest.mark.gpu


# --------------------------------------------------------------------------
# paged attention
# --------------------------------------------------------------------------
# one tile of 64 tokens (written by the CTA that has it), pairs cut into a tile per CTA, pairs of many tiles per CTA
PAGED_NAN = [(5, 64), (0, 5, 777), (40000,), (300, 20000, 1)]


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths", PAGED_NAN)
def test_paged_nan_query(gpu, dtype, lengths):
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, len(lengths), 8, 2, 128, 16, list(lengths), sum(lengths))
    want, wlse = api.paged_attention(q, kc, vc, table, n, scale)
    q[:, 3, 17] = math.nan
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    some = n > 0
    assert bool(out[some, 3].isnan().all()) and bool(lse[some, 3].isnan().all())
    assert bool((out[~some] == 0).all()) and bool((lse[~some] == -math.inf).all())
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(out[:, keep], want[:, keep]) and torch.equal(lse[:, keep], wlse[:, keep])


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("length,first,last", [(777, 64, 128), (777, 0, 64), (40000, 12800, 13312), (40000, 39999, 40000)])
def test_paged_nan_keys(gpu, dtype, length, first, last):
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, 1, 8, 2, 128, 16, [length], length)
    want, wlse = api.paged_attention(q, kc, vc, table, n, scale)
    for j in range(first, last):
        kc[int(table[0, j // 16]), 1, j % 16] = math.nan
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    assert bool(out[0, 4:].isnan().all()) and bool(lse[0, 4:].isnan().all())
    assert torch.equal(out[0, :4], want[0, :4]) and torch.equal(lse[0, :4], wlse[0, :4])


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("length,at", [(5, 4), (777, 300), (40000, 12803)])
def test_paged_nan_values(gpu, dtype, length, at):
    q, kc, vc, table, n, scale = paged_inputs(gpu, dtype, 1, 8, 2, 128, 16, [length], length)
    want, wlse = api.paged_attention(q, kc, vc, table, n, scale)
    vc[int(table[0, at // 16]), 0, at % 16, 9] = math.nan
    out, lse = api.paged_attention(q, kc, vc, table, n, scale)
    hit = torch.zeros(8, 128, dtype=torch.bool, device=gpu)
    hit[:4, 9] = True
    assert torch.equal(lse, wlse) and bool(out[0][hit].isnan().all()) and torch.equal(out[0][~hit], want[0][~hit])


# --------------------------------------------------------------------------
# linear attention: what is no number stays in the state
# --------------------------------------------------------------------------
LINEAR_NAN = [  # T, decay, token, n: in one segment and in several, with what the token leaves decayed to nothing
    (150, -0.3, 20, 150), (3000, -0.5, 100, 3000), (3000, -20.0, 1000, 3000), (3000, -0.5, 1500, 2500),
    (3000, -math.inf, 700, 3000), (3000, -0.01, 100, 3000), (20000, -1.0, 5000, 19999),
]


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("T,g,t,n", LINEAR_NAN)
@pytest.mark.parametrize("which", ["k", "v"])
def test_linear_keeps_what_is_no_number(gpu, dtype, bad, T, g, t, n, which):
    q, k, v, _, scale = linear_inputs(gpu, dtype, 2, T, 2, 64, 72, T)
    ld = torch.tensor([g, -0.05], device=gpu)
    lens = torch.tensor([n, T], device=gpu).int()
    want, wlast = api.linear_attention(q, k, v, ld, scale, lengths=lens)
    (k if which == "k" else v)[0, t, 0, 5] = bad
    out, last = api.linear_attention(q, k, v, ld, scale, lengths=lens)
    # by the recurrence: a row of the state (k) or a column of it (v) is no number from token t on, so every output
    # after it is none (k) or its element 5 (v); tokens before t in its chunk of 64 may be either
    cols = slice(None) if which == "k" else slice(5, 6)
    assert not bool(torch.isfinite(out[0, t:n, 0, cols]).any())
    row = last[0, 0, 5] if which == "k" else last[0, 0, :, 5]
    assert not bool(torch.isfinite(row).any())
    # all else is as before
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[0, t // 64 * 64:n, 0, cols] = False
    assert torch.equal(out[rest], want[rest])
    rest = torch.ones_like(last, dtype=torch.bool)
    if which == "k":
        rest[0, 0, 5] = False
    else:
        rest[0, 0, :, 5] = False
    assert torch.equal(last[rest], wlast[rest])


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,g,t,n", LINEAR_NAN)
def test_linear_backward_keeps_what_is_no_number(gpu, dtype, T, g, t, n):
    q, k, v, _, scale = linear_inputs(gpu, dtype, 1, T, 2, 64, 72, T)
    ld = torch.tensor([g, -0.05], device=gpu)
    lens = torch.tensor([n], device=gpu).int()
    go = rand(wk.generator(5, gpu), 1, T, 2, 72, dtype=dtype)
    state = rand(wk.generator(6, gpu), 1, 2, 64, 72, dtype=F32)
    at = n - 1 - t                                           # far from the sequence's end, near its beginning, or neither
    want = api.linear_attention_backward(q, k, v, ld, scale, go, state=state, lengths=lens)
    go[0, at, 0, 5] = math.nan
    dq, dk, dv, ds = api.linear_attention_backward(q, k, v, ld, scale, go, state=state, lengths=lens)
    # the gradient of the state has its column 5 lost for all tokens up to `at`
    assert bool(dk[0, :at + 1, 0].isnan().all()) and bool(dv[0, :at + 1, 0, 5].isnan().all())
    assert bool(ds[0, 0, :, 5].isnan().all())
    # tokens behind it only where they share a chunk with it: 64 tokens counted from the sequence's end
    late = n - t // 64 * 64
    for got, ref in ((dk, want[1]), (dv, want[2])):
        assert torch.equal(got[0, late:, 0], ref[0, late:, 0]) and torch.equal(got[:, :, 1], ref[:, :, 1])
    keep = [i for i in range(72) if i != 5]
    assert torch.equal(dv[..., keep], want[2][..., keep]) and torch.equal(ds[0, 0][:, keep], want[3][0, 0][:, keep])
    assert bool(dq[0, at, 0].isnan().all())
    rest = [i for i in range(T) if i // 64 != at // 64]
    assert torch.equal(dq[0, rest], want[0][0, rest])


@gpu_only
def test_linear_captured_calls_and_streams_with_what_is_no_number(gpu):
    """A captured forward and backward pass in several segments, replayed with a NaN that has decayed away and without
    it again, and the same calls on three streams at once, each with a workspace of its own."""
    q, k, v, _, scale = linear_inputs(gpu, BF, 2, 3000, 3, 128, 128, 41)
    ld = torch.tensor([-20.0, -0.7, -0.01], device=gpu)
    go = rand(wk.generator(5, gpu), 2, 3000, 3, 128)

    def run():
        out, last = api.linear_attention(q, k, v, ld, scale)
        return (out, last, *api.linear_attention_backward(q, k, v, ld, scale, go, grad_state=last, want_initial=True))
    clean = [t.clone() for t in run()]
    v1 = v.clone()
    v1[0, 200, 0, 7] = math.nan
    v0 = v.clone()
    v.copy_(v1)
    spoilt = [t.clone() for t in run()]
    assert bool(spoilt[0][0, 200:, 0, 7].isnan().all()) and bool(spoilt[1][0, 0, :, 7].isnan().all())
    v.copy_(v0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for now, want in ((v0, clean), (v1, spoilt), (v1, spoilt), (v0, clean)):
        v.copy_(now)
        graph.replay()
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) and torch.equal(a.isnan(), b.isnan())
                   for a, b in zip(got, want))
    v.copy_(v1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for s in streams:
        with torch.cuda.stream(s):
            results.append(run())
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) and torch.equal(a.isnan(), b.isnan())
                   for a, b in zip(r, spoilt))


# --------------------------------------------------------------------------
# linear attention: gradients by value under any decay, and with any scale
# --------------------------------------------------------------------------
def check_gradients(gpu, dtype, q, k, v, ld, scale, go, state, n, gs):
    got = api.linear_attention_backward(q, k, v, ld, scale, go, state=state, lengths=n, grad_state=gs)
    want = linear_grad_ref(q, k, v, ld, scale, go, state, n, gs)
    absn = lambda t: None if t is None else t.abs()  # noqa: E731
    mags = linear_grad_ref(q.abs(), k.abs(), v.abs(), ld, abs(scale), go.abs(), absn(state), n, absn(gs))
    # as in test_linear_backward: fp32 roundings in units of the absolute sums (a decay's exponent among them, at most
    # 100 E before it underflows), for bf16 the masked products and the state rounded once on their way into a product;
    # 1e-36: products of decays below fp32's smallest normal number are zero
    f = (max(q.shape[-1], v.shape[-1]) + 64 + 100 + 2 * q.shape[1] / 64) * E
    for i, (a, b, m) in enumerate(zip(got, want, mags)):
        rounding = 2.0 ** -8 if dtype is BF and i < 3 else 0.0
        within(a, b, (U[dtype] if i < 3 else E) * b.abs() + (f + rounding) * m + 1e-36, "qkvs"[i])
    return got


@gpu_only
@pytest.mark.parametrize("dtype,B,T,H,dk,dv,lengths,with_state", [
    (BF, 1, 150, 2, 64, 64, None, True), (BF, 2, 129, 4, 96, 80, [64, 129], False), (BF, 1, 1500, 2, 128, 128, None, True),
    (BF, 1, 2100, 2, 128, 128, None, True), (BF, 2, 1300, 3, 128, 96, [1300, 700], True),
    (BF, 2, 1000, 2, 72, 128, [100, 993], False), (F32, 1, 150, 2, 64, 64, None, True),
    (F32, 1, 257, 1, 128, 128, None, True), (F32, 2, 1100, 1, 64, 64, [1100, 513], True),
])
@pytest.mark.parametrize("decay", [0.0, -0.7, -3.0, -math.inf])
def test_linear_gradients_under_any_decay(gpu, dtype, B, T, H, dk, dv, lengths, with_state, decay):
    q, k, v, ld, scale = linear_inputs(gpu, dtype, B, T, H, dk, dv, B + T + dv, decay)
    g = wk.generator(8, gpu)
    n = None if lengths is None else torch.tensor(lengths, device=gpu).int()
    state = rand(g, B, H, dk, dv, dtype=F32, scale=2.0) if with_state else None
    gs = rand(g, B, H, dk, dv, dtype=F32) if with_state else None
    check_gradients(gpu, dtype, q, k, v, ld, scale, rand(g, B, T, H, dv, dtype=dtype), state, n, gs)


@gpu_only
@pytest.mark.parametrize("dtype,T,lengths", [(BF, 150, None), (BF, 1500, [1500, 700]), (F32, 200, None),
                                             (F32, 700, [0, 700])])
@pytest.mark.parametrize("scale", [1e-30, -0.3, 7.0])
def test_linear_gradients_with_any_scale(gpu, dtype, T, lengths, scale):
    # what reaches the state's gradient through the outputs is scale grad_out, some 1e6 for the smallest one
    q, k, v, ld, _ = linear_inputs(gpu, dtype, 2, T, 2, 64, 64, T)
    g = wk.generator(9, gpu)
    n = None if lengths is None else torch.tensor(lengths, device=gpu).int()
    small = abs(scale) < 1e-20
    state, gs = (rand(g, 2, 2, 64, 64, dtype=F32, scale=x) for x in (1.0, 1e10 if small else 1.0))
    go = rand(g, 2, T, 2, 64, dtype=dtype, scale=1e36 if small else 1.0)
    check_gradients(gpu, dtype, q, k, v, ld, scale, go, state, n, gs)


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0, 100, 1500])
def test_linear_gradient_of_an_unused_state_is_the_state_gradient(gpu, dtype, T):
    q, k, v, ld, _ = linear_inputs(gpu, dtype, 3, T, 2, 64, 64, T)
    g = wk.generator(9, gpu)
    state, gs = (rand(g, 3, 2, 64, 64, dtype=F32) for _ in range(2))
    n = torch.tensor([0, T, 0], device=gpu).int()
    _, last = api.linear_attention(q, k, v, ld, 0.3, state=state, lengths=n)
    assert torch.equal(last[::2], state[::2])
    ds = api.linear_attention_backward(q, k, v, ld, 0.3, v.clone(), state=state, lengths=n, grad_state=gs)[3]
    assert torch.equal(ds[::2], gs[::2])


# --------------------------------------------------------------------------
# head norm
# --------------------------------------------------------------------------
def at(i):
    return 0x7F0000000000 + (i << 24)      # a stand-in for a device pointer of its own (never dereferenced)


def test_rotate_outputs_that_are_other_inputs_are_refused():
    """In place is an output on its own input, row by row; on any other input, or with other rows, calls would read what
    others have written.  Refused before any launch."""
    value = -8                              # ATTNRES_ERR_VALUE

    def rotate(q=at(0), k=at(1), qo=at(2), ko=at(3), qos=256, kos=256, T=2):
        return _lib.lib().attnres_head_norm_rotate(q, k, 1, T, 4, 4, 64, 1, 512, 512, None, None, None, None, 0, 0, 1e-6,
                                                   qo, ko, qos, kos, None)
    assert rotate(qo=at(1)) == value and rotate(ko=at(0)) == value and rotate(ko=at(2)) == value
    assert rotate(qo=at(1), qos=512) == value and rotate(qo=at(0)) == value and rotate(ko=at(1)) == value

    def append(q=at(0), k=at(1), v=at(2), qo=at(3), kc=at(4), vc=at(5), qos=256):
        return _lib.lib().attnres_head_norm_rotate_append(q, k, v, 1, 2, 4, 4, 64, 1, 512, 512, 512, None, None, None, None,
                                                          0, 0, 1e-6, qo, qos, kc, vc, 8, 16, at(6), 4, None)
    assert append(qo=at(1)) == value and append(qo=at(2)) == value and append(qo=at(0)) == value
    assert append(kc=at(5)) == value and append(kc=at(0)) == value and append(vc=at(2)) == value and append(vc=at(3)) == value

    def backward(dq=at(4), dk=at(5), qs=512, gs=512):
        return _lib.lib().attnres_head_norm_rotate_backward(at(0), at(1), 1, 2, 4, 4, 64, 1, qs, 512, None, None, None, None,
                                                            0, 0, 1e-6, at(2), at(3), gs, 512, dq, dk, None, None, None, 0,
                                                            None)
    assert backward(dq=at(0)) == value and backward(dq=at(2)) == value and backward(dk=at(1)) == value
    assert backward(dq=at(1)) == value and backward(dq=at(3)) == value and backward(dk=at(0)) == value
    assert backward(dk=at(2)) == value and backward(dq=at(5)) == value and backward(dq=at(1), qs=256) == value


@gpu_only
def test_rotate_outputs_that_are_other_inputs_are_refused_by_the_wrappers(gpu):
    q, k, v, wq, wk_, pos, fr = norm_inputs(gpu, BF, 2, 5, 4, 4, 64, 64, 3, packed=False)
    before = [t.clone() for t in (q, k, v)]
    kc, vc = (torch.zeros(4, 4, 16, 64, dtype=BF, device=gpu) for _ in range(2))
    table = torch.arange(4, device=gpu).view(2, 2).int()
    wide = torch.cat((q, k), 2)             # q with rows of its own, and with rows of this one
    for call in (lambda: api.head_norm_rotate(q, k, wq, wk_, pos, fr, q_out=k),
                 lambda: api.head_norm_rotate(q, k, wq, wk_, pos, fr, k_out=q),
                 lambda: api.head_norm_rotate(q, k, wq, wk_, pos, fr, q_out=v, k_out=v),
                 lambda: api.head_norm_rotate(wide[:, :, :4], k, wq, wk_, pos, fr,
                                              q_out=wide.view(-1)[:q.numel()].view(q.shape)),
                 lambda: api.head_norm_rotate_append(q, k, v, wq, wk_, pos, fr, kc, vc, table, q_out=k),
                 lambda: api.head_norm_rotate_append(q, k, v, wq, wk_, pos, fr, kc, kc, table)):
        with pytest.raises(_lib.AttnResError):
            call()
    assert all(torch.equal(a, b) for a, b in zip((q, k, v), before)) and not bool(kc.any())
    # each on its own input, rows apart as they are
    want = api.head_norm_rotate(q, k, wq, wk_, pos, fr)
    qv, kv = wide[:, :, :4], wide[:, :, 4:]
    api.head_norm_rotate(qv, kv, wq, wk_, pos, fr, q_out=qv, k_out=kv)
    assert torch.equal(qv, want[0]) and torch.equal(kv, want[1])
    qa = api.head_norm_rotate_append(q, k, v, wq, wk_, pos, fr, kc, vc, table, q_out=q)
    assert qa is q and torch.equal(q, want[0])


@gpu_only
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_rotate_frequencies_that_are_no_number(gpu, dtype, inter):
    q, k, _, wq, wk_, pos, fr = norm_inputs(gpu, dtype, 2, 5, 3, 2, 64, 64, 7)
    pos[0, 0] = 0
    want = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS, interleaved=inter)
    lost = [3, 9, 30]
    fr[3], fr[9], fr[30] = math.nan, math.inf, -math.inf
    got = api.head_norm_rotate(q, k, wq, wk_, pos, fr, EPS, interleaved=inter)
    cols = [2 * i + j for i in lost for j in (0, 1)] if inter else [i + j for i in lost for j in (0, 32)]
    rest = [i for i in range(64) if i not in cols]
    for a, b in zip(got, want):
        assert bool(a[..., cols].isnan().all()) and torch.equal(a[..., rest], b[..., rest])


# --------------------------------------------------------------------------
# the build
# --------------------------------------------------------------------------
def test_build_checks_the_planned_registers():
    from transformer_depth_wise_gb300 import build as b
    log = "".join(f"ptxas info    : Compiling entry function '_ZN7attnres{name}' for 'sm_103a'\n"
                  f"ptxas info    : Function properties for _ZN7attnres{name}\n    0 bytes stack frame\n"
                  f"ptxas info    : Used {n} registers, used 2 barriers\n"
                  for name, n in (("16linear_tc_kernelILb0EE", 72), ("5otherE", 40), ("16linear_tc_kernelILb1EE", 72)))
    b.check_registers(log, "linear_tc_kernel", 72)
    for bad in (log.replace("72", "70", 1), log.replace("Used 72", "Used 80"), ""):
        with pytest.raises(RuntimeError):
            b.check_registers(bad, "linear_tc_kernel", 72)
    for name in b.REGISTER_SHARES:
        assert b.planned_registers(f"{b.CSRC}/{name}") % 8 == 0
