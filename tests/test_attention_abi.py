"""Refusals of the attention sublayer's entry points, on the CPU: the C checks come before any launch, the wrappers'
before any C call."""
import math

import pytest
import torch

from transformer_depth_wise_gb300 import _lib, api

FAKE = 0x7F0000000000      # 16-byte aligned stand-in for a device pointer (never dereferenced)
OK, NULL, SHAPE, DTYPE, ALIGN, CAP, VALUE = 0, -1, -2, -3, -4, -7, -8


def rotate(q=FAKE, k=FAKE, B=1, T=2, Hq=4, Hk=2, d=64, dtype=1, qs=256, ks=128, wq=None, pos=None, fr=FAKE, rot=64,
           inter=0, eps=1e-6, qo=FAKE, ko=FAKE, qos=256, kos=128):
    return _lib.lib().attnres_head_norm_rotate(q, k, B, T, Hq, Hk, d, dtype, qs, ks, wq, None, pos, fr, rot, inter, eps,
                                               qo, ko, qos, kos, None)


def test_rotate_refusals():
    assert rotate(dtype=2) == DTYPE
    assert rotate(B=-1) == SHAPE and rotate(T=-1) == SHAPE and rotate(Hq=0) == SHAPE and rotate(Hk=0) == SHAPE
    assert rotate(d=72) == ALIGN and rotate(d=0) == SHAPE and rotate(d=528) == SHAPE
    assert rotate(rot=8) == ALIGN and rotate(rot=80) == SHAPE and rotate(rot=-16) == SHAPE
    assert rotate(dtype=0, d=264, rot=0) == SHAPE and rotate(dtype=0, d=68, rot=0) == ALIGN
    assert rotate(qs=252) == ALIGN and rotate(qs=-256) == SHAPE and rotate(qos=248) == SHAPE and rotate(kos=0) == SHAPE
    assert rotate(inter=2) == VALUE and rotate(eps=-1.0) == VALUE and rotate(eps=math.nan) == VALUE
    assert rotate(q=None) == NULL and rotate(k=None) == NULL and rotate(qo=None) == NULL and rotate(fr=None) == NULL
    assert rotate(q=FAKE + 8) == ALIGN and rotate(ko=FAKE + 2) == ALIGN and rotate(wq=FAKE + 4) == ALIGN
    assert rotate(pos=FAKE + 2) == ALIGN and rotate(fr=FAKE + 4) == ALIGN
    assert rotate(B=0, q=None) == OK and rotate(T=0, qo=None) == OK


def append(q=FAKE, v=FAKE, B=1, T=1, Hk=2, vs=128, kc=FAKE, vc=FAKE, num=4, page=16, table=FAKE, maxp=2, qos=256, qo=FAKE):
    return _lib.lib().attnres_head_norm_rotate_append(q, FAKE, v, B, T, 4, Hk, 64, 1, 256, 128, vs, None, None, None,
                                                      FAKE, 64, 0, 1e-6, qo, qos, kc, vc, num, page, table, maxp, None)


def test_append_refusals():
    assert append(page=0) == SHAPE and append(num=-1) == SHAPE and append(maxp=-1) == SHAPE
    assert append(page=1 << 20, maxp=1 << 12) == SHAPE and append(page=1 << 20, maxp=1025) == SHAPE
    assert append(vs=4) == ALIGN and append(qos=128) == SHAPE
    assert append(v=None) == NULL and append(kc=None) == NULL and append(vc=None) == NULL and append(table=None) == NULL
    assert append(kc=FAKE + 8) == ALIGN and append(table=FAKE + 2) == ALIGN
    assert append(B=0, kc=None) == OK


def rotate_bwd(gq=FAKE, dq=FAKE, gw=FAKE, ws=FAKE, rows=2, gqs=256, B=1, T=1):
    return _lib.lib().attnres_head_norm_rotate_backward(FAKE, FAKE, B, T, 4, 2, 64, 1, 256, 128, None, None, None, FAKE,
                                                        64, 0, 1e-6, gq, FAKE, gqs, 128, dq, FAKE, gw, None, ws, rows,
                                                        None)


def test_rotate_backward_refusals():
    assert rotate_bwd(gq=None) == NULL and rotate_bwd(dq=None) == NULL and rotate_bwd(ws=None) == NULL
    assert rotate_bwd(rows=1) == CAP and rotate_bwd(gqs=4) == ALIGN and rotate_bwd(gw=FAKE + 4) == ALIGN
    assert rotate_bwd(B=0, gw=None, gq=None) == OK
    assert _lib.lib().attnres_head_norm_rotate_backward_workspace_rows() >= 2


def paged(q=FAKE, qs=512, kc=FAKE, vc=FAKE, num=8, page=16, table=FAKE, maxp=4, n=FAKE, B=2, Hq=8, Hk=2, d=64, dtype=1,
          scale=0.1, out=FAKE, lse=None, ws=FAKE, bytes_=1 << 40):
    return _lib.lib().attnres_paged_attention(q, qs, kc, vc, num, page, table, maxp, n, B, Hq, Hk, d, dtype, scale, out,
                                              lse, ws, bytes_, None)


def test_paged_refusals():
    size = _lib.lib().attnres_paged_attention_workspace_bytes
    assert size(8, 2, 64, 1) > 0 and size(8, 2, 64, 5) == DTYPE and size(8, 3, 64, 1) == SHAPE
    assert size(17, 1, 64, 1) == SHAPE and size(8, 0, 64, 1) == SHAPE and size(8, 2, 60, 1) == ALIGN
    assert size(8, 2, 264, 1) == SHAPE and size(0, 2, 64, 1) == SHAPE
    assert paged(dtype=3) == DTYPE and paged(B=-1) == SHAPE and paged(page=0) == SHAPE and paged(maxp=-1) == SHAPE
    assert paged(Hq=34, qs=34 * 64) == SHAPE and paged(Hq=7) == SHAPE and paged(d=4) == ALIGN
    assert paged(scale=math.inf) == VALUE and paged(scale=math.nan) == VALUE
    assert paged(q=None) == NULL and paged(kc=None) == NULL and paged(n=None) == NULL and paged(out=None) == NULL
    assert paged(table=None) == NULL and paged(ws=None) == NULL
    assert paged(bytes_=size(8, 2, 64, 1) - 1) == CAP
    assert paged(q=FAKE + 8) == ALIGN and paged(vc=FAKE + 4) == ALIGN and paged(lse=FAKE + 2) == ALIGN
    assert paged(qs=516) == ALIGN and paged(B=0, q=None, out=None) == OK


def linear(q=FAKE, B=1, T=100, H=2, dk=64, dv=64, dtype=1, qs=128, g=FAKE, scale=0.1, n=None, state=None, out=FAKE,
           last=None, ws=FAKE, bytes_=1 << 40):
    return _lib.lib().attnres_linear_attention(q, FAKE, FAKE, B, T, H, dk, dv, dtype, qs, 128, 128, g, scale, n, state,
                                               out, last, ws, bytes_, None)


def test_linear_refusals():
    assert linear(dtype=9) == DTYPE and linear(B=-1) == SHAPE and linear(H=0) == SHAPE and linear(dk=136) == SHAPE
    assert linear(dv=136) == SHAPE and linear(dk=60) == ALIGN and linear(dv=0) == SHAPE and linear(T=1 << 31) == SHAPE
    assert linear(B=1 << 30, T=0) == SHAPE
    assert linear(scale=0.0) == VALUE and linear(scale=math.inf) == VALUE and linear(scale=1e-45) == VALUE
    assert linear(q=None) == NULL and linear(g=None) == NULL and linear(out=None) == NULL
    assert linear(qs=4) == ALIGN and linear(q=FAKE + 8) == ALIGN and linear(state=FAKE + 8) == ALIGN
    assert linear(g=FAKE + 2) == ALIGN and linear(n=FAKE + 1) == ALIGN
    assert linear(qs=64) == SHAPE and linear(qs=0) == SHAPE                # overlapping rows
    assert linear(B=0, q=None, g=None, out=None, ws=None) == OK and linear(T=0, q=None, out=None) == OK
    assert linear(out=FAKE) == VALUE                                       # out is q, k and v
    size = _lib.lib().attnres_linear_attention_workspace_bytes
    assert size(1, 100, 2, 64, 64, 1) >= 0 and size(1, 100, 0, 64, 64, 1) == SHAPE and size(1, 1, 1, 4, 8, 1) == ALIGN


def linear_bwd(go=FAKE, gs=None, dq=FAKE, ds=None, B=1, T=100, gos=128, scale=0.1, bytes_=1 << 40):
    return _lib.lib().attnres_linear_attention_backward(FAKE, FAKE, FAKE, B, T, 2, 64, 64, 1, 128, 128, 128, FAKE, scale,
                                                        None, None, go, gos, gs, dq, FAKE, FAKE, ds, FAKE, bytes_, None)


def test_linear_backward_refusals():
    assert linear_bwd(go=None) == NULL and linear_bwd(dq=None) == NULL and linear_bwd(gos=12) == ALIGN
    assert linear_bwd(gs=FAKE, ds=FAKE) == VALUE and linear_bwd(scale=0.0) == VALUE and linear_bwd(B=0) == OK
    assert linear_bwd(T=0) == OK
    assert linear_bwd(dq=FAKE) == VALUE                                    # the gradients are the inputs


def test_step_refusals():
    def step(q=FAKE, B=1, H=2, dk=64, dv=64, dtype=1, qs=128, scale=0.1, state=FAKE, new=FAKE, out=FAKE):
        return _lib.lib().attnres_linear_attention_step(q, FAKE, FAKE, B, H, dk, dv, dtype, qs, 128, 128, FAKE, scale,
                                                        state, new, out, None)
    assert step(q=None) == NULL and step(state=None) == NULL and step(new=None) == NULL and step(out=None) == NULL
    assert step(dk=256) == SHAPE and step(dv=4) == ALIGN and step(scale=math.nan) == VALUE and step(qs=2) == ALIGN
    assert step(state=FAKE + 4) == ALIGN and step(B=0, q=None) == OK


def test_wrappers_refuse_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(1, 2, 3, 64)
    for call in (lambda: api.head_norm_rotate(x, x), lambda: api.head_norm_rotate(x[0], x),
                 lambda: api.linear_attention(x, x, x, torch.zeros(3), 1.0),
                 lambda: api.linear_attention_step(x[0], x[0], x[0], torch.zeros(3), 1.0, None),
                 lambda: api.linear_attention_step(x, x, x, torch.zeros(3), 1.0, None),
                 lambda: api.paged_attention(x[0], x, x, torch.zeros(2, 1), torch.zeros(2), 1.0),
                 lambda: api.paged_attention(None, x, x, None, None, 1.0)):
        with pytest.raises(ValueError):
            call()


def test_rotary_frequencies():
    f = api.rotary_frequencies(8, 10000.0, "cpu")
    assert f.dtype == torch.float64 and f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-14)


@pytest.mark.gpu
def test_wrappers_refuse_gpu_tensors_of_the_wrong_kind(gpu):
    bf = torch.bfloat16
    q = torch.zeros(2, 3, 4, 64, dtype=bf, device=gpu)
    ld = torch.zeros(4, device=gpu)
    pos = torch.zeros(2, 3, dtype=torch.int32, device=gpu)
    fr = api.rotary_frequencies(64, device=gpu)
    kc = torch.zeros(4, 2, 16, 64, dtype=bf, device=gpu)
    table = torch.zeros(2, 2, dtype=torch.int32, device=gpu)
    n = torch.zeros(2, dtype=torch.int32, device=gpu)
    wide = torch.zeros(2, 3, 4, 128, dtype=bf, device=gpu)
    for err, call in (
            (TypeError, lambda: api.head_norm_rotate(q.half(), q.half())),
            (TypeError, lambda: api.head_norm_rotate(q, q.float())),
            (ValueError, lambda: api.head_norm_rotate(q, q[:1])),
            (ValueError, lambda: api.head_norm_rotate(wide[..., ::2], q)),
            (ValueError, lambda: api.head_norm_rotate(q.transpose(0, 1), q.transpose(0, 1))),
            (ValueError, lambda: api.head_norm_rotate(wide[..., :64], wide[..., :64])),
            (TypeError, lambda: api.head_norm_rotate(q, q, positions=pos.long())),
            (ValueError, lambda: api.head_norm_rotate(q, q, positions=pos[:1])),
            (TypeError, lambda: api.head_norm_rotate(q, q, positions=pos, inv_freq=fr.float())),
            (TypeError, lambda: api.head_norm_rotate(q, q, q_weight=torch.ones(64, dtype=bf, device=gpu))),
            (ValueError, lambda: api.head_norm_rotate_append(q, q, q, None, None, pos, fr, kc, kc, table)),
            (ValueError, lambda: api.paged_attention(q[:, 0].contiguous(), kc, kc, table[:1], n, 1.0)),
            (TypeError, lambda: api.paged_attention(q[:, 0].contiguous(), kc, kc, table, n.long(), 1.0)),
            (TypeError, lambda: api.paged_attention(q[:, 0].contiguous(), kc.float(), kc, table, n, 1.0)),
            (_lib.AttnResError, lambda: api.paged_attention(q[:, 0], kc, kc, table, n, math.inf)),
            (_lib.AttnResError, lambda: api.paged_attention(q[:, 0], kc, kc, table, n, 1.0,
                                                            workspace=torch.empty(16, device=gpu))),
            (TypeError, lambda: api.linear_attention(q, q, q.float(), ld, 1.0)),
            (ValueError, lambda: api.linear_attention(q, q, q, ld[:3], 1.0)),
            (TypeError, lambda: api.linear_attention(q, q, q, ld, 1.0, lengths=n.long())),
            (ValueError, lambda: api.linear_attention(q, q, q, ld, 1.0, state=torch.zeros(2, 4, 64, 32, device=gpu))),
            (_lib.AttnResError, lambda: api.linear_attention(wide, wide, wide, ld, 0.0)),
            (ValueError, lambda: api.linear_attention_backward(q, q, q, ld, 1.0, q[:, :2])),
            (TypeError, lambda: api.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], ld, 1.0,
                                                          torch.zeros(2, 4, 64, 64, dtype=bf, device=gpu)))):
        with pytest.raises(err):
            call()
