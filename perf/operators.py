"""The attention sublayer's operators: their plain forms and the cases that are measured.

Three groups of operators stand between two depth aggregations of a hybrid decoder layer:

* ``rotate``, ``append``, ``rotate_bwd``: the RMS norm of every query and key head with the position rotation in the
  same pass; its serving form, which puts the new keys and values into a paged cache; its backward pass;
* ``paged``: attention of one new token per sequence over the paged cache;
* ``linear``, ``linear_train``, ``step``: linear attention with one decay per head, over prompts, with its backward pass,
  and for single tokens.

``run`` computes them from elementary torch operations in 32 bits (angles in 64) where ``own`` is false and calls the
framework where it is true; ``exact`` computes the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def _rotate(op, B, T, Hq, Hk, d, rot, interleaved, dtype, start=0, page=0, cached=0):
    return {"op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot, "interleaved": interleaved,
            "dtype": dtype, "start": start, "page": page, "cached": cached}


def _paged(B, Hq, Hk, d, page, shortest, longest, dtype):
    return {"op": "paged", "B": B, "Hq": Hq, "Hk": Hk, "d": d, "page": page, "shortest": shortest,
            "longest": longest, "dtype": dtype}


def _linear(op, B, T, H, dk, dv, ragged, state, dtype):
    return {"op": op, "B": B, "T": T, "H": H, "dk": dk, "dv": dv, "ragged": ragged, "state": state, "dtype": dtype}


def listed():
    return [
        # the queries and keys of a 64K-token prompt, width 7168 (56 heads of 128, 8 key heads)
        {"name": "rotate_prefill", **_rotate("rotate", 1, 65536, 56, 8, 128, 128, False, "bf16")},
        # fp32 rows of width 256 as an accuracy run has them, a few of them: latency
        {"name": "rotate_few_f32", **_rotate("rotate", 3, 111, 4, 2, 64, 32, True, "f32", start=100000)},
        # one decoded token for each of 256 sequences: q, k and v of the token, the latter two into the cache
        {"name": "append_decode", **_rotate("append", 256, 1, 56, 8, 128, 128, False, "bf16", page=64, cached=100)},
        # a training step's gradient through norm and rotation, width 2048, half of each head rotated
        {"name": "rotate_backward", **_rotate("rotate_bwd", 4, 4096, 16, 16, 128, 64, True, "bf16")},
        # one user's chat of 777 tokens, every query head with its own keys: latency
        {"name": "paged_one", **_paged(1, 16, 16, 128, 16, 777, 777, "bf16")},
        # a full serving batch of 256 sequences of very different lengths, seven query heads to a key head
        {"name": "paged_batch", **_paged(256, 56, 8, 128, 64, 1, 8192, "bf16")},
        # two very long documents, width 4096: few rows, a long axis
        {"name": "paged_long", **_paged(2, 32, 4, 128, 64, 65537, 131071, "bf16")},
        # a 64K-token prompt through linear attention, width 4096, from an empty state
        {"name": "linear_prefill", **_linear("linear", 1, 65536, 32, 128, 128, False, False, "bf16")},
        # a padded batch of prompts that go on from earlier states, narrow key heads
        {"name": "linear_ragged", **_linear("linear", 8, 1023, 16, 64, 128, True, True, "bf16")},
        # forward and backward of a training step, width 2048
        {"name": "linear_train", **_linear("linear_train", 4, 4096, 16, 128, 128, False, False, "bf16")},
        # one decoded token for four sequences: latency
        {"name": "step_few", **_linear("step", 4, 1, 16, 128, 128, False, True, "bf16")},
        # one decoded token for 256 sequences, width 4096
        {"name": "step_batch", **_linear("step", 256, 1, 32, 128, 128, False, True, "bf16")},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "rotate_bwd", "paged", "paged", "linear", "linear", "linear_train", "step"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op in ("rotate", "append", "rotate_bwd"):
        d = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([d, d // 32 * 16])
        Hk = rng.choice([1, 2, 4, 7, 8, 16])
        Hq = Hk * rng.choice([1, 1, 3, 4, 7])
        most = 300_000_000 if op == "rotate" else 60_000_000
        rows = _log_int(rng, 1, min(65536, most // ((Hq + Hk) * d)))
        if op == "append":
            B, T = _log_int(rng, 1, 256), 1
            if rng.random() < 0.3:
                B, T = min(B, 16), _log_int(rng, 2, 333)
        else:
            B = rng.choice([1, 1, 2, 5])
            T = max(1, rows // B)
        return _rotate(op, B, T, Hq, Hk, d, rot, rng.random() < 0.4, dtype, start=rng.choice([0, 0, 4097, 1_000_000]),
                       page=rng.choice([16, 32, 64, 128]), cached=_log_int(rng, 1, 200))
    if op == "paged":
        d = rng.choice([64, 128, 128, 128, 96, 256])
        Hk = rng.choice([1, 2, 4, 5, 8, 16])
        G = rng.choice([1, 2, 4, 7, 8, 16])
        longest = _log_int(rng, 1, 131072)
        most = 4_000_000_000 // (2 * Hk * d * (4 if dtype == "f32" else 2))      # bytes of the whole cache
        B = _log_int(rng, 1, max(1, min(256, most // longest)))
        return _paged(B, G * Hk, Hk, d, rng.choice([16, 32, 64, 128]), rng.choice([0, 1, longest // 2, longest]), longest,
                      dtype)
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (96, 80), (128, 64)])
    H = rng.choice([1, 3, 4, 8, 16, 32])
    if op == "step":
        return _linear(op, _log_int(rng, 1, 256), 1, H, dk, dv, False, True, dtype)
    most = (100_000_000 if op == "linear" else 16_000_000) // (4 if dtype == "f32" else 1)
    T = _log_int(rng, 1, 65536 if op == "linear" else 8192)
    B = _log_int(rng, 1, max(1, min(16, most // (T * H * (dk + dv)))))
    T = max(1, min(T, most // (B * H * (dk + dv))))
    return _linear(op, B, T, H, dk, dv, rng.random() < 0.4, rng.random() < 0.5, dtype)


def _lengths(case, seed):
    """The lengths of a batch's sequences, from the seed: whole numbers between the case's shortest and longest."""
    g = torch.Generator().manual_seed(seed * 7 + 3)
    lo, hi = case["shortest"], case["longest"]
    n = torch.randint(lo, hi + 1, (case["B"],), generator=g)
    n[-1] = hi
    if case["B"] > 1:
        n[0] = lo
    return n


def _mean_length(case):
    return case["longest"] if case["B"] == 1 else (case["shortest"] + case["longest"]) / 2


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op, B = case["op"], case["B"]
    if op in ("rotate", "append", "rotate_bwd"):
        rows, Hq, Hk, d = B * case["T"], case["Hq"], case["Hk"], case["d"]
        elems = rows * (Hq + Hk) * d
        if op == "rotate":
            return {"bytes": 2 * elems * e + 4 * rows, "flops": 7 * elems}
        if op == "append":
            return {"bytes": 2 * (elems + rows * Hk * d) * e + 8 * rows, "flops": 7 * elems}
        return {"bytes": 3 * elems * e + 4 * rows, "flops": 16 * elems}
    if op == "paged":
        tokens, d = B * _mean_length(case), case["d"]
        return {"bytes": int(2 * tokens * case["Hk"] * d * e + 2 * B * case["Hq"] * d * e + 4 * B * case["Hq"]),
                "flops": int(4 * tokens * case["Hq"] * d)}
    T, H, dk, dv = case["T"], case["H"], case["dk"], case["dv"]
    tokens = B * T * (0.5 if case["ragged"] else 1.0)
    states = B * H * dk * dv * 4
    if op == "step":
        return {"bytes": 2 * states + B * H * (2 * dk + 2 * dv) * e, "flops": 5 * B * H * dk * dv}
    first = tokens * H * (2 * dk + dv) * e + B * T * H * dv * e      # rows behind a sequence are written, not read
    if op == "linear":
        return {"bytes": int(first + states * (2 if case["state"] else 1)), "flops": int(4 * tokens * H * dk * dv)}
    second = tokens * H * (2 * dk + 2 * dv) * e + B * T * H * (2 * dk + dv) * e
    return {"bytes": int(first + second + states * (2 if case["state"] else 0)),
            "flops": int(14 * tokens * H * dk * dv)}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    dt = TYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=dt):
        x = torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)
        return x if scale == 1.0 else x.mul_(scale)

    s = {"case": case}
    op, B = case["op"], case["B"]
    if op in ("rotate", "append", "rotate_bwd"):
        T, Hq, Hk, d, rot = case["T"], case["Hq"], case["Hk"], case["d"], case["rot"]
        # one projection's output holds the queries, keys and values of a token side by side; q, k and v are views of it
        qkv = normal(B, T, (Hq + 2 * Hk) * d)
        s["q"] = qkv[..., :Hq * d].unflatten(-1, (Hq, d))
        s["k"] = qkv[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
        s["v"] = qkv[..., (Hq + Hk) * d:].unflatten(-1, (Hk, d))
        s["q"].mul_(3.0)
        s["wq"] = normal(d, scale=0.1, dtype=torch.float32).add_(1.0)
        s["wk"] = normal(d, scale=0.1, dtype=torch.float32).add_(1.0)
        s["inv_freq"] = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / max(rot, 1))
        if op == "append":
            # every sequence has some tokens in the cache already, its pages lie scattered in the pool
            page = case["page"]
            have = torch.randint(0, case["cached"] + 1, (B, 1), device=dev, generator=g)
            s["positions"] = (have + torch.arange(T, device=dev)).int()
            per = -(-(case["cached"] + T) // page)
            s["table"] = torch.randperm(B * per, device=dev, generator=g).view(B, per).int()
            s["k_cache"] = normal(B * per, Hk, page, d)
            s["v_cache"] = normal(B * per, Hk, page, d)
        else:
            s["positions"] = (case["start"] + torch.arange(T, device=dev)).int().expand(B, T).contiguous()
        if op == "rotate_bwd":
            s["gq"], s["gk"] = normal(B, T, Hq, d), normal(B, T, Hk, d)
        return s
    if op == "paged":
        Hq, Hk, d, page = case["Hq"], case["Hk"], case["d"], case["page"]
        per = max(1, -(-case["longest"] // page))
        s["q"] = normal(B, Hq, d, scale=1.5)
        s["k_cache"] = normal(B * per, Hk, page, d)
        s["v_cache"] = normal(B * per, Hk, page, d)
        s["table"] = torch.randperm(B * per, device=dev, generator=g).view(B, per).int()
        s["lengths"] = _lengths(case, seed).int().to(dev)
        s["scale"] = 1.0 / math.sqrt(d)
        return s
    T, H, dk, dv = case["T"], case["H"], case["dk"], case["dv"]
    shape = (B, H) if op == "step" else (B, T, H)
    s["q"], s["k"], s["v"] = normal(*shape, dk), normal(*shape, dk), normal(*shape, dv)
    s["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H)
    s["scale"] = 1.0 / math.sqrt(dk)
    s["state"] = normal(B, H, dk, dv, scale=3.0, dtype=torch.float32) if case["state"] else None
    if op == "step":
        s["state_out"] = torch.empty_like(s["state"])
        return s
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, T + 1, (B,), device=dev, generator=g)
        n[0] = T
        s["lengths"] = n.int()
    if op == "linear_train":
        s["go"] = normal(B, T, H, dv)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------------------
def _angles(s):
    a = s["positions"].double()[..., None] * s["inv_freq"]                    # [B, T, rot / 2]
    return a.cos().float()[:, :, None], a.sin().float()[:, :, None]


def _halves(x, rot, interleaved):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def _joined(a, b, rest, interleaved):
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1)


def _norm_rotate(x, w, cos, sin, case):
    x = x.float()
    z = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    a, b = _halves(z, case["rot"], case["interleaved"])
    return _joined(a * cos - b * sin, b * cos + a * sin, z[..., case["rot"]:], case["interleaved"])


def _norm_rotate_bwd(x, w, cos, sin, grad, case):
    x, grad = x.float(), grad.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    a, b = _halves(grad, case["rot"], case["interleaved"])
    dz = _joined(a * cos + b * sin, b * cos - a * sin, grad[..., case["rot"]:], case["interleaved"])
    n = x * r
    dn = dz * w
    return r * (dn - n * (dn * n).mean(-1, keepdim=True)), (dz * n).sum((0, 1, 2))


def _paged_plain(s):
    case = s["case"]
    Hk, d = case["Hk"], case["d"]
    t = s["table"].long()
    k = s["k_cache"][t].transpose(1, 2).flatten(2, 3).float()                 # [B, Hk, most tokens, d]
    v = s["v_cache"][t].transpose(1, 2).flatten(2, 3).float()
    q = s["q"].float().unflatten(1, (Hk, -1))
    x = q @ k.transpose(-1, -2) * s["scale"]                                  # [B, Hk, G, tokens]
    seen = torch.arange(k.shape[2], device=k.device) < s["lengths"][:, None, None, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = (p @ v) / z.clamp_min(1e-30)
    lse = torch.where(z > 0, m + torch.log(z), -math.inf)
    return o.flatten(1, 2).to(s["q"].dtype), lse.flatten(1)


CHUNK = 256


def _decayed(a, b, c, g, first, lengths):
    """sum_{s <= t} e^{g (t - s)} (a_t . b_s) c_s + e^{g (t + 1)} a_t . first, all [B, H, T, d], in chunks of the time axis.

    Rows behind a sequence are zero in b and c already."""
    B, H, T, _ = a.shape
    C = min(CHUNK, T)
    n = -(-T // C)
    pad = (0, 0, 0, n * C - T)
    a, b, c = (torch.nn.functional.pad(x, pad).unflatten(2, (n, C)) for x in (a, b, c))
    i = torch.arange(C, device=a.device, dtype=torch.float32)
    g = g[:, None, None]
    near = torch.where(i[:, None] >= i, torch.exp(g * (i[:, None] - i).clamp_min(0)), 0.0)       # [H, C, C]
    out = (a @ b.transpose(-1, -2) * near[:, None]) @ c
    w = torch.exp(g * (C - 1 - i)[:, None])                                                      # [H, C, 1]
    sums = ((b * w[:, None]).transpose(-1, -2) @ c).flatten(3)                                   # [B, H, n, dk dv]
    j = torch.arange(n, device=a.device, dtype=torch.float32)
    far = torch.where(j[:, None] > j, torch.exp(g * C * (j[:, None] - j - 1).clamp_min(0)), 0.0)  # [H, n, n]
    before = far @ sums
    if first is not None:
        before = before + torch.exp(g * C * j[:, None]) * first.flatten(2)[:, :, None]
    before = before.unflatten(3, (b.shape[-1], c.shape[-1]))
    out = out + (a @ before) * torch.exp(g * (i + 1)[:, None])[:, None]
    return out.flatten(2, 3)[:, :, :T]


def _seen(s, T, dev):
    if s["lengths"] is None:
        return torch.ones(1, 1, T, 1, device=dev)
    return (torch.arange(T, device=dev) < s["lengths"][:, None])[:, None, :, None].float()


def _linear_plain(s):
    T, dt = s["case"]["T"], s["q"].dtype
    seen = _seen(s, T, s["q"].device)
    q, k, v = ((s[n].transpose(1, 2).float() * seen) for n in ("q", "k", "v"))
    g = s["log_decay"]
    o = _decayed(q * s["scale"], k, v, g, s["state"], s["lengths"]) * seen
    n = torch.full((1,), T, device=q.device) if s["lengths"] is None else s["lengths"]
    back = (n[:, None] - 1 - torch.arange(T, device=q.device)).clamp_min(0).float()               # [B, T]
    state = (k * torch.exp(g[:, None] * back[:, None])[..., None]).transpose(-1, -2) @ v
    if s["state"] is not None:
        state = state + s["state"] * torch.exp(g * n[:, None].float())[..., None, None]
    return o.transpose(1, 2).to(dt), state


def _linear_bwd_plain(s):
    T, dt, g = s["case"]["T"], s["q"].dtype, s["log_decay"]
    seen = _seen(s, T, s["q"].device)
    q, k, v, go = ((s[n].transpose(1, 2).float() * seen) for n in ("q", "k", "v", "go"))
    go = go * s["scale"]
    first = None if s["state"] is None else s["state"].transpose(-1, -2)
    dq = _decayed(go, v, k, g, first, s["lengths"]) * seen
    q, k, v, go = (x.flip(2) for x in (q, k, v, go))
    dk = _decayed(v, go, q, g, None, None).flip(2) * seen
    dv = _decayed(k, q, go, g, None, None).flip(2) * seen
    out = [x.transpose(1, 2).to(dt) for x in (dq, dk, dv)]
    if s["state"] is not None:
        q, go = q.flip(2), go.flip(2)
        i = torch.arange(1, T + 1, device=q.device, dtype=torch.float32)
        out.append((q * torch.exp(g[:, None] * i)[..., None]).transpose(-1, -2) @ go)
    return out


def _step_plain(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    torch.addcmul(s["state"] * torch.exp(s["log_decay"])[:, None, None], k[..., None], v[..., None, :], out=s["state_out"])
    o = (q[..., None] * s["state_out"]).sum(-2) * s["scale"]
    return o.to(s["q"].dtype), s["state_out"]


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "rotate":
        cos, sin = _angles(s)
        return tuple(_norm_rotate(s[n], s["w" + n], cos, sin, case).to(s[n].dtype) for n in ("q", "k"))
    if op == "append":
        cos, sin = _angles(s)
        q, k = (_norm_rotate(s[n], s["w" + n], cos, sin, case).to(s[n].dtype) for n in ("q", "k"))
        p = s["positions"].long()
        pages, slots = s["table"].long().gather(1, p // case["page"]), p % case["page"]
        s["k_cache"][pages, :, slots] = k
        s["v_cache"][pages, :, slots] = s["v"]
        return q, s["k_cache"], s["v_cache"]
    if op == "rotate_bwd":
        cos, sin = _angles(s)
        dq, dwq = _norm_rotate_bwd(s["q"], s["wq"], cos, sin, s["gq"], case)
        dk, dwk = _norm_rotate_bwd(s["k"], s["wk"], cos, sin, s["gk"], case)
        return dq.to(s["q"].dtype), dk.to(s["k"].dtype), dwq, dwk
    if op == "paged":
        return _paged_plain(s)
    if op == "linear":
        return _linear_plain(s)
    if op == "linear_train":
        return (_linear_plain(s)[0], *_linear_bwd_plain(s))
    return _step_plain(s)


# ---------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------------------------------
def _framework(s):
    from transformer_depth_wise_gb300 import api
    case, op = s["case"], s["case"]["op"]
    if op == "rotate":
        return api.head_norm_rotate(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], EPS,
                                    interleaved=case["interleaved"])
    if op == "append":
        q = api.head_norm_rotate_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["positions"], s["inv_freq"],
                                        s["k_cache"], s["v_cache"], s["table"], EPS, interleaved=case["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    if op == "rotate_bwd":
        return api.head_norm_rotate_backward(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], EPS,
                                             s["gq"], s["gk"], interleaved=case["interleaved"])
    if op == "paged":
        return api.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["scale"])
    if op == "linear":
        return api.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], state=s["state"],
                                    lengths=s["lengths"])
    if op == "linear_train":
        o, _ = api.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], state=s["state"],
                                    lengths=s["lengths"], want_state=False)
        dq, dk, dv, ds = api.linear_attention_backward(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], s["go"],
                                                       state=s["state"], lengths=s["lengths"])
        return (o, dq, dk, dv) if ds is None else (o, dq, dk, dv, ds)
    o = api.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], s["state"],
                                  state_out=s["state_out"])
    return o, s["state_out"]


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _turned(x, w, s, sign, norm=True):
    """Heads x [B, T, H, d] normed (or not) and turned by sign * position * inv_freq, as complex products."""
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    x = x.double()
    if norm:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    z = x[..., :rot].unflatten(-1, (rot // 2, 2) if inter else (2, rot // 2))
    z = torch.view_as_complex((z if inter else z.transpose(-1, -2)).contiguous())
    a = s["positions"].double()[..., None, None] * s["inv_freq"] * sign
    z = torch.view_as_real(z * torch.polar(torch.ones_like(a), a))
    z = (z if inter else z.transpose(-1, -2)).flatten(-2)
    return torch.cat((z, x[..., rot:]), -1)


def _exact_norm_bwd(x, w, s, grad):
    dz = _turned(grad, None, s, -1, norm=False)
    x, w = x.double(), w.double()
    rms = (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    u = dz * w
    return u / rms - x * (u * x).mean(-1, keepdim=True) / rms ** 3, (dz * x / rms).flatten(0, 2).sum(0)


def _exact_paged(s):
    out, lses = [], []
    for b, n in enumerate(s["lengths"].tolist()):
        Hk = s["case"]["Hk"]
        q = s["q"][b].double().unflatten(0, (Hk, -1))
        if n == 0:
            out.append(torch.zeros_like(q).flatten(0, 1))
            lses.append(torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device).flatten())
            continue
        pages = s["table"][b, :-(-n // s["case"]["page"])].long()
        k, v = (s[c][pages].transpose(0, 1).flatten(1, 2)[:, :n].double() for c in ("k_cache", "v_cache"))
        x = torch.einsum("hgd,htd->hgt", q, k) * s["scale"]
        lse = torch.logsumexp(x, -1)
        out.append(torch.einsum("hgt,htd->hgd", torch.exp(x - lse[..., None]), v).flatten(0, 1))
        lses.append(lse.flatten())
    return torch.stack(out), torch.stack(lses)


def _exact_linear(s, backward):
    """The recurrence S_t = e^g S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, token by token, and its reverse."""
    case, lens = s["case"], s["lengths"]
    B, T, H, dk, dv = (case[n] for n in ("B", "T", "H", "dk", "dv"))
    dev = s["q"].device
    q, k, v = (s[n].double().transpose(0, 1).contiguous() for n in ("q", "k", "v"))                # [T, B, H, d]
    lam = s["log_decay"].double().exp()[:, None, None]
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=dev) if s["state"] is None else s["state"].double().clone()
    n = torch.full((B,), T, device=dev) if lens is None else lens
    live = (torch.arange(T, device=dev)[:, None] < n).double()[:, :, None, None]                   # [T, B, 1, 1]
    keep = lam * live[..., None] + (1 - live[..., None])                                            # [T, B, H, 1, 1]
    k = k * live
    go = s["go"].double().transpose(0, 1).contiguous() * live if backward else None
    o, dq, ds, rows = torch.empty_like(v), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(T):
        S.mul_(keep[t]).add_(k[t][..., None] * v[t][..., None, :])
        o[t] = (q[t][..., None, :] @ S)[..., 0, :]
        if backward:
            dq[t] = (S @ go[t][..., None])[..., 0]
    o = (o * live * s["scale"]).transpose(0, 1)
    if not backward:
        return o, S
    G = torch.zeros_like(S)
    for t in range(T - 1, -1, -1):
        G.add_(q[t][..., None] * go[t][..., None, :])
        ds[t] = (G @ v[t][..., None])[..., 0]
        rows[t] = (k[t][..., None, :] @ G)[..., 0, :]
        G.mul_(keep[t])
    grads = [(x * live * s["scale"]).transpose(0, 1) for x in (dq, ds, rows)]
    return (o, *grads) if s["state"] is None else (o, *grads, G * s["scale"])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        return _turned(s["q"], s["wq"], s, 1), _turned(s["k"], s["wk"], s, 1)
    if op == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k, page = _turned(s["k"], s["wk"], s, 1), case["page"]
        for b, row in enumerate(s["positions"].tolist()):
            for t, p in enumerate(row):
                at = int(s["table"][b, p // page])
                kc[at, :, p % page] = k[b, t]
                vc[at, :, p % page] = s["v"][b, t].double()
        return _turned(s["q"], s["wq"], s, 1), kc, vc
    if op == "rotate_bwd":
        dq, dwq = _exact_norm_bwd(s["q"], s["wq"], s, s["gq"])
        dk, dwk = _exact_norm_bwd(s["k"], s["wk"], s, s["gk"])
        return dq, dk, dwq, dwk
    if op == "paged":
        return _exact_paged(s)
    if op in ("linear", "linear_train"):
        return _exact_linear(s, op == "linear_train")
    S = s["state"].double() * s["log_decay"].double().exp()[:, None, None]
    S = S + torch.einsum("bhk,bhv->bhkv", s["k"].double(), s["v"].double())
    return torch.einsum("bhk,bhkv->bhv", s["q"].double(), S) * s["scale"], S
