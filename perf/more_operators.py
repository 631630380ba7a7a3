"""A serving layer's operators around its attention: their plain forms and the cases that are measured.

Three groups, in the order in which a decoder layer over text and images runs them:

* ``norm``, ``norm8``, ``norm_bwd``: the RMS norm with the residual's addition, its form with an output in 8 bits (e4m3)
  and scales, and its backward pass;
* ``axes``, ``axes_append``, ``axes_bwd``: the head norm with a rotation whose positions have several axes (time, height,
  width), its form that puts keys and values into a paged cache, and its backward pass;
* ``shared``: attention of one new token per sequence of a batch that shares a long prefix in the paged cache, each
  sequence going on with pages of its own.

``run`` computes them from elementary torch operations in 32 bits (angles in 64) where ``own`` is false and calls the
framework where it is true; ``exact`` computes the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
TOP = 448.0                              # the largest e4m3 value
LEAST = 2.0 ** -126                      # the smallest scale


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def _norm(op, rows, D, group, residual, dtype):
    return {"op": op, "rows": rows, "D": D, "group": group, "residual": residual, "dtype": dtype}


def _axes(op, B, T, Hq, Hk, d, rot, axes, mixed, interleaved, dtype, start=0, page=0, cached=0):
    return {"op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot, "axes": axes, "mixed": mixed,
            "interleaved": interleaved, "dtype": dtype, "start": start, "page": page, "cached": cached}


def _shared(B, Hq, Hk, d, page, prefix, shortest, longest, dtype):
    return {"op": "shared", "B": B, "Hq": Hq, "Hk": Hk, "d": d, "page": page, "prefix": prefix, "shortest": shortest,
            "longest": longest, "dtype": dtype}


def listed():
    return [
        # a 32K-token prompt's residual stream of width 7168 on its way into an 8-bit projection, a scale per 128 values
        {"name": "norm8_prompt", **_norm("norm8", 32768, 7168, 128, True, "bf16")},
        # one decoded token for each of 256 sequences, a scale per token: latency
        {"name": "norm8_decode", **_norm("norm8", 256, 7168, 0, True, "bf16")},
        # fp32 rows of width 256 as an accuracy run has them, a few of them: latency
        {"name": "norm_few_f32", **_norm("norm", 333, 256, 0, True, "f32")},
        # a training step's gradient through the addition and the norm, 4 x 4096 tokens of width 4096
        {"name": "norm_backward", **_norm("norm_bwd", 16384, 4096, 0, True, "bf16")},
        # the queries and keys of 64K tokens of text and images, width 7168, three axes in sections of the pairs
        {"name": "axes_prefill", **_axes("axes", 1, 65536, 56, 8, 128, 128, 3, False, False, "bf16")},
        # one decoded token for each of 256 sequences: q, k and v of the token, the latter two into the cache
        {"name": "axes_append_decode", **_axes("axes_append", 256, 1, 56, 8, 128, 128, 3, True, False, "bf16", page=64,
                                               cached=100)},
        # four images of 777 patches each into the cache, height and width, fp32
        {"name": "axes_append_f32", **_axes("axes_append", 4, 777, 16, 4, 64, 64, 2, False, True, "f32", start=5000,
                                            page=16, cached=33)},
        # a training step's gradient through norm and rotation, width 2048, half of each head rotated
        {"name": "axes_backward", **_axes("axes_bwd", 4, 4096, 16, 16, 128, 64, 3, True, False, "bf16")},
        # a serving batch of 256 chats behind one 8K system prompt, seven query heads to a key head
        {"name": "shared_batch", **_shared(256, 56, 8, 128, 64, 8192, 1, 2048, "bf16")},
        # four short chats behind a short system prompt, every query head with its own keys: latency
        {"name": "shared_few", **_shared(4, 16, 16, 128, 16, 1111, 0, 100, "bf16")},
        # 64 questions about one very long document, width 4096, eight query heads to a key head
        {"name": "shared_long", **_shared(64, 32, 4, 128, 64, 131071, 1, 512, "bf16")},
        # fp32 with narrow heads, as an accuracy run has them
        {"name": "shared_f32", **_shared(33, 8, 2, 64, 32, 4097, 0, 300, "f32")},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "norm8", "norm_bwd", "axes", "axes_append", "axes_bwd", "shared", "shared",
                     "shared", "shared"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op in ("norm", "norm8", "norm_bwd"):
        D = 8 * _log_int(rng, 8, 1024)
        group = 0
        if op == "norm8":
            group = rng.choice([0, 32, 64, 128])
            D = max(D // 128, 1) * 128 if group else D
        most = 200_000_000 if op == "norm8" else 50_000_000
        return _norm(op, _log_int(rng, 1, min(65536, most // D)), D, group, rng.random() < 0.8, dtype)
    if op in ("axes", "axes_append", "axes_bwd"):
        d = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([d, d // 32 * 16])
        Hk = rng.choice([1, 2, 4, 7, 8, 16])
        Hq = Hk * rng.choice([1, 1, 3, 4, 7])
        most = 300_000_000 if op == "axes" else 60_000_000
        rows = _log_int(rng, 1, min(65536, most // ((Hq + Hk) * d)))
        if op == "axes_append":
            B, T = _log_int(rng, 1, 256), 1
            if rng.random() < 0.3:
                B, T = min(B, 16), _log_int(rng, 2, 333)
        else:
            B = rng.choice([1, 1, 2, 5])
            T = max(1, rows // B)
        return _axes(op, B, T, Hq, Hk, d, rot, rng.choice([2, 3, 3, 4]), rng.random() < 0.5, rng.random() < 0.4, dtype,
                     start=rng.choice([0, 0, 4097, 1_000_000]), page=rng.choice([16, 32, 64, 128]),
                     cached=_log_int(rng, 1, 200))
    d = rng.choice([64, 128, 128, 128, 80, 96])
    Hk = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 2, 4, 7, 8, 16])
    B = _log_int(rng, 1, 256)
    scores = (16_000_000 if dtype == "f32" else 200_000_000) // (B * G * Hk)       # of each query with the prefix
    prefix = _log_int(rng, 1, max(1, min(131072, scores)))
    own_most = (400_000_000 if dtype == "f32" else 2_000_000_000) // (2 * Hk * d * 2 * B)   # bytes of the sequences' pages
    longest = _log_int(rng, 1, max(1, min(4096, own_most)))
    return _shared(B, G * Hk, Hk, d, rng.choice([16, 32, 64, 128]), prefix,
                   rng.choice([0, 1, longest // 2, longest]), longest, dtype)


def _lengths(case, seed):
    """The sequences' own lengths, from the seed: whole numbers between the case's shortest and longest."""
    g = torch.Generator().manual_seed(seed * 7 + 3)
    lo, hi = case["shortest"], case["longest"]
    n = torch.randint(lo, hi + 1, (case["B"],), generator=g)
    n[-1] = hi
    if case["B"] > 1:
        n[0] = lo
    return n


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op in ("norm", "norm8", "norm_bwd"):
        rows, D = case["rows"], case["D"]
        n = rows * D
        tensors = (3 if case["residual"] else 1) if op != "norm_bwd" else (4 if case["residual"] else 3)
        extra = 4 * D
        if op == "norm":
            extra += n * e
        elif op == "norm8":
            extra += n + 4 * rows * (D // case["group"] if case["group"] else 1)
        else:
            extra += 4 * D                                            # the weight's gradient
        return {"bytes": tensors * n * e + extra, "flops": (10 if op == "norm_bwd" else 6) * n}
    B, Hq, Hk, d = case["B"], case["Hq"], case["Hk"], case["d"]
    if op == "shared":
        mean = case["longest"] if B == 1 else (case["shortest"] + case["longest"]) / 2
        tokens = case["prefix"] + B * mean
        return {"bytes": int(2 * tokens * Hk * d * e + 2 * B * Hq * d * e + 4 * B * Hq),
                "flops": int(4 * B * (case["prefix"] + mean) * Hq * d)}
    rows = B * case["T"]
    elems = rows * (Hq + Hk) * d
    if op == "axes":
        return {"bytes": 2 * elems * e + 4 * case["axes"] * rows, "flops": 7 * elems}
    if op == "axes_append":
        return {"bytes": 2 * (elems + rows * Hk * d) * e + 4 * (case["axes"] + 2) * rows, "flops": 7 * elems}
    return {"bytes": 3 * elems * e + 4 * case["axes"] * rows, "flops": 16 * elems}


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
    op = case["op"]
    if op in ("norm", "norm8", "norm_bwd"):
        rows, D = case["rows"], case["D"]
        s["w"] = normal(D, scale=0.1, dtype=torch.float32).add_(1.0)
        if op == "norm_bwd":
            s["s"], s["gy"] = normal(rows, D, scale=3.0), normal(rows, D)
            s["gs"] = normal(rows, D) if case["residual"] else None
        else:
            s["x"] = normal(rows, D)
            # a residual stream: a few channels much larger than the rest
            s["residual"] = normal(rows, D, scale=3.0) if case["residual"] else None
            if case["residual"]:
                s["residual"][:, ::97].mul_(8.0)
        return s
    B, Hq, Hk, d = case["B"], case["Hq"], case["Hk"], case["d"]
    if op == "shared":
        page = case["page"]
        first, per = -(-case["prefix"] // page), max(1, -(-case["longest"] // page))
        pages = torch.randperm(first + B * per, device=dev, generator=g).int()
        s["prefix_table"], s["table"] = pages[:first].contiguous(), pages[first:].view(B, per).contiguous()
        s["q"] = normal(B, Hq, d, scale=1.5)
        s["k_cache"] = normal(first + B * per, Hk, page, d)
        s["v_cache"] = normal(first + B * per, Hk, page, d)
        s["prefix"] = torch.tensor([case["prefix"]], dtype=torch.int32, device=dev)
        s["lengths"] = _lengths(case, seed).int().to(dev)
        s["scale"] = 1.0 / math.sqrt(d)
        return s
    T, rot, A = case["T"], case["rot"], case["axes"]
    # one projection's output holds the queries, keys and values of a token side by side; q, k and v are views of it
    qkv = normal(B, T, (Hq + 2 * Hk) * d)
    s["q"] = qkv[..., :Hq * d].unflatten(-1, (Hq, d))
    s["k"] = qkv[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    s["v"] = qkv[..., (Hq + Hk) * d:].unflatten(-1, (Hk, d))
    s["q"].mul_(3.0)
    s["wq"] = normal(d, scale=0.1, dtype=torch.float32).add_(1.0)
    s["wk"] = normal(d, scale=0.1, dtype=torch.float32).add_(1.0)
    pairs = rot // 2
    s["inv_freq"] = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / max(rot, 1))
    # the axis of each pair: taking turns, or a section of the pairs to each axis
    i = torch.arange(pairs, device=dev)
    s["axes"] = (i % A if case["mixed"] else (i * A).div(max(pairs, 1), rounding_mode="floor")).int()
    # images of 32 x 32 patches between runs of 32 text tokens, whose axes are all equal
    t = torch.arange(T, device=dev).expand(B, T) + torch.arange(B, device=dev)[:, None] * 77
    run, at = t // 1056, t % 1056
    patch = (at - 32).clamp_min(0)
    text = at < 32
    base = case["start"] + run * 65 + 32
    place = [torch.where(text, base - 32 + at, base)]
    place += [torch.where(text, base - 32 + at, base + x) for x in (patch // 32, patch % 32, patch % 7)]
    s["positions"] = torch.stack([place[0]] + place[-(A - 1):] if A == 2 else place[:A], -1).int()
    if op == "axes_append":
        # every sequence has some tokens in the cache already, its pages lie scattered in the pool
        page = case["page"]
        have = torch.randint(0, case["cached"] + 1, (B, 1), device=dev, generator=g)
        s["places"] = (have + torch.arange(T, device=dev)).int()
        per = -(-(case["cached"] + T) // page)
        s["table"] = torch.randperm(B * per, device=dev, generator=g).view(B, per).int()
        s["k_cache"] = normal(B * per, Hk, page, d)
        s["v_cache"] = normal(B * per, Hk, page, d)
    if op == "axes_bwd":
        s["gq"], s["gk"] = normal(B, T, Hq, d), normal(B, T, Hk, d)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------------------
def _add_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"]
    return y, x


def _in_8_bits(y, group):
    z = y.unflatten(-1, (-1, group or y.shape[-1]))
    scale = (z.abs().amax(-1) / TOP).clamp_min(LEAST)
    return (z / scale[..., None]).flatten(-2).to(F8), scale


def _norm_plain(s):
    case = s["case"]
    if case["op"] == "norm_bwd":
        x, gy = s["s"].float(), s["gy"].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n, u = x * r, gy * s["w"]
        dx = r * (u - n * (u * n).mean(-1, keepdim=True))
        if s["gs"] is not None:
            dx = dx + s["gs"].float()
        return dx.to(s["s"].dtype), (gy * n).sum(0)
    y, x = _add_norm(s)
    total = [x.to(s["x"].dtype)] if s["residual"] is not None else []
    if case["op"] == "norm":
        return [y.to(s["x"].dtype)] + total
    return [*_in_8_bits(y, case["group"])] + total


def _angles(s):
    a = s["positions"].double()[..., s["axes"].long()] * s["inv_freq"]        # [B, T, rot / 2]
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


def _axes_plain(s):
    case, op = s["case"], s["case"]["op"]
    cos, sin = _angles(s)
    if op == "axes_bwd":
        dq, dwq = _norm_rotate_bwd(s["q"], s["wq"], cos, sin, s["gq"], case)
        dk, dwk = _norm_rotate_bwd(s["k"], s["wk"], cos, sin, s["gk"], case)
        return dq.to(s["q"].dtype), dk.to(s["k"].dtype), dwq, dwk
    q, k = (_norm_rotate(s[n], s["w" + n], cos, sin, case).to(s[n].dtype) for n in ("q", "k"))
    if op == "axes":
        return q, k
    p = s["places"].long()
    pages, slots = s["table"].long().gather(1, p // case["page"]), p % case["page"]
    s["k_cache"][pages, :, slots] = k
    s["v_cache"][pages, :, slots] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _shared_plain(s):
    Hk, B, P = s["case"]["Hk"], s["case"]["B"], s["case"]["prefix"]
    t, f = s["table"].long(), s["prefix_table"].long()
    q = s["q"].float().unflatten(1, (Hk, -1)) * s["scale"]                    # [B, Hk, G, d]
    G = q.shape[2]
    k, v = (s[c][f].transpose(0, 1).flatten(1, 2)[:, :P].float() for c in ("k_cache", "v_cache"))   # [Hk, P, d]
    rows = q.transpose(0, 1).flatten(1, 2)                                    # [Hk, B G, d]: one product for all sequences
    x = (rows @ k.transpose(-1, -2)).unflatten(1, (B, G)).transpose(0, 1)     # [B, Hk, G, P]
    ko, vo = (s[c][t].transpose(1, 2).flatten(2, 3).float() for c in ("k_cache", "v_cache"))        # [B, Hk, own, d]
    y = q @ ko.transpose(-1, -2)
    seen = torch.arange(ko.shape[2], device=ko.device) < s["lengths"][:, None, None, None]
    y = torch.where(seen, y, -math.inf)
    m = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    x, y = torch.exp(x - m), torch.exp(y - m)
    z = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
    o = (x.transpose(0, 1).flatten(1, 2) @ v).unflatten(1, (B, G)).transpose(0, 1) + y @ vo
    return (o / z).flatten(1, 2).to(s["q"].dtype), (m + torch.log(z)).flatten(1)


def _plain(s):
    op = s["case"]["op"]
    if op == "shared":
        return _shared_plain(s)
    return _norm_plain(s) if op.startswith("norm") else _axes_plain(s)


# ---------------------------------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------------------------------
def _framework(s):
    from transformer_depth_wise_gb300 import api
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        y, total = api.add_rms_norm(s["x"], s["residual"], s["w"], EPS)
        return [y] if total is None else [y, total]
    if op == "norm8":
        y, scale, total = api.add_rms_norm_8bit(s["x"], s["residual"], s["w"], EPS, group=case["group"])
        return [y, scale] if total is None else [y, scale, total]
    if op == "norm_bwd":
        return api.add_rms_norm_backward(s["s"], s["w"], EPS, s["gy"], s["gs"])
    if op == "axes":
        return api.head_norm_rotate(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], EPS,
                                    interleaved=case["interleaved"], axes=s["axes"])
    if op == "axes_append":
        q = api.head_norm_rotate_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["positions"], s["inv_freq"],
                                        s["k_cache"], s["v_cache"], s["table"], EPS, interleaved=case["interleaved"],
                                        axes=s["axes"], places=s["places"])
        return q, s["k_cache"], s["v_cache"]
    if op == "axes_bwd":
        return api.head_norm_rotate_backward(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], EPS,
                                             s["gq"], s["gk"], interleaved=case["interleaved"], axes=s["axes"])
    return api.shared_prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix"], s["table"],
                                       s["lengths"], s["scale"])


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _exact_norm(s):
    case, w = s["case"], s["w"].double()
    if case["op"] == "norm_bwd":
        x, gy = s["s"].double(), s["gy"].double()
        ms = x.square().mean(-1, keepdim=True) + EPS
        dot = (gy * w * x).mean(-1, keepdim=True)
        dx = (gy * w - x * (dot / ms)) / ms.sqrt()
        return dx if s["gs"] is None else dx + s["gs"].double(), (gy * x / ms.sqrt()).sum(0)
    x = s["x"].double()
    if s["residual"] is not None:
        x = x + s["residual"].double()
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    total = [] if s["residual"] is None else [x]
    if case["op"] == "norm":
        return [y] + total
    rows, D = y.shape
    z = y.view(rows, -1, case["group"] or D)
    scale = torch.clamp(z.abs().amax(2) / TOP, min=LEAST)
    return [(z / scale.unsqueeze(2)).view(rows, D), scale] + total


def _turned(x, w, s, sign, norm=True):
    """Heads x [B, T, H, d] normed (or not) and turned by sign * their pairs' angles, as complex products."""
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    x = x.double()
    if norm:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    z = x[..., :rot].unflatten(-1, (rot // 2, 2) if inter else (2, rot // 2))
    z = torch.view_as_complex((z if inter else z.transpose(-1, -2)).contiguous())
    one = torch.nn.functional.one_hot(s["axes"].long(), s["case"]["axes"]).double()                  # [rot / 2, axes]
    a = torch.einsum("bta,pa,p->btp", s["positions"].double(), one, s["inv_freq"])[:, :, None] * sign
    z = torch.view_as_real(z * torch.polar(torch.ones_like(a), a))
    z = (z if inter else z.transpose(-1, -2)).flatten(-2)
    return torch.cat((z, x[..., rot:]), -1)


def _exact_axes(s):
    op = s["case"]["op"]
    if op == "axes_bwd":
        out = []
        for x, w, grad in ((s["q"], s["wq"], s["gq"]), (s["k"], s["wk"], s["gk"])):
            dz = _turned(grad, None, s, -1, norm=False)
            x, u = x.double(), dz * w.double()
            rms = (x.square().mean(-1, keepdim=True) + EPS).sqrt()
            out.append((u / rms - x * (u * x).mean(-1, keepdim=True) / rms ** 3, (dz * x / rms).flatten(0, 2).sum(0)))
        return out[0][0], out[1][0], out[0][1], out[1][1]
    q, k = _turned(s["q"], s["wq"], s, 1), _turned(s["k"], s["wk"], s, 1)
    if op == "axes":
        return q, k
    kc, vc, page = s["k_cache"].double(), s["v_cache"].double(), s["case"]["page"]
    table = s["table"].tolist()
    for b, row in enumerate(s["places"].tolist()):
        for t, p in enumerate(row):
            at = table[b][p // page]
            kc[at, :, p % page] = k[b, t]
            vc[at, :, p % page] = s["v"][b, t].double()
    return q, kc, vc


def _exact_shared(s):
    out, lses = [], []
    Hk, page, P = s["case"]["Hk"], s["case"]["page"], s["case"]["prefix"]
    kp, vp = (s[c][s["prefix_table"].long()].transpose(0, 1).flatten(1, 2)[:, :P].double() for c in ("k_cache", "v_cache"))
    for b, n in enumerate(s["lengths"].tolist()):
        q = s["q"][b].double().unflatten(0, (Hk, -1))
        pages = s["table"][b, :-(-n // page)].long()
        k, v = (s[c][pages].transpose(0, 1).flatten(1, 2)[:, :n].double() for c in ("k_cache", "v_cache"))
        x = torch.cat((q @ kp.transpose(1, 2), q @ k.transpose(1, 2)), -1) * s["scale"]
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[..., None])
        out.append((p[..., :P] @ vp + p[..., P:] @ v).flatten(0, 1))
        lses.append(lse.flatten())
    return torch.stack(out), torch.stack(lses)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "shared":
        return _exact_shared(s)
    return _exact_norm(s) if case["op"].startswith("norm") else _exact_axes(s)
