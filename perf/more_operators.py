"""What is measured of the 4-bit products beyond a few tokens' experts and beyond q4_K: the
products of a mixture-of-experts layer grouped by expert, for any number of tokens and any
raggedness, the sort of the (token, slot) pairs that they read, and matrix-vector products with
4-bit weights that carry one scale (and zero) per group of values.

Every operator here is given in its plain form (elementary torch operations in float32) and as
the calls a program makes of the package, chosen by `own`.

The grouped products take q4_K blocks: 256 values in 144 bytes (f16 d, f16 dmin, twelve bytes of
6-bit scales sc and mins m, 128 bytes of nibbles v), value = d*sc*v - dmin*m. Activations are
float32 and enter each product as q8_1: per 32 values d = amax/127, q = round-half-away(x * (1/d)),
value = f16(d) * q, the divisions and the product rounded to float32.

The matrix-vector products take nibbles v [N, K/2] (the even value in the low four bits) with a
scale s per row and group of values and, optionally, a zero z of the scale's type, value =
s * (v - z) with z = 8 where there is none. Activations are float32, float16 or bfloat16, and so
is the result, each rounded once.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def _in(M, E, k, D, F, act="silu", gated=True, padded=0, skew=0.5):
    return {"op": "grouped_in", "M": M, "E": E, "k": k, "D": D, "F": F, "act": act,
            "gated": gated, "padded": padded, "skew": skew}


def _out(M, E, k, D, F, residual=True, padded=0, skew=0.5):
    return {"op": "grouped_out", "M": M, "E": E, "k": k, "D": D, "F": F, "residual": residual,
            "padded": padded, "skew": skew}


def _group(M, E, k, padded=0, skew=0.5):
    return {"op": "group", "M": M, "E": E, "k": k, "padded": padded, "skew": skew}


def _vec(M, N, K, group, x="f16", scale="f16", zeros=True, y=None, act="none", bias=False,
         residual=False):
    return {"op": "matvec", "M": M, "N": N, "K": K, "group": group, "x": x, "scale": scale,
            "zeros": zeros, "y": y or x, "act": act, "bias": bias, "residual": residual}


def listed():
    return [
        # a short prompt through 8 of 64 small experts: about 12 rows an expert
        dict(_in(100, 64, 8, 2048, 1024), name="in 100 of 64"),
        # experts without a gate, one device's column share of an odd width, a ragged batch
        # whose last tokens are padding
        dict(_in(300, 8, 2, 4096, 1376, act="gelu", gated=False, padded=13, skew=1.0),
             name="in 300 of 8, ungated share"),
        # a 2k-token prefill through 2 of 8 large experts: the largest case
        dict(_in(2048, 8, 2, 4096, 11008), name="in 2048 of 8"),
        dict(_out(100, 64, 8, 2048, 1024), name="out 100 of 64"),
        # a ragged prefill, an inner width of an odd number of blocks, some experts liked by most
        dict(_out(777, 64, 6, 2048, 1280, padded=9, skew=1.0), name="out 777 of 64"),
        dict(_out(2048, 8, 2, 4096, 11008), name="out 2048 of 8"),
        # the pairs of a short prompt, and of a long prefill over many experts
        dict(_group(100, 64, 8), name="group 100 of 64"),
        dict(_group(8192, 256, 8, padded=100, skew=1.0), name="group 8192 of 256"),
        # one decoded token: an attention output projection added to the residual stream
        dict(_vec(1, 4096, 4096, 128, x="f16", scale="f16", zeros=True, residual=True),
             name="matvec 1x4096x4096 f16"),
        # and a down projection in float32 with small symmetric groups
        dict(_vec(1, 4096, 11008, 32, x="f32", scale="f16", zeros=False),
             name="matvec 1x4096x11008 f32"),
        # a column share of an up projection with bias for three streams
        dict(_vec(3, 1376, 4096, 64, x="bf16", scale="bf16", zeros=False, act="gelu", bias=True),
             name="matvec 3x1376x4096 bf16"),
        # a decode batch of sixteen through a wide projection, results in float32
        dict(_vec(16, 11008, 4096, 128, x="bf16", scale="bf16", zeros=True, y="f32", act="silu"),
             name="matvec 16x11008x4096 bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("grouped_in", "grouped_out", "group", "matvec"))
    if op == "matvec":
        M, N = _log(rng, 1, 16), _log(rng, 16, 22016)
        K = 32 * _log(rng, 2, 344)
        t = rng.choice(tuple(TYPES))
        return _vec(M, N, K, rng.choice((32, 64, 128, 256, K)), t, rng.choice(("f16", "bf16")),
                    rng.random() < 0.5, rng.choice((t, "f32")), rng.choice(ACTS),
                    rng.random() < 0.5, rng.random() < 0.5)
    E = _log(rng, 4, 256 if op == "group" else 128)
    k = rng.randint(1, min(8, E))
    skew = rng.uniform(0.0, 1.5)
    if op == "group":
        M = _log(rng, 1, 16384)
        return _group(M, E, k, rng.randint(0, M // 8), skew)
    D = 256 * _log(rng, 2, 16)
    # all experts' weights together, and the products' work, stay below the largest listed
    most = max(1, min(16, (8 * 4096 * 11008) // (E * D * 256)))
    F = 256 * _log(rng, 1, most)
    M = _log(rng, 1, 4096)
    M = max(1, min(M, 2048 * 2 * 4096 * 11008 // (k * D * F)))
    padded = rng.randint(0, M // 8)
    if op == "grouped_out":
        return _out(M, E, k, D, F, rng.random() < 0.5, padded, skew)
    return _in(M, E, k, D, F if rng.random() < 0.5 else max(16, F - rng.randint(1, 255)),
               rng.choice(ACTS[1:]), rng.random() < 0.7, padded, skew)


# ---------------------------------------------------------------- inputs

def _q4k(rows, K, g, dev):
    """q4_K blocks [rows, K/256, 144] fitted to N(0, 0.02) weights, as a quantizer writes them:
    per 32 values the range [min(0, least), greatest] on 16 levels."""
    w = torch.randn(rows, K // 256, 8, 32, generator=g, device=dev).mul_(0.02)
    lo = w.amin(-1).clamp_(max=0.0)
    step = (w.amax(-1) - lo) / 15.0
    d = (step.amax(-1, keepdim=True) / 63.0).half()
    dmin = ((-lo).amax(-1, keepdim=True) / 63.0).half()
    sc = (step / d.float()).round_().nan_to_num_(0.0).clamp_(0, 63)
    m = (-lo / dmin.float()).round_().nan_to_num_(0.0).clamp_(0, 63)
    low, size = (dmin.float() * m).unsqueeze(-1), (d.float() * sc).unsqueeze(-1)
    v = ((w + low) / size).nan_to_num_(0.0, 0.0, 0.0).round_().clamp_(0, 15).to(torch.uint8)
    sc, m = sc.to(torch.uint8), m.to(torch.uint8)
    out = torch.empty(rows, K // 256, 144, dtype=torch.uint8, device=dev)
    out[..., 0:2] = d.view(torch.uint8)
    out[..., 2:4] = dmin.view(torch.uint8)
    out[..., 4:8] = sc[..., :4] | ((sc[..., 4:] >> 4) << 6)
    out[..., 8:12] = m[..., :4] | ((m[..., 4:] >> 4) << 6)
    out[..., 12:16] = (sc[..., 4:] & 15) | ((m[..., 4:] & 15) << 4)
    out[..., 16:] = (v[..., 0::2, :] | (v[..., 1::2, :] << 4)).flatten(-2)
    return out


def _q4g(N, K, group, scale, zeros, g, dev):
    """Nibbles [N, K/2], scales and zeros [N, ceil(K/group)] (zeros None where symmetric) fitted
    to N(0, 0.02) weights; a zero is the whole number that the quantizer rounds it to."""
    n = -(-K // group)
    w = torch.zeros(N, n * group, device=dev)
    w[:, :K] = torch.randn(N, K, generator=g, device=dev).mul_(0.02)
    w = w.unflatten(1, (n, group))
    if zeros:
        lo, hi = w.amin(-1).clamp_(max=0.0), w.amax(-1).clamp_(min=0.0)
        s = ((hi - lo) / 15.0).to(TYPES[scale])
        z = (-lo / s.float()).round_().nan_to_num_(0.0).clamp_(0, 15).to(TYPES[scale])
        v = (w / s.float().unsqueeze(-1) + z.float().unsqueeze(-1)).nan_to_num_(0.0)
    else:
        s = (w.abs().amax(-1) / 7.5).to(TYPES[scale])
        z = None
        v = (w / s.float().unsqueeze(-1)).nan_to_num_(0.0) + 8.0
    v = v.round_().clamp_(0, 15).to(torch.uint8).flatten(1)[:, :K]
    return (v[:, 0::2] | (v[:, 1::2] << 4)).contiguous(), s, z


def _acts(rows, K, g, dev):
    """N(0, 1) activations with one value in a thousand twenty times as large, as the residual
    stream of a language model has them."""
    x = torch.randn(rows, K, generator=g, device=dev)
    return torch.where(torch.rand(rows, K, generator=g, device=dev) < 0.001, 20.0 * x, x)


def _top(c, g, dev):
    """The experts of each token, int32 [M, k], and their logits; `skew` is how far the tokens
    agree. Tokens of the padding, the last ones, name no expert."""
    M, E = c["M"], c["E"]
    logits = (1.5 * torch.randn(M, E, generator=g, device=dev)
              + c["skew"] * torch.randn(E, generator=g, device=dev))
    top = logits.topk(c["k"], dim=1)
    ids = top.indices.to(torch.int32)
    if c["padded"]:
        ids[M - c["padded"]:] = -1
    return ids, top.values


def _package():
    import q4_q8_int8_amd as mmq
    return mmq


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    op, M = case["op"], case["M"]
    s = {"case": dict(case)}
    if op == "matvec":
        N, K = case["N"], case["K"]
        s["x"] = _acts(M, K, g, dev).to(TYPES[case["x"]])
        s["w"], s["scale"], s["zero"] = _q4g(N, K, case["group"], case["scale"], case["zeros"],
                                             g, dev)
        s["bias"] = 0.1 * torch.randn(N, generator=g, device=dev) if case["bias"] else None
        s["residual"] = (_acts(M, N, g, dev).to(TYPES[case["y"]]) if case["residual"] else None)
    elif op == "group":
        s["ids"] = _top(case, g, dev)[0]
    else:
        E, k, D, F = case["E"], case["k"], case["D"], case["F"]
        s["ids"], best = _top(case, g, dev)
        if op == "grouped_in":
            s["x"] = _acts(M, D, g, dev)
            s["up"] = torch.stack([_q4k(F, D, g, dev) for _ in range(E)])
            s["gate"] = (torch.stack([_q4k(F, D, g, dev) for _ in range(E)])
                         if case["gated"] else None)
        else:
            a = torch.randn(M * k, F, generator=g, device=dev)
            s["h"] = a * torch.sigmoid(a) * torch.randn(M * k, F, generator=g, device=dev)
            s["weights"] = torch.softmax(best, dim=1)
            s["residual"] = _acts(M, D, g, dev) if case["residual"] else None
            s["down"] = torch.stack([_q4k(D, F, g, dev) for _ in range(E)])
        # the pairs of every expert that has some, as the plain form wants them
        flat = s["ids"].flatten().cpu()
        s["pairs"] = [(e, (flat == e).nonzero().flatten().to(dev)) for e in range(E)
                      if bool((flat == e).any())]
    if own:
        _keep(s, dev)
    return s


def _keep(s, dev):
    """What a program keeps beside its inputs: repacked weights, scratch, output buffers and,
    for the experts' products, the pairs sorted by expert."""
    mmq, c = _package(), s["case"]
    op, M = c["op"], c["M"]

    def raw(n):
        return torch.empty(max(n, 16), dtype=torch.uint8, device=dev)

    if op == "matvec":
        N, K = c["N"], c["K"]
        s["format"] = mmq.q4G_format(c["group"], TYPES[c["scale"]], c["zeros"])
        s["rep"] = raw(mmq.mmq_q4G_repacked_bytes(N, K, s["format"]))
        mmq.repack_q4_G(s["w"], s["scale"], s["zero"], N, K, s["format"], s["rep"])
        s["y"] = torch.empty(M, N, dtype=TYPES[c["y"]], device=dev)
        s["act"] = mmq.ACTIVATIONS[c["act"]]
        return
    E, k = c["E"], c["k"]
    s["groups"] = torch.empty(mmq.mmq_moe_group_bytes(M, E, k) // 4, dtype=torch.int32,
                              device=dev)
    if op == "group":
        return
    mmq.mmq_moe_group(M, E, k, s["ids"], s["groups"])
    D, F = c["D"], c["F"]
    if op == "grouped_in":
        if c["gated"]:
            n = mmq.mmq_q4K_pair_bytes(F, D)
            s["rep"] = raw(E * n)
            for e in range(E):
                mmq.repack_q4_K_pair(s["gate"][e], s["up"][e], F, D, s["rep"][e * n:(e + 1) * n])
        else:
            n = mmq.mmq_q4K_repacked_bytes(F, D)
            s["rep"] = raw(E * n)
            for e in range(E):
                mmq.repack_q4_K(s["up"][e], F, D, s["rep"][e * n:(e + 1) * n])
        s["q8"] = raw(mmq.mmq_q8_1_bytes(M, D))
        # rows of pairs without an expert stay as they are
        s["H"] = torch.zeros(M * k, F, dtype=torch.float32, device=dev)
        s["act"] = mmq.ACTIVATIONS[c["act"]]
    else:
        n = mmq.mmq_q4K_repacked_bytes(D, F)
        s["rep"] = raw(E * n)
        for e in range(E):
            mmq.repack_q4_K(s["down"][e], D, F, s["rep"][e * n:(e + 1) * n])
        s["workspace"] = raw(mmq.mmq_grouped_down_workspace_bytes(M, E, k, D, F))
        s["out"] = torch.empty(M, D, dtype=torch.float32, device=dev)


# ---------------------------------------------------------------- the operators

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    mmq, c = _package(), s["case"]
    op, M = c["op"], c["M"]
    if op == "matvec":
        mmq.mmq_q4G(M, c["N"], c["K"], s["x"], s["rep"], s["format"], s["y"], bias=s["bias"],
                    residual=s["residual"], act=s["act"])
        return s["y"]
    E, k = c["E"], c["k"]
    if op == "group":
        mmq.mmq_moe_group(M, E, k, s["ids"], s["groups"])
        offsets, order, place = mmq.moe_groups(s["groups"], M, E, k)
        return {"offsets": offsets, "order": order, "place": place}
    if op == "grouped_in":
        call = mmq.mmq_q4K_grouped_gated if c["gated"] else mmq.mmq_q4K_grouped
        call(M, E, k, c["F"], c["D"], s["x"], s["groups"], s["rep"], s["H"], s["q8"],
             act=s["act"])
        return s["H"]
    mmq.mmq_q4K_grouped_down(M, E, k, c["D"], c["F"], s["h"], s["groups"], s["weights"],
                             s["rep"], s["out"], s["workspace"], residual=s["residual"])
    return s["out"]


def _q8(x):
    """The values that q8_1 holds for x [rows, K]. The quotients are taken in float64 and
    rounded to float32, which is their correctly rounded float32 value."""
    b = x.unflatten(-1, (-1, 32))
    d = (b.abs().amax(-1, keepdim=True).double() / 127.0).float()
    inv = torch.where(d > 0, (1.0 / d.double()).float(), 0.0)
    p = b * inv
    t = p.trunc()
    q = (t + torch.where((p - t).abs() >= 0.5, p.sign(), 0.0)).clamp(-127.0, 127.0)
    return (q * d.half().float()).flatten(-2)


def _decode(w):
    """float32 values [..., rows, K] of q4_K blocks [..., rows, K/256, 144]."""
    head = w[..., :4].contiguous().view(torch.float16).float()
    s = w[..., 4:16]
    sc = torch.cat((s[..., 0:4] & 63, (s[..., 8:12] & 15) | ((s[..., 0:4] >> 6) << 4)), -1)
    m = torch.cat((s[..., 4:8] & 63, (s[..., 8:12] >> 4) | ((s[..., 4:8] >> 6) << 4)), -1)
    n = w[..., 16:].unflatten(-1, (4, 32))
    v = torch.stack((n & 15, n >> 4), -2).flatten(-3, -2).float()
    scale = (head[..., 0:1] * sc.float()).unsqueeze(-1)
    low = (head[..., 1:2] * m.float()).unsqueeze(-1)
    return (v * scale - low).flatten(-3)


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)
        return v / (1.0 + torch.exp(-2.0 * u))
    return v


def _run_plain(s):
    c = s["case"]
    op, M = c["op"], c["M"]
    if op == "matvec":
        y = s["x"].float() @ _matrix(s, c).T
        if s["bias"] is not None:
            y = y + s["bias"]
        y = _act(y, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(TYPES[c["y"]])
    if op == "group":
        return _group_plain(s["ids"].flatten(), c["E"])
    k, D, F = c["k"], c["D"], c["F"]
    if op == "grouped_in":
        a = _q8(s["x"])
        h = torch.zeros(M * k, F, device=a.device)
        for e, p in s["pairs"]:
            rows = a[p // k]
            u = rows @ _decode(s["up"][e]).T
            h[p] = (_act(rows @ _decode(s["gate"][e]).T, c["act"]) * u if c["gated"]
                    else _act(u, c["act"]))
        return h
    a = _q8(s["h"])
    y = torch.zeros(M * k, D, device=a.device)
    for e, p in s["pairs"]:
        y[p] = a[p] @ _decode(s["down"][e]).T
    y = (y.unflatten(0, (M, k)) * s["weights"].unsqueeze(-1)).sum(1)
    return y if s["residual"] is None else y + s["residual"]


def _matrix(s, c):
    """float32 values [N, K] of the weights of a matrix-vector product."""
    v = torch.stack((s["w"] & 15, s["w"] >> 4), -1).flatten(1).float()
    each = torch.arange(c["K"], device=v.device) // c["group"]
    z = 8.0 if s["zero"] is None else s["zero"].float()[:, each]
    return (v - z) * s["scale"].float()[:, each]


def _group_plain(flat, E):
    """Where each expert's pairs begin, the pairs sorted by expert (those without one are -1, at
    the end) and the place of every pair among them (-1 without one)."""
    P, dev = flat.numel(), flat.device
    named = (flat >= 0) & (flat < E)
    count = (flat == torch.arange(E, device=dev).unsqueeze(1)).sum(1)
    offsets = torch.cat((torch.zeros_like(count[:1]), count.cumsum(0)))
    order = torch.sort(torch.where(named, flat, E), stable=True).indices
    at = torch.arange(P, device=dev)
    place = torch.empty_like(order)
    place[order] = at
    return {"offsets": offsets.to(torch.int32),
            "order": torch.where(at < offsets[-1], order, -1).to(torch.int32),
            "place": torch.where(named, place, -1).to(torch.int32)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, M = case["op"], case["M"]
    if op == "matvec":
        N, K = case["N"], case["K"]
        size = {"f32": 4, "f16": 2, "bf16": 2}
        read = N * K // 2 + N * -(-K // case["group"]) * (4 if case["zeros"] else 2)
        read += size[case["x"]] * M * K + (4 * N if case["bias"] else 0)
        read += size[case["y"]] * M * N if case["residual"] else 0
        return {"bytes": read + size[case["y"]] * M * N, "flops": 2 * M * N * K}
    E, k = case["E"], case["k"]
    P = M * k
    if op == "group":
        return {"bytes": 12 * P + 4 * (E + 1), "flops": P}
    D, F = case["D"], case["F"]
    used = E * (1.0 - (1.0 - k / E) ** M)  # experts that at least one of M tokens names
    P -= case["padded"] * k
    if op == "grouped_in":
        n = 2 if case["gated"] else 1
        return {"bytes": 4 * M * D + int(used * n * F * D * 144 / 256) + 4 * P * (F + 1),
                "flops": 2 * n * P * F * D}
    return {"bytes": (4 * P * (F + 2) + int(used * F * D * 144 / 256)
                      + (8 if case["residual"] else 4) * M * D),
            "flops": 2 * P * F * D}


# ---------------------------------------------------------------- the definition in 64 bits

def _values64(w):
    """float64 values of q4_K blocks, sub-block by sub-block from the format's definition."""
    b = w.to(torch.int32)
    d = w[..., 0:2].contiguous().view(torch.float16)[..., 0].double()
    dmin = w[..., 2:4].contiguous().view(torch.float16)[..., 0].double()
    parts = []
    for j in range(8):
        if j < 4:
            sc, m = b[..., 4 + j] % 64, b[..., 8 + j] % 64
        else:
            sc = b[..., 8 + j] % 16 + 16 * (b[..., j] // 64)
            m = b[..., 8 + j] // 16 + 16 * (b[..., 4 + j] // 64)
        n = b[..., 16 + 32 * (j // 2):48 + 32 * (j // 2)]
        v = n // 16 if j % 2 else n % 16
        parts.append((d * sc).unsqueeze(-1) * v - (dmin * m).unsqueeze(-1))
    return torch.cat(parts, -1).reshape(*w.shape[:-2], -1)


def _tokens64(x):
    """float64 values of the q8_1 blocks of x; the scale, its reciprocal and the scaled value
    are float32 by the format's definition."""
    b = x.reshape(x.shape[0], -1, 32).double()
    d = (b.abs().max(-1, keepdim=True).values / 127.0).float().double()
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d)).float().double()
    p = (b * inv).float().double()
    q = torch.copysign(torch.floor(p.abs() + 0.5), p).clamp(-127.0, 127.0)
    return (q * d.to(torch.float16).double()).reshape(x.shape)


def _act64(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op, M = case["op"], case["M"]
    if op == "group":
        return None
    if op == "matvec":
        N, K, group = case["N"], case["K"], case["group"]
        x = s["x"].double()
        y = torch.zeros(M, N, dtype=torch.float64, device=x.device)
        b = s["w"].to(torch.int32)
        v = torch.empty(N, K, dtype=torch.float64, device=x.device)
        v[:, 0::2], v[:, 1::2] = (b % 16).double(), (b // 16).double()
        for i, k0 in enumerate(range(0, K, group)):
            z = 8.0 if s["zero"] is None else s["zero"][:, i:i + 1].double()
            part = x[:, k0:k0 + group] @ (v[:, k0:k0 + group] - z).T
            y += part * s["scale"][:, i].double()
        y = _act64(y if s["bias"] is None else y + s["bias"].double(), case["act"])
        return y if s["residual"] is None else y + s["residual"].double()
    k, D, F = case["k"], case["D"], case["F"]
    ids = s["ids"].flatten().tolist()
    pairs = {}
    for p, e in enumerate(ids):
        if e >= 0:
            pairs.setdefault(e, []).append(p)
    dev = s["ids"].device
    if op == "grouped_in":
        a = _tokens64(s["x"])
        h = torch.zeros(M * k, F, dtype=torch.float64, device=dev)
        for e, ps in pairs.items():
            at = torch.tensor(ps, device=dev)
            t = a[torch.tensor([p // k for p in ps], device=dev)]
            u = t @ _values64(s["up"][e]).T
            h[at] = (_act64(t @ _values64(s["gate"][e]).T, case["act"]) * u if case["gated"]
                     else _act64(u, case["act"]))
        return h
    a = _tokens64(s["h"])
    out = (torch.zeros(M, D, dtype=torch.float64, device=dev) if s["residual"] is None
           else s["residual"].double())
    weights = s["weights"].flatten().double()
    for e, ps in pairs.items():
        at = torch.tensor(ps, device=dev)
        y = (a[at] @ _values64(s["down"][e]).T) * weights[at].unsqueeze(1)
        out.index_add_(0, torch.tensor([p // k for p in ps], device=dev), y)
    return out
