"""Measured cases of the operators around attention and of the 4-bit layer:

  rms        residual update and root-mean-square norm, bf16 to bf16
  rms_layer  the norm to int8 codes with scales, then the W8A8 layer on them
  rotary     root-mean-square norm of each head of q and k, then rotary positions of several axes
  mx_linear  activation, microscaled 4-bit quantisation (MXFP4) and the product with MXFP4 weights
  block      residual update and norm to MXFP4, the QKV product, then norm and rotary of q and k

With `own` false, `run` computes the plain forms with elementary torch operations in fp32 (the
angles in fp64); with `own` true it calls the framework.  `exact` holds the definitions in fp64.
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the AdaNorm conditioning layer of two requests on 4-bit weights: the smallest product,
        # latency counts
        dict(name="mx_cond_2", op="mx_linear", rows=2, K=1536, N=9216, act="silu"),
        # text tokens' QKV projection
        dict(name="mx_text", op="mx_linear", rows=77, K=1536, N=4608, act="none"),
        # joint-attention out-projection, image and text tokens: ragged rows
        dict(name="mx_attn_out", op="mx_linear", rows=4429, K=1536, N=1536, act="none"),
        # FFN down-projection behind its GELU
        dict(name="mx_ffn_fc2", op="mx_linear", rows=4096, K=6144, N=1536, act="gelu"),
        # the large compute-bound product
        dict(name="mx_large", op="mx_linear", rows=9216, K=12288, N=4608, act="gelu"),
        # a text stream's tokens before their projection
        dict(name="rms_text", op="rms", rows=77, K=1536, residual=False),
        # long packed sequences with the residual update
        dict(name="rms_packed", op="rms", rows=36864, K=1536, residual=True),
        # the norm in front of a W8A8 out-projection with two K-segments
        dict(name="rms_layer", op="rms_layer", rows=333, K=1536, first=1024, residual=True, N=1536),
        # q and k of a text stream, one axis, 24 heads of 64
        dict(name="rotary_text", op="rotary", B=1, text=77, grid="0,0,0", start=0, Hq=24, Hk=24,
             D=64, widths="64", style="halves", norm=True, heads_first=False, own_pos=False),
        # joint attention: 333 text tokens before a 64x64 image, out of the packed projection
        dict(name="rotary_joint", op="rotary", B=1, text=333, grid="1,64,64", start=0, Hq=24,
             Hk=24, D=64, widths="16,24,24", style="pairs", norm=True, heads_first=False,
             own_pos=False),
        # a video far into its stream: 21 frames of 30x52, heads before tokens
        dict(name="rotary_video", op="rotary", B=1, text=0, grid="21,30,52", start=100000, Hq=12,
             Hk=12, D=128, widths="44,42,42", style="halves", norm=True, heads_first=True,
             own_pos=False),
        # transformer block entry: residual, norm, 4-bit QKV projection, norm and rotary of q and k
        dict(name="rms_qkv_rotary", op="block", B=1, text=333, grid="1,64,64", start=0, K=1536,
             Hq=24, Hk=24, D=64, widths="16,24,24", style="pairs", norm=True, own_pos=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["mx_linear", "mx_linear", "mx_linear", "rms", "rms_layer", "rotary", "rotary",
                     "block"])
    if op == "mx_linear":
        rows, K = log(1, 9216), 64 * log(1, 192)
        N = 16 * log(1, max(1, min(576, (1 << 38) // (16 * rows * K))))
        return dict(op=op, rows=rows, K=K, N=N, act=rng.choice(["none", "none", "silu", "gelu"]))
    if op == "rms":
        rows = log(1, 36864)
        K = 8 * log(1, max(1, min(2560, (1 << 25) // (4 * rows)))) - rng.choice([0, 0, 3])
        return dict(op=op, rows=rows, K=K, residual=rng.random() < 0.5)
    if op == "rms_layer":
        K = 64 * log(1, 96)
        return dict(op=op, rows=log(1, 4608), K=K, first=64 * rng.randint(1, K // 64),
                    residual=rng.random() < 0.5, N=16 * log(1, 192))
    D = rng.choice([64, 64, 128, 128, 72, 96, 40, 256])
    pairs = rng.choice([D, D, D // 2]) // 16 * 8
    axes = rng.choice([1, 2, 3, 3])
    cuts = sorted(rng.randint(0, pairs) for _ in range(axes - 1))  # an axis may have no pair
    ends = [0] + cuts + [pairs]
    widths = ",".join(str(2 * (b - a)) for a, b in zip(ends, ends[1:]))
    Hk = rng.choice([1, 2, 3, 8, 12, 24])
    Hq = Hk * rng.choice([1, 1, 1, 2, 4])
    text, kind = log(1, 512), rng.choice(["text", "image", "joint", "video"])
    side = log(1, 96)
    grid = dict(text="0,0,0", image="1,%d,%d" % (side, log(1, 96)),
                joint="1,%d,%d" % (side, side),
                video="%d,%d,%d" % (log(1, 24), log(1, 40), log(1, 56)))[kind]
    if kind in ("image", "video"):
        text = 0
    tokens = text + math.prod(map(int, grid.split(",")))
    B = max(1, min(rng.choice([1, 1, 2, 3]), (1 << 26) // (tokens * (Hq + Hk) * D)))
    common = dict(B=B, text=text, grid=grid, start=rng.choice([0, 0, log(1, 1 << 24)]), Hq=Hq,
                  Hk=Hk, D=D, widths=widths, style=rng.choice(["pairs", "halves"]),
                  norm=rng.random() < 0.7, own_pos=rng.random() < 0.3)
    if op == "rotary":
        return dict(op=op, **common, heads_first=rng.random() < 0.4)
    common.update(Hq=min(Hq, 24), Hk=min(Hk, 24), D=max(64, min(D, 128)), widths="16,24,24")
    if common["Hq"] * common["D"] % 16 or common["Hk"] * common["D"] % 16:
        common["D"] = 64
    return dict(op=op, **common, K=64 * log(1, 48))


# ---------------------------------------------------------------- prepare --
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ceil8(n):
    return -(-n // 8) * 8


def _rows(g, M, K, spread=None):
    """bf16 [M][K] of rows a multiple of 8 elements apart, the channels' spreads uneven."""
    out = torch.empty(M, _ceil8(K), device=DEV, dtype=BF)[:, :K]
    spread = torch.exp(0.5 * _normal(g, K)) if spread is None else spread
    step = max(1, (1 << 26) // max(1, K))
    for i in range(0, M, step):
        part = out[i:i + step]
        part.copy_(_normal(g, *part.shape).mul_(spread))
    return out


def _mx_weight(c, g, s, K, N):
    """An MXFP4 weight: codes 0..15 [N][K] (sign in bit 3) and block exponents [N][K / 32], and
    both in the layer's tiles."""
    w = _normal(g, N, K).mul_(torch.exp(0.5 * _normal(g, N, 1))).mul_(0.02)
    block = w.view(N, K // 32, 32)
    e = (torch.frexp(block.abs().amax(2)).exponent - 3).clamp(min=-127)
    block.mul_(torch.exp2(-e.float())[:, :, None])
    size = torch.bucketize(w.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0],
                                                 device=DEV)).to(torch.uint8)
    s["w_code"] = size + 8 * (w < 0).to(torch.uint8)
    s["w_exp"] = e.to(torch.int16)
    # tiles of 16 rows x 128 k; a byte holds two neighbours in k, the first in its low half
    kt, ks = -(-K // 128), -(-K // 512)
    code = torch.zeros(N, kt * 128, device=DEV, dtype=torch.uint8)
    code[:, :K] = s["w_code"]
    code = code[:, ::2] | code[:, 1::2] << 4
    code = code.view(N // 16, 16, kt, 4, 16).permute(0, 2, 3, 1, 4).contiguous().view(-1)
    scale = torch.zeros(N, ks * 16, device=DEV, dtype=torch.uint8)
    scale[:, :K // 32] = (e + 127).to(torch.uint8)
    scale = scale.view(N // 16, 16, ks, 4, 4).permute(0, 2, 4, 1, 3).contiguous().view(-1)
    s["w"] = (code, scale)


def _heads(c, g, s):
    """Positions of the tokens, frequencies of the pairs, and the norms' weights."""
    T, H, W = map(int, c["grid"].split(","))
    widths = [int(w) for w in c["widths"].split(",")]
    s["widths"], axes = widths, len(widths)
    at = torch.stack(torch.meshgrid(*(torch.arange(n, device=DEV) for n in (T, H, W)),
                                    indexing="ij"), -1).view(-1, 3)
    at[:, 0] += c["start"]
    words = torch.zeros(c["text"], 3, device=DEV, dtype=at.dtype)  # text counts on the first axis
    words[:, 0] = torch.arange(c["text"], device=DEV) + (c["start"] if not T else 0)
    at = torch.cat([words, at])
    at = at[:, :axes] if axes != 2 or not T else at[:, 1:]
    if c["own_pos"]:  # every sample from a place of its own
        move = torch.randint(0, 1000, (c["B"], 1, axes), generator=g, device=DEV)
        at = at + move
    s["pos"] = at.to(torch.int32).contiguous()
    s["freq"] = torch.cat([10000.0 ** (-torch.arange(0, w, 2, device=DEV, dtype=torch.float64) / w)
                           if w else torch.zeros(0, device=DEV, dtype=torch.float64)
                           for w in widths])
    for name in ("gq", "gk"):
        s[name] = 1 + 0.2 * _normal(g, c["D"]) if c["norm"] else None
    return at.shape[-2]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * int(seed) + 29)
    s = {"case": c}
    op = c["op"]
    if op == "mx_linear":
        s["z"] = _rows(g, c["rows"], c["K"])
        _mx_weight(c, g, s, c["K"], c["N"])
        s["y"] = torch.empty(c["rows"], c["N"], device=DEV, dtype=BF)
        return s
    if op in ("rotary", "block"):
        L = _heads(c, g, s)
        M, wide = c["B"] * L, (c["Hq"] + 2 * c["Hk"]) * c["D"]
        if op == "rotary":  # q and k as the projection left them
            y = _rows(g, M, wide).view(c["B"], L, -1)
            nq, nk = c["Hq"] * c["D"], c["Hk"] * c["D"]
            s["q"] = y[..., :nq].unflatten(-1, (c["Hq"], c["D"]))
            s["k"] = y[..., nq:nq + nk].unflatten(-1, (c["Hk"], c["D"]))
            for name in ("q", "k"):
                B, L, H, D = s[name].shape
                if c["heads_first"]:
                    out = torch.empty(B, H, L, D, device=DEV, dtype=BF).transpose(1, 2)
                else:
                    out = torch.empty(B, L, H, D, device=DEV, dtype=BF)
                s[name + "_out"] = out
            return s
        c["rows"], c["N"], c["residual"], c["L"] = M, wide, True, L
    M, K = c["rows"], c["K"]
    s["h"] = _rows(g, M, K)
    s["gamma"] = 1 + 0.2 * _normal(g, K)
    if c["residual"]:
        s["branch"] = _rows(g, M, K, 0.7)
        s["h_out"] = torch.empty(M, _ceil8(K), device=DEV, dtype=BF)[:, :K]
    if op == "rms":
        s["x"] = torch.empty(M, _ceil8(K), device=DEV, dtype=BF)[:, :K]
        return s
    N = c["N"]
    s["y"] = torch.empty(M, N, device=DEV, dtype=BF)
    if op == "block":
        _mx_weight(c, g, s, K, N)
        return s
    # the W8A8 layer: int8 weight (row major and in the layer's tiles), scales
    s["kseg"] = [c["first"]] + ([K - c["first"]] if c["first"] < K else [])
    s["wq"] = torch.randint(-127, 128, (K, N), generator=g, device=DEV, dtype=torch.int8)
    s["w_packed"] = (s["wq"].view(K // 64, 4, 16, N // 16, 16).permute(3, 0, 1, 4, 2)
                     .contiguous().view(-1))
    n = len(s["kseg"])
    s["w_scale"] = (0.5 + torch.rand(n, N, generator=g, device=DEV)) / (64 * math.sqrt(K))
    top = 4.5 * (0.9 + 0.2 * torch.rand(2, n, generator=g, device=DEV))
    q = torch.tensor([[127.0], [128.0]], device=DEV)
    s["act"] = torch.cat([top / q, q / top])  # s+, s-, inv+, inv-
    return s


# -------------------------------------------------------------- plain form --
def _act(t, kind):
    if kind == "silu":
        return t * torch.sigmoid(t)
    if kind == "gelu":
        return 0.5 * t * torch.special.erfc(t * -math.sqrt(0.5))
    return t


def _mx_round(x):
    """The values that bf16 x [M][K] has as MXFP4, fp32."""
    b = x.float().unflatten(1, (-1, 32))
    e = (torch.frexp(b.abs().amax(2, keepdim=True)).exponent - 3).clamp(min=-127)
    up = torch.exp2(-e.float())
    b = b * up
    v = b.abs()
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    v = (torch.round(v / step) * step).clamp(max=6.0)
    return (torch.copysign(v, b) / up).flatten(1)


def _mx_product(s, x):
    size = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    w = torch.cat([size, -size])[s["w_code"].int()].unflatten(1, (-1, 32))
    w = (w * torch.exp2(s["w_exp"].float())[:, :, None]).flatten(1)
    return (_mx_round(x) @ w.t()).to(BF)


def _rms(s):
    """h' (None without a residual) and x."""
    h, stored = s["h"].float(), None
    if s["case"]["residual"]:
        stored = (h + s["branch"].float()).to(BF)
        h = stored.float()
    x = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["gamma"]
    return stored, x.to(BF)


def _rotary(s, t, gamma):
    """t: bf16 [B][L][H][D]"""
    c, t = s["case"], t.float()
    if gamma is not None:
        t = t * torch.rsqrt(t.square().mean(3, keepdim=True) + EPS) * gamma
    R = sum(s["widths"])
    axis = torch.repeat_interleave(torch.arange(len(s["widths"]), device=DEV),
                                   torch.tensor(s["widths"], device=DEV) // 2, output_size=R // 2)
    angle = s["pos"].double()[..., axis] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if angle.dim() == 2:
        cos, sin = cos[None], sin[None]
    cos, sin = cos[:, :, None], sin[:, :, None]
    r = t[..., :R]
    a, b = (r[..., ::2], r[..., 1::2]) if c["style"] == "pairs" else r.chunk(2, 3)
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([a, b], -1).flatten(3) if c["style"] == "pairs" else torch.cat([a, b], 3)
    return torch.cat([r, t[..., R:]], 3).to(BF)


def _w8a8(s, x):
    sp, sn, ip, ineg = s["act"].repeat_interleave(
        torch.tensor(s["kseg"], device=DEV), 1, output_size=x.shape[1])
    x = x.float()
    q = torch.where(x < 0, x * ineg, x * ip).clamp(-128, 127).round()
    w = s["wq"].float() * s["w_scale"].repeat_interleave(
        torch.tensor(s["kseg"], device=DEV), 0, output_size=x.shape[1])
    return ((torch.where(q < 0, q * sn, q * sp)) @ w).to(BF)


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "mx_linear":
        return _mx_product(s, _act(s["z"].float(), c["act"]).to(BF))
    if op == "rotary":
        return {"q": _rotary(s, s["q"], s["gq"]), "k": _rotary(s, s["k"], s["gk"])}
    h, x = _rms(s)
    out = {} if h is None else {"h": h}
    if op == "rms":
        out["x"] = x
    elif op == "rms_layer":
        out["y"] = _w8a8(s, x)
    else:
        y = _mx_product(s, x).view(c["B"], c["L"], c["N"])
        nq, nk = c["Hq"] * c["D"], c["Hk"] * c["D"]
        q = _rotary(s, y[..., :nq].unflatten(2, (c["Hq"], c["D"])), s["gq"])
        k = _rotary(s, y[..., nq:nq + nk].unflatten(2, (c["Hk"], c["D"])), s["gk"])
        out["y"] = torch.cat([q.flatten(2), k.flatten(2), y[..., nq + nk:]], 2).view(-1, c["N"])
    return out


# ------------------------------------------------------------ the framework --
def _framework(s):
    import segmented_dual_scale_amd as S
    c, op = s["case"], s["case"]["op"]
    if op == "mx_linear":
        act = {"none": S.SEGQ_ACT_NONE, "silu": S.SEGQ_ACT_SILU, "gelu": S.SEGQ_ACT_GELU}[c["act"]]
        return S.segquant_gemm_mxfp4(s["z"], s["w"], c["N"], act_kind=act, out=s["y"])
    if op in ("rotary", "block"):
        style = {"pairs": S.SEGQ_ROTARY_PAIRS, "halves": S.SEGQ_ROTARY_HALVES}[c["style"]]
        head = dict(positions=s["pos"], freq=s["freq"], widths=s["widths"], style=style,
                    q_gamma=s["gq"], k_gamma=s["gk"], eps=EPS, norm=c["norm"])
    if op == "rotary":
        q, k = S.segquant_qk_rotary(s["q"], s["k"], q_out=s["q_out"], k_out=s["k_out"], **head)
        return {"q": q, "k": k}
    norm = dict(eps=EPS, gamma=s["gamma"], branch=s.get("branch"), h_out=s.get("h_out"))
    if op == "rms":
        _, x, h, _ = S.segquant_rmsnorm_quantize(s["h"], x_out=s["x"], **norm)
        return {"x": x} if h is None else {"h": h, "x": x}
    if op == "rms_layer":
        codes, _, h, _ = S.segquant_rmsnorm_quantize(s["h"], act_scales=s["act"], kseg=s["kseg"],
                                                     **norm)
        y = S.segquant_gemm_w8a8_seg(None, s["w_packed"], s["w_scale"], s["act"], s["kseg"],
                                     xq=codes, out=s["y"])
        return {"y": y} if h is None else {"h": h, "y": y}
    _, _, h, mx = S.segquant_rmsnorm_quantize(s["h"], mx_out=True, **norm)
    y = S.segquant_gemm_mxfp4(None, s["w"], c["N"], K=c["K"], xq=mx, out=s["y"])
    nq, nk, t = c["Hq"] * c["D"], c["Hk"] * c["D"], y.view(c["B"], c["L"], c["N"])
    q = t[..., :nq].unflatten(2, (c["Hq"], c["D"]))
    k = t[..., nq:nq + nk].unflatten(2, (c["Hk"], c["D"]))
    S.segquant_qk_rotary(q, k, q_out=q, k_out=k, **head)
    return {"h": h, "y": y}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------- work --
def work(case):
    c, op = case, case["op"]
    if op == "mx_linear":
        M, K, N = c["rows"], c["K"], c["N"]
        return {"bytes": 2 * M * K + N * K * 17 // 32 + 2 * M * N,
                "flops": 2 * M * K * N + 8 * M * K}
    if op in ("rotary", "block"):
        L = c["text"] + math.prod(map(int, c["grid"].split(",")))
        axes, n = len(c["widths"].split(",")), c["B"] * L * (c["Hq"] + c["Hk"]) * c["D"]
        pos = 4 * L * axes * (c["B"] if c["own_pos"] else 1)
        if op == "rotary":
            return {"bytes": 4 * n + pos, "flops": (7 if c["norm"] else 3) * n}
        M, K, N = c["B"] * L, c["K"], (c["Hq"] + 2 * c["Hk"]) * c["D"]
        return {"bytes": 6 * M * K + N * K * 17 // 32 + 2 * M * N + pos,
                "flops": 2 * M * K * N + 12 * M * K + 7 * n}
    M, K = c["rows"], c["K"]
    total = (8 if c["residual"] else 4) * M * K + 4 * K
    if op == "rms":
        return {"bytes": total, "flops": 5 * M * K}
    N = c["N"]
    return {"bytes": total - 2 * M * K + K * N + 2 * M * N, "flops": 4 * M * K * N + 9 * M * K}


# ------------------------------------------------------------------- exact --
def _exact_act(t, kind):
    if kind == "silu":
        return t / (1 + torch.exp(-t))
    if kind == "gelu":
        return torch.erfc(-t / math.sqrt(2.0)) * t / 2
    return t


def _exact_mx(s, x):
    """y of the bf16 activation x: both factors decoded by table, the sum in fp64."""
    M, K = x.shape
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    y = torch.zeros(M, s["w_code"].shape[0], dtype=torch.float64, device=DEV)
    for at in range(0, K, 2048):
        part = x[:, at:at + 2048].double()
        n = part.shape[1] // 32
        top = part.view(M, n, 32).abs().max(2).values
        # the largest power of two not above `top`, over 4, the largest one of the 4-bit values
        power = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
        power = power + (torch.exp2(power + 1) <= top).double() - (torch.exp2(power) > top).double()
        unit = torch.exp2(torch.clamp(power - 2, min=-127)).repeat_interleave(32, 1)
        v = part.abs() / unit
        # halfway cases go to the even code
        up = ((v > 0.25).long() + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5)
              + (v > 5))
        part = table[up] * unit * torch.sign(part)
        code = s["w_code"][:, at:at + 2048].long()
        w = table[code % 8] * (1 - 2 * (code // 8))
        w = w * torch.exp2(s["w_exp"][:, at // 32:at // 32 + n].double()).repeat_interleave(32, 1)
        y += part @ w.t()
    return y


def _exact_rms(s):
    h = s["h"].double()
    out = {}
    if s["case"]["residual"]:
        h = h + s["branch"].double()
        out["h"] = h
        h = h.to(BF).double()  # the norm reads the residual stream as it is stored
    out["x"] = h / torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + EPS) * s["gamma"].double()
    return out


def _exact_rotary(s, t, gamma):
    c, widths = s["case"], s["widths"]
    out = t.double()
    if gamma is not None:
        out = out / torch.sqrt((out * out).sum(3, keepdim=True) / c["D"] + EPS) * gamma.double()
    src, R, at = out.clone(), sum(widths), 0
    for axis, w in enumerate(widths):
        for j in range(w // 2):
            theta = s["pos"][..., axis].double() * 10000.0 ** (-2 * j / w)
            cos, sin = torch.cos(theta)[..., None], torch.sin(theta)[..., None]
            i = at + j
            lo, hi = (2 * i, 2 * i + 1) if c["style"] == "pairs" else (i, i + R // 2)
            out[..., lo] = src[..., lo] * cos - src[..., hi] * sin
            out[..., hi] = src[..., hi] * cos + src[..., lo] * sin
        at += w // 2
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    if op == "mx_linear":
        return _exact_mx(s, _exact_act(s["z"].double(), c["act"]).to(BF))
    if op == "rotary":
        return {"q": _exact_rotary(s, s["q"], s["gq"]), "k": _exact_rotary(s, s["k"], s["gk"])}
    out = _exact_rms(s)
    if op == "rms":
        return out
    x = out.pop("x").to(BF)
    if op == "block":
        y = _exact_mx(s, x).to(BF).double().view(c["B"], c["L"], -1)
        at = 0
        for heads, gamma in ((c["Hq"], s["gq"]), (c["Hk"], s["gk"])):
            n = heads * c["D"]
            t = y[..., at:at + n].unflatten(2, (heads, c["D"]))
            y[..., at:at + n] = _exact_rotary(s, t, gamma).flatten(2)
            at += n
        out["y"] = y.view(c["rows"], -1)
        return out
    y, at, act = 0, 0, s["act"].double()
    for i, width in enumerate(s["kseg"]):
        v = x[:, at:at + width].double()
        plus = torch.round(v.clamp(min=0) * act[2, i]).clamp(max=127) * act[0, i]
        minus = torch.round(v.clamp(max=0) * act[3, i]).clamp(min=-128) * act[1, i]
        y = y + (plus + minus) @ s["wq"][at:at + width].double() * s["w_scale"][i].double()
        at += width
    out["y"] = y
    return out
