"""Cases and plain forms of the operators around the 8-bit projection:

  norm   residual addition + RMS norm, forward (bf16 rows, the same rows in e4m3 with one scale per 128
         columns, 1/rms) and backward (with the gradient of the residual stream)
  mm     matrix product of e4m3 operands, row scales per 128 columns and weight scales per 128 x 128 block,
         in both directions: Y = X W^T and dX = dY W
  step   one LoRA projection over a frozen e4m3 weight, forward and backward
  rope   rotary positions on the heads of a row-strided matrix, forward and backward

``run`` computes them in plain torch where ``own`` is false, and through qlora_fine_tuning_nf4_b200.ops where it
is true.  ``exact`` computes them in 64 bits, written apart from the plain form."""

import math

import torch

own = False

BLOCK = 128    # columns (rows x columns of a weight) that share a scale
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the norm in front of a projection at a full training batch (4 x 2048 tokens, width 4096)
        {"name": "norm_q8_batch", "op": "norm", "bwd": False, "M": 8192, "d": 4096, "plus_one": False},
        # the same norm for a single token
        {"name": "norm_q8_token", "op": "norm", "bwd": False, "M": 1, "d": 4096, "plus_one": False},
        # backward on a packed batch: odd row count, a width whose last block of 128 is 8 wide, gain 1 + w
        {"name": "norm_bwd_ragged", "op": "norm", "bwd": True, "M": 5003, "d": 2056, "plus_one": True},
        # gate projection of a 4096 -> 11008 MLP at a full batch: the largest product
        {"name": "mm_gate", "op": "mm", "bwd": False, "M": 8192, "K": 4096, "N": 11008},
        # input gradient of a 4096 -> 14336 projection: the reduction runs over the outputs
        {"name": "mm_dx", "op": "mm", "bwd": True, "M": 4096, "K": 4096, "N": 14336},
        # a few tokens: the weight's bytes and the launch count
        {"name": "mm_tokens", "op": "mm", "bwd": False, "M": 16, "K": 4096, "N": 4096},
        # nothing a multiple of a tile: a reduction that ends inside a block of 128, ragged rows and columns
        {"name": "mm_ragged", "op": "mm", "bwd": False, "M": 333, "K": 1040, "N": 2064},
        # one training step of an attention projection on one sequence
        {"name": "step_seq", "op": "step", "M": 2048, "K": 4096, "N": 4096, "r": 16},
        # one training step of a grouped-query k projection on a short sequence, rank 64
        {"name": "step_short", "op": "step", "M": 64, "K": 4096, "N": 1024, "r": 64},
        # the q and k heads of a fused Q/K/V output (32 + 8 heads of 128 in rows of 6144), packed sequences
        {"name": "rope_qkv", "op": "rope", "bwd": False, "M": 8192, "heads": 40, "D": 128, "rot": 128, "ld": 6144,
         "interleaved": False, "scaling": "none", "top": 2048},
        # one token at a far position
        {"name": "rope_token", "op": "rope", "bwd": False, "M": 1, "heads": 40, "D": 128, "rot": 128, "ld": 6144,
         "interleaved": False, "scaling": "linear", "top": 131072},
        # gradients of interleaved, partly rotated heads with frequencies stretched for far positions
        {"name": "rope_bwd_long", "op": "rope", "bwd": True, "M": 4099, "heads": 12, "D": 96, "rot": 64, "ld": 1200,
         "interleaved": True, "scaling": "llama3", "top": 1048576},
    ]


def _log(rng, lo, hi, mult=1):
    """A multiple of ``mult`` in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // mult * mult))


def draw(rng):
    op = rng.choice(["norm", "norm", "mm", "mm", "step", "rope", "rope"])
    if op == "norm":
        M, d = _log(rng, 1, 8192), _log(rng, 8, 16384, 8)
        while M * d > 8192 * 8192:
            M = (M + 1) // 2
        return {"op": op, "bwd": rng.random() < 0.4, "M": M, "d": d, "plus_one": rng.random() < 0.5}
    if op == "mm":
        M, K, N = _log(rng, 1, 8192), _log(rng, 64, 14336, 16), _log(rng, 16, 14336, 16)
        while M * K * N > 8192 * 4096 * 11008:
            M = (M + 1) // 2
        return {"op": op, "bwd": rng.random() < 0.5, "M": M, "K": K, "N": N}
    if op == "step":
        M, K, N = _log(rng, 1, 4096), _log(rng, 64, 8192, 16), _log(rng, 16, 8192, 16)
        while M * K * N > 2048 * 4096 * 11008:
            M = (M + 1) // 2
        return {"op": op, "M": M, "K": K, "N": N, "r": rng.choice([16, 32, 64])}
    D = rng.choice([32, 64, 80, 96, 128, 256])
    rot = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
    heads = rng.randint(1, 64)
    return {"op": op, "bwd": rng.random() < 0.5, "M": _log(rng, 1, 8192), "heads": heads, "D": D, "rot": rot,
            "ld": heads * D + 8 * rng.choice([0, 0, 1, 32, 128]), "interleaved": rng.random() < 0.5,
            "scaling": rng.choice(["none", "linear", "llama3"]), "top": _log(rng, 16, 1 << 20)}


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["M"] * c["d"]
        if c["bwd"]:  # reads H, dY, dH, 1/rms and the gain, writes dX
            return {"bytes": 8 * n + 4 * c["M"] + 2 * c["d"], "flops": 8 * n}
        # reads X, R and the gain, writes H, Y, the codes, their scales and 1/rms
        return {"bytes": 9 * n + 4 * c["M"] * _blocks(c["d"]) + 4 * c["M"] + 2 * c["d"], "flops": 8 * n}
    if c["op"] == "mm":
        M, K, N = c["M"], c["K"], c["N"]
        red, out = (N, K) if c["bwd"] else (K, N)
        return {"bytes": M * red + K * N + 4 * M * _blocks(red) + 4 * _blocks(K) * _blocks(N) + 2 * M * out,
                "flops": 2 * M * K * N}
    if c["op"] == "step":
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        return {"bytes": K * N + 4 * _blocks(K) * _blocks(N) + 4 * M * (K + N) + 4 * r * (K + N),
                "flops": 4 * M * K * N + 6 * M * r * (K + N)}
    n = c["M"] * c["heads"] * c["D"]
    return {"bytes": 4 * n + 8 * c["M"], "flops": 3 * c["M"] * c["heads"] * c["rot"]}


# ----------------------------------------------------------------- inputs --

def _quantized_rows(x):
    """bf16 [M, K] -> (e4m3 [M, K], fp32 scales [ceil(K / 128), M]), as a user's program has them in hand."""
    M, K = x.shape
    kb = _blocks(K)
    pad = torch.zeros(M, kb * BLOCK, device=x.device)
    pad[:, :K] = x
    t = pad.view(M, kb, BLOCK)
    scale = (t.abs().amax(2) / E4M3_MAX).clamp_min(2.0 ** -126)
    codes = (t / scale[:, :, None]).view(M, kb * BLOCK)[:, :K].contiguous().to(torch.float8_e4m3fn)
    return codes, scale.t().contiguous()


def _quantized_weight(w):
    """fp32 [N, K] -> (e4m3 [N, K], fp32 scales [ceil(N / 128), ceil(K / 128)])."""
    N, K = w.shape
    nb, kb = _blocks(N), _blocks(K)
    pad = torch.zeros(nb * BLOCK, kb * BLOCK, device=w.device)
    pad[:N, :K] = w
    t = pad.view(nb, BLOCK, kb, BLOCK)
    scale = (t.abs().amax((1, 3)) / E4M3_MAX).clamp_min(2.0 ** -126)
    codes = (t / scale[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:N, :K].contiguous()
    return codes.to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
    bf = torch.bfloat16
    if c["op"] == "norm":
        M, d = c["M"], c["d"]
        # hidden states: rows of different norm, a few channels far larger than the rest
        chan = torch.where(torch.rand(d, device=dev, generator=g) < 0.01, 12.0, 1.0)
        rows = 0.5 + torch.rand(M, 1, device=dev, generator=g)
        s = {"X": (normal(M, d) * 0.3).to(bf), "R": (normal(M, d) * chan * rows).to(bf),
             "w": (normal(d) * 0.1 + (0.0 if c["plus_one"] else 1.0)).to(bf)}
        if c["bwd"]:
            H = (s.pop("X").float() + s.pop("R").float()).to(bf)
            s |= {"H": H, "rstd": (1.0 / torch.sqrt(H.double().square().mean(1) + 1e-5)).float(),
                  "dY": normal(M, d).to(bf), "dH": normal(M, d).to(bf)}
    elif c["op"] == "mm":
        M, red = c["M"], c["N"] if c["bwd"] else c["K"]
        codes, scale = _quantized_rows((normal(M, red) * (0.5 + torch.rand(M, 1, device=dev, generator=g))).to(bf))
        wc, ws = _quantized_weight(normal(c["N"], c["K"]) * 0.02)
        s = {"codes": codes, "scale": scale, "w_codes": wc, "w_scale": ws}
    elif c["op"] == "step":
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        wc, ws = _quantized_weight(normal(N, K) * 0.02)
        s = {"w_codes": wc, "w_scale": ws, "X": normal(M, K).to(bf), "dY": normal(M, N).to(bf),
             "A": ((torch.rand(K, r, device=dev, generator=g) * 2 - 1) / math.sqrt(K)).to(bf),
             "B": (normal(r, N) * 0.02).to(bf), "s": 16.0 / r}
    else:
        full = normal(c["M"], c["ld"]).to(bf)
        s = {"X": full[:, :c["heads"] * c["D"]],  # rows of the fused projection's output, in place of a copy
             "positions": torch.randint(0, c["top"], (c["M"],), device=dev, generator=g)}
    return {"case": dict(case), **s}


# ------------------------------------------------------------- plain form --

def _pow2_scale(amax):
    """Smallest power of two s >= 2^-126 with amax / s <= 448, from the fp32 bits of amax."""
    e = ((amax.view(torch.int32) + 0x1FFFFF) >> 23) - 8
    return (e.clamp_min(1) << 23).view(torch.float32)


def _plain_quantize(x):
    """fp32 [M, K] -> (e4m3 values as e4m3, scales [ceil(K / 128), M]); powers of two divide exactly."""
    M, K = x.shape
    kb = _blocks(K)
    t = torch.nn.functional.pad(x, (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    scale = _pow2_scale(t.abs().amax(2))
    codes = (t / scale[:, :, None]).view(M, kb * BLOCK)[:, :K].contiguous().to(torch.float8_e4m3fn)
    return codes, scale.t().contiguous()


def _plain_rows(codes, scale):
    """e4m3 rows and their scales -> fp32 values."""
    return codes.float() * scale.t().repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _plain_weight(codes, scale):
    s = scale.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
    return codes.float() * s[:codes.shape[0], :codes.shape[1]]


def _plain_freq(c, dev):
    """Radians per position of each rotated pair."""
    f = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float64) / c["rot"])
    if c["scaling"] == "linear":
        return f / 8.0
    if c["scaling"] == "llama3":  # factor 8, low 1, high 4, trained at 8192
        wave = 2 * math.pi / f
        blend = ((8192.0 / wave - 1.0) / 3.0).clamp(0.0, 1.0)
        return (1 - blend) * f / 8.0 + blend * f
    return f


def _plain_norm(st):
    c = st["case"]
    g = st["w"].float() + (1.0 if c["plus_one"] else 0.0)
    if c["bwd"]:
        h, gdy, rstd = st["H"].float(), st["dY"].float() * g, st["rstd"][:, None]
        n = h * rstd
        return {"dX": (st["dH"].float() + rstd * (gdy - n * (n * gdy).mean(1, keepdim=True))).to(torch.bfloat16)}
    H = (st["X"].float() + st["R"].float()).to(torch.bfloat16)
    # the mean and the root in 64 bits: rstd then rounds alike in any order of the sum, and with it every value
    # that lies next to a border of the 8-bit format
    rstd = (1.0 / torch.sqrt(H.double().square().mean(1) + 1e-5)).float()
    Y = (H.float() * rstd[:, None] * g).to(torch.bfloat16)
    codes, scale = _plain_quantize(Y.float())
    return {"H": H, "Y": Y, "rstd": rstd, "codes": codes, "scale": scale}


def _plain_mm(st):
    x, w = _plain_rows(st["codes"], st["scale"]), _plain_weight(st["w_codes"], st["w_scale"])
    return {"out": (x @ w if st["case"]["bwd"] else x @ w.t()).to(torch.bfloat16)}


def _plain_step(st):
    X, dY, A, B, s = st["X"].float(), st["dY"].float(), st["A"].float(), st["B"].float(), st["s"]
    W = _plain_weight(st["w_codes"], st["w_scale"])
    XA, G = X @ A, dY @ B.t()
    out = {"Y": _plain_rows(*_plain_quantize(X)) @ W.t() + s * (XA @ B), "XA": XA,
           "dX": _plain_rows(*_plain_quantize(dY)) @ W + s * (G @ A.t()), "dA": s * (X.t() @ G),
           "dB": s * (XA.t() @ dY)}
    return {k: v.to(torch.bfloat16) for k, v in out.items()}


def _plain_rope(st):
    c, X = st["case"], st["X"]
    M, H, D, rot = c["M"], c["heads"], c["D"], c["rot"]
    angle = st["positions"].double()[:, None] * _plain_freq(c, X.device)  # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["bwd"]:
        sin = -sin
    x = X.reshape(M, H, D).float()
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).reshape(M, H, rot) if c["interleaved"] else torch.cat((u, v), -1)
    return {"out": torch.cat((r, x[..., rot:]), -1).reshape(M, H * D).to(torch.bfloat16)}


# ----------------------------------------------------------- own kernels --

def _own(st):
    from qlora_fine_tuning_nf4_b200 import ops
    c = st["case"]
    if c["op"] == "norm":
        if c["bwd"]:
            return {"dX": ops.qlora_add_rmsnorm_bwd(st["H"], st["w"], st["rstd"], st["dY"], dH=st["dH"],
                                                    plus_one=c["plus_one"])}
        H, Y, rstd, Y8 = ops.qlora_add_rmsnorm_fwd(st["X"], st["R"], st["w"], 1e-5, plus_one=c["plus_one"],
                                                   quantize=True)
        return {"H": H, "Y": Y, "rstd": rstd, "codes": Y8.codes, "scale": Y8.scale}
    if c["op"] == "rope":
        if "plan" not in st:  # the frequencies of a model, kept for all its layers and steps
            scaling = {"none": None, "linear": {"type": "linear", "factor": 8.0},
                       "llama3": {"type": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0,
                                  "original_max_position": 8192}}[c["scaling"]]
            st["plan"] = ops.rope_plan(c["rot"], base=10000.0, scaling=scaling)
        f = ops.qlora_rope_bwd if c["bwd"] else ops.qlora_rope_fwd
        return {"out": f(st["X"], c["heads"], c["D"], st["plan"], positions=st["positions"],
                         interleaved=c["interleaved"])}
    if "ws" not in st:  # the workspace a program keeps for all its calls
        st["ws"] = ops.Workspace()
    w = ops.FP8Weight(st["w_codes"], st["w_scale"])
    if c["op"] == "mm":
        f = ops.fp8_matmul_t if c["bwd"] else ops.fp8_matmul
        return {"out": f(ops.FP8Rows(st["codes"], st["scale"]), w, st["ws"])}
    lin = ops.LoraLinear8(w, st["A"], st["B"], st["s"])
    Y, XA = ops.qlora_linear8_fwd(lin, st["X"], st["ws"])
    dX, dA, dB = ops.qlora_linear8_bwd(lin, st["X"], XA, st["dY"], st["ws"])
    return {"Y": Y, "XA": XA, "dX": dX, "dA": dA, "dB": dB}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "mm": _plain_mm, "step": _plain_step, "rope": _plain_rope}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact --

def _exact_e4m3(x):
    """64-bit [M, K] -> (values on the e4m3 grid in units of the block's scale, scales [M, blocks])."""
    M, K = x.shape
    q, scales = torch.empty_like(x), []
    for lo in range(0, K, BLOCK):
        t = x[:, lo:lo + BLOCK]
        m, e = torch.frexp(t.abs().max(1).values)        # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
        p = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-126)
        p = torch.where(m == 0, torch.full_like(p, -126), p)
        s = torch.ldexp(torch.ones_like(m), p)
        v = t / s[:, None]
        ulp = torch.ldexp(torch.ones_like(v), torch.frexp(v)[1].clamp_min(-5) - 4)  # 4 significant bits, 2^-9 at least
        q[:, lo:lo + BLOCK] = torch.round(v / ulp) * ulp
        scales.append(s)
    return q, torch.stack(scales, 1)


def _exact_spread(scale, rows, cols, n, k):
    """Scales of blocks of rows x cols -> one per element of [n, k]."""
    i = torch.arange(n, device=scale.device) // rows
    j = torch.arange(k, device=scale.device) // cols
    return scale.double()[i][:, j]


def exact(case, seed):
    c, st = case, prepare(case, seed)
    f8 = lambda t: t.double()  # noqa: E731
    if c["op"] == "norm":
        gain = f8(st["w"]) + float(c["plus_one"])
        if c["bwd"]:
            h, dy = f8(st["H"]), f8(st["dY"])
            r = torch.rsqrt((h * h).sum(1) / c["d"] + 1e-5)
            dot = (h * dy * gain).sum(1) / c["d"]
            return {"dX": f8(st["dH"]) + r[:, None] * gain * dy - h * (r ** 3 * dot)[:, None]}
        h = (f8(st["X"]) + f8(st["R"])).to(torch.bfloat16).double()  # the stream is kept in bf16
        r = torch.rsqrt((h * h).sum(1) / c["d"] + 1e-5)
        y = h * r[:, None] * gain
        codes, _ = _exact_e4m3(y.to(torch.bfloat16).double())
        # a scale is a power of two: next to a border it has no value in real numbers
        return {"H": h, "Y": y, "rstd": r, "codes": codes, "scale": None}
    if c["op"] == "mm":
        M, K, N = c["M"], c["K"], c["N"]
        red = N if c["bwd"] else K
        x = f8(st["codes"].float()) * _exact_spread(st["scale"].t(), 1, BLOCK, M, red)
        w = f8(st["w_codes"].float()) * _exact_spread(st["w_scale"], BLOCK, BLOCK, N, K)
        return {"out": torch.matmul(x, w if c["bwd"] else w.transpose(0, 1))}
    if c["op"] == "step":
        M, K, N = c["M"], c["K"], c["N"]
        w = f8(st["w_codes"].float()) * _exact_spread(st["w_scale"], BLOCK, BLOCK, N, K)
        x, dy, a, b, s = f8(st["X"]), f8(st["dY"]), f8(st["A"]), f8(st["B"]), st["s"]
        qx, sx = _exact_e4m3(x)
        qd, sd = _exact_e4m3(dy)
        xv, dv = qx * _exact_spread(sx, 1, BLOCK, M, K), qd * _exact_spread(sd, 1, BLOCK, M, N)
        xa = torch.matmul(x, a)
        gb = torch.matmul(dy, b.transpose(0, 1))
        return {"Y": torch.matmul(xv, w.transpose(0, 1)) + s * torch.matmul(xa, b), "XA": xa,
                "dX": torch.matmul(dv, w) + s * torch.matmul(gb, a.transpose(0, 1)),
                "dA": s * torch.matmul(x.transpose(0, 1), gb), "dB": s * torch.matmul(xa.transpose(0, 1), dy)}
    M, H, D, rot = c["M"], c["heads"], c["D"], c["rot"]
    theta = []
    for i in range(rot // 2):
        t = math.exp(-2.0 * i / rot * math.log(10000.0))
        if c["scaling"] == "linear":
            t /= 8.0
        elif c["scaling"] == "llama3":
            turns = 8192.0 * t / (2.0 * math.pi)  # full turns within the trained length
            mix = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
            t = t * mix + t / 8.0 * (1.0 - mix)
        theta.append(t)
    theta = torch.tensor(theta, dtype=torch.float64, device="cuda")
    phi = st["positions"].double().view(M, 1, 1) * theta * (-1.0 if c["bwd"] else 1.0)
    turn = torch.complex(torch.cos(phi), torch.sin(phi))
    x = f8(st["X"].contiguous()).view(M, H, D)
    out = x.clone()
    i = torch.arange(rot // 2, device="cuda")
    re, im = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
    z = torch.complex(x[:, :, re], x[:, :, im]) * turn
    out[:, :, re], out[:, :, im] = z.real, z.imag
    return {"out": out.view(M, H * D)}
