"""What is measured of the layer's linear maps and their 8-bit activation checkpoints.

Operators (n tokens, `cin` input channels, `cout` output channels):

  fwd      Y = act(X W^T + b) + R, the matrix product with bias, activation and residual in its epilogue;
           optionally the pre-activation Z = X W^T + b is saved too (bf16)
  bwd      dZ = dY * act'(Z), dX = dZ W, dW = dZ^T X, db = column sums of dZ; X and Z are held in bf16
           or as 8-bit checkpoints
  train    fwd that saves X and Z as 8-bit checkpoints, and the bwd that uses them
  roundtrip, unpack   the checkpoint of an activation written and read back, or read back alone

A checkpoint holds signed 8-bit codes and one power-of-two scale 2^(s - 127) per block of 32 channels of a
row: s is the smallest exponent >= 1 with max|x| <= 127 * 2^(s - 127), and a code is x / scale rounded to
nearest, ties to even.  Rows of codes are padded to a multiple of 128 channels.
"""
import math

import torch

own = False

BLOCK = 32
ACTS = ("none", "relu", "silu", "gelu")  # gelu: the tanh form


def listed():
    return [
        # the step embedding of a sampler: one token through a small MLP's first matrix; latency
        dict(name="fwd_one_token", op="fwd", n=1, cin=1024, cout=4096, act="silu", bias=True, residual=False, save=False),
        # an odd number of prompt tokens, odd channel counts, pre-activation kept for the backward
        dict(name="fwd_ragged", op="fwd", n=1003, cin=1000, cout=1416, act="gelu", bias=True, residual=True, save=True),
        # output projection of the 24x48x80 grid, 8 heads of 128, added to the residual stream
        dict(name="fwd_out_proj", op="fwd", n=92160, cin=1024, cout=1024, act="none", bias=True, residual=True, save=False),
        # feed-forward expansion of the same grid
        dict(name="fwd_ffn_up", op="fwd", n=92160, cin=1024, cout=4096, act="gelu", bias=True, residual=False, save=False),
        # feed-forward contraction of the 16x24x40 grid
        dict(name="fwd_ffn_down", op="fwd", n=15360, cin=4096, cout=1024, act="none", bias=True, residual=True, save=False),
        # gradients of the query projection of the 8x16x16 grid, three heads of 64
        dict(name="bwd_tiny_grid", op="bwd", n=2048, cin=192, cout=192, act="none", x8=False, z8=False, bias=False, fp32=True),
        # gradients of the output projection of the 24x48x80 grid, X saved in bf16, weight gradient in fp32
        dict(name="bwd_out_proj", op="bwd", n=92160, cin=1024, cout=1024, act="none", x8=False, z8=False, bias=True, fp32=True),
        # the feed-forward expansion's gradients from 8-bit checkpoints
        dict(name="bwd_ffn_up_ckpt", op="bwd", n=92160, cin=1024, cout=4096, act="gelu", x8=True, z8=True, bias=True, fp32=False),
        # a training step of a ragged batch through checkpoints
        dict(name="train_ragged", op="train", n=2011, cin=520, cout=1288, act="silu", bias=True, residual=True),
        # an attention tensor of the 32x72x120 grid (8 heads of 128) saved in the forward and restored in the backward
        dict(name="roundtrip_1080p", op="roundtrip", n=276480, width=1024, pad=0),
        # a few strided rows (one head group of a fused projection)
        dict(name="roundtrip_strided", op="roundtrip", n=1003, width=328, pad=696),
        # a feed-forward pre-activation restored
        dict(name="unpack_ffn", op="unpack", n=92160, width=4096, pad=0),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _channels(rng):
    return max(64, min(4096, int(_log(rng, 64, 4096)) // 8 * 8))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "bwd", "train", "roundtrip", "unpack"))
    if op in ("roundtrip", "unpack"):
        width = _channels(rng)
        n = max(1, min(int(_log(rng, 1, 300000)), 377_000_000 // width))
        return dict(op=op, n=n, width=width, pad=rng.choice((0, 0, 8, 264)))
    cin, cout = _channels(rng), _channels(rng)
    act = rng.choice(ACTS)
    # at most the work of the largest listed backward
    n = max(1, min(int(_log(rng, 1, 100000)), 386_000_000_000 // (cin * cout) // (2 if op == "train" else 1)))
    if op == "fwd":
        return dict(op=op, n=n, cin=cin, cout=cout, act=act, bias=rng.random() < 0.7, residual=rng.random() < 0.5,
                    save=rng.random() < 0.3)
    if op == "bwd":
        return dict(op=op, n=n, cin=cin, cout=cout, act=act, x8=rng.random() < 0.5, z8=act != "none" and rng.random() < 0.5,
                    bias=rng.random() < 0.7, fp32=act == "none" and rng.random() < 0.7)
    return dict(op=op, n=n, cin=cin, cout=cout, act=act, bias=True, residual=rng.random() < 0.5)


def work(case):
    n = case["n"]
    if case["op"] in ("roundtrip", "unpack"):
        w = case["width"]
        held, plain = n * (w + -(-w // BLOCK)), 2 * n * w
        # unpack: codes and scales read, values written; roundtrip: values read and written, and what is held
        # written once and read once
        return {"bytes": held + plain if case["op"] == "unpack" else 2 * held + 2 * plain, "flops": 0}
    ci, co = case["cin"], case["cout"]
    x, w, y = n * ci, ci * co, n * co

    def eight(k, c):
        return n * (c + -(-c // BLOCK)) if k else 2 * n * c

    if case["op"] == "fwd":
        by = 2 * (x + w + y) + (2 * co if case["bias"] else 0) + (2 * y if case["residual"] else 0) + (2 * y if case["save"] else 0)
        return {"bytes": by, "flops": 2 * n * ci * co}
    has_z = case["act"] != "none"
    g = 4 if case.get("fp32") else 2
    bwd = 2 * y + eight(case.get("x8", True), ci) + 2 * w + 2 * x + g * w + (g * co if case["bias"] else 0)
    bwd += eight(case.get("z8", True), co) if has_z else 0
    if case["op"] == "bwd":
        return {"bytes": bwd, "flops": 4 * n * ci * co}
    fwd = 2 * (x + w + y) + 2 * co + (2 * y if case["residual"] else 0) + eight(True, ci) + (eight(True, co) if has_z else 0)
    return {"bytes": fwd + bwd, "flops": 6 * n * ci * co}


# --------------------------------------------------------------------------------------------- inputs


def _activations(n, c, g, pad=0):
    """Normal values whose channels differ in size, a few of them much larger, as activations have."""
    scale = torch.exp(0.5 * torch.randn(c, generator=g, device="cuda"))
    scale[torch.randint(0, c, (max(1, c // 128),), generator=g, device="cuda")] *= 8
    x = torch.empty(n, c + pad, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // c)
    for at in range(0, n, step):
        m = min(step, n - at)
        x[at:at + m, :c] = torch.randn(m, c, generator=g, device="cuda") * scale
        if pad:
            x[at:at + m, c:] = 0
    return x[:, :c]


def _held(x):
    """A checkpoint of x for the cases that start from one: codes [n, ld] int8 and scales [n, ld / 32] uint8."""
    n, c = x.shape
    ld = -(-c // 128) * 128
    codes = torch.zeros(n, ld, dtype=torch.int8, device=x.device)
    scales = torch.ones(n, ld // BLOCK, dtype=torch.uint8, device=x.device)
    step = max(1, (1 << 26) // ld)
    for at in range(0, n, step):
        q, s = _codes(x[at:at + step].float())
        codes[at:at + step] = q.to(torch.int8).reshape(-1, ld)
        scales[at:at + step] = s.to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    n = case["n"]
    if case["op"] in ("roundtrip", "unpack"):
        x = _activations(n, case["width"], g, case["pad"])
        if case["op"] == "roundtrip":
            s["x"] = x
        else:
            s["codes"], s["scales"] = _held(x)
            s["room"] = torch.empty(n, case["width"] + case["pad"], dtype=torch.bfloat16, device="cuda")[:, :case["width"]]
        return s
    ci, co = case["cin"], case["cout"]
    x = _activations(n, ci, g)
    s["w"] = (torch.randn(co, ci, generator=g, device="cuda") / ci ** 0.5).to(torch.bfloat16)
    s["b"] = (0.5 * torch.randn(co, generator=g, device="cuda")).to(torch.bfloat16) if case["bias"] else None
    if case.get("residual"):
        s["r"] = torch.randn(n, co, generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] != "fwd":
        s["dy"] = torch.randn(n, co, generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] == "bwd":
        s["x"] = _held(x) if case["x8"] else x
        if case["act"] != "none":
            z = torch.randn(n, co, generator=g, device="cuda").to(torch.bfloat16) * 1.5
            s["z"] = _held(z) if case["z8"] else z
    else:
        s["x"] = x
    return s


# ----------------------------------------------------------------------------------------- plain forms


def _codes(x):
    """x fp32 [n, c] -> codes [n, blocks, 32] and biased exponents [n, blocks] over rows padded to 128."""
    n, c = x.shape
    ld = -(-c // 128) * 128
    b = torch.nn.functional.pad(x, (0, ld - c)).reshape(n, ld // BLOCK, BLOCK)
    top = b.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1
    s = torch.where(m > 127 / 128, e - 6, e - 7).clamp(min=-126)
    s = torch.where(top > 0, s, torch.full_like(s, -126))
    # division by a power of two, in two steps so that the factor itself stays representable
    half = torch.div(s, 2, rounding_mode="floor")
    q = torch.ldexp(torch.ldexp(b, -half[..., None]), -(s - half)[..., None])
    return torch.round(q), s + 127


def _values(codes, scales, c):
    n = codes.shape[0]
    q = codes.reshape(n, -1, BLOCK).float()
    return torch.ldexp(q, (scales.to(torch.int32) - 127)[..., None]).reshape(n, -1)[:, :c]


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    v = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
    return z / (1 + torch.exp(-v))


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    k = math.sqrt(2 / math.pi)
    v, dv = (z, 1.0) if act == "silu" else (2 * k * (z + 0.044715 * z * z * z), 2 * k * (1 + 3 * 0.044715 * z * z))
    p, q = 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
    return p + z * p * q * dv


def _plain_fwd(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s.get("residual"):
        y = y + s["r"].float()
    return z, y.to(torch.bfloat16)


def _plain_bwd(s, x, z):
    dz = s["dy"].float()
    if s["act"] != "none":
        dz = dz * _slope(z, s["act"])
    out = torch.float32 if s.get("fp32") else torch.bfloat16
    r = {"dX": (dz @ s["w"].float()).to(torch.bfloat16), "dW": (dz.t() @ x).to(out)}
    if s["bias"]:
        r["db"] = dz.double().sum(0).to(out)
    return r


def _run_plain(s):
    if s["op"] == "roundtrip":
        return _values(*_codes(s["x"].float()), s["width"]).to(torch.bfloat16)
    if s["op"] == "unpack":
        return _values(s["codes"], s["scales"], s["width"]).to(torch.bfloat16)
    if s["op"] == "fwd":
        z, y = _plain_fwd(s)
        return {"Y": y, "Z": z.to(torch.bfloat16)} if s["save"] else {"Y": y}
    if s["op"] == "bwd":
        x = _values(*s["x"], s["cin"]) if s["x8"] else s["x"].float()
        z = None
        if s["act"] != "none":
            z = _values(*s["z"], s["cout"]) if s["z8"] else s["z"].float()
        return _plain_bwd(s, x, z)
    z, y = _plain_fwd(s)
    held = _values(*_codes(z), s["cout"]) if s["act"] != "none" else None
    return {"Y": y, **_plain_bwd(s, _values(*_codes(s["x"].float()), s["cin"]), held)}


# ------------------------------------------------------------------------------- the framework's calls


def _run_own(s):
    from dynamic_block_sparse_stats_b200 import api
    op = s["op"]
    if op == "roundtrip":
        return api.ckpt8_unpack(api.ckpt8_pack(s["x"]))
    if op == "unpack":
        return api.ckpt8_unpack(api.Ckpt8(s["codes"], s["scales"], s["width"]), out=s["room"])
    act = {"none": api.ACT_NONE, "relu": api.ACT_RELU, "silu": api.ACT_SILU, "gelu": api.ACT_GELU}[s["act"]]
    need = ("dX", "dW", "db") if s["bias"] else ("dX", "dW")

    def held(v, c, is8):
        return api.Ckpt8(*v, c) if is8 else v

    if op == "fwd":
        f = api.linear_fwd(s["x"], s["w"], s["b"], act=act, residual=s.get("r"), save="bf16" if s["save"] else None)
        return {"Y": f.Y, "Z": f.Z} if s["save"] else {"Y": f.Y}
    if op == "bwd":
        z = held(s["z"], s["cout"], s["z8"]) if s["act"] != "none" else None
        b = api.linear_bwd(s["dy"], held(s["x"], s["cin"], s["x8"]), s["w"], Z=z, act=act, need=need, grad_fp32=s["fp32"])
        r = {}
    else:
        x8 = api.ckpt8_pack(s["x"])
        f = api.linear_fwd(s["x"], s["w"], s["b"], act=act, residual=s.get("r"), save="ckpt8" if s["act"] != "none" else None)
        b = api.linear_bwd(s["dy"], x8, s["w"], Z=f.Z, act=act, need=need)
        r = {"Y": f.Y}
    r.update(dX=b.dX, dW=b.dW)
    if s["bias"]:
        r["db"] = b.db
    return r


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------- in 64 bits


def _exact_round8(x):
    """The values that a checkpoint of x (float64) stands for."""
    n, c = x.shape
    b = torch.zeros(n, -(-c // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    b[:, :c] = x
    b = b.view(n, -1, BLOCK)
    e = torch.ceil(torch.log2(b.abs().amax(-1, keepdim=True) / 127))
    e = torch.where(torch.isfinite(e), e, torch.full_like(e, -126)).clamp(min=-126)
    # the logarithm is rounded: settle the two neighbours by the definition itself
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 127 * torch.exp2(e), e + 1, e)
    e = torch.where((top <= 127 * torch.exp2(e - 1)) & (e > -126), e - 1, e)
    q = torch.exp2(e)
    return (torch.round(b / q) * q).view(n, -1)[:, :c]


def _exact_restore(codes, scales, c):
    q = torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, dim=1)
    return (codes.double() * q)[:, :c]


def _exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _exact_slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "roundtrip":
        return torch.cat([_exact_round8(p.double()) for p in s["x"].split(32768)])
    if op == "unpack":
        return torch.cat([_exact_restore(q, p, s["width"]) for q, p in zip(s["codes"].split(32768), s["scales"].split(32768))])
    w = s["w"].double()
    r = {}
    z = None
    if op != "bwd":
        x = s["x"].double()
        z = x @ w.t() + (s["b"].double() if s["b"] is not None else 0)
        y = _exact_act(z, s["act"])
        r["Y"] = y + s["r"].double() if s.get("residual") else y
        if op == "fwd":
            if s["save"]:
                r["Z"] = z
            return r
        x, z = _exact_round8(x), _exact_round8(z)
    else:
        x = _exact_restore(*s["x"], s["cin"]) if s["x8"] else s["x"].double()
        if s["act"] != "none":
            z = _exact_restore(*s["z"], s["cout"]) if s["z8"] else s["z"].double()
    dz = s["dy"].double()
    if s["act"] != "none":
        dz = dz * _exact_slope(z, s["act"])
    r.update(dX=dz @ w, dW=dz.t() @ x)
    if s["bias"]:
        r["db"] = dz.sum(0)
    return r
