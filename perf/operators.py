"""Cases of the operators around a gated feed-forward block: what a pass computes and costs.

Five operators, each with a plain form in elementary torch operations (``own = False``) and the call
of the library that a user makes (``own = True``):

  matvec         y = x W^T for a few tokens x (bf16), W held as NVFP4 (serving: any linear layer)
  gated_matvec   h = act(x Wg^T) * (x Wu^T) for a few tokens (serving: a block's first half)
  gated          h, and gate and up for the backward pass, from quantized operands (training)
  gated_backward the gradients of gate and up from the quantized output gradient (training)
  clip           the global 2-norm of many gradients, and the gradients scaled to a largest norm

NVFP4: E2M1 codes, two to a byte (low nibble first), an E4M3 scale for each 16 elements of a row and an
fp32 scale S for the tensor or for each row; the value is code * scale / S.  MXFP8: E4M3 codes, an
E8M0 scale for each 32.  "slab": MXFP8 codes of each band of 256 rows stored as consecutive slabs of
64 columns.
"""
import math
import random

import torch

own = False

ACTS = ("silu", "gelu", "gelu_tanh")
HIDDEN, FFN = 4096, 14336   # the benchmark's layer


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the smallest layer of the tests: one token, nothing but latency
        dict(name="matvec 1x256x256", op="matvec", m=1, n=256, k=256, rows=False, out="bf16"),
        # the down projection of the benchmark's layer while one sequence decodes
        dict(name="matvec 1x4096x14336", op="matvec", m=1, n=HIDDEN, k=FFN, rows=False, out="bf16"),
        # a batch of 16 sequences, a vocabulary-like odd number of rows, row-scaled weights, logits in fp32
        dict(name="matvec 16x6151x4112 rows f32", op="matvec", m=16, n=6151, k=4112, rows=True, out="f32"),
        # gate and up projections of the benchmark's layer while one sequence decodes
        dict(name="gated_mv 1x14336x4096", op="gated_matvec", act="silu", m=1, n=FFN, k=HIDDEN, rows=False),
        # a handful of drafted tokens through a small block with odd sizes
        dict(name="gated_mv 5x1033x2064 tanh", op="gated_matvec", act="gelu_tanh", m=5, n=1033, k=2064, rows=True),
        # the benchmark's training step: 16384 tokens, gate and up kept for the backward pass
        dict(name="gated nvfp4 16384 save", op="gated", fmt="nvfp4", act="silu", m=16384, n=FFN, k=HIDDEN, save=True,
             slab=False),
        # a ragged microbatch in MXFP8, evaluation (nothing kept)
        dict(name="gated mxfp8 1000 ragged", op="gated", fmt="mxfp8", act="gelu", m=1000, n=2056, k=1056, save=False,
             slab=False),
        # the backward pass of the benchmark's training step, the gradient in MXFP8 as its recipe has it
        dict(name="gated_bwd mxfp8 16384 slab", op="gated_backward", fmt="mxfp8", act="silu", m=16384, n=FFN, k=HIDDEN,
             slab=True),
        # the backward pass of a ragged microbatch, all in NVFP4
        dict(name="gated_bwd nvfp4 333 ragged", op="gated_backward", fmt="nvfp4", act="gelu_tanh", m=333, n=1003,
             k=2080, slab=False),
        # biases and norms: few elements at odd places of a flat bucket
        dict(name="clip 37 small tensors", op="clip", tensors=37, total=30000, kind="f32", active=True),
        # the fp32 weight gradients of two of the benchmark's blocks
        dict(name="clip 2 ffn blocks f32", op="clip", tensors=4, total=2 * 3 * HIDDEN * FFN, kind="f32", active=True),
        # a model's mixed gradients whose norm is below the bound: read, and left as they are
        dict(name="clip 300 mixed inactive", op="clip", tensors=300, total=60_000_000, kind="mixed", active=False),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["matvec", "matvec", "gated_matvec", "gated_matvec", "gated", "gated_backward", "clip"])
    act = rng.choice(ACTS)
    if op == "matvec":
        return dict(op=op, m=_spread(rng, 1, 64), n=_spread(rng, 16, 16384), k=_spread(rng, 64, 16384, 16),
                    rows=rng.random() < 0.4, out=rng.choice(["bf16", "f32"]))
    if op == "gated_matvec":
        return dict(op=op, act=act, m=_spread(rng, 1, 64), n=_spread(rng, 16, 14336), k=_spread(rng, 64, 8192, 16),
                    rows=rng.random() < 0.4)
    if op == "clip":
        return dict(op=op, tensors=_spread(rng, 1, 400), total=_spread(rng, 1000, 200_000_000),
                    kind=rng.choice(["f32", "bf16", "mixed"]), active=rng.random() < 0.7)
    fmt = rng.choice(["nvfp4", "mxfp8"])
    slab = fmt == "mxfp8" and rng.random() < 0.5
    c = dict(op=op, fmt=fmt, act=act, m=_spread(rng, 16, 16384), n=_spread(rng, 64, 14336),
             k=_spread(rng, 512, 4096, 512) if slab else _spread(rng, 64, 4096, 32), slab=slab)
    if op == "gated":
        c["save"] = rng.random() < 0.5
    return c


def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(numel for _, numel in _tensors(case))
        per = sum(numel * (4 if kind == "f32" else 2) for kind, numel in _tensors(case))
        return {"bytes": per * (2 if case["active"] else 1), "flops": 3.0 * n}
    m, n, k = case["m"], case["n"], case["k"]
    per = 0.5 + 1 / 16 if case.get("fmt", "nvfp4") == "nvfp4" else 1 + 1 / 32   # bytes of an operand's element
    if op == "matvec":
        return {"bytes": n * k * per + 2.0 * m * k + m * n * (4 if case["out"] == "f32" else 2), "flops": 2.0 * m * n * k}
    if op == "gated_matvec":
        return {"bytes": 2 * n * k * per + 2.0 * m * k + 2.0 * m * n, "flops": 4.0 * m * n * k}
    if op == "gated":
        return {"bytes": (m + 2 * n) * k * per + m * n * (6.0 if case["save"] else 2.0), "flops": 4.0 * m * n * k}
    return {"bytes": (m + n) * k * per + 8.0 * m * n, "flops": 2.0 * m * n * k}


def _tensors(case):
    """(kind, elements) of each gradient: sizes between a few elements and a large share of the total."""
    count, total = case["tensors"], case["total"]
    if count == 4 and total == 2 * 3 * HIDDEN * FFN:   # two blocks: [gate; up] and down
        sizes = [2 * FFN * HIDDEN, HIDDEN * FFN] * 2
    else:
        r = random.Random(count * 1000003 + total)
        parts = [math.exp(r.uniform(0.0, 6.0)) for _ in range(count)]
        sizes = [max(1, int(total * p / sum(parts))) for p in parts]
    return [("bf16" if case["kind"] == "bf16" or (case["kind"] == "mixed" and i % 3) else "f32", s)
            for i, s in enumerate(sizes)]


# ---------------------------------------------------------------- inputs

def _nvfp4(v, rows):
    """Codes, scale bytes and S of v [R, K] in fp32 as a quantizer leaves them."""
    r, k = v.shape
    amax = v.abs().amax(1) if rows else v.abs().amax().reshape(1)
    s = 2688.0 / amax.clamp_min(1e-30)
    b = v.reshape(r, k // 16, 16)
    sb = (b.abs().amax(2) * s.reshape(-1, 1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = sb.float()
    t = b * (s.reshape(-1, 1, 1) / f.clamp_min(2.0 ** -9).unsqueeze(2)) * (f > 0).unsqueeze(2)
    a = t.abs()
    code = torch.zeros(a.shape, dtype=torch.uint8, device=v.device)
    for edge in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += a > edge
    code += (t < 0).to(torch.uint8) * 8
    code = code.reshape(r, k // 2, 2)
    return {"codes": (code[..., 0] | (code[..., 1] << 4)).contiguous(), "scales": sb.view(torch.uint8).contiguous(),
            "s_enc": s.contiguous()}


def _mxfp8(v, slab):
    r, k = v.shape
    b = v.reshape(r, k // 32, 32)
    e = torch.floor(torch.log2(b.abs().amax(2).clamp_min(2.0 ** -100))) - 8
    codes = (b * torch.exp2(-e).unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(r, k)
    scales = (e + 127).to(torch.uint8)
    if slab:
        codes = torch.cat([codes[b0:b0 + 256].reshape(-1, k // 64, 64).transpose(0, 1).reshape(-1, k)
                           for b0 in range(0, r, 256)])
    return {"codes": codes.contiguous(), "scales": scales.contiguous(), "s_enc": None}


def _operand(case, gen, r, k, std, rows=False):
    v = torch.randn((r, k), generator=gen, device="cuda").mul_(std).to(torch.bfloat16).float()
    return _nvfp4(v, rows) if case.get("fmt", "nvfp4") == "nvfp4" else _mxfp8(v, case["slab"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": dict(case)}
    op = case["op"]
    if op == "clip":
        flat = {}
        for kind, dt in (("f32", torch.float32), ("bf16", torch.bfloat16)):
            n = sum(s for t, s in _tensors(case) if t == kind)
            if n:
                flat[kind] = torch.randn(n, generator=g, device="cuda").mul_(0.01).to(dt)
        total = sum(float(f.double().square().sum()) for f in flat.values())
        # an active bound sits well below the norm, an inactive one above it
        st["max_norm"] = math.sqrt(total) * (0.3 if case["active"] else 2.0)
        st["flat"] = flat
        st["out_flat"] = {t: torch.empty_like(f) for t, f in flat.items()} if case["active"] else flat

        def views(buf):
            at, got = {t: 0 for t in buf}, []
            for t, s in _tensors(case):
                got.append(buf[t][at[t]:at[t] + s])
                at[t] += s
            return got
        st["grads"] = views(flat)
        st["out"] = views(st["out_flat"]) if case["active"] else None
        return st
    m, n, k = case["m"], case["n"], case["k"]
    if op in ("matvec", "gated_matvec"):
        st["x"] = torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16)
        for w in ("w",) if op == "matvec" else ("gate", "up"):
            st[w] = _operand(case, g, n, k, 0.03, case["rows"])
        return st
    if op == "gated":
        st["a"] = _operand(case, g, m, k, 1.0)
        st["gate"] = _operand(case, g, n, k, 0.03)
        st["up"] = _operand(case, g, n, k, 0.03)
        return st
    st["dy"] = _operand(case, g, m, k, 0.01)
    st["wd"] = _operand(case, g, n, k, 0.02)   # the down projection's weight, stored along the block's output
    st["gate_up"] = torch.randn((m, 2 * n), generator=g, device="cuda").mul_(1.5).to(torch.bfloat16)
    return st


# ---------------------------------------------------------------- the plain forms, in 32 bits

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _values(q, slab):
    """Codes times block scales in fp32 (exact), without the tensor scale."""
    c = q["codes"]
    if q["s_enc"] is not None:
        lut = torch.tensor(_E2M1, device=c.device)
        v = torch.stack([lut[(c & 15).int()], lut[(c >> 4).int()]], 2).reshape(c.shape[0], -1)
        return v * q["scales"].view(torch.float8_e4m3fn).float().repeat_interleave(16, 1)
    if slab:
        k = c.shape[1]
        c = torch.cat([c[b0:b0 + 256].reshape(k // 64, -1, 64).transpose(0, 1).reshape(-1, k)
                       for b0 in range(0, c.shape[0], 256)])
    return c.view(torch.float8_e4m3fn).float() * torch.exp2(q["scales"].float() - 127.0).repeat_interleave(32, 1)


def _product(a, sa, b, sb, slab=False):
    """a b^T over the scales; a is a tensor of values or a quantized operand."""
    av = a.float() if isinstance(a, torch.Tensor) else _values(a, slab)
    y = av @ _values(b, slab).t()
    if sb is not None:
        y = y / (sb.reshape(1, -1) if sa is None else sa.reshape(-1, 1) * sb.reshape(1, -1))
    return y


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        p = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    s = 1.0 / (1.0 + torch.exp(-2.0 * c * (g + 0.044715 * g * g * g)))
    return g * s, s + g * s * (1.0 - s) * (2.0 * c * (1.0 + 3 * 0.044715 * g * g))


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for t in st["grads"]:
            total = total + t.double().square().sum()
        norm = total.sqrt()
        scale = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        if st["out"] is None:
            for t in st["grads"]:
                t.copy_(t.float() * scale)
        else:
            for t, o in zip(st["grads"], st["out"]):
                o.copy_(t.float() * scale)
        return {"norm": norm.float().reshape(1), "grads": st["out_flat"]}
    if op == "matvec":
        y = _product(st["x"], None, st["w"], st["w"]["s_enc"])
        return y if case["out"] == "f32" else y.to(torch.bfloat16)
    if op == "gated_matvec":
        g = _product(st["x"], None, st["gate"], st["gate"]["s_enc"])
        u = _product(st["x"], None, st["up"], st["up"]["s_enc"])
        return (_act(g, case["act"])[0] * u).to(torch.bfloat16)
    if op == "gated":
        a = st["a"]
        g = _product(a, a["s_enc"], st["gate"], st["gate"]["s_enc"], case["slab"])
        u = _product(a, a["s_enc"], st["up"], st["up"]["s_enc"], case["slab"])
        h = (_act(g, case["act"])[0] * u).to(torch.bfloat16)
        return {"h": h, "gate_up": torch.cat([g, u], 1).to(torch.bfloat16)} if case["save"] else {"h": h}
    dh = _product(st["dy"], st["dy"]["s_enc"], st["wd"], st["wd"]["s_enc"], case["slab"])
    n = case["n"]
    g, u = st["gate_up"][:, :n].float(), st["gate_up"][:, n:].float()
    f, df = _act(g, case["act"])
    return torch.cat([dh * u * df, dh * f], 1).to(torch.bfloat16)


# ---------------------------------------------------------------- the library's calls

def _own(st):
    import block_scaled_precision_nvfp4_amd as bsq
    case = st["case"]
    op = case["op"]
    if op == "clip":
        norm = bsq.clip_grad_norm(st["grads"], st["max_norm"], out=st["out"])
        return {"norm": norm, "grads": st["out_flat"]}
    if op == "matvec":
        w = st["w"]
        return bsq.nvfp4_matvec(st["x"], w["codes"], w["scales"], w["s_enc"],
                                out_dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    act = {"silu": bsq.ACT_SILU, "gelu": bsq.ACT_GELU, "gelu_tanh": bsq.ACT_GELU_TANH}[case["act"]]
    if op == "gated_matvec":
        g, u = st["gate"], st["up"]
        return bsq.nvfp4_gated_matvec(act, st["x"], g["codes"], g["scales"], g["s_enc"], u["codes"], u["scales"],
                                      u["s_enc"])
    fmt = bsq.FMT_NVFP4 if case["fmt"] == "nvfp4" else bsq.FMT_MXFP8 | (bsq.FMT_MX_SLAB if case["slab"] else 0)
    if op == "gated":
        a, g, u = st["a"], st["gate"], st["up"]
        r = bsq.blockscaled_gated_gemm(fmt, act, a["codes"], a["scales"], a["s_enc"], g["codes"], g["scales"],
                                       g["s_enc"], u["codes"], u["scales"], u["s_enc"], save_gate_up=case["save"])
        return {"h": r[0], "gate_up": r[1]} if case["save"] else {"h": r}
    dy, wd = st["dy"], st["wd"]
    return bsq.blockscaled_gated_gemm_backward(fmt, act, dy["codes"], dy["scales"], dy["s_enc"], wd["codes"],
                                               wd["scales"], wd["s_enc"], st["gate_up"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition, in 64 bits

def _ldexp(m, e):
    return m.double() * torch.pow(2.0, e.double())


def _e4m3(b):
    b = b.to(torch.int64)
    e, f = (b >> 3) & 15, b & 7
    v = torch.where(e == 0, _ldexp(f, torch.full_like(f, -9)), _ldexp(8 + f, e - 10))
    return torch.where(b > 127, -v, v)


def _decode(q, slab):
    c = q["codes"].to(torch.int64)
    if q["s_enc"] is not None:
        nib = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.int64, device=c.device)
        nib[:, 0::2], nib[:, 1::2] = c % 16, c // 16
        e, f = (nib >> 1) & 3, nib & 1
        v = torch.where(e == 0, f.double() / 2, _ldexp(2 + f, e - 2))
        v = torch.where(nib > 7, -v, v)
        v = v.reshape(c.shape[0], -1, 16) * _e4m3(q["scales"]).unsqueeze(2)
        return v.reshape(c.shape[0], -1) / q["s_enc"].double().reshape(-1, 1)
    v = _e4m3(q["codes"])
    if slab:
        r, k = v.shape
        w = torch.empty_like(v)
        for b0 in range(0, r, 256):
            rows = min(256, r - b0)
            band = v.reshape(-1)[b0 * k:(b0 + rows) * k]
            for s in range(k // 64):
                w[b0:b0 + rows, 64 * s:64 * s + 64] = band[s * rows * 64:(s + 1) * rows * 64].reshape(rows, 64)
        v = w
    r, k = v.shape
    return (v.reshape(r, -1, 32) * torch.pow(2.0, q["scales"].double() - 127).unsqueeze(2)).reshape(r, k)


def _activation64(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if act == "gelu":
        p = torch.special.erfc(-g / math.sqrt(2.0)) / 2
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    dz = math.sqrt(8 / math.pi) * (1 + 0.134145 * g ** 2)
    return g * torch.sigmoid(z), torch.sigmoid(z) + g * torch.sigmoid(z) * torch.sigmoid(-z) * dz


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(math.fsum(float(f.double().pow(2).sum()) for f in st["flat"].values()))
        c = min(1.0, st["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64),
                "grads": {t: f.double() * c for t, f in st["flat"].items()}}
    if op == "matvec":
        return torch.mm(st["x"].double(), _decode(st["w"], False).t())
    if op == "gated_matvec":
        x = st["x"].double()
        g, u = torch.mm(x, _decode(st["gate"], False).t()), torch.mm(x, _decode(st["up"], False).t())
        return _activation64(g, case["act"])[0] * u
    if op == "gated":
        a = _decode(st["a"], case["slab"])
        g = torch.mm(a, _decode(st["gate"], case["slab"]).t())
        u = torch.mm(a, _decode(st["up"], case["slab"]).t())
        h = _activation64(g, case["act"])[0] * u
        return {"h": h, "gate_up": torch.cat([g, u], 1)} if case["save"] else {"h": h}
    dh = torch.mm(_decode(st["dy"], case["slab"]), _decode(st["wd"], case["slab"]).t())
    g, u = st["gate_up"].double().chunk(2, 1)
    f, df = _activation64(g, case["act"])
    return torch.cat([dh * u * df, dh * f], 1)
