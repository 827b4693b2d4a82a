"""Cases of the operators for tokens that have weights of their own: what a pass computes and costs.

Five operators, each with a plain form in elementary torch operations (``own = False``) and the call of the
library that a user makes (``own = True``):

  sort              the order of token slots by expert, each expert's rows padded to a multiple (any mixture of experts)
  gather            tokens copied to their experts' rows, as bf16 or as the quantized operand of a grouped product
  combine           the experts' rows weighted and added up for each token
  combine_backward  the gradients of the experts' rows and of the weights
  lora              each token's low-rank adapter beside a projection: added to a given output, or beside
                    NVFP4 weights that all tokens share

A token t has k slots, slot t k + j being its j-th expert's.  ``positions`` [T, k] holds each slot's row in the order by
expert (-1: dropped), ``source`` [R] each row's slot (-1: none).  NVFP4: E2M1 codes, two to a byte (low nibble
first), an E4M3 scale for each 16 elements and an fp32 scale S for the tensor or for each row; the value is
code * scale / S.  MXFP8: E4M3 codes, an E8M0 scale for each 32.
"""
import math

import torch

own = False

HIDDEN, FFN, TOKENS = 4096, 14336, 16384   # the benchmark's layer


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a small batch, two of eight experts each: nothing but latency
        dict(name="sort 37x2 of 8", op="sort", tokens=37, k=2, experts=8, align=1, drop=False),
        # a training step's tokens, eight of 128 experts each, some over their expert's capacity; padded for
        # products grouped along the contraction
        dict(name="sort 16384x8 of 128 pad 32", op="sort", tokens=TOKENS, k=8, experts=128, align=32, drop=True),
        # a decoding batch's operand of the experts' forward products
        dict(name="gather nvfp4 64x8 h4096", op="gather", fmt="nvfp4", tokens=64, k=8, experts=128, align=1, hidden=HIDDEN,
             drop=False),
        # the training step's tokens as they are (the weight gradients quantize them along the tokens)
        dict(name="gather bf16 16384x2 h4096", op="gather", fmt="bf16", tokens=TOKENS, k=2, experts=8, align=32,
             hidden=HIDDEN, drop=False),
        # many small experts, an odd number of tokens, experts that are full
        dict(name="gather mxfp8 8191x8 h2080", op="gather", fmt="mxfp8", tokens=8191, k=8, experts=64, align=32, hidden=2080,
             drop=True),
        # one token decoding
        dict(name="combine 1x2 h4096", op="combine", tokens=1, k=2, experts=8, align=1, hidden=HIDDEN, drop=False,
             y="bf16", weights=True),
        # the training step's way back
        dict(name="combine 16384x2 h4096", op="combine", tokens=TOKENS, k=2, experts=8, align=32, hidden=HIDDEN, drop=False,
             y="bf16", weights=True),
        # the gradients of that way back
        dict(name="combine_bwd 16384x2 h4096", op="combine_backward", tokens=TOKENS, k=2, experts=8, align=32,
             hidden=HIDDEN, drop=False, y="bf16"),
        # a ragged microbatch over many experts, their outputs kept in fp32
        dict(name="combine_bwd 333x6 h1032 f32", op="combine_backward", tokens=333, k=6, experts=60, align=1, hidden=1032,
             drop=True, y="f32"),
        # sixteen requests with an adapter each, decoding through the gate projection of the benchmark's layer
        dict(name="lora nvfp4 16x14336x4096 r16", op="lora", base="nvfp4", m=16, n=FFN, k=HIDDEN, r=16, adapters=32, used=16,
             runs=False, rows=False, y="bf16"),
        # a few requests, one without an adapter, small odd sizes, fp32 logits
        dict(name="lora nvfp4 5x1033x2064 r8", op="lora", base="nvfp4", m=5, n=1033, k=2064, r=8, adapters=4, used=3,
             runs=False, rows=True, y="f32"),
        # the prompts of eight requests
        dict(name="lora add 4096x4096x4096 r64", op="lora", base="add", m=4096, n=HIDDEN, k=HIDDEN, r=64, adapters=8, used=8,
             runs=True, rows=False, y="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["sort", "gather", "gather", "combine", "combine", "combine_backward", "lora", "lora", "lora"])
    if op == "lora":
        base = rng.choice(["nvfp4", "add"])
        m = _spread(rng, 1, 64) if base == "nvfp4" else _spread(rng, 1, 4096)
        adapters = _spread(rng, 1, 32)
        return dict(op=op, base=base, m=m, n=_spread(rng, 16, 14336), k=_spread(rng, 64, 8192, 16),
                    r=rng.choice([8, 16, 16, 24, 32, 64, 128]), adapters=adapters, used=rng.randint(1, min(adapters, m)),
                    runs=rng.random() < 0.5 if m < 256 else True, rows=base == "nvfp4" and rng.random() < 0.4,
                    y=rng.choice(["bf16", "f32"]))
    k = rng.randint(1, 8)
    c = dict(op=op, tokens=_spread(rng, 1, 16384 if op == "sort" else 65536 // k), k=k, experts=_spread(rng, max(2, k), 128),
             align=rng.choice([1, 16, 32, 128]), drop=rng.random() < 0.5)
    if op == "sort":
        return c
    if op == "gather":
        c["fmt"] = rng.choice(["bf16", "nvfp4", "mxfp8"])
        c["hidden"] = _spread(rng, 64, 4096, 32 if c["fmt"] == "mxfp8" else 16)
    else:
        c["hidden"] = _spread(rng, 64, 4096, 8)
        c["y"] = rng.choice(["bf16", "bf16", "f32"])
        if op == "combine":
            c["weights"] = rng.random() < 0.7
    return c


def _rows(case):
    n, a = case["tokens"] * case["k"], case["align"]
    return (n + min(n, case["experts"]) * (a - 1)) // a * a


def work(case):
    op = case["op"]
    if op == "lora":
        m, n, k, r = case["m"], case["n"], case["k"], case["r"]
        b = 2.0 * m * k + 2.0 * case["used"] * r * (k + n) + 4.0 * m + m * n * (4 if case["y"] == "f32" else 2)
        f = 2.0 * m * r * (k + n)
        if case["base"] == "nvfp4":
            return {"bytes": b + n * k * (0.5 + 1 / 16), "flops": f + 2.0 * m * n * k}
        return {"bytes": b + m * n * (4 if case["y"] == "f32" else 2), "flops": f}
    t, n, rows = case["tokens"], case["tokens"] * case["k"], _rows(case)
    if op == "sort":
        return {"bytes": 12.0 * n + 4.0 * rows + 8.0 * (case["experts"] + 1), "flops": 0.0}
    h = case["hidden"]
    index = 4.0 * n + 4.0 * rows
    if op == "gather":
        per = {"bf16": 2 * h, "nvfp4": h // 2 + h // 16 + 4, "mxfp8": h + h // 32}[case["fmt"]]
        return {"bytes": 2.0 * t * h + rows * per + index, "flops": 0.0}
    y = 4 if case["y"] == "f32" else 2
    if op == "combine":
        return {"bytes": float(n) * h * y + 2.0 * t * h + n * (8 if case["weights"] else 4), "flops": 2.0 * n * h}
    return {"bytes": 2.0 * t * h + float(n) * h * y + float(rows) * h * y + index + 8.0 * n, "flops": 3.0 * n * h}


# ---------------------------------------------------------------- inputs

def _order(experts, count, align, rows):
    """offsets, positions and source of the order by expert."""
    t, k = experts.shape
    e = experts.reshape(-1)
    hit = torch.arange(count, device=e.device).reshape(-1, 1) == e   # an expert's slots along a row
    upto = hit.cumsum(1, dtype=torch.int32)
    padded = (upto[:, -1].long() + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    kept = (e >= 0) & (e < count)
    at = e.clamp(0, count - 1)
    p = torch.where(kept, offsets[at] + upto[at, torch.arange(t * k, device=e.device)] - 1, -1)
    source = torch.full((rows + 1,), -1, dtype=torch.int32, device=e.device)
    source[torch.where(p < 0, rows, p)] = torch.arange(t * k, dtype=torch.int32, device=e.device)
    return offsets, p.reshape(t, k).to(torch.int32), source[:rows].contiguous()


def _nvfp4_weight(v, rows):
    """Codes, scale bytes and S of v [N, K] as a quantizer leaves them."""
    n, k = v.shape
    s = 2688.0 / (v.abs().amax(1) if rows else v.abs().amax().reshape(1))
    codes, scale = _nvfp4_codes(v, s.reshape(-1, 1))
    return {"codes": codes, "scales": scale.view(torch.uint8), "s_enc": s.contiguous()}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    st = {"case": dict(case)}
    if case["op"] == "lora":
        m, n, k, r, count, used = (case[x] for x in ("m", "n", "k", "r", "adapters", "used"))
        st["x"] = randn(m, k).to(torch.bfloat16)
        st["a"] = randn(count, r, k).mul_(k ** -0.5).to(torch.bfloat16)
        st["b"] = randn(count, n, r).mul_(r ** -0.5).to(torch.bfloat16)
        st["scales"] = torch.rand(count, generator=g, device="cuda") + 0.5
        ids = torch.randperm(count, generator=g, device="cuda")[:used]
        which = torch.arange(m, device="cuda") * used // m   # runs of tokens of one request
        if not case["runs"]:
            which = which[torch.randperm(m, generator=g, device="cuda")]
        st["adapters"] = ids[which].to(torch.int32)
        if m > 4:
            st["adapters"][m // 3] = -1   # a request without one
        if case["base"] == "nvfp4":
            st["w"] = _nvfp4_weight(randn(n, k).mul_(k ** -0.5).to(torch.bfloat16).float(), case["rows"])
        else:
            dt = torch.float32 if case["y"] == "f32" else torch.bfloat16
            st["y"] = randn(m, n).to(dt)
            st["out"] = torch.empty_like(st["y"])
        return st
    t, k, count = case["tokens"], case["k"], case["experts"]
    # k different experts of each token, some experts far more often than others
    score = torch.rand((t, count), generator=g, device="cuda") + torch.rand(count, generator=g, device="cuda")
    experts = score.topk(k, 1).indices
    if case["drop"]:
        experts = torch.where(torch.rand((t, k), generator=g, device="cuda") < 0.03, -1, experts)
    if case["op"] == "sort":
        st["experts"] = experts
        return st
    _, st["positions"], st["source"] = _order(experts, count, case["align"], _rows(case))
    h = case["hidden"]
    x = randn(t, h).to(torch.bfloat16)
    if case["op"] == "gather":
        st["x"] = x
        if case["fmt"] == "nvfp4":
            word = torch.arange(65536, device="cuda").unsqueeze(1) >> torch.tensor([0, 4, 8, 12], device="cuda")
            st["quads"] = torch.tensor(_E2M1, device="cuda", dtype=torch.bfloat16)[word & 15].view(torch.int64).reshape(-1)
        return st
    st["y"] = randn(_rows(case), h).to(torch.float32 if case["y"] == "f32" else torch.bfloat16)
    w = torch.rand((t, k), generator=g, device="cuda") + 0.05
    st["weights"] = w / w.sum(1, keepdim=True) if case.get("weights", True) else None
    if case["op"] == "combine_backward":
        st["dout"] = x
    return st


# ---------------------------------------------------------------- the plain forms, in 32 bits

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _nvfp4_codes(v, s):
    """Packed codes and E4M3 block scales of v [R, H] (fp32) under S (a column of them, or one)."""
    b = v.reshape(v.shape[0], -1, 16)
    # divided by a tensor: torch takes a number's reciprocal, which rounds twice
    scale = (b.abs().amax(2) * s / s.new_full((1,), 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = scale.float()
    q = b * torch.where(f > 0, s / f, 0.0).unsqueeze(2)
    a = q.abs()
    # ties go to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + ((b < 0) & (f > 0).unsqueeze(2)) * 8).to(torch.uint8).reshape(v.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), scale


def _e2m1_values(st, codes):
    """The codes' values as bf16 [R, H], four at a time from the table of all 16-bit words: what the bytes stand for."""
    return st["quads"][codes.view(torch.int16).to(torch.int32) & 65535].view(torch.bfloat16)


def _with_zero_row(rows, source, k):
    """rows[source // k], and zeros where there is none."""
    return torch.cat([rows, rows.new_zeros((1, rows.shape[1]))])[torch.where(source < 0, rows.shape[0], source // k)]


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "sort":
        o, p, s = _order(st["experts"], case["experts"], case["align"], _rows(case))
        return {"offsets": o, "positions": p, "source": s}
    if op == "gather":
        x, src, k = st["x"], st["source"], case["k"]
        if case["fmt"] == "bf16":
            return _with_zero_row(x, src, k)
        v = x.float()
        if case["fmt"] == "nvfp4":
            amax = v.abs().amax(1, keepdim=True)
            s = torch.where(amax > 0, amax.new_full((1,), 2688.0) / amax, 1.0).clamp(max=torch.finfo(torch.float32).max)
            codes, scale = _nvfp4_codes(v, s)
            one = torch.where(src < 0, 1.0, s[src.clamp(min=0) // k, 0])
            return {"codes": _e2m1_values(st, _with_zero_row(codes, src, k)),
                    "scales": _with_zero_row(scale.view(torch.uint8), src, k).view(torch.float8_e4m3fn), "s_enc": one}
        b = v.reshape(v.shape[0], -1, 32)
        m = b.abs().amax(2)
        e = (torch.frexp(m).exponent - 9).clamp(-127, 127)   # frexp's mantissa lies in [1/2, 1)
        power = ((127 - e) << 23).view(torch.float32)   # 2^-e
        codes = (b * power.unsqueeze(2)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        scale = torch.where(m > 0, e + 127, 0).to(torch.uint8)
        return {"codes": _with_zero_row(codes.view(torch.uint8).reshape(v.shape), src, k).view(torch.float8_e4m3fn),
                "scales": _with_zero_row(scale, src, k).view(torch.float8_e8m0fnu)}
    if op == "lora":
        m, r, count = case["m"], case["r"], case["adapters"]
        mine = st["adapters"].reshape(-1, 1) == torch.arange(count, device="cuda")
        t = st["x"].float() @ st["a"].reshape(count * r, -1).float().t()
        t = t.reshape(m, count, r) * (mine * st["scales"]).unsqueeze(2)
        add = t.reshape(m, count * r) @ st["b"].float().transpose(1, 2).reshape(count * r, -1)
        if case["base"] == "add":
            return (st["y"].float() + add).to(st["y"].dtype)
        w = st["w"]
        lut = torch.tensor(_E2M1, device="cuda")
        c = w["codes"]
        wv = torch.stack([lut[(c & 15).int()], lut[(c >> 4).int()]], 2).reshape(c.shape[0], -1)
        wv = wv * w["scales"].view(torch.float8_e4m3fn).float().repeat_interleave(16, 1)
        y = st["x"].float() @ wv.t() / w["s_enc"] + add
        return y if case["y"] == "f32" else y.to(torch.bfloat16)
    y, p = st["y"], st["positions"]
    rows = torch.where((p < 0).unsqueeze(2), 0.0, y[p.clamp(min=0).reshape(-1)].float().reshape(*p.shape, -1))
    if op == "combine":
        if st["weights"] is not None:
            rows = rows * st["weights"].unsqueeze(2)
        return rows.sum(1).to(torch.bfloat16)
    d = st["dout"].float()
    dw = (rows * d.unsqueeze(1)).sum(2)
    w = torch.cat([st["weights"].reshape(-1), d.new_zeros(1)])[st["source"]]   # -1: the zero at the end
    return {"dy": (d[st["source"].clamp(min=0) // case["k"]] * w.unsqueeze(1)).to(y.dtype), "dweights": dw}


# ---------------------------------------------------------------- the library's calls

def _own(st):
    import block_scaled_precision_nvfp4_amd as bsq
    case = st["case"]
    op = case["op"]
    if op == "sort":
        return bsq.moe_sort(st["experts"], case["experts"], case["align"])
    if op == "gather":
        x, p, s = st["x"], st["positions"], st["source"]
        if case["fmt"] == "bf16":
            return bsq.moe_gather(x, p, s)
        if case["fmt"] == "nvfp4":
            q = bsq.moe_gather_nvfp4_rowscaled(x, p, s)
            return {"codes": _e2m1_values(st, q["codes"]), "scales": q["scales"].view(torch.float8_e4m3fn), "s_enc": q["s_enc"]}
        q = bsq.moe_gather_mxfp8(x, p, s)
        return {"codes": q["row_codes"].view(torch.float8_e4m3fn), "scales": q["row_scales"].view(torch.float8_e8m0fnu)}
    if op == "combine":
        return bsq.moe_combine(st["y"], st["positions"], st["weights"])
    if op == "combine_backward":
        dy, dw = bsq.moe_combine_backward(st["dout"], st["y"], st["positions"], st["source"], st["weights"])
        return {"dy": dy, "dweights": dw}
    if case["base"] == "add":
        return bsq.lora_add(st["y"], st["x"], st["adapters"], st["a"], st["b"], st["scales"], out=st["out"])
    w = st["w"]
    return bsq.nvfp4_lora_matvec(st["x"], w["codes"], w["scales"], w["s_enc"], st["adapters"], st["a"], st["b"], st["scales"],
                                 out_dtype=torch.float32 if case["y"] == "f32" else torch.bfloat16)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition, in 64 bits

def _f32(v):
    """v rounded to binary32, where the definition says so."""
    return v.to(torch.float32).double()


def _two_to(e):
    """2^e for whole e in binary64's normal range, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _log2(v):
    """floor(log2 v) of binary64 values in the normal range."""
    return (v.view(torch.int64) >> 52) - 1023


def _e4m3(v):
    """v to the nearest E4M3 value, ties to even, at most 448."""
    a = v.abs()
    step = _two_to(_log2(a.clamp_min(2.0 ** -20)).clamp_min(-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def _e2m1(v):
    a = v.abs()
    r = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    return torch.copysign(r.clamp(max=6.0), v)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        return None   # whole numbers only
    if op == "lora":
        x, ad = st["x"].double(), st["adapters"]
        if case["base"] == "add":
            out = st["y"].double().clone()
        else:
            w = st["w"]
            n, k = case["n"], case["k"]
            c = w["codes"].long()
            nib = torch.stack([c % 16, c // 16], 2).reshape(n, k)
            e, f = (nib >> 1) & 3, (nib & 1).double()
            mag = torch.where(e == 0, f / 2, (2 + f) * _two_to(e - 2))
            v = torch.where(nib > 7, -mag, mag).reshape(n, k // 16, 16) * w["scales"].view(torch.float8_e4m3fn).double().unsqueeze(2)
            out = torch.mm(x, v.reshape(n, k).t()) / w["s_enc"].double().reshape(1, -1)
        for a in range(case["adapters"]):
            at = (ad == a).nonzero().reshape(-1)
            if at.numel():
                t = torch.mm(x[at], st["a"][a].double().t()) * st["scales"][a].double()
                out[at] += torch.mm(t, st["b"][a].double().t())
        return out
    p, src, k = st["positions"].long(), st["source"].long(), case["k"]
    live = (src >= 0).nonzero().reshape(-1)
    token = src[live] // k
    rows = src.numel()
    if op == "gather":
        x = st["x"].double()
        t, h = x.shape

        def spread(v, fill=0.0):
            o = torch.full((rows,) + tuple(v.shape[1:]), fill, dtype=torch.float64, device="cuda")
            o[live] = v[token]
            return o
        if case["fmt"] == "bf16":
            return spread(x)
        if case["fmt"] == "nvfp4":
            top = x.abs().max(1, keepdim=True).values
            s = torch.where(top > 0, _f32(torch.full_like(top, 2688.0) / top), 1.0)
            b = x.reshape(t, h // 16, 16)
            scale = _e4m3(_f32(_f32(b.abs().max(2).values * s) / 6.0))
            mul = torch.where(scale > 0, _f32(s / scale), 0.0)
            return {"codes": spread(_e2m1(_f32(b * mul.unsqueeze(2))).reshape(t, h)), "scales": spread(scale),
                    "s_enc": spread(s, 1.0).reshape(-1)}
        b = x.reshape(t, h // 32, 32)
        top = b.abs().max(2).values
        unit = _two_to((_log2(top.clamp_min(2.0 ** -140)) - 8).clamp_min(-127))
        low = 2.0 ** -127   # the scale byte 0, of blocks without a value
        return {"codes": spread(_e4m3(b / unit.unsqueeze(2)).reshape(t, h)),
                "scales": spread(torch.where(top > 0, unit, low), low)}
    if op == "combine":
        out = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            at = (p[:, j] >= 0).nonzero().reshape(-1)
            w = 1.0 if st["weights"] is None else st["weights"][at, j].double().unsqueeze(1)
            out[at] += st["y"][p[at, j]].double() * w
        return out
    d, w = st["dout"].double(), st["weights"].double()
    dy = torch.zeros((rows, case["hidden"]), dtype=torch.float64, device="cuda")
    dy[live] = d[token] * w.reshape(-1)[src[live]].unsqueeze(1)
    dw = torch.zeros_like(w)
    for j in range(k):
        at = (p[:, j] >= 0).nonzero().reshape(-1)
        dw[at, j] = (d[at] * st["y"][p[at, j]].double()).sum(1)
    return {"dy": dy, "dweights": dw}
