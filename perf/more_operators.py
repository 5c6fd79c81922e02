"""The feed-forward block's first product with its gated unit, both directions, and the clipping of its gradients:
cases, plain forms, exact values.

Four operators of the library are measured:

* ``gated``       gemm_gated_run: A = silu(X·Wgᵀ) * (X·Wuᵀ) in one kernel, 16-bit or block-scaled e4m3 operands, with an
                  8-bit checkpoint of both products for the backward pass.
* ``gated_back``  gemm_gated_back_run: dA = dY·W2 and, from the checkpoint, the gradients of both products and A again, in one
                  kernel.
* ``gated_few``   gemm_gated_matvec_run: the same as ``gated`` for 1 to 16 rows.
* ``clip``        gemm_clip_run: the Euclidean norm of many tensors together, and the tensors scaled to a largest norm.

Where ``own`` is false ``run`` computes them with elementary torch operations in 32 bits, rounded once at
the end; where it is true it makes the library's calls.  Values held in 8 bits come back as float8 tensors
(e4m3 for the codes, e8m0 for the scales).
"""
import math
import random

import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
SCALED = 1                # gemm.GEMM_SCALE_UE8M0_32
CLIP_WORKSPACE = 16384    # bytes: gemm.GEMM_CLIP_WORKSPACE


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through the first product of a 4096-wide block: 134 MB of weights
        dict(name="gated_few 1x8192x4096 bf16", op="gated_few", M=1, F=8192, K=4096, x="bf16", w="bf16", a="bf16"),
        # a few tokens of a narrow block, sizes that are multiples of nothing wide
        dict(name="gated_few 5x1040x2064 f16", op="gated_few", M=5, F=1040, K=2064, x="f16", w="f16", a="f16"),
        # a batch of decoded tokens with the training run's 8-bit weights
        dict(name="gated_few 16x8192x8192 e4m3", op="gated_few", M=16, F=8192, K=8192, x="bf16", w="e4m3", a="bf16"),
        # a short ragged batch
        dict(name="gated 333x1040x2064 bf16", op="gated", M=333, F=1040, K=2064, x="bf16", a="bf16", keep=False),
        # a serving batch past the few-row form, 8-bit operands in and out
        dict(name="gated 64x8192x4096 e4m3", op="gated", M=64, F=8192, K=4096, x="e4m3", a="e4m3", keep=False),
        # a middle-sized training batch in 16 bits, both products kept for the backward pass
        dict(name="gated 2048x4096x4096 f16", op="gated", M=2048, F=4096, K=4096, x="f16", a="f16", keep=True),
        # a training batch on block-scaled operands, both products kept
        dict(name="gated 4096x8192x8192 e4m3", op="gated", M=4096, F=8192, K=8192, x="e4m3", a="e4m3", keep=True),
        # the backward pass of a short ragged batch, without the operand again
        dict(name="gated_back 200x1040x528 f16", op="gated_back", M=200, F=1040, N=528, x="f16", again=False),
        # the backward pass of a training batch, with the second product's operand again for its weight's gradient
        dict(name="gated_back 4096x8192x8192 bf16", op="gated_back", M=4096, F=8192, N=8192, x="bf16", again=True),
        # the gradients of a small model's biases and norms: a launch's latency
        dict(name="clip 9 f32", op="clip", count=9, total=20011, type="f32", factor=0.5),
        # a middle-sized model's gradients in both types, within their limit: nothing to scale
        dict(name="clip 291 mixed", op="clip", count=291, total=40000003, type="mixed", factor=2.0),
        # the gradients of a 4096-wide block with 8192 inner channels
        dict(name="clip 3 f32", op="clip", count=3, total=100667392, type="f32", factor=0.25),
    ]


def _size(rng, low, high, step=1):
    """A multiple of step, spread over the logarithm of low..high."""
    v = math.exp(rng.uniform(math.log(low), math.log(max(low, high))))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_back", "gated_few", "gated_few", "clip"])
    if op == "gated":
        F, K = _size(rng, 16, 8192, 16), _size(rng, 16, 8192, 16)
        x = rng.choice(["bf16", "f16", "e4m3", "e4m3"])
        return dict(op=op, M=_size(rng, 1, 4096), F=F, K=K, x=x, a=rng.choice(["e4m3", "bf16", "f16"] if x == "e4m3" else
                                                                              ["e4m3", x, x]), keep=rng.random() < 0.6)
    if op == "gated_back":
        return dict(op=op, M=_size(rng, 1, 4096), F=_size(rng, 16, 8192, 16), N=_size(rng, 8, 8192, 8),
                    x=rng.choice(["bf16", "bf16", "f16"]), again=rng.random() < 0.5)
    if op == "gated_few":
        x, w = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
        K = _size(rng, 16, 16384, 16)
        return dict(op=op, M=rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 11, 16]), F=_size(rng, 1, min(16384, (1 << 26) // K)), K=K,
                    x=x, w=w, a=x)
    total = _size(rng, 100, 100000000)
    return dict(op=op, count=_size(rng, 1, min(600, total // 10)), total=total, type=rng.choice(["f32", "bf16", "mixed"]),
                factor=rng.choice([0.1, 0.5, 2.0]))


# ------------------------------------------------------------------------------------------ inputs

def _blocks(n):
    return (n + 31) // 32


def _activations(M, K, gen):
    """Normal, with every 97th channel ten times wider (as residual streams have)."""
    v = torch.randn(M, K, generator=gen, device="cuda")
    v[:, ::97] *= 10.0
    return v


def _sizes(count, total):
    """Sizes of `count` tensors, `total` elements together: a few large ones and many small, odd ones among them."""
    r = random.Random(count)
    weight = [math.exp(r.uniform(0.0, 6.0)) for _ in range(count)]
    sizes = [max(1, int(total * w / sum(weight))) for w in weight]
    sizes[0] += max(0, total - sum(sizes))
    return sizes


def _type_of(case, i):
    return ("bf16", "f32")[i % 2] if case["type"] == "mixed" else case["type"]


def _places(case):
    """{type: [elements of its buffer, (first element, size) of each tensor in it]}: a buffer of each type holds its tensors
    one behind the other, each on a line of its own."""
    out = {}
    for i, n in enumerate(_sizes(case["count"], case["total"])):
        kind = out.setdefault(_type_of(case, i), [0])
        kind.append((kind[0], n))
        kind[0] += (n + 63) // 64 * 64
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case, stream=torch.cuda.current_stream())

    def new(dtype, *shape):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op in ("gated", "gated_few"):
        M, F, K = case["M"], case["F"], case["K"]
        x = _activations(M, K, gen)
        w = torch.randn(2 * F, K, generator=gen, device="cuda") / math.sqrt(K)
        weights = case["x"] if op == "gated" else case["w"]
        s["X"], s["SFX"] = _to_e4m3(x) if case["x"] == "e4m3" else (x.to(TORCH[case["x"]]), None)
        s["W"], s["SFW"] = _to_e4m3(w) if weights == "e4m3" else (w.to(TORCH[weights]), None)
        s["A"] = new(TORCH[case["a"]], M, F)
        if op == "gated":
            s["SFA"] = new(torch.float8_e8m0fnu, M, _blocks(F)) if case["a"] == "e4m3" else None
            s["CK"] = new(torch.float8_e4m3fn, M, 2 * F) if case["keep"] else None
            s["SFCK"] = new(torch.float8_e8m0fnu, M, 2 * _blocks(F)) if case["keep"] else None
            if own:
                from blackwell_tensor_core_tma_gb300 import gemm
                s["plan"] = gemm.GatedPlan(M, F, K, case["x"], case["a"], SCALED if case["x"] == "e4m3" else 0)
    elif op == "gated_back":
        M, F, N = case["M"], case["F"], case["N"]
        dt = TORCH[case["x"]]
        s["DY"] = (torch.randn(M, N, generator=gen, device="cuda") * 0.02).to(dt)
        s["W2"] = (torch.randn(N, F, generator=gen, device="cuda") / math.sqrt(F)).to(dt)
        z = torch.randn(M, 2 * F, generator=gen, device="cuda")
        halves = [_to_e4m3(z[:, :F]), _to_e4m3(z[:, F:])]
        s["CK"] = torch.cat([c.view(torch.uint8) for c, _ in halves], 1).view(torch.float8_e4m3fn)
        s["SFCK"] = torch.cat([c.view(torch.uint8) for _, c in halves], 1).view(torch.float8_e8m0fnu)
        s["DZ"] = new(dt, M, 2 * F)
        s["A"] = new(dt, M, F) if case["again"] else None
        if own:
            from blackwell_tensor_core_tma_gb300 import gemm
            s["plan"] = gemm.GatedBackPlan(M, F, N, case["x"])
    else:
        places, held = _places(case), 0
        s["G"], s["C"], tensors = [], [], []
        for kind, (length, *spans) in places.items():
            flat = torch.zeros(length, dtype=TORCH[kind], device="cuda")
            for at, n in spans:
                flat[at:at + n] = torch.randn(n, generator=gen, device="cuda") * 1e-3
                held += n
            s["G"].append(flat)
            s["C"].append(torch.zeros_like(flat))
            tensors += [(s["G"][-1][at:at + n], s["C"][-1][at:at + n], kind) for at, n in spans]
        s["limit"] = case["factor"] * 1e-3 * math.sqrt(held)      # of the norm that such gradients have
        s["NORM"] = new(torch.float32, 1)
        s["workspace"] = new(torch.uint8, CLIP_WORKSPACE)
        if own:
            from blackwell_tensor_core_tma_gb300 import gemm
            s["tensors"] = gemm.clip_tensors(tensors)
    return s


# ------------------------------------------------------------------------------------- plain forms

def _to_e4m3(v):
    """(codes, scales) of rows of 32-bit values: per 32 elements the smallest power of two s with
    max |v| <= 448 s, and v / s rounded to e4m3."""
    M, F = v.shape
    n = _blocks(F)
    p = torch.nn.functional.pad(v, (0, n * 32 - F)).view(M, n, 32)
    bits = p.abs().amax(2).view(torch.int32)
    code = (((bits + 0x1FFFFF) >> 23) - 8).clamp(min=0)          # + 1 where the mantissa passes 448's 1.75
    inverse = ((254 - code) << 23).view(torch.float32)
    q = (p * inverse[:, :, None]).view(M, n * 32)[:, :F].to(torch.float8_e4m3fn)
    return q, code.to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(q, sf):
    """An operand's values in 32 bits: codes times their blocks' scales, or 16-bit values as they are."""
    if sf is None:
        return q.float()
    M, F = q.shape
    n = _blocks(F)
    p = torch.nn.functional.pad(q.float(), (0, n * 32 - F)).view(M, n, 32)
    return (p * sf.float()[:, :, None]).view(M, n * 32)[:, :F]


def _plain(s):
    op = s["op"]
    if op in ("gated", "gated_few"):
        F = s["F"]
        z = _values(s["X"], s["SFX"]) @ _values(s["W"], s["SFW"]).t()
        g, u = z[:, :F], z[:, F:]
        a = g / (1.0 + torch.exp(-g)) * u
        if s["a"] == "e4m3":
            q, sf = _to_e4m3(a)
            out = {"a": q, "sf": sf}
        else:
            out = {"a": a.to(TORCH[s["a"]])}
        if op == "gated" and s["keep"]:
            (qg, sg), (qu, su) = _to_e4m3(g), _to_e4m3(u)
            out["ck"] = [qg, qu]
            out["sfck"] = [sg, su]
        return out
    if op == "gated_back":
        F, n = s["F"], _blocks(s["F"])
        g = _values(s["CK"][:, :F], s["SFCK"][:, :n])
        u = _values(s["CK"][:, F:], s["SFCK"][:, n:])
        da = s["DY"].float() @ s["W2"].float()
        sg = 1.0 / (1.0 + torch.exp(-g))
        dz = torch.cat([da * u * sg * (1.0 + g * (1.0 - sg)), da * g * sg], 1)
        out = {"dz": dz.to(TORCH[s["x"]])}
        if s["again"]:
            out["a"] = (g * sg * u).to(TORCH[s["x"]])
        return out
    norm = sum(g.float().square().sum(dtype=torch.float64) for g in s["G"]).sqrt()
    scale = torch.clamp(s["limit"] / norm, max=1.0).float()
    return {"norm": norm.float(), "c": [(g.float() * scale).to(g.dtype) for g in s["G"]]}


# ------------------------------------------------------------------------------ the library's calls

def _own(s):
    from blackwell_tensor_core_tma_gb300 import gemm
    op, stream = s["op"], s["stream"]
    if op == "gated":
        F, n = s["F"], _blocks(s["F"])
        s["plan"].run(s["X"], s["W"], s["A"], s["SFX"], s["SFW"], s["SFA"], s["CK"], s["SFCK"], stream)
        out = {"a": s["A"]}
        if s["SFA"] is not None:
            out["sf"] = s["SFA"]
        if s["keep"]:
            out["ck"] = [s["CK"][:, :F], s["CK"][:, F:]]
            out["sfck"] = [s["SFCK"][:, :n], s["SFCK"][:, n:]]
        return out
    if op == "gated_back":
        s["plan"].run(s["DY"], s["W2"], s["CK"], s["SFCK"], s["DZ"], s["A"], stream)
        out = {"dz": s["DZ"]}
        if s["again"]:
            out["a"] = s["A"]
        return out
    if op == "gated_few":
        gemm.gemm_gated_matvec_run(s["M"], s["F"], s["K"], s["x"], s["w"], s["a"], s["X"], s["W"], s["SFW"], s["A"], stream)
        return {"a": s["A"]}
    gemm.gemm_clip_run(s["tensors"], s["limit"], s["NORM"], s["workspace"], CLIP_WORKSPACE, stream)
    return {"norm": s["NORM"][0], "c": s["C"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ work and exact

def work(case):
    """Each input read once and each output written once; multiplies and adds of the formulas."""
    op = case["op"]
    if op == "clip":
        sizes = _sizes(case["count"], case["total"])
        b = sum(2 * n * BYTES[_type_of(case, i)] for i, n in enumerate(sizes))
        return {"bytes": b + 4, "flops": 3 * sum(sizes)}
    M, F = case["M"], case["F"]
    if op == "gated_back":
        N = case["N"]
        b = 2 * M * N + 2 * N * F + M * F * (2 + 4 + (2 if case["again"] else 0)) + 2 * M * _blocks(F)
        return {"bytes": b, "flops": 2 * M * N * F + 14 * M * F}
    K = case["K"]
    w = case["x"] if op == "gated" else case["w"]
    b = M * K * BYTES[case["x"]] + 2 * F * K * BYTES[w] + M * F * BYTES[case["a"]]
    b += (M * _blocks(K) if case["x"] == "e4m3" else 0) + (2 * F * _blocks(K) if w == "e4m3" else 0)
    b += M * _blocks(F) if case["a"] == "e4m3" else 0
    if op == "gated" and case["keep"]:
        b += 2 * M * F + 2 * M * _blocks(F)
    return {"bytes": b, "flops": 4 * M * F * K + 6 * M * F}


def _wide(codes, scales):
    """An operand in 64 bits."""
    v = codes.double()
    if scales is not None:
        v *= torch.repeat_interleave(scales.double(), 32, dim=1)[:, :v.shape[1]]
    return v


def _exact_scales(v):
    """Each block's power of two for 64-bit values, and the values over it (before rounding to 8 bits)."""
    M, F = v.shape
    n = _blocks(F)
    p = torch.zeros(M, n * 32, dtype=torch.float64, device=v.device)
    p[:, :F] = v
    p = p.view(M, n, 32)
    top = p.abs().amax(2) / 448.0
    mantissa, exponent = torch.frexp(top)              # top = mantissa * 2^exponent, 0.5 <= mantissa < 1
    exponent = exponent.double() - (mantissa == 0.5).double()
    exponent = torch.where(top == 0, torch.full_like(exponent, -127.0), exponent.clamp(min=-127.0))
    scale = torch.pow(torch.full_like(exponent, 2.0), exponent)
    return (p / scale[:, :, None]).view(M, n * 32)[:, :F], scale


def exact(case, seed):
    """The definition in 64 bits: what is rounded to fewer bits on its way out is left unrounded."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        flats = [g.double() for g in s["G"]]
        norm = math.hypot(*(float(torch.linalg.vector_norm(f)) for f in flats))
        return {"norm": norm, "c": [f * min(1.0, s["limit"] / norm) for f in flats]}
    if op == "gated_back":
        F, n = case["F"], _blocks(case["F"])
        g, u = _wide(s["CK"][:, :F], s["SFCK"][:, :n]), _wide(s["CK"][:, F:], s["SFCK"][:, n:])
        da = torch.einsum("mn,nf->mf", s["DY"].double(), s["W2"].double())
        sg = torch.sigmoid(g)
        dsilu = sg + g * sg * torch.sigmoid(-g)
        out = {"dz": torch.hstack([da * u * dsilu, da * g * sg])}
        if case["again"]:
            out["a"] = g * sg * u
        return out
    x, w = _wide(s["X"], s["SFX"]), _wide(s["W"], s["SFW"])
    g, u = (torch.einsum("mk,fk->mf", x, half) for half in torch.tensor_split(w, 2))
    a = g * torch.sigmoid(g) * u
    out = {"a": a}
    if case["a"] == "e4m3":
        out["a"], out["sf"] = _exact_scales(a)
    if op == "gated" and case["keep"]:
        (qg, sg), (qu, su) = _exact_scales(g), _exact_scales(u)
        out["ck"], out["sfck"] = [qg, qu], [sg, su]
    return out
