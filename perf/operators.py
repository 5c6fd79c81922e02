"""The feed-forward block's operators around the block-scaled product: cases, plain forms, exact values.

Five entry points of the library are measured:

* ``norm``       gemm_norm_run: residual addition and root-mean-square norm, written as the block-scaled
                 e4m3 operand of the next product or as a 16-bit one.
* ``norm_back``  gemm_norm_backward: its gradients (and the 16-bit operand again).
* ``gate``       gemm_gate_run: silu(g) * u between the two products, with an 8-bit checkpoint of g and u.
* ``gate_back``  gemm_gate_backward: the gradients of g and u from that checkpoint alone.
* ``matvec``     gemm_matvec_run: 1 to 16 rows times 4-bit weights with scales.

Where ``own`` is false ``run`` computes them with elementary torch operations in 32 bits, rounded once at
the end; where it is true it makes the library's calls.  Values held in 8 bits come back as float8 tensors
(e4m3 for the codes, e8m0 for the scales).
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
EPS = 1e-6
NORM_PARTS = 512          # rows of K floats in gemm_norm_backward's workspace
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token of a 4096-wide residual stream, 16-bit operand for the matrix-vector product
        dict(name="norm 1x4096 bf16", op="norm", M=1, K=4096, x="bf16", h="bf16", y="bf16", residual=True, save=False),
        # a training batch of 8192 tokens, e4m3 operand, statistics kept for the backward pass
        dict(name="norm 8192x8192 e4m3", op="norm", M=8192, K=8192, x="bf16", h="bf16", y="e4m3", residual=True, save=True),
        # a short ragged batch in 32 bits: rows that end inside a scale block's 32 elements
        dict(name="norm_back 333x2064 f32", op="norm_back", M=333, K=2064, dy="f32", h="f32", y="bf16", again=False),
        # the backward pass of a training batch, with the operand again for the weight gradient
        dict(name="norm_back 4096x8192 bf16", op="norm_back", M=4096, K=8192, dy="bf16", h="bf16", y="bf16", again=True),
        # one decoded token between two matrix-vector products: no checkpoint
        dict(name="gate 1x8192 bf16", op="gate", M=1, F=8192, z="bf16", a="bf16", save=False),
        # a training batch: e4m3 operand and the 8-bit checkpoint
        dict(name="gate 4096x8192 e4m3", op="gate", M=4096, F=8192, z="bf16", a="e4m3", save=True),
        # ragged rows, 32-bit gradients in and out
        dict(name="gate_back 77x2064 f32", op="gate_back", M=77, F=2064, da="f32", dz="f32", a="bf16", again=False),
        # the backward pass of a training batch, with the second product's operand again
        dict(name="gate_back 4096x8192 bf16", op="gate_back", M=4096, F=8192, da="bf16", dz="bf16", a="bf16", again=True),
        # one token through a square projection, scales per 16
        dict(name="matvec 1x4096x4096 ue4m3", op="matvec", M=1, N=4096, K=4096, x="bf16", d="bf16", scales=2, c=False),
        # a few tokens, sizes that are multiples of nothing wide
        dict(name="matvec 5x1000x2080 ue8m0", op="matvec", M=5, N=1000, K=2080, x="f16", d="f32", scales=1, c=True),
        # one token through the widest layer: 134 MB of weights
        dict(name="matvec 1x32768x8192 ue4m3", op="matvec", M=1, N=32768, K=8192, x="bf16", d="bf16", scales=2, c=False),
        # a batch of decoded tokens with a residual added in 32 bits
        dict(name="matvec 16x8192x16384 ue8m0", op="matvec", M=16, N=8192, K=16384, x="bf16", d="f32", scales=1, c=True),
    ]


def _size(rng, low, high, step=1):
    """A multiple of step, spread over the logarithm of low..high."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "gate", "gate_back", "matvec", "matvec"])
    if op == "norm":
        K = _size(rng, 16, 16384, 16)
        return dict(op=op, M=_size(rng, 1, min(16384, (1 << 26) // K)), K=K, x=rng.choice(["bf16", "f32"]),
                    h=rng.choice(["bf16", "f32"]), y=rng.choice(["e4m3", "e4m3", "bf16", "f16"]),
                    residual=rng.random() < 0.75, save=rng.random() < 0.5)
    if op == "norm_back":
        K = _size(rng, 16, 16384, 16)
        return dict(op=op, M=_size(rng, 1, min(16384, (1 << 25) // K)), K=K, dy=rng.choice(["bf16", "f32"]),
                    h=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "f16"]), again=rng.random() < 0.5)
    if op in ("gate", "gate_back"):
        F = _size(rng, 16, 32768, 16)
        M = _size(rng, 1, min(16384, (1 << 25) // F))
        if op == "gate":
            return dict(op=op, M=M, F=F, z=rng.choice(["bf16", "f32"]), a=rng.choice(["e4m3", "e4m3", "bf16", "f16"]),
                        save=rng.random() < 0.6)
        return dict(op=op, M=M, F=F, da=rng.choice(["bf16", "f32"]), dz=rng.choice(["bf16", "f32"]),
                    a=rng.choice(["bf16", "f16"]), again=rng.random() < 0.5)
    K = _size(rng, 32, 32768, 32)
    return dict(op=op, M=rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 11, 16]), N=_size(rng, 16, min(65536, (1 << 28) // K)), K=K,
                x=rng.choice(["bf16", "f16"]), d=rng.choice(["bf16", "f32"]), scales=rng.choice([1, 2]),
                c=rng.random() < 0.3)


# ------------------------------------------------------------------------------------------ inputs

def _stream_like(M, K, gen, dtype, outliers=True):
    """Activations: normal, with every 97th channel ten times wider (as residual streams have)."""
    v = torch.randn(M, K, generator=gen, device="cuda")
    if outliers:
        v[:, ::97] *= 10.0
    return v.to(dtype)


def _blocks(F):
    return (F + 31) // 32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M = case["op"], case["M"]
    s = dict(case, stream=torch.cuda.current_stream())

    def new(dtype, *shape):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op == "norm":
        K = case["K"]
        s["X"] = _stream_like(M, K, gen, TORCH[case["x"]], outliers=False)
        s["R"] = _stream_like(M, K, gen, TORCH[case["h"]]) if case["residual"] else None
        s["W"] = 1.0 + 0.1 * torch.randn(K, generator=gen, device="cuda")
        s["H"] = new(TORCH[case["h"]], M, K) if case["residual"] or case["save"] else None
        s["Y"] = new(TORCH[case["y"]], M, K)
        s["SFY"] = new(torch.float8_e8m0fnu, M, _blocks(K)) if case["y"] == "e4m3" else None
        s["RSTD"] = new(torch.float32, M) if case["save"] else None
    elif op == "norm_back":
        K = case["K"]
        s["DY"] = (torch.randn(M, K, generator=gen, device="cuda") * 0.02).to(TORCH[case["dy"]])
        s["DH"] = (torch.randn(M, K, generator=gen, device="cuda") * 0.02).to(TORCH[case["h"]])
        s["H"] = _stream_like(M, K, gen, TORCH[case["h"]])
        s["W"] = 1.0 + 0.1 * torch.randn(K, generator=gen, device="cuda")
        s["RSTD"] = 1.0 / torch.sqrt(s["H"].float().square().mean(1) + EPS)
        s["DX"] = new(TORCH[case["h"]], M, K)
        s["DW"] = new(torch.float32, K)
        s["Y"] = new(TORCH[case["y"]], M, K) if case["again"] else None
        s["workspace"] = new(torch.float32, min(M, NORM_PARTS), K)
    elif op == "gate":
        F = case["F"]
        s["Z"] = _stream_like(M, 2 * F, gen, TORCH[case["z"]], outliers=False)
        s["A"] = new(TORCH[case["a"]], M, F)
        s["SFA"] = new(torch.float8_e8m0fnu, M, _blocks(F)) if case["a"] == "e4m3" else None
        s["CK"] = new(torch.float8_e4m3fn, M, 2 * F) if case["save"] else None
        s["SFCK"] = new(torch.float8_e8m0fnu, M, 2 * _blocks(F)) if case["save"] else None
    elif op == "gate_back":
        F = case["F"]
        s["DA"] = (torch.randn(M, F, generator=gen, device="cuda") * 0.02).to(TORCH[case["da"]])
        z = torch.randn(M, 2 * F, generator=gen, device="cuda")
        halves = [_to_e4m3(z[:, :F]), _to_e4m3(z[:, F:])]
        s["CK"] = torch.cat([c.view(torch.uint8) for c, _ in halves], 1).view(torch.float8_e4m3fn)
        s["SFCK"] = torch.cat([c.view(torch.uint8) for _, c in halves], 1).view(torch.float8_e8m0fnu)
        s["DZ"] = new(TORCH[case["dz"]], M, 2 * F)
        s["A"] = new(TORCH[case["a"]], M, F) if case["again"] else None
    else:
        N, K = case["N"], case["K"]
        block = 32 if case["scales"] == 1 else 16
        s["X"] = (_stream_like(M, K, gen, torch.float32) / math.sqrt(K)).to(TORCH[case["x"]])
        w = torch.randn(N, K // block, block, generator=gen, device="cuda")
        amax = w.abs().amax(2)
        if case["scales"] == 1:      # powers of two: the smallest that brings the block within 6
            code = torch.ceil(torch.log2(amax / 6.0)).clamp_(-127, 127) + 127.0
            scale = torch.exp2(code - 127.0)
            s["SFB"] = code.to(torch.uint8)
        else:                        # three mantissa bits: the nearest to the block's maximum / 6
            scale = (amax / 6.0).clamp_(min=2.0 ** -9).to(torch.float8_e4m3fn)
            s["SFB"] = scale.view(torch.uint8)
            scale = scale.float()
        level = torch.bucketize((w / scale[:, :, None]).abs_(),
                                torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda"), out_int32=True)
        code = (level.to(torch.uint8) | ((w < 0).to(torch.uint8) << 3)).view(N, K // 2, 2)
        s["B"] = code[:, :, 0] | (code[:, :, 1] << 4)
        s["C"] = torch.randn(M, N, generator=gen, device="cuda") if case["c"] else None
        s["D"] = new(TORCH[case["d"]], M, N)
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


def _from_e4m3(q, sf):
    M, F = q.shape
    n = _blocks(F)
    p = torch.nn.functional.pad(q.float(), (0, n * 32 - F)).view(M, n, 32)
    return (p * sf.float()[:, :, None]).view(M, n * 32)[:, :F]


def _operand(v, kind):
    """An operand's values in its type: {"y": ...} and its scales where it has some."""
    if kind == "e4m3":
        q, sf = _to_e4m3(v)
        return {"y": q, "sf": sf}
    return {"y": v.to(TORCH[kind])}


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = s["X"].float() if s["R"] is None else s["X"].float() + s["R"].float()
        h = h.to(TORCH[s["h"]])
        v = h.float()
        rstd = 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
        out = _operand(v * rstd * s["W"], s["y"])
        if s["H"] is not None:
            out["h"] = h
        if s["save"]:
            out["rstd"] = rstd[:, 0]
        return out
    if op == "norm_back":
        dy, h, rstd = s["DY"].float(), s["H"].float(), s["RSTD"][:, None]
        g = dy * s["W"]
        n = h * rstd
        dx = s["DH"].float() + rstd * (g - n * (g * n).mean(1, keepdim=True))
        out = {"dx": dx.to(TORCH[s["h"]]), "dw": (dy * n).sum(0)}
        if s["again"]:
            out["y"] = (n * s["W"]).to(TORCH[s["y"]])
        return out
    if op == "gate":
        F = s["F"]
        z = s["Z"].float()
        g, u = z[:, :F], z[:, F:]
        out = _operand(g / (1.0 + torch.exp(-g)) * u, s["a"])
        if s["save"]:
            (qg, sg), (qu, su) = _to_e4m3(g), _to_e4m3(u)
            out["ck"] = [qg, qu]
            out["sfck"] = [sg, su]
        return out
    if op == "gate_back":
        F, n = s["F"], _blocks(s["F"])
        g = _from_e4m3(s["CK"][:, :F], s["SFCK"][:, :n])
        u = _from_e4m3(s["CK"][:, F:], s["SFCK"][:, n:])
        da = s["DA"].float()
        sg = 1.0 / (1.0 + torch.exp(-g))
        dz = torch.cat([da * u * sg * (1.0 + g * (1.0 - sg)), da * g * sg], 1)
        out = {"dz": dz.to(TORCH[s["dz"]])}
        if s["again"]:
            out["y"] = (g * sg * u).to(TORCH[s["a"]])
        return out
    N, K = s["N"], s["K"]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], 1)      # byte -> its two values
    w = torch.index_select(pairs, 0, s["B"].view(-1).int())
    if s["scales"] == 1:
        scale = s["SFB"].view(torch.float8_e8m0fnu).float()
        w = w.view(N, K // 32, 32)
    else:
        scale = s["SFB"].view(torch.float8_e4m3fn).float()
        w = w.view(N, K // 16, 16)
    w = (w * scale[:, :, None]).view(N, K)
    d = s["X"].float() @ w.t()
    if s["C"] is not None:
        d = d + s["C"]
    return {"d": d.to(TORCH[s["d"]])}


# ------------------------------------------------------------------------------ the library's calls

def _own(s):
    from blackwell_tensor_core_tma_gb300 import gemm
    op, M, stream = s["op"], s["M"], s["stream"]
    if op == "norm":
        gemm.gemm_norm_run(M, s["K"], s["x"], s["h"], s["y"], EPS, s["X"], s["R"], s["W"], s["H"], s["Y"], s["SFY"],
                           s["RSTD"], stream)
        out = {"y": s["Y"]}
        if s["SFY"] is not None:
            out["sf"] = s["SFY"]
        if s["H"] is not None:
            out["h"] = s["H"]
        if s["save"]:
            out["rstd"] = s["RSTD"]
        return out
    if op == "norm_back":
        gemm.gemm_norm_backward(M, s["K"], s["dy"], s["h"], s["y"], s["DY"], s["DH"], s["H"], s["RSTD"], s["W"], s["DX"],
                                s["DW"], s["Y"], s["workspace"], s["workspace"].numel() * 4, stream)
        out = {"dx": s["DX"], "dw": s["DW"]}
        if s["again"]:
            out["y"] = s["Y"]
        return out
    if op == "gate":
        F, n = s["F"], _blocks(s["F"])
        gemm.gemm_gate_run(M, F, s["z"], s["a"], s["Z"], s["A"], s["SFA"], s["CK"], s["SFCK"], stream)
        out = {"y": s["A"]}
        if s["SFA"] is not None:
            out["sf"] = s["SFA"]
        if s["save"]:
            out["ck"] = [s["CK"][:, :F], s["CK"][:, F:]]
            out["sfck"] = [s["SFCK"][:, :n], s["SFCK"][:, n:]]
        return out
    if op == "gate_back":
        gemm.gemm_gate_backward(M, s["F"], s["da"], s["dz"], s["a"], s["DA"], s["CK"], s["SFCK"], s["DZ"], s["A"], stream)
        out = {"dz": s["DZ"]}
        if s["again"]:
            out["y"] = s["A"]
        return out
    gemm.gemm_matvec_run(M, s["N"], s["K"], s["x"], s["d"], s["scales"], s["X"], s["B"], s["SFB"], s["C"], s["D"], stream)
    return {"d": s["D"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ work and exact

def work(case):
    """Each input read once and each output written once; multiplies and adds of the formulas."""
    op, M = case["op"], case["M"]
    if op == "norm":
        K = case["K"]
        per = BYTES[case["x"]] + BYTES[case["y"]] + (BYTES[case["h"]] if case["residual"] else 0)
        if case["residual"] or case["save"]:
            per += BYTES[case["h"]]
        b = M * K * per + 4 * K + (M * _blocks(K) if case["y"] == "e4m3" else 0) + (4 * M if case["save"] else 0)
        return {"bytes": b, "flops": 5 * M * K}
    if op == "norm_back":
        K = case["K"]
        per = BYTES[case["dy"]] + 3 * BYTES[case["h"]] + (BYTES[case["y"]] if case["again"] else 0)
        return {"bytes": M * K * per + 8 * K + 4 * M, "flops": 10 * M * K}
    if op == "gate":
        F = case["F"]
        b = M * F * (2 * BYTES[case["z"]] + BYTES[case["a"]] + (2 if case["save"] else 0))
        b += M * _blocks(F) * ((1 if case["a"] == "e4m3" else 0) + (2 if case["save"] else 0))
        return {"bytes": b, "flops": 6 * M * F}
    if op == "gate_back":
        F = case["F"]
        per = 2 + BYTES[case["da"]] + 2 * BYTES[case["dz"]] + (BYTES[case["a"]] if case["again"] else 0)
        return {"bytes": M * F * per + 2 * M * _blocks(F), "flops": 14 * M * F}
    N, K = case["N"], case["K"]
    b = N * K // 2 + N * (K // (32 if case["scales"] == 1 else 16)) + M * K * 2 + M * N * BYTES[case["d"]]
    return {"bytes": b + (4 * M * N if case["c"] else 0), "flops": 2 * M * N * K}


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
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point() and k in
         ("X", "R", "W", "DY", "DH", "H", "RSTD", "Z", "DA", "C")}
    if op == "norm":
        # h is defined as rounded to the stream's type; the norm takes the rounded values
        h = (s["X"].double() if s["R"] is None else s["X"].double() + s["R"].double()).to(TORCH[case["h"]]).double()
        rstd = torch.rsqrt((h * h).sum(1) / case["K"] + EPS)
        y = torch.einsum("mk,m,k->mk", h, rstd, d["W"])
        out = {"y": y}
        if case["y"] == "e4m3":
            out["y"], out["sf"] = _exact_scales(y)
        if s["H"] is not None:
            out["h"] = h
        if case["save"]:
            out["rstd"] = rstd
        return out
    if op == "norm_back":
        inner = torch.einsum("mk,mk,k->m", d["DY"], d["H"], d["W"]) / case["K"]
        dx = d["DH"] + torch.einsum("mk,k,m->mk", d["DY"], d["W"], d["RSTD"]) \
            - torch.einsum("mk,m->mk", d["H"], d["RSTD"] ** 3 * inner)
        out = {"dx": dx, "dw": torch.einsum("mk,mk,m->k", d["DY"], d["H"], d["RSTD"])}
        if case["again"]:
            out["y"] = torch.einsum("mk,m,k->mk", d["H"], d["RSTD"], d["W"])
        return out
    if op == "gate":
        g, u = torch.tensor_split(d["Z"], 2, dim=1)
        a = g * torch.sigmoid(g) * u
        out = {"y": a}
        if case["a"] == "e4m3":
            out["y"], out["sf"] = _exact_scales(a)
        if case["save"]:
            (qg, sg), (qu, su) = _exact_scales(g), _exact_scales(u)
            out["ck"], out["sfck"] = [qg, qu], [sg, su]
        return out
    if op == "gate_back":
        F, n = case["F"], _blocks(case["F"])
        spread = torch.repeat_interleave(s["SFCK"].double().view(case["M"], 2, n), 32, dim=2)[:, :, :F]
        g, u = torch.unbind(s["CK"].double().view(case["M"], 2, F) * spread, 1)
        sg = torch.sigmoid(g)
        dsilu = sg + g * sg * torch.sigmoid(-g)
        out = {"dz": torch.hstack([d["DA"] * u * dsilu, d["DA"] * g * sg])}
        if case["again"]:
            out["y"] = g * sg * u
        return out
    N, K, M = case["N"], case["K"], case["M"]
    byte = s["B"]
    w = torch.empty(N, K, dtype=torch.float64, device="cuda")
    for half in (0, 1):                                # sign, two exponent bits (bias 1), one mantissa bit
        code = (byte >> (4 * half)) & 15
        e, m = ((code >> 1) & 3).double(), (code & 1).double()
        mag = torch.where(e == 0, 0.5 * m, torch.exp2(e - 1) * (1 + 0.5 * m))
        w[:, half::2] = torch.where(code >= 8, -mag, mag)
    sf = s["SFB"].double()
    if case["scales"] == 1:
        sf = torch.exp2(sf - 127)
    else:                                              # four exponent bits (bias 7), three mantissa bits
        c = s["SFB"]
        e, m = (c >> 3).double(), (c & 7).double()
        sf = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e - 7) * (1 + m / 8))
    w.view(N, sf.shape[1], -1).mul_(sf[:, :, None])
    out = torch.einsum("mk,nk->mn", d["X"], w)
    return {"d": out + d["C"] if case["c"] else out}
