"""Cases of the expert-grouped and the scaled int8 operators, for measuring them.

Four operators, each in its plain form (`own` false: elementary torch
operations in 32 bits, rounded once at the end) and as the library's calls
(`own` true):

  grouped   D[rows of g] = act(A[rows of g] B_g + bias_g): the products of the
            tokens with the weights of the expert each was sent to, tokens
            sorted by expert.  With the weights read the other way round it is
            the gradient of the tokens.
  wgrad     D_g = A[rows of g]^T B[rows of g] (+ D_g): the gradient of the
            experts' weights.
  quantize  rows of int8 and a scale for each from rows of 16- or 32-bit numbers.
  i8        D = act(scaleA_i scaleB_j sum_k A_ik B_kj + bias_j): the product of
            int8 rows with int8 weights, a scale for each token and each
            output channel.
"""
import math
import random

import torch

own = False

_FLOAT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_CODE = {"f16": 0, "bf16": 1, "f32": 3}
_ACT = {"none": 0, "relu": 1, "gelu_tanh": 2}


def listed():
    return [
        # decoding: a few tokens, two experts each, through the experts' first
        # layer of the library's MLP configuration; the weights' bytes are the cost
        dict(name="grouped decode 8x14336x4096", op="grouped", rows=16, groups=8, n=14336, k=4096, dtype="bf16",
             weights="nk", act="gelu_tanh", bias=True, skew=0.5),
        # a small layer with few tokens, some experts without any: latency
        dict(name="grouped decode 16x1024x1024", op="grouped", rows=9, groups=16, n=1024, k=1024, dtype="f16",
             weights="nk", act="none", bias=False, skew=0.5),
        # a chunk of a prompt over many experts: ragged groups of a few dozen tokens
        dict(name="grouped chunk 64x1536x2048", op="grouped", rows=4099, groups=64, n=1536, k=2048, dtype="bf16",
             weights="nk", act="relu", bias=True, skew=0.7),
        # training: forward of a large batch, weights stored inputs first
        dict(name="grouped train 8x4096x4096", op="grouped", rows=16384, groups=8, n=4096, k=4096, dtype="bf16",
             weights="kn", act="none", bias=False, skew=0.3),
        # training: gradient of the tokens (the forward's weights read the other way)
        dict(name="grouped dgrad 8x4096x8192", op="grouped", rows=8191, groups=8, n=4096, k=8192, dtype="f16",
             weights="nk", act="none", bias=False, skew=0.3),
        # training: gradient of the weights, added to 32-bit sums over micro-batches
        dict(name="wgrad train 8x4096x4096", op="wgrad", rows=16384, groups=8, n=4096, k=4096, dtype="bf16",
             out="f32", accumulate=True, skew=0.3),
        # the same for many small experts, a few rows each, in the weights' own type
        dict(name="wgrad small 32x1024x1000", op="wgrad", rows=1023, groups=32, n=1000, k=1024, dtype="bf16",
             out="bf16", accumulate=False, skew=0.7),
        # activations of a decoding step
        dict(name="quantize 16x4096", op="quantize", rows=16, cols=4096, dtype="bf16"),
        # activations of a training-sized batch
        dict(name="quantize 8192x14336", op="quantize", rows=8192, cols=14336, dtype="bf16"),
        # one token through a quantized layer
        dict(name="i8 1x14336x4096", op="i8", m=1, n=14336, k=4096, out="bf16", act="none", bias=False),
        # a decoding batch
        dict(name="i8 24x8192x8192", op="i8", m=24, n=8192, k=8192, out="bf16", act="none", bias=True),
        # a prompt through the library's MLP configuration
        dict(name="i8 8192x14336x4096", op="i8", m=8192, n=14336, k=4096, out="bf16", act="gelu_tanh", bias=True),
    ]


def _log(rng, lo, hi, steps=(1, 1, 8, 64)):
    """A size spread over the logarithm of [lo, hi], often a multiple of one of `steps`."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice(steps)
    return max(lo, min(hi, max(1, v // step) * step))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 8 to 128, now and then any number."""
    return _log(rng, lo, hi, (1, 8, 16, 32, 64, 64, 128, 128))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "wgrad", "quantize", "i8", "i8"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_width(rng, 64, 14336), dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "i8":
        return dict(op=op, m=_log(rng, 1, 8192), n=_width(rng, 512, 14336), k=_width(rng, 512, 4096), out=rng.choice(["bf16", "f16", "f32"]),
                    act=rng.choice(["none", "relu", "gelu_tanh"]), bias=rng.random() < 0.5)
    c = dict(op=op, rows=_log(rng, 1, 16384), groups=rng.choice([2, 4, 7, 8, 16, 32, 64]), n=_width(rng, 512, 4096),
             k=_width(rng, 512, 4096), dtype=rng.choice(["bf16", "f16"]), skew=round(rng.uniform(0.0, 1.0), 2))
    if op == "wgrad":
        c.update(groups=min(c["groups"], 16), out=rng.choice(["f32", c["dtype"]]), accumulate=rng.random() < 0.5)
    else:
        c.update(weights=rng.choice(["nk", "kn"]), act=rng.choice(["none", "relu", "gelu_tanh"]), bias=rng.random() < 0.5)
    return c


def _offsets(case):
    """Where each group's rows start and end: groups + 1 numbers.  Shares of the
    rows are drawn unevenly (`skew`), and with many groups some get none."""
    r = random.Random("%(rows)d %(groups)d %(skew)s" % case)
    share = [math.exp(3.0 * case["skew"] * r.gauss(0.0, 1.0)) * (0.0 if r.random() < 0.1 else 1.0) for _ in range(case["groups"])]
    if not any(share):
        share[0] = 1.0
    total, at, out = sum(share), 0.0, [0]
    for s in share:
        at += s
        out.append(min(case["rows"], max(out[-1], int(round(case["rows"] * at / total)))))
    out[-1] = case["rows"]
    return out


def _active(case):
    o = _offsets(case)
    return sum(1 for a, b in zip(o, o[1:]) if b > a)


def work(case):
    if case["op"] == "quantize":
        e, size = 4 if case["dtype"] == "f32" else 2, case["rows"] * case["cols"]
        return {"bytes": size * (e + 1) + 4 * case["rows"], "flops": 3 * size}
    if case["op"] == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        e = 4 if case["out"] == "f32" else 2
        return {"bytes": m * k + n * k + e * m * n + 4 * (m + n) + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    m, n, k, g = case["rows"], case["n"], case["k"], case["groups"]
    if case["op"] == "wgrad":
        e = 4 if case["out"] == "f32" else 2
        # every group's gradient is written, an empty group's too; what it is added to is read
        return {"bytes": 2 * m * (n + k) + e * n * k * g * (2 if case["accumulate"] else 1) + 4 * (g + 1), "flops": 2 * m * n * k}
    a = _active(case)
    return {"bytes": 2 * m * (n + k) + 2 * n * k * a + (4 * n * a if case["bias"] else 0) + 4 * (g + 1), "flops": 2 * m * n * k}


def _normal(gen, shape, scale, dtype):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(scale))
    return x


def _activations(gen, rows, cols, dtype):
    """Rows of different sizes, and a few channels much larger than the others, as between a model's layers."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device="cuda"))
    x *= torch.where(torch.rand((1, cols), generator=gen, device="cuda") < 0.01, 8.0, 1.0)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        s["x"] = _activations(gen, case["rows"], case["cols"], _FLOAT[case["dtype"]])
        s["q"] = torch.empty((case["rows"], case["cols"]), dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(case["rows"], device="cuda")
    elif op == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        # what quantize gives for normal tokens, and weights with a scale for each output channel
        s["a"] = _normal(gen, (m, k), 36.0, torch.float32).round_().clamp_(-127, 127).to(torch.int8)
        s["b"] = _normal(gen, (n, k), 36.0, torch.float32).round_().clamp_(-127, 127).to(torch.int8)
        s["scale_a"] = 0.028 * torch.exp(0.5 * torch.randn(m, generator=gen, device="cuda"))
        s["scale_b"] = (0.028 / math.sqrt(k)) * torch.exp(0.2 * torch.randn(n, generator=gen, device="cuda"))
        s["bias_v"] = _normal(gen, (n,), 0.5, torch.float32) if case["bias"] else None
        s["d"] = torch.empty((m, n), dtype=_FLOAT[case["out"]], device="cuda")
        s["ws"] = None
    else:
        m, n, k, g = case["rows"], case["n"], case["k"], case["groups"]
        dt = _FLOAT[case["dtype"]]
        s["ends"] = _offsets(case)
        s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda")
        s["a"] = _activations(gen, m, k, dt)
        if op == "wgrad":
            s["b"] = _normal(gen, (m, n), 0.1, dt)
            out = _FLOAT[case["out"]]
            # what earlier micro-batches have added
            s["d0"] = _normal(gen, (g, k, n), 0.5, out) if case["accumulate"] else None
            s["d"] = torch.empty((g, k, n), dtype=out, device="cuda")
        else:
            s["b"] = _normal(gen, (g, n, k) if case["weights"] == "nk" else (g, k, n), 1.0 / math.sqrt(k), dt)
            s["bias_v"] = _normal(gen, (g, n), 0.5, torch.float32) if case["bias"] else None
            s["d"] = torch.empty((m, n), dtype=dt, device="cuda")
    if own:
        import tiled_tensor_core_02_gb300 as ttc
        s["lib"] = ttc
        if op == "i8":
            m, n, k = case["m"], case["n"], case["k"]
            need = ttc.ttc_gemm_i8_scaled_workspace_size(m, n, k, s["a"].data_ptr(), k, s["b"].data_ptr(), k,
                                                         s["d"].data_ptr(), n, _CODE[case["out"]])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return s


def _act(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["x"].float()
        top = x.abs().amax(dim=1)
        scale = top / torch.full_like(top, 127.0)
        scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
        inverse = torch.where(scale > 0, torch.ones_like(scale) / scale, torch.zeros_like(scale))
        return {"q": torch.round(x * inverse[:, None]).clamp(-127, 127).to(torch.int8), "scale": scale}
    if op == "i8":
        v = (s["a"].float() @ s["b"].float().t()) * s["scale_a"][:, None] * s["scale_b"][None, :]
        if s["bias_v"] is not None:
            v = v + s["bias_v"]
        return _act(v, s["act"]).to(s["d"].dtype)
    ends, d = s["ends"], s["d"]
    if op == "wgrad":
        for g in range(s["groups"]):
            lo, hi = ends[g], ends[g + 1]
            v = s["a"][lo:hi].float().t() @ s["b"][lo:hi].float()
            d[g] = v + s["d0"][g].float() if s["d0"] is not None else v
        return d
    for g in range(s["groups"]):
        lo, hi = ends[g], ends[g + 1]
        if hi > lo:
            w = s["b"][g].float()
            v = s["a"][lo:hi].float() @ (w.t() if s["weights"] == "nk" else w)
            if s["bias_v"] is not None:
                v = v + s["bias_v"][g]
            d[lo:hi] = _act(v, s["act"])
    return d


def run(s):
    if not own:
        return _plain(s)
    ttc, op = s["lib"], s["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "quantize":
        st = ttc.ttc_quantize_rows(s["rows"], s["cols"], s["x"].data_ptr(), s["cols"], _CODE[s["dtype"]],
                                   s["q"].data_ptr(), s["cols"], s["scale"].data_ptr(), stream)
        out = {"q": s["q"], "scale": s["scale"]}
    elif op == "i8":
        m, n, k, ws, bias = s["m"], s["n"], s["k"], s["ws"], s["bias_v"]
        st = ttc.ttc_gemm_i8_scaled(m, n, k, s["a"].data_ptr(), k, s["scale_a"].data_ptr(), s["b"].data_ptr(), k,
                                    s["scale_b"].data_ptr(), s["d"].data_ptr(), n,
                                    None if bias is None else bias.data_ptr(), _ACT[s["act"]], _CODE[s["out"]],
                                    None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), stream)
        out = s["d"]
    elif op == "wgrad":
        m, n, k, c = s["rows"], s["n"], s["k"], s["d0"]
        st = ttc.ttc_gemm_grouped_wgrad(s["groups"], m, n, k, s["a"].data_ptr(), k, s["b"].data_ptr(), n,
                                        s["offsets"].data_ptr(), None if c is None else c.data_ptr(), n, n * k,
                                        s["d"].data_ptr(), n, n * k, 1.0, 0.0 if c is None else 1.0,
                                        _CODE[s["dtype"]], _CODE[s["out"]], stream)
        out = s["d"]
    else:
        m, n, k, bias = s["rows"], s["n"], s["k"], s["bias_v"]
        nk = s["weights"] == "nk"
        st = ttc.ttc_gemm_grouped(s["groups"], m, n, k, s["a"].data_ptr(), k, s["offsets"].data_ptr(),
                                  s["b"].data_ptr(), k if nk else n, n * k, ttc.COL_MAJOR if nk else ttc.ROW_MAJOR,
                                  s["d"].data_ptr(), n, 1.0, None if bias is None else bias.data_ptr(), n,
                                  _ACT[s["act"]], _CODE[s["dtype"]], stream)
        out = s["d"]
    if st != 0:
        raise RuntimeError("%s: %s" % (op, ttc.ttc_status_string(st)))
    return out


def exact(case, seed):
    """The definitions in 64 bits, a block of rows or columns at a time."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        # a value half way between two steps goes either way with the last bit
        # of the scale, so the steps themselves have no exact value
        return {"q": None, "scale": (s["x"].double().abs().max(dim=1).values / 127.0)}

    def finish(v):
        if case["act"] == "relu":
            return v.clamp_min(0.0)
        if case["act"] == "gelu_tanh":
            return v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
        return v

    if op == "i8":
        out = torch.empty((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        a = s["a"].double()
        for j in range(0, case["n"], 2048):
            cols = slice(j, min(j + 2048, case["n"]))
            v = torch.matmul(a, s["b"][cols].double().transpose(0, 1))
            v = torch.einsum("ij,i,j->ij", v, s["scale_a"].double(), s["scale_b"][cols].double())
            out[:, cols] = finish(v if s["bias_v"] is None else v + s["bias_v"][cols].double())
        return out
    start, stop = s["ends"][:-1], s["ends"][1:]
    if op == "wgrad":
        out = torch.zeros((case["groups"], case["k"], case["n"]), dtype=torch.float64, device="cuda")
        if s["d0"] is not None:
            out.copy_(s["d0"])
        for g, (lo, hi) in enumerate(zip(start, stop)):
            out[g] += torch.einsum("mk,mn->kn", s["a"][lo:hi].double(), s["b"][lo:hi].double())
        return out
    out = torch.empty((case["rows"], case["n"]), dtype=torch.float64, device="cuda")
    form = "mk,nk->mn" if case["weights"] == "nk" else "mk,kn->mn"
    for g, (lo, hi) in enumerate(zip(start, stop)):
        v = torch.einsum(form, s["a"][lo:hi].double(), s["b"][g].double())
        out[lo:hi] = finish(v if s["bias_v"] is None else v + s["bias_v"][g].double())
    return out
