"""Cases of the gated feed-forward and the block-scaled fp8 operators, for measuring them.

Four operators, each in its plain form (`own` false: elementary torch
operations in 32 bits, rounded once at the end) and as the library's calls
(`own` true):

  gated     D = act(A Bg) * (A Bu): both projections of a gated feed-forward
            block, the activation and the product; for training with the two
            projections themselves.  Dense, or grouped by expert as the
            library's grouped products are (rows of group g by its weights).
  grad      with dH = A B, the gradient of D: dG = dH * U * act'(G) and
            dU = dH * act(G), and D again for the next weights' gradient.  A is
            the gradient of the block's result, B its last projection.
  quantize  8-bit floats with a fp32 scale for each block of 128 elements of a
            row, or of 128 x 128, of a matrix or of its transpose.
  f8        D[i, j] = act(sum over blocks b of 128 k: sA[i, b] sB[j, b] sum of
            A[i, k] B[j, k] over the block, + C[i, j]): the product of such
            rows, sB by rows or by blocks of 128 rows.
"""
import math
import random

import torch

own = False

_FLOAT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_CODE = {"f16": 0, "bf16": 1, "f32": 3, "e4m3": 4, "e5m2": 5}
_TOP = {"e4m3": 448.0, "e5m2": 57344.0}  # the largest finite values
_ACT = {"none": 0, "relu": 1, "gelu_tanh": 2, "silu": 3}


def listed():
    return [
        # one token through the library's MLP configuration, gated: the weights' bytes are the cost
        dict(name="gated 1x14336x4096", op="gated", rows=1, groups=1, n=14336, k=4096, dtype="bf16", weights="nk", act="silu",
             save=False, skew=0.0),
        # a decoding batch over small experts, some without a token: latency
        dict(name="gated decode 16x1024x1024", op="gated", rows=24, groups=16, n=1024, k=1024, dtype="f16", weights="nk",
             act="gelu_tanh", save=False, skew=0.5),
        # a chunk of a prompt, ragged in every direction, weights stored inputs first
        dict(name="gated chunk 1001x2728x1016", op="gated", rows=1001, groups=1, n=2728, k=1016, dtype="f16", weights="kn",
             act="silu", save=False, skew=0.0),
        # training: a large batch forward, the projections kept for the backward pass
        dict(name="gated train 8192x14336x4096", op="gated", rows=8192, groups=1, n=14336, k=4096, dtype="bf16", weights="nk",
             act="silu", save=True, skew=0.0),
        # its backward pass
        dict(name="grad train 8192x14336x4096", op="grad", rows=8192, groups=1, n=14336, k=4096, dtype="bf16", weights="kn",
             act="silu", save=True, skew=0.0),
        # the backward pass of a layer of small experts, ragged groups
        dict(name="grad 2047 of 16, 1536x2048", op="grad", rows=2047, groups=16, n=1536, k=2048, dtype="f16", weights="kn",
             act="gelu_tanh", save=False, skew=0.5),
        # activations of a decoding step
        dict(name="quantize 16x4096", op="quantize", rows=16, cols=4096, dtype="bf16", q="e4m3", block=1, turn=False),
        # activations of a training batch for the gradient of the weights: blocks along the tokens
        dict(name="quantize 8192x14336 turned", op="quantize", rows=8192, cols=14336, dtype="bf16", q="e4m3", block=1, turn=True),
        # one token through a quantized layer
        dict(name="f8 1x14336x4096", op="f8", rows=1, groups=1, n=14336, k=4096, ta="e4m3", tb="e4m3", block=128, out="bf16",
             act="none", add=False, skew=0.0),
        # a chunk of a prompt over many quantized experts: ragged groups of some dozen tokens
        dict(name="f8 4099 of 64, 1536x2048", op="f8", rows=4099, groups=64, n=1536, k=2048, ta="e4m3", tb="e4m3", block=128,
             out="bf16", act="none", add=False, skew=0.7),
        # a prompt through the library's MLP configuration
        dict(name="f8 8192x14336x4096", op="f8", rows=8192, groups=1, n=14336, k=4096, ta="e4m3", tb="e4m3", block=128, out="bf16",
             act="gelu_tanh", add=False, skew=0.0),
        # training: the gradient of the weights, both operands scaled along the tokens, added to 32-bit sums
        dict(name="f8 wgrad 4096x4096x8192", op="f8", rows=4096, groups=1, n=4096, k=8192, ta="e4m3", tb="e5m2", block=1, out="f32",
             act="none", add=True, skew=0.0),
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
    op = rng.choice(["gated", "gated", "grad", "quantize", "f8", "f8"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_width(rng, 64, 14336), dtype=rng.choice(["bf16", "f16", "f32"]),
                    q=rng.choice(["e4m3", "e4m3", "e5m2"]), block=rng.choice([1, 1, 128]), turn=rng.random() < 0.4)
    groups = rng.choice([1, 1, 1, 2, 7, 8, 16, 32, 64])
    rows = _log(rng, 1, 8192)
    big = groups == 1
    c = dict(op=op, rows=rows, groups=groups, n=_width(rng, 512, 14336 if big else 4096), k=_width(rng, 512, 4096),
             skew=round(rng.uniform(0.0, 1.0), 2))
    if op == "f8":
        add = big and rng.random() < 0.3
        c.update(ta=rng.choice(["e4m3", "e4m3", "e5m2"]), tb=rng.choice(["e4m3", "e4m3", "e5m2"]), block=rng.choice([1, 128, 128]),
                 out=rng.choice(["bf16", "bf16", "f16", "f32"]), act="none" if add else rng.choice(["none", "none", "relu", "gelu_tanh"]),
                 add=add)
    else:
        c.update(dtype=rng.choice(["bf16", "f16"]), weights=rng.choice(["nk", "kn"]), act=rng.choice(["silu", "silu", "gelu_tanh", "relu", "none"]),
                 save=rng.random() < 0.5)
    return c


def _offsets(case):
    """Where each group's rows start and end: groups + 1 numbers.  Shares of the
    rows are drawn unevenly (`skew`), and with many groups some get none."""
    if case["groups"] == 1:
        return [0, case["rows"]]
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


def _blocks(x):
    return -(-x // 128)


def work(case):
    if case["op"] == "quantize":
        e, size = 4 if case["dtype"] == "f32" else 2, case["rows"] * case["cols"]
        return {"bytes": size * (e + 1) + 4 * size // (128 * case["block"]), "flops": 3 * size}
    m, n, k, a = case["rows"], case["n"], case["k"], _active(case)
    if case["op"] == "gated":
        return {"bytes": 2 * m * k + 4 * n * k * a + 2 * m * n * (3 if case["save"] else 1), "flops": 4 * m * n * k + 2 * m * n}
    if case["op"] == "grad":
        # gate and up are read, their gradients written, and D where it is asked for
        return {"bytes": 2 * m * k + 2 * n * k * a + 2 * m * n * (5 if case["save"] else 4), "flops": 2 * m * n * k + 6 * m * n}
    e = 4 if case["out"] == "f32" else 2
    scales = m * _blocks(k) + a * (n if case["block"] == 1 else _blocks(n)) * _blocks(k)
    return {"bytes": m * k + n * k * a + 4 * scales + e * m * n * (2 if case["add"] else 1), "flops": 2 * m * n * k}


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


def _f8(gen, shape, kind, block):
    """8-bit values and scales as a quantizer leaves them: (values with rows on 16-byte boundaries, scales)."""
    rows, k = shape[-2:]
    # values of a block reach its largest one; scales of some spread
    pitch = -(-k // 16) * 16
    q = torch.empty((*shape[:-1], pitch), dtype=_FLOAT[kind], device="cuda")[..., :k]
    flat = q.view(-1, k) if pitch == k else q.flatten(0, -2)
    step = max(1, (1 << 27) // k)
    for i in range(0, flat.shape[0], step):
        part = flat[i:i + step]
        v = torch.randn(part.shape, generator=gen, device="cuda").mul_(_TOP[kind] / 4.0)
        part.copy_(v.clamp_(-_TOP[kind], _TOP[kind]))
    s = torch.exp(0.3 * torch.randn((*shape[:-2], -(-rows // block), _blocks(k)), generator=gen, device="cuda"))
    return q, s * (4.0 / _TOP[kind])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        s["x"] = _activations(gen, case["rows"], case["cols"], _FLOAT[case["dtype"]])
        r, c = (case["cols"], case["rows"]) if case["turn"] else (case["rows"], case["cols"])
        s["d"] = torch.empty((r, -(-c // 16) * 16), dtype=_FLOAT[case["q"]], device="cuda")[:, :c]
        s["scale"] = torch.empty((-(-r // case["block"]), _blocks(c)), device="cuda")
        return s
    m, n, k, g = case["rows"], case["n"], case["k"], case["groups"]
    s["ends"] = _offsets(case)
    s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda") if g > 1 else None
    if op == "f8":
        s["a"], s["scale_a"] = _f8(gen, (m, k), case["ta"], 1)
        s["b"], s["scale_b"] = _f8(gen, (g, n, k), case["tb"], case["block"])
        s["scale_b"] /= math.sqrt(k)
        out = _FLOAT[case["out"]]
        # what earlier micro-batches have added
        s["c"] = _normal(gen, (m, n), 0.5, out) if case["add"] else None
        s["d"] = torch.empty((m, n), dtype=out, device="cuda")
        return s
    dt = _FLOAT[case["dtype"]]
    s["a"] = _activations(gen, m, k, dt)
    shape = (g, n, k) if case["weights"] == "nk" else (g, k, n)
    s["b"] = _normal(gen, shape, 1.0 / math.sqrt(k), dt)
    s["d"] = torch.empty((m, n), dtype=dt, device="cuda") if op == "gated" or case["save"] else None
    if op == "gated":
        s["b_up"] = _normal(gen, shape, 1.0 / math.sqrt(k), dt)
        s["pre"] = torch.empty((m, 2 * n), dtype=dt, device="cuda") if case["save"] else None
    else:
        s["pre"] = _normal(gen, (m, 2 * n), 1.0, dt)  # what the forward pass kept: gate and up side by side
        s["dpre"] = torch.empty((m, 2 * n), dtype=dt, device="cuda")
    return s


def _act(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _slope(v, act):
    """The derivative of _act."""
    if act == "relu":
        return torch.where(v > 0, torch.ones_like(v), torch.zeros_like(v))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * (c + 3.0 * 0.044715 * c * v * v)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    return torch.ones_like(v)


def _values(q, scale, block):
    """The numbers that blocks of 8-bit floats stand for, in 32 bits."""
    by_column = scale.repeat_interleave(128, dim=-1)[..., :q.shape[-1]]
    return q.float() * (by_column if block == 1 else by_column.repeat_interleave(128, dim=-2)[..., :q.shape[-2], :])


def _quantize(s):
    x = s["x"].t() if s["turn"] else s["x"]
    rows, cols = x.shape
    top, block = _TOP[s["q"]], s["block"]
    x = torch.nn.functional.pad(x.float(), (0, -cols % 128, 0, -rows % block))
    x = x.reshape(x.shape[0] // block, block, x.shape[1] // 128, 128)
    scale = x.abs().amax(dim=(1, 3)) / torch.full((1, 1), top, device="cuda")
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inverse = torch.where(scale > 0, torch.ones_like(scale) / scale, torch.zeros_like(scale))
    q = (x * inverse[:, None, :, None]).clamp(-top, top).to(_FLOAT[s["q"]])
    return {"q": q.reshape(q.shape[0] * block, -1)[:rows, :cols], "scale": scale}


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _quantize(s)
    outs, dt = {}, s["a"].dtype
    if op == "f8":
        d = s["d"]
    elif op == "gated":
        d, pre, n = s["d"], s["pre"], s["n"]
    else:
        d, pre, dpre, n = s["d"], s["pre"], s["dpre"], s["n"]
    for g in range(s["groups"]):  # one turn for a dense layer
        lo, hi = s["ends"][g], s["ends"][g + 1]
        if hi == lo:
            continue
        if op == "f8":
            v = _values(s["a"][lo:hi], s["scale_a"][lo:hi], 1) @ _values(s["b"][g], s["scale_b"][g], s["block"]).t()
            d[lo:hi] = _act(v if s["c"] is None else v + s["c"][lo:hi].float(), s["act"])
            continue
        w = s["b"][g].float()
        v = s["a"][lo:hi].float() @ (w.t() if s["weights"] == "nk" else w)
        if op == "gated":
            w = s["b_up"][g].float()
            u = s["a"][lo:hi].float() @ (w.t() if s["weights"] == "nk" else w)
            d[lo:hi] = _act(v, s["act"]) * u
            if pre is not None:
                pre[lo:hi, :n], pre[lo:hi, n:] = v, u
        else:
            gate, up = pre[lo:hi, :n].float(), pre[lo:hi, n:].float()
            a = _act(gate, s["act"])
            dpre[lo:hi, :n], dpre[lo:hi, n:] = v * up * _slope(gate, s["act"]), v * a
            if d is not None:
                d[lo:hi] = a * up
    if op == "f8":
        return d
    outs["d"] = d
    if op == "gated":
        outs["pre"] = pre
    else:
        outs["dpre"] = dpre
    return {k: v for k, v in outs.items() if v is not None}


def _address(t, column=0):
    return None if t is None else t.data_ptr() + column * t.element_size()


def run(s):
    if not own:
        return _plain(s)
    import tiled_tensor_core_02_gb300 as ttc

    op = s["op"]
    stream = torch.cuda.current_stream().cuda_stream
    d = s["d"]
    if op == "quantize":
        x, scale = s["x"], s["scale"]
        st = ttc.ttc_quantize_blocks(s["rows"], s["cols"], x.data_ptr(), s["cols"], _CODE[s["dtype"]], s["block"], int(s["turn"]),
                                     d.data_ptr(), d.stride(0), _CODE[s["q"]], scale.data_ptr(), scale.shape[1], stream)
        out = {"q": d, "scale": scale}
    elif op == "f8":
        m, n, k, g, a, b, sa, sb = s["rows"], s["n"], s["k"], s["groups"], s["a"], s["b"], s["scale_a"], s["scale_b"]
        st = ttc.ttc_gemm_f8_blocks(g, m, n, k, a.data_ptr(), a.stride(0), _CODE[s["ta"]], sa.data_ptr(), sa.shape[1],
                                    _address(s["offsets"]), b.data_ptr(), b.stride(1), b.stride(0), _CODE[s["tb"]], sb.data_ptr(),
                                    sb.shape[2], sb.stride(0), s["block"], _address(s["c"]), n, d.data_ptr(), n, None, 0,
                                    _ACT[s["act"]], _CODE[s["out"]], stream)
        out = d
    else:
        m, n, k, g, a, b, pre = s["rows"], s["n"], s["k"], s["groups"], s["a"], s["b"], s["pre"]
        ldb, layout = (k, ttc.COL_MAJOR) if s["weights"] == "nk" else (n, ttc.ROW_MAJOR)
        if op == "gated":
            st = ttc.ttc_gemm_gated(g, m, n, k, a.data_ptr(), k, _address(s["offsets"]), b.data_ptr(), s["b_up"].data_ptr(), ldb,
                                    n * k, layout, d.data_ptr(), n, _address(pre), _address(pre, n), 2 * n, _ACT[s["act"]],
                                    _CODE[s["dtype"]], stream)
            out = {"d": d} if pre is None else {"d": d, "pre": pre}
        else:
            dpre = s["dpre"]
            st = ttc.ttc_gemm_gated_grad(g, m, n, k, a.data_ptr(), k, _address(s["offsets"]), b.data_ptr(), ldb, n * k, layout,
                                         _address(pre), _address(pre, n), 2 * n, _address(dpre), _address(dpre, n), 2 * n,
                                         _address(d), n, _ACT[s["act"]], _CODE[s["dtype"]], stream)
            out = {"dpre": dpre} if d is None else {"d": d, "dpre": dpre}
    if st != 0:
        raise RuntimeError("%s: %s" % (op, ttc.ttc_status_string(st)))
    return out


def exact(case, seed):
    """The definitions in 64 bits, a block of columns at a time."""
    s = prepare(case, seed)
    op, act = case["op"], case.get("act")
    if op == "quantize":
        # a value half way between two steps goes either way with the last bit of the
        # scale, so the steps themselves have no exact value
        x = s["x"].t() if case["turn"] else s["x"]
        (rows, cols), b = x.shape, case["block"]
        most = torch.zeros((-(-rows // b) * b, _blocks(cols) * 128), dtype=torch.float64, device="cuda")
        most[:rows, :cols] = x.double().abs()
        return {"q": None, "scale": most.unflatten(1, (-1, 128)).unflatten(0, (-1, b)).amax(dim=(1, 3)) / _TOP[case["q"]]}

    def sigmoid(v):
        return torch.special.expit(v)

    def logistic_gelu(v):  # (1 + tanh(z)) / 2 = sigmoid(2 z)
        return sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))

    def value(v):
        return {"none": lambda: v, "relu": lambda: v.clamp_min(0.0), "silu": lambda: v * sigmoid(v),
                "gelu_tanh": lambda: v * logistic_gelu(v)}[act]()

    def derivative(v):
        if act == "silu":
            return sigmoid(v) + v * sigmoid(v) * sigmoid(-v)
        if act == "gelu_tanh":
            q = logistic_gelu(v)
            return q + 2.0 * math.sqrt(2.0 / math.pi) * v * q * (1.0 - q) * (1.0 + 0.134145 * v ** 2)
        return (v > 0).double() if act == "relu" else torch.ones_like(v)

    m, n = case["rows"], case["n"]

    def wide(q, scale, rows_of_a_block):
        v = q.double()
        for b in range(scale.shape[-1]):
            by_row = scale[..., b].double()
            if rows_of_a_block > 1:
                by_row = by_row.unsqueeze(-1).expand(-1, rows_of_a_block).flatten()[:q.shape[0]]
            v[:, 128 * b:128 * b + 128].mul_(by_row.unsqueeze(-1))
        return v

    names = {"f8": ("d",), "gated": ("d", "gate", "up") if case.get("save") else ("d",),
             "grad": ("dgate", "dup", "d") if case.get("save") else ("dgate", "dup")}[op]
    out = {name: torch.empty((m, n), dtype=torch.float64, device="cuda") for name in names}
    for g, (lo, hi) in enumerate(zip(s["ends"][:-1], s["ends"][1:])):
        a = wide(s["a"][lo:hi], s["scale_a"][lo:hi], 1) if op == "f8" else s["a"][lo:hi].double()
        for j in range(0, n if hi > lo else 0, 2048):
            cols = slice(j, min(j + 2048, n))
            if op == "f8":
                by = case["block"]
                b = wide(s["b"][g][cols], s["scale_b"][g][(j // by):-(-cols.stop // by)], by)
                v = torch.einsum("mk,nk->mn", a, b)
                out["d"][lo:hi, cols] = value(v if s["c"] is None else v + s["c"][lo:hi, cols].double())
                continue
            pick = (lambda w: w[g][cols].double()) if case["weights"] == "nk" else (lambda w: w[g][:, cols].double().t())
            v = torch.einsum("mk,nk->mn", a, pick(s["b"]))
            if op == "gated":
                u = torch.einsum("mk,nk->mn", a, pick(s["b_up"]))
                out["d"][lo:hi, cols] = value(v) * u
                if case["save"]:
                    out["gate"][lo:hi, cols], out["up"][lo:hi, cols] = v, u
            else:
                gate, up = s["pre"][lo:hi, cols].double(), s["pre"][lo:hi, n + j:n + cols.stop].double()
                out["dgate"][lo:hi, cols] = torch.einsum("ij,ij,ij->ij", v, up, derivative(gate))
                out["dup"][lo:hi, cols] = v * value(gate)
                if case["save"]:
                    out["d"][lo:hi, cols] = value(gate) * up
    if op == "f8":
        return out["d"]
    if op == "gated":
        return {"d": out["d"], "pre": torch.cat((out["gate"], out["up"]), 1)} if case["save"] else {"d": out["d"]}
    return {"dpre": torch.cat((out["dgate"], out["dup"]), 1), **({"d": out["d"]} if case["save"] else {})}
