"""The operators of 8-bit floating-point tensor-parallel layers, measured at real sizes.

Between two blocks of a decoder layer a serving step adds the t partial sums of the last
row-parallel layer to the residual stream and norms the rows into 8 bits (`norm`); what the
attention leaves is brought to 8 bits by itself (`quant`, which also makes the weights' codes
when a model is loaded); the column- and row-parallel layers multiply 8-bit rows by 8-bit
weights (`col`, `row`), and the MLP block runs both with its hidden rows in 8 bits (`mlp`).

Values are e4m3 codes (torch.float8_e4m3fn) with float32 scales.  A row of k columns has a
scale for each group of 128 columns (the last may be shorter), held [ceil(k/128), rows]; a
weight [out, k] has one for each block of 128 x 128, held [ceil(out/128), ceil(k/128)]; a
merged [gate; up] weight has the blocks of its gate rows, then those of its up rows.  The scale
of a group is max(its largest |x|, 2^-100) / 448 and a code is x / scale rounded to the
nearest e4m3 value.
"""

import math

import torch

own = False

G = 128                     # columns of a group, rows and columns of a weight's block
TOP = 448.0                 # largest e4m3 value
LEAST = 2.0 ** -100         # a group's largest value counts as at least this


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token between the layers of a model of 8192, partials of 4 shards: latency counts
        dict(name="norm_one", kind="norm", t=4, n=1, h=8192, f32=False, residual=True),
        # a prefill's rows between the same layers
        dict(name="norm_prefill", kind="norm", t=4, n=8192, h=8192, f32=False, residual=True),
        # the attention's output of a decode batch, before o_proj of 8 shards
        dict(name="quant_decode", kind="quant", t=8, n=64, k=1024, weight=False),
        # the same of a prefill
        dict(name="quant_prefill", kind="quant", t=4, n=8192, k=2048, weight=False),
        # a shard of a gate_up weight as a model is loaded
        dict(name="quant_weight", kind="quant", t=1, n=14336, k=8192, weight=True),
        # QKV projection of a decode batch, 8 shards
        dict(name="qkv_decode", kind="col", t=8, n=16, k=8192, out=1280, gated=False, f32=False),
        # gate_up of an odd chunk of a prompt, hidden rows in 8 bits
        dict(name="gate_up_chunk", kind="col", t=8, n=333, k=8192, out=3584, gated=True, f32=False),
        # o_proj of one token over 8 shards, and of a chunk
        dict(name="o_proj_one", kind="row", t=8, n=1, k=1024, out=8192, f32=False),
        dict(name="o_proj_chunk", kind="row", t=4, n=1000, k=2048, out=8192, f32=True),
        # the MLP block of a small model for a few tokens, of a large one in decode and in prefill
        dict(name="mlp_small", kind="mlp", t=2, n=8, h=1024, f=4096),
        dict(name="mlp_decode", kind="mlp", t=4, n=32, h=8192, f=28672),
        dict(name="mlp_prefill", kind="mlp", t=4, n=4096, h=8192, f=28672),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, step * round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)))


def draw(rng):
    kind = rng.choice(["norm", "quant", "col", "col", "row", "row", "mlp", "mlp"])
    t = rng.choice([1, 2, 4, 8])
    if kind == "norm":
        return dict(kind=kind, t=t, n=_log(rng, 1, 8192), h=_log(rng, 512, 8192, 16), f32=rng.random() < 0.3,
                    residual=rng.random() < 0.8)
    if kind == "quant":
        weight = rng.random() < 0.3
        return dict(kind=kind, t=t, n=_log(rng, 100, 14336) if weight else _log(rng, 1, 8192),
                    k=_log(rng, 256, 8192 // t, 16), weight=weight)
    if kind == "col":
        gated = rng.random() < 0.5
        return dict(kind=kind, t=t, n=_log(rng, 1, 4096), k=_log(rng, 512, 8192, 16), out=_log(rng, 128, 28672 // t, 16),
                    gated=gated, f32=not gated and rng.random() < 0.5)
    if kind == "row":
        return dict(kind=kind, t=t, n=_log(rng, 1, 4096), k=_log(rng, 256, 28672 // t, 16), out=_log(rng, 512, 8192, 8),
                    f32=rng.random() < 0.3)
    return dict(kind=kind, t=t, n=_log(rng, 1, 4096), h=_log(rng, 512, 8192, 16), f=t * _log(rng, 128, 28672 // t, 16))


def _groups(k):
    return -(-k // G)


def work(c):
    kind, t, n = c["kind"], c["t"], c["n"]
    if kind == "norm":
        h = c["h"]
        io = t * (4 if c["f32"] else 2) + 2 * c["residual"] + 2 + 1
        return {"bytes": n * h * io + 4 * n * _groups(h) + 2 * h, "flops": n * h * (t + 6)}
    if kind == "quant":
        k = c["k"]
        scales = _groups(n) * _groups(k) if c["weight"] else n * _groups(k)
        return {"bytes": t * (3 * n * k + 4 * scales), "flops": 3 * t * n * k}
    if kind == "col":
        k, out = c["k"], c["out"]
        rows = out * (2 if c["gated"] else 1)
        y = n * out * (4 if c["f32"] else 2) if not c["gated"] else n * out + 4 * n * _groups(out)
        return {"bytes": n * k + 4 * n * _groups(k) + t * (rows * k + y + 4 * _groups(rows) * _groups(k)),
                "flops": 2 * t * n * rows * k}
    if kind == "row":
        k, out = c["k"], c["out"]
        return {"bytes": t * (n * k + 4 * n * _groups(k) + out * k + 4 * _groups(out) * _groups(k))
                + n * out * (4 if c["f32"] else 2), "flops": 2 * t * n * out * k}
    h, f = c["h"], c["f"]
    return {"bytes": n * h + 4 * n * _groups(h) + 3 * h * f + 12 * _groups(h) * _groups(f) + 2 * n * h,
            "flops": 6 * n * h * f}


# ------------------------------------------------------------------ inputs

def _scale(amax):
    return amax.clamp(min=LEAST) / torch.full((), TOP, device=amax.device)     # by a tensor: a true division


def _pad(x, *sides):
    """x with zeros behind its last two sizes, up to multiples of sides."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % sides[1], 0, -x.shape[-2] % sides[0]))


def _quantise_rows(x):
    """Codes [n, k] and scales [groups, n] of float rows [n, k]."""
    n, k = x.shape
    v = _pad(x, 1, G).view(n, -1, G)
    s = _scale(v.abs().amax(-1, keepdim=True))
    return (v / s).view(n, -1)[:, :k].to(torch.float8_e4m3fn), s.squeeze(-1).t().contiguous()


def _quantise_weight(w):
    """Codes [out, k] and scales [blocks, groups] of a float weight [out, k]."""
    out, k = w.shape
    v = _pad(w, G, G)
    v = v.view(v.shape[0] // G, G, v.shape[1] // G, G)
    s = _scale(v.abs().amax((1, 3), keepdim=True))
    codes = (v / s).view(v.shape[0] * G, -1)[:out, :k].to(torch.float8_e4m3fn).contiguous()
    return codes, s.view(s.shape[0], s.shape[2]).contiguous()


def _rows(codes, scales):
    """float32 rows that codes [n, k] and scales [groups, n] stand for."""
    n, k = codes.shape
    return codes.float() * scales.t().repeat_interleave(G, 1)[:, :k]


def _weight(codes, scales):
    """float32 weight that codes [out, k] and scales [blocks, groups] stand for."""
    out, k = codes.shape
    v = _pad(codes.float(), G, G)
    v = v.view(v.shape[0] // G, G, v.shape[1] // G, G) * scales[:, None, :, None]
    return v.view(scales.shape[0] * G, -1)[:out, :k]


def _gated(codes, scales):
    half, blocks = codes.shape[0] // 2, scales.shape[0] // 2
    return _weight(codes[:half], scales[:blocks]), _weight(codes[half:], scales[blocks:])


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    kind, t, n = c["kind"], c["t"], c["n"]
    s = {"case": dict(c)}

    def rows(n, k, dtype=torch.bfloat16):          # activations: some channels are louder
        loud = torch.exp(0.6 * torch.randn(k, device=dev, generator=g))
        return (torch.randn((n, k), device=dev, generator=g) * loud).to(dtype)

    def weight(out, k):
        return torch.randn((out, k), device=dev, generator=g) * 0.02

    def gate_up(os, k):
        a, b = _quantise_weight(weight(os, k)), _quantise_weight(weight(os, k))
        return torch.cat([a[0].view(torch.uint8), b[0].view(torch.uint8)]).view(torch.float8_e4m3fn), torch.cat([a[1], b[1]])

    def split(pairs):
        return [p[0] for p in pairs], [p[1] for p in pairs]

    if kind == "norm":
        dt = torch.float32 if c["f32"] else torch.bfloat16
        s["partials"] = [rows(n, c["h"], dt) * 0.3 for _ in range(t)]
        s["residual"] = rows(n, c["h"]) if c["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(c["h"], device=dev, generator=g)).to(torch.bfloat16)
    elif kind == "quant":
        s["x"] = [weight(n, c["k"]).to(torch.bfloat16) if c["weight"] else rows(n, c["k"]) for _ in range(t)]
    elif kind == "col":
        s["x"], s["xs"] = _quantise_rows(rows(n, c["k"]).float())
        s["w"], s["ws"] = split([gate_up(c["out"], c["k"]) if c["gated"] else _quantise_weight(weight(c["out"], c["k"]))
                                 for _ in range(t)])
    elif kind == "row":
        s["x"], s["xs"] = split([_quantise_rows(rows(n, c["k"]).float()) for _ in range(t)])
        s["w"], s["ws"] = split([_quantise_weight(weight(c["out"], c["k"])) for _ in range(t)])
    else:
        h, fs = c["h"], c["f"] // t
        s["x"], s["xs"] = _quantise_rows(rows(n, h).float())
        s["a"], s["as"] = split([gate_up(fs, h) for _ in range(t)])
        s["b"], s["bs"] = split([_quantise_weight(weight(h, fs)) for _ in range(t)])
    if own:                                    # the checked and marshalled call that a serving loop repeats
        s["call"] = _handle(s)
    return s


def _handle(s):
    import megatron_tensor_layers_gb300 as tp

    c = s["case"]
    dt = torch.float32 if c.get("f32") else torch.bfloat16
    if c["kind"] == "norm":
        return tp.prepare(tp.tp_fp8_rmsnorm, s["partials"], s["weight"], residual=s["residual"])
    if c["kind"] == "quant":
        return tp.prepare(tp.tp_fp8_quantize_weight if c["weight"] else tp.tp_fp8_quantize, s["x"])
    if c["kind"] == "col":
        if c["gated"]:
            return tp.prepare(tp.tp_fp8_linear_col, s["x"], s["xs"], s["w"], s["ws"], act="silu", y_dtype=torch.float8_e4m3fn)
        return tp.prepare(tp.tp_fp8_linear_col, s["x"], s["xs"], s["w"], s["ws"], y_dtype=dt)
    if c["kind"] == "row":
        return tp.prepare(tp.tp_fp8_linear_row, s["x"], s["xs"], s["w"], s["ws"], mode="fused", y_dtype=dt)
    return tp.prepare(tp.tp_fp8_mlp_forward, s["x"], s["xs"], s["a"], s["as"], s["b"], s["bs"], mode="fused")


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return s["call"]()
    return {"norm": _plain_norm, "quant": _plain_quant, "col": _plain_col, "row": _plain_row, "mlp": _plain_mlp}[s["case"]["kind"]](s)


def _act(g):
    return g / (1.0 + torch.exp(-g))


def _plain_norm(s):
    r = s["partials"][0].float()
    for p in s["partials"][1:]:
        r = r + p.float()
    if s["residual"] is not None:
        r = s["residual"].float() + r
    y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    codes, scales = _quantise_rows(y)
    return r.to(torch.bfloat16), codes, scales


def _plain_quant(s):
    f = _quantise_weight if s["case"]["weight"] else _quantise_rows
    both = [f(x.float()) for x in s["x"]]
    return [b[0] for b in both], [b[1] for b in both]


def _plain_col(s):
    c, x = s["case"], _rows(s["x"], s["xs"])
    if not c["gated"]:
        dt = torch.float32 if c["f32"] else torch.bfloat16
        return [(x @ _weight(w, ws).t()).to(dt) for w, ws in zip(s["w"], s["ws"])]
    both = [_quantise_rows(_plain_gated(x, w, ws)) for w, ws in zip(s["w"], s["ws"])]
    return [b[0] for b in both], [b[1] for b in both]


def _plain_gated(x, w, ws):
    gate, up = _gated(w, ws)
    return _act(x @ gate.t()) * (x @ up.t())


def _plain_row(s):
    y = 0.0
    for x, xs, w, ws in zip(s["x"], s["xs"], s["w"], s["ws"]):
        y = y + _rows(x, xs) @ _weight(w, ws).t()
    return y.to(torch.float32 if s["case"]["f32"] else torch.bfloat16)


def _plain_mlp(s):
    x, y = _rows(s["x"], s["xs"]), 0.0
    for a, sa, b, sb in zip(s["a"], s["as"], s["b"], s["bs"]):
        hidden = _rows(*_quantise_rows(_plain_gated(x, a, sa)))
        y = y + hidden @ _weight(b, sb).t()
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ the definition in 64 bits

def _nearest(v):
    """float64 v rounded to the nearest e4m3 value, ties to the even one."""
    _, e = torch.frexp(v.abs())                                    # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _each(k):
    """The group of every column."""
    return torch.arange(k, device="cuda") // G


def _code_rows(v):
    """(code values, scales [groups, n]) of float64 rows."""
    n, k = v.shape
    top = torch.zeros((n, _groups(k)), dtype=v.dtype, device=v.device)
    top.scatter_reduce_(1, _each(k).expand(n, k), v.abs(), "amax")
    s = (torch.clamp(top, min=LEAST) / TOP).float().double()       # a scale is held in float32
    return _nearest(v / s[:, _each(k)]), s.t()


def _spread(codes, scales, by_row):
    """float64 values of codes: scales [groups, n] of rows, or [blocks, groups] of a weight."""
    v = codes.double()
    if by_row:
        return v * scales.double()[_each(codes.shape[1])].t()
    return v * scales.double()[_each(codes.shape[0])][:, _each(codes.shape[1])]


def exact(c, seed):
    s = prepare(c, seed)
    kind = c["kind"]
    if kind == "norm":
        r = sum(p.double() for p in s["partials"])
        if s["residual"] is not None:
            r = r + s["residual"].double()
        y = r * torch.rsqrt((r * r).sum(-1, keepdim=True) / c["h"] + 1e-6) * s["weight"].double()
        return (r, *_code_rows(y))
    if kind == "quant":
        if not c["weight"]:
            both = [_code_rows(x.double()) for x in s["x"]]
        else:
            both = []
            for x in s["x"]:
                v, rows, cols = x.double(), _each(c["n"]), _each(c["k"])
                top = torch.zeros((_groups(c["n"]), c["k"]), dtype=v.dtype, device=v.device)
                top.scatter_reduce_(0, rows[:, None].expand_as(v), v.abs(), "amax")
                sc = torch.zeros((_groups(c["n"]), _groups(c["k"])), dtype=v.dtype, device=v.device)
                sc.scatter_reduce_(1, cols.expand_as(top), top, "amax")
                sc = (torch.clamp(sc, min=LEAST) / TOP).float().double()
                both.append((_nearest(v / sc[rows][:, cols]), sc))
        return [b[0] for b in both], [b[1] for b in both]
    if kind == "row":
        return sum(_spread(x, xs, True) @ _spread(w, ws, False).T for x, xs, w, ws in zip(s["x"], s["xs"], s["w"], s["ws"]))
    x = _spread(s["x"], s["xs"], True)

    def hidden(w, ws):
        half, blocks = w.shape[0] // 2, ws.shape[0] // 2
        gate = x @ _spread(w[:half], ws[:blocks], False).T
        return gate * torch.sigmoid(gate) * (x @ _spread(w[half:], ws[blocks:], False).T)

    if kind == "col":
        if not c["gated"]:
            return [x @ _spread(w, ws, False).T for w, ws in zip(s["w"], s["ws"])]
        both = [_code_rows(hidden(w, ws)) for w, ws in zip(s["w"], s["ws"])]
        return [b[0] for b in both], [b[1] for b in both]
    y = 0.0
    for a, sa, b, sb in zip(s["a"], s["as"], s["b"], s["bs"]):
        codes, sc = _code_rows(hidden(a, sa))
        y = y + _spread(codes, sc, True) @ _spread(b, sb, False).T
    return y
