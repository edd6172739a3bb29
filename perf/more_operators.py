"""Cases of the operators of a gated feed-forward block, with the operators'
plain forms.

Four operators, each in its directions and types:

  * ``gated``: both projections of a gated block, the activation and their
    product, from E4M3 operands, dense or per expert; the result in bf16, or
    quantized 1x128 together with the projections themselves as a checkpoint
    in 8 bits.
  * ``grad``: the gradient of the activation and the product from the
    checkpoint (8 bits or bf16), as it is, or quantized for the input gradient
    and for the weight gradients.
  * ``read`` and ``turn``: a checkpoint in 8 bits read back, and turned into the
    128x1 groups that a weight gradient sums over.
  * ``dgrad``: input gradients of the experts' products.

With ``own`` false, ``run`` computes a pass with elementary torch operations
in 32 bits, rounded once at the end; with ``own`` true, with this package's
entry points.
"""
import math

import torch

own = False

BF16, F32, F8, F64 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float64
TYPES = {"bf16": BF16, "f32": F32}
E4M3_MAX = 448.0

# Largest work of a case: products in multiplications, the others in values.
MOST_PRODUCT = 4096 * 4096 * 7168
MOST_VALUES = 4096 * 7168


# ---- cases -------------------------------------------------------------------

def _gated(name, rows, inner, width, act="silu", result="quant", keep=False, scales="f32",
           experts=0, spare=0):
    return {"name": name, "kind": "gated", "rows": rows, "inner": inner, "width": width,
            "act": act, "result": result, "keep": keep, "scales": scales, "experts": experts,
            "spare": spare}


def _grad(name, rows, inner, act="silu", kept="e4m3", da="bf16", result="all"):
    return {"name": name, "kind": "grad", "rows": rows, "inner": inner, "act": act, "kept": kept,
            "da": da, "result": result}


def _stored(name, kind, rows, width, result="bf16", scales="f32"):
    return {"name": name, "kind": kind, "rows": rows, "width": width, "result": result,
            "scales": scales}


def _dgrad(name, rows, experts, out, inner, scales="f32", spare=0):
    return {"name": name, "kind": "dgrad", "rows": rows, "experts": experts, "out": out,
            "inner": inner, "scales": scales, "spare": spare}


def listed():
    return [
        # one sequence generating, a shared expert of 2048; all latency and
        # the weights' bytes
        _gated("gated_one_token", 1, 2048, 7168, result="bf16"),
        # a decode batch of 256 tokens through 2 x 1024 columns, quantized for
        # the down projection
        _gated("gated_decode_256", 256, 1024, 7168),
        # a small model's odd batch, GELU, power-of-two scales, projections kept
        _gated("gated_ragged_333", 333, 640, 896, act="gelu_tanh", keep=True, scales="pow2"),
        # training step over 4096 tokens: quantized, projections kept in 8 bits
        _gated("gated_train_4096", 4096, 2048, 7168, keep=True),
        # sixteen tokens to 8 of 32 experts each
        _gated("gated_experts_decode", 128, 2048, 7168, experts=32),
        # prefill of 8192 rows over 32 experts, projections kept in 8 bits
        _gated("gated_experts_8192", 8192, 2048, 7168, keep=True, experts=32),
        # gradient of a small odd batch from bf16 projections, fp32 da
        _grad("grad_ragged_333", 333, 640, act="gelu_tanh", kept="bf16", da="f32",
              result="dense"),
        # training step over 4096 tokens: everything that the input and weight
        # gradients take
        _grad("grad_train_4096", 4096, 2048),
        # an odd matrix read back from 8 bits
        _stored("read_ragged_1037", "read", 1037, 1001, result="f32"),
        # a layer's 4096 stored input rows, turned for its weight gradient
        _stored("turn_4096", "turn", 4096, 7168),
        # a small model's experts, some rows behind the last expert's
        _dgrad("dgrad_ragged_1037", 1037, 10, 1024, 896, spare=37),
        # down projections of 32 experts, 8192 rows
        _dgrad("dgrad_experts_8192", 8192, 32, 7168, 2048),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _blocks(rng, low, high):
    return max(1, _log(rng, low, high) // 128) * 128


def draw(rng):
    what = rng.choice(("gated", "gated", "experts", "grad", "read", "turn", "dgrad"))
    if what in ("gated", "experts"):
        inner, width = _blocks(rng, 128, 2048), _blocks(rng, 256, 7168)
        rows = _log(rng, 1, min(8192, MOST_PRODUCT // (2 * inner * width)))
        experts = _log(rng, 2, 32) if what == "experts" else 0
        spare = rng.choice((0, 0, rng.randint(1, rows))) if experts else 0
        result = rng.choice(("bf16", "quant", "quant"))
        case = _gated("", rows, inner, width, rng.choice(("silu", "silu", "gelu_tanh")), result,
                      result == "quant" and rng.random() < 0.5,
                      rng.choice(("f32", "f32", "pow2")), experts, spare)
    elif what == "grad":
        inner = _blocks(rng, 128, 2048)
        rows = _log(rng, 1, MOST_VALUES // 4 // inner)
        case = _grad("", rows, inner, rng.choice(("silu", "silu", "gelu_tanh")),
                     rng.choice(("e4m3", "e4m3", "bf16")), rng.choice(("bf16", "bf16", "f32")),
                     rng.choice(("dense", "rows", "all")))
    elif what == "dgrad":
        out, inner = _blocks(rng, 256, 7168), _blocks(rng, 128, 4096)
        experts = _log(rng, 2, 32)
        rows = _log(rng, 1, min(8192, MOST_PRODUCT // (out * inner)))
        case = _dgrad("", rows, experts, out, inner, rng.choice(("f32", "f32", "pow2")),
                      rng.choice((0, 0, rng.randint(1, rows))))
    else:
        width = _log(rng, 64, 7168)
        if rng.random() < 0.5:
            width = max(128, width // 128 * 128)
        case = _stored("", what, _log(rng, 1, MOST_VALUES // width), width,
                       rng.choice(("bf16", "f32")) if what == "read" else "bf16",
                       rng.choice(("f32", "pow2")) if what == "read" else "f32")
    del case["name"]
    return case


# ---- inputs ------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _normal(g, shape, dtype=F32, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _activations(g, rows, width):
    """N(0, 1) with about 0.1% of the channels 100 times as large, as
    activations have them."""
    x = torch.randn((rows, width), generator=g, device="cuda")
    far = torch.rand(width, generator=g, device="cuda") < 1e-3
    return (x * torch.where(far, 100.0, 1.0)).to(BF16).float()


def _groups(v):
    """v [..., width] as [..., groups, 128], zeros past the end."""
    width = v.shape[-1]
    groups = (width + 127) // 128
    if width % 128:
        v = torch.nn.functional.pad(v, (0, groups * 128 - width))
    return v.reshape(*v.shape[:-1], groups, 128)


def _scale(amax, scales):
    """amax / 448, or the smallest power of two (2^-126 at least) that is no
    smaller."""
    if scales == "f32":
        return amax / E4M3_MAX
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, -126).clamp_min(-126)
    return torch.ldexp(torch.ones_like(amax), e)


def _codes(v, s):
    return torch.where(s > 0, v / s, 0.0).clamp(-E4M3_MAX, E4M3_MAX).to(F8)


def _quantized(v, scales="f32"):
    """1x128 E4M3 values and scales of fp32 v [..., width]."""
    grouped = _groups(v)
    s = _scale(grouped.abs().amax(-1), scales)
    q = _codes(grouped, s[..., None])
    return q.reshape(*v.shape[:-1], -1)[..., :v.shape[-1]].contiguous(), s


def _quantized_blocks(w, scales):
    """128x128 E4M3 bytes and scales of fp32 w [out][inner], both multiples of
    128."""
    n, k = w.shape
    blocks = w.reshape(n // 128, 128, k // 128, 128)
    s = _scale(blocks.abs().amax((1, 3)), scales)
    return _codes(blocks, s[:, None, :, None]).reshape(n, k).view(torch.uint8), s


def _weights(g, out, inner, experts, scales):
    parts = [_quantized_blocks(_normal(g, (out, inner), sigma=inner ** -0.5), scales)
             for _ in range(max(1, experts))]
    if not experts:
        return parts[0]
    return torch.stack([q for q, _ in parts]), torch.stack([s for _, s in parts])


def _offsets(g, rows, experts):
    """Where each expert's rows begin, popular experts (Zipf, s = 1.1) with
    more; and the largest count."""
    popular = -1.1 * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=F32))
    chosen = popular.softmax(0).multinomial(rows, replacement=True, generator=g)
    counts = (chosen[:, None] == torch.arange(experts, device="cuda")).sum(0)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, int(counts.max())


def _zeros(*shape, dtype):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _prepare_gated(case, g):
    rows, inner, width, experts = case["rows"], case["inner"], case["width"], case["experts"]
    s = {"case": case}
    q, s["x_scales"] = _quantized(_activations(g, rows, width), case["scales"])
    s["x"] = q.view(torch.uint8)
    s["w"], s["w_scales"] = _weights(g, 2 * inner, width, experts, case["scales"])
    if experts:
        s["group_offsets"], s["most"] = _offsets(g, rows - case["spare"], experts)
        # rows behind the last expert's stay as they are: zero
        if case["result"] == "bf16":
            s["to"] = {"out": _zeros(rows, inner, dtype=BF16)}
        else:
            s["to"] = {"q": _zeros(rows, inner, dtype=torch.uint8),
                       "scales": _zeros(rows, inner // 128, dtype=F32)}
            if case["keep"]:
                s["to"]["h"] = _zeros(rows, 2 * inner, dtype=torch.uint8)
                s["to"]["h_scales"] = _zeros(rows, inner // 64, dtype=F32)
    return s


def _prepare_grad(case, g):
    rows, inner = case["rows"], case["inner"]
    s = {"case": case, "da": _normal(g, (rows, inner), TYPES[case["da"]])}
    h = _normal(g, (rows, 2 * inner), sigma=2.0)
    if case["kept"] == "e4m3":
        q, s["h_scales"] = _quantized(h)
        s["h"] = q.view(torch.uint8)
    else:
        s["h"], s["h_scales"] = h.to(BF16), None
    return s


def _prepare_stored(case, g):
    q, scales = _quantized(_activations(g, case["rows"], case["width"]), case["scales"])
    return {"case": case, "q": q.view(torch.uint8), "scales": scales}


def _prepare_dgrad(case, g):
    rows, out, inner, experts = case["rows"], case["out"], case["inner"], case["experts"]
    s = {"case": case}
    q, s["dy_scales"] = _quantized(_normal(g, (rows, out)), case["scales"])
    s["dy"] = q.view(torch.uint8)
    s["w"], s["w_scales"] = _weights(g, out, inner, experts, case["scales"])
    s["group_offsets"], s["most"] = _offsets(g, rows - case["spare"], experts)
    s["dx"] = _zeros(rows, inner, dtype=BF16)
    return s


PREPARE = {"gated": _prepare_gated, "grad": _prepare_grad, "read": _prepare_stored,
           "turn": _prepare_stored, "dgrad": _prepare_dgrad}


def prepare(case, seed):
    return PREPARE[case["kind"]](case, _generator(seed))


# ---- plain forms ---------------------------------------------------------------

def _values(q, scales):
    """What 1x128 codes and scales stand for, fp32."""
    v = _groups(q.view(F8).float()) * scales[..., None]
    return v.reshape(*q.shape[:-1], -1)[..., :q.shape[-1]]


def _block_values(w, scales):
    *lead, n, k = w.shape
    v = w.view(F8).float().reshape(*lead, n // 128, 128, k // 128, 128)
    return (v * scales[..., :, None, :, None]).reshape(w.shape)


def _kept(v, scales):
    """v after a trip through 1x128 E4M3, as bf16."""
    return _values(*_quantized(v, scales)).to(BF16)


def _placed(s, x):
    """x's rows as columns of their expert's matrix, [experts][width][most];
    and (expert, place, whether it is an expert's) of each row."""
    at = torch.arange(x.shape[0], device=x.device)
    ends = s["group_offsets"][1:].contiguous()
    full = at < ends[-1]
    expert = torch.searchsorted(ends, at.int(), right=True).clamp_max(ends.shape[0] - 1)
    place = torch.where(full, at - s["group_offsets"][expert], s["most"])
    placed = torch.zeros((ends.shape[0], x.shape[1], s["most"] + 1), device=x.device)
    placed[expert, :, place] = x
    return placed, expert, place, full


def _by_expert(s, x, w):
    """Row r of x times w[expert of r]^T; zeros behind the last expert's."""
    placed, expert, place, full = _placed(s, x)
    y = torch.bmm(w, placed)
    return torch.where(full[:, None], y[expert, :, place], 0.0)


def _act(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _act_slope(v, act):
    if act == "silu":
        e = 1 / (1 + torch.exp(-v))
        return e * (1 + v * (1 - e))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v * v * v))
    return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)


def _plain_gated(s):
    case = s["case"]
    x, w = _values(s["x"], s["x_scales"]), _block_values(s["w"], s["w_scales"])
    h = _by_expert(s, x, w) if case["experts"] else x @ w.t()
    a = _act(h[:, :case["inner"]], case["act"]) * h[:, case["inner"]:]
    if case["result"] == "bf16":
        return {"a": a.to(BF16)}
    r = {"a": _kept(a, case["scales"])}
    if case["keep"]:
        r["h"] = _kept(h, case["scales"])
    return r


def _plain_grad(s):
    case = s["case"]
    h = s["h"].float() if s["h_scales"] is None else _values(s["h"], s["h_scales"])
    g, u = h[:, :case["inner"]], h[:, case["inner"]:]
    da, a = s["da"].float(), _act(g, case["act"])
    dh = torch.cat((da * u * _act_slope(g, case["act"]), da * a), dim=1)
    if case["result"] == "dense":
        return {"dh": dh.to(BF16)}
    r = dict(zip(("q", "scales"), _quantized(dh)))
    if case["result"] == "all":
        r["q_t"], r["scales_t"] = _quantized(dh.t())
        r["a_t"], r["a_scales_t"] = _quantized((a * u).t())
    return r


def _plain_read(s):
    return {"x": _values(s["q"], s["scales"]).to(TYPES[s["case"]["result"]])}


def _plain_turn(s):
    return dict(zip(("q_t", "scales_t"), _quantized(_values(s["q"], s["scales"]).t())))


def _plain_dgrad(s):
    dy, w = _values(s["dy"], s["dy_scales"]), _block_values(s["w"], s["w_scales"])
    return {"dx": _by_expert(s, dy, w.transpose(1, 2).contiguous()).to(BF16)}


PLAIN = {"gated": _plain_gated, "grad": _plain_grad, "read": _plain_read, "turn": _plain_turn,
         "dgrad": _plain_dgrad}


# ---- the package's operators -----------------------------------------------------

def _own_gated(s):
    import fp8_fine_grained_token_amd as F
    case = s["case"]
    args = [s["x"], s["x_scales"], s["w"], s["w_scales"]]
    pow2, grouped, to = case["scales"] == "pow2", case["experts"] > 0, s.get("to", {})
    if grouped:
        args.append(s["group_offsets"])
    if case["result"] == "bf16":
        if grouped:
            call = F.fp8_block_grouped_gemm_gated_pow2 if pow2 else F.fp8_block_grouped_gemm_gated
        else:
            call = F.fp8_block_gemm_gated_pow2 if pow2 else F.fp8_block_gemm_gated
        return {"a": call(*args, activation=case["act"], **to)}
    if grouped:
        call = (F.fp8_block_grouped_gemm_gated_quant_1x128_pow2 if pow2
                else F.fp8_block_grouped_gemm_gated_quant_1x128)
    else:
        call = (F.fp8_block_gemm_gated_quant_1x128_pow2 if pow2
                else F.fp8_block_gemm_gated_quant_1x128)
    q, scales, h, h_scales = call(*args, activation=case["act"], checkpoint=case["keep"], **to)
    r = {"a": F.fp8_dequant_act_1x128(q, scales)}
    if case["keep"]:
        r["h"] = F.fp8_dequant_act_1x128(h, h_scales)
    return r


def _own_grad(s):
    import fp8_fine_grained_token_amd as F
    case = s["case"]
    args = (s["da"], s["h"], s["h_scales"], case["act"])
    if case["result"] == "dense":
        return {"dh": F.fp8_gated_grad(*args)}
    if case["result"] == "rows":
        q, scales = F.fp8_gated_grad_quant_1x128(*args)
        return {"q": q.view(F8), "scales": scales}
    q, scales, q_t, scales_t, a_t, a_scales_t = F.fp8_gated_grad_quant(*args)
    return {"q": q.view(F8), "scales": scales, "q_t": q_t.view(F8), "scales_t": scales_t,
            "a_t": a_t.view(F8), "a_scales_t": a_scales_t}


def _own_read(s):
    import fp8_fine_grained_token_amd as F
    return {"x": F.fp8_dequant_act_1x128(s["q"], s["scales"], out_dtype=s["case"]["result"])}


def _own_turn(s):
    import fp8_fine_grained_token_amd as F
    q_t, scales_t = F.fp8_requant_act_128x1_t(s["q"], s["scales"])
    return {"q_t": q_t.view(F8), "scales_t": scales_t}


def _own_dgrad(s):
    import fp8_fine_grained_token_amd as F
    call = (F.fp8_block_grouped_gemm_dgrad_pow2 if s["case"]["scales"] == "pow2"
            else F.fp8_block_grouped_gemm_dgrad)
    return {"dx": call(s["dy"], s["dy_scales"], s["w"], s["w_scales"], s["group_offsets"],
                       dx=s["dx"])}


OWN = {"gated": _own_gated, "grad": _own_grad, "read": _own_read, "turn": _own_turn,
       "dgrad": _own_dgrad}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["kind"]](state)


# ---- work ----------------------------------------------------------------------

def _used(rows, experts):
    """Experts that at least one row goes to, on average."""
    if not experts:
        return 1
    p = [(e + 1) ** -1.1 for e in range(experts)]
    return sum(1 - (1 - v / sum(p)) ** rows for v in p)


def work(case):
    rows = case["rows"] - case.get("spare", 0)
    e4m3 = 1 + 4 / 128
    if case["kind"] == "gated":
        inner, width = case["inner"], case["width"]
        out = 2 if case["result"] == "bf16" else e4m3 * (3 if case["keep"] else 1)
        return {"bytes": rows * width * e4m3 + rows * inner * out
                + _used(rows, case["experts"]) * 2 * inner * width,
                "flops": 4 * rows * inner * width}
    if case["kind"] == "dgrad":
        out, inner = case["out"], case["inner"]
        return {"bytes": rows * out * e4m3 + rows * inner * 2
                + _used(rows, case["experts"]) * out * inner,
                "flops": 2 * rows * out * inner}
    if case["kind"] == "grad":
        values = rows * case["inner"]
        put = {"dense": 4, "rows": 2 * e4m3, "all": 5 * e4m3}[case["result"]]
        get = (2 if case["da"] == "bf16" else 4) + (2 * e4m3 if case["kept"] == "e4m3" else 4)
        return {"bytes": values * (get + put), "flops": 20 * values}
    values = rows * case["width"]
    put = e4m3 if case["kind"] == "turn" else 2 if case["result"] == "bf16" else 4
    return {"bytes": values * (e4m3 + put), "flops": 2 * values}


# ---- the definitions in 64 bits ----------------------------------------------------

def _exact_rounded(v):
    """v to the nearest E4M3 value, ties to even."""
    v = v.clamp(-448, 448)
    e = torch.frexp(v.abs().clamp_min(2.0 ** -6))[1] - 1
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return torch.round(v / step) * step


def _exact_scales(v, scales):
    """Scales of v's groups of 128 along its last axis."""
    parts = torch.split(v, 128, dim=-1)
    s = torch.stack([p.abs().amax(-1) for p in parts], dim=-1) / 448
    if scales == "pow2":
        s = torch.exp2(torch.ceil(torch.log2(s.clamp_min(2.0 ** -126))))
    return s


def _exact_kept(v, scales):
    s = _exact_scales(v, scales).repeat_interleave(128, dim=-1)[..., :v.shape[-1]]
    return _exact_rounded(torch.where(s > 0, v / s, 0.0)) * s


def _exact_input(q, scales):
    return q.view(F8).to(F64) * scales.to(F64).repeat_interleave(128, dim=-1)[..., :q.shape[-1]]


def _exact_weights(q, scales):
    s = scales.to(F64).repeat_interleave(128, dim=0).repeat_interleave(128, dim=1)
    return q.view(F8).to(F64) * s


def _exact_act(v, act):
    """(act(v), act'(v)) as v sigmoid(z) and its differential."""
    if act == "silu":
        z, dz = v, 1.0
    else:
        c = 2 * (2 / math.pi) ** 0.5
        z, dz = c * (v + 0.044715 * v.pow(3)), c * (1 + 0.134145 * v.pow(2))
    s = torch.sigmoid(z)
    return v * s, s + v * dz * s * torch.sigmoid(-z)


def _exact_product(s, x, turned):
    """Each row of x times its expert's weights (the only ones' if there are no
    experts), as they are or turned."""
    grouped = "group_offsets" in s
    ends = s["group_offsets"].tolist() if grouped else [0, x.shape[0]]
    wide = s["w"].shape[-1] if turned else s["w"].shape[-2]
    y = torch.zeros((x.shape[0], wide), dtype=F64, device="cuda")
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a < b:
            w = (_exact_weights(s["w"][e], s["w_scales"][e]) if grouped
                 else _exact_weights(s["w"], s["w_scales"]))
            y[a:b] = x[a:b] @ (w if turned else w.t())
    return y


def _exact_gated(s):
    case = s["case"]
    h = _exact_product(s, _exact_input(s["x"], s["x_scales"]), False)
    a = _exact_act(h[:, :case["inner"]], case["act"])[0] * h[:, case["inner"]:]
    if case["result"] == "bf16":
        return {"a": a}
    r = {"a": _exact_kept(a, case["scales"])}
    if case["keep"]:
        r["h"] = _exact_kept(h, case["scales"])
    return r


def _exact_grad(s):
    case = s["case"]
    h = s["h"].to(F64) if s["h_scales"] is None else _exact_input(s["h"], s["h_scales"])
    g, u = h.split(case["inner"], dim=1)
    a, slope = _exact_act(g, case["act"])
    da = s["da"].to(F64)
    dh = torch.cat((da * u * slope, da * a), dim=1)
    if case["result"] == "dense":
        return {"dh": dh}
    r = {"q": None, "scales": _exact_scales(dh, "f32")}
    if case["result"] == "all":
        r.update(q_t=None, scales_t=_exact_scales(dh.t(), "f32"), a_t=None,
                 a_scales_t=_exact_scales((a * u).t(), "f32"))
    return r


def _exact_read(s):
    return {"x": _exact_input(s["q"], s["scales"])}


def _exact_turn(s):
    return {"q_t": None, "scales_t": _exact_scales(_exact_input(s["q"], s["scales"]).t(), "f32")}


def _exact_dgrad(s):
    return {"dx": _exact_product(s, _exact_input(s["dy"], s["dy_scales"]), True)}


EXACT = {"gated": _exact_gated, "grad": _exact_grad, "read": _exact_read, "turn": _exact_turn,
         "dgrad": _exact_dgrad}


def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["kind"]](s)
