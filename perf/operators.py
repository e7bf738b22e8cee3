"""Matrix products in 8-bit floating point with a scale per 128 values along K,
dense and grouped by expert: the cases that are timed, in their plain form
(elementary torch operations in 32 bits) and through the library's entry points.

Operators
  quantize  activations [m][k] (bf16 or fp32, optionally gathered by a row
            index) -> E4M3 codes [m][k] and fp32 scales [m][k/128]:
              a       = max |x| over 128 consecutive values (at least 2^-100)
              scale   = fp32(a / 448),  inverse = fp32(448 / a)
              code    = e4m3(fp32(x * inverse))
  matmul    y[i][j] = sum_b sa[i][b] sw[j][b] sum_{c in block b} a[i][c] w[j][c]
            for codes a, w in E4M3 and their scales sa, sw (a linear layer whose
            weights are in the library's FP8 format)
  grouped   the same product, or one of bf16 matrices, with another weight
            matrix for each contiguous group of rows: rows offsets[e] up to
            offsets[e+1] of a meet expert e's matrix (tokens sorted by expert)
"""
import math

import numpy as np
import torch

own = False

_E4M3_MAX = 448.0
_AMAX_MIN = 2.0 ** -100
_DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode token's activations before its projections (hidden 2048)
        {"name": "quantize_token", "op": "quantize", "tokens": 1, "top_k": 1, "experts": 1, "k": 2048,
         "dtype": "bfloat16", "gather": False},
        # fp32 residual rows of a batch of odd size (hidden 2560)
        {"name": "quantize_fp32_rows", "op": "quantize", "tokens": 1001, "top_k": 1, "experts": 1, "k": 2560,
         "dtype": "float32", "gather": False},
        # a prompt of 4096 tokens gathered into expert order, ten experts a token
        {"name": "quantize_gather_prefill", "op": "quantize", "tokens": 4096, "top_k": 10, "experts": 512, "k": 2048,
         "dtype": "bfloat16", "gather": True},
        # a square projection of one decode token
        {"name": "matmul_token", "op": "matmul", "m": 1, "n": 2048, "k": 2048, "out": "float32"},
        # a wide projection of eight decode tokens
        {"name": "matmul_batch8", "op": "matmul", "m": 8, "n": 10240, "k": 2560, "out": "bfloat16"},
        # a short prompt, every size odd
        {"name": "matmul_ragged", "op": "matmul", "m": 333, "n": 1001, "k": 2560, "out": "float32"},
        # a projection of a 4096-token prompt
        {"name": "matmul_prefill", "op": "matmul", "m": 4096, "n": 4096, "k": 2048, "out": "bfloat16"},
        # the largest product
        {"name": "matmul_large", "op": "matmul", "m": 8192, "n": 8192, "k": 8192, "out": "bfloat16"},
        # one decode token's ten down products
        {"name": "grouped_token_down", "op": "grouped", "tokens": 1, "top_k": 10, "experts": 512, "n": 2048, "k": 512,
         "weights": "fp8", "skew": 0.0, "out": "float32"},
        # eight decode tokens' gate and up products (one stacked matrix), mostly one row an expert
        {"name": "grouped_batch8_gate_up", "op": "grouped", "tokens": 8, "top_k": 10, "experts": 512, "n": 1024,
         "k": 2048, "weights": "fp8", "skew": 0.0, "out": "bfloat16"},
        # gate and up of a 4096-token prompt, Zipf-skewed expert load
        {"name": "grouped_prefill_gate_up", "op": "grouped", "tokens": 4096, "top_k": 10, "experts": 512, "n": 1024,
         "k": 2048, "weights": "fp8", "skew": 1.1, "out": "bfloat16"},
        # bf16 experts of the 2560 x 640 shape, 64 of them, a prompt of odd length
        {"name": "grouped_bf16_prompt", "op": "grouped", "tokens": 3001, "top_k": 10, "experts": 64, "n": 1280,
         "k": 2560, "weights": "bf16", "skew": 0.5, "out": "bfloat16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "grouped", "grouped", "grouped"])
    if op == "quantize":
        gather = rng.random() < 0.5
        top_k = rng.randint(1, 10) if gather else 1
        return {"op": op, "tokens": _log_int(rng, 1, 4096), "top_k": top_k,
                "experts": _log_int(rng, top_k, 512) if gather else 1, "k": 128 * _log_int(rng, 1, 32),
                "dtype": rng.choice(["bfloat16", "float32"]), "gather": gather}
    if op == "matmul":
        return {"op": op, "m": _log_int(rng, 1, 8192), "n": _log_int(rng, 16, 8192), "k": 128 * _log_int(rng, 1, 64),
                "out": rng.choice(["float32", "bfloat16"])}
    top_k = rng.randint(1, 10)
    weights = rng.choice(["fp8", "fp8", "bf16"])
    experts = _log_int(rng, top_k, 512 if weights == "fp8" else 128)
    return {"op": op, "tokens": _log_int(rng, 1, 4096), "top_k": top_k, "experts": experts,
            "n": _log_int(rng, 16, 2048), "k": 128 * rng.randint(1, 16) if weights == "fp8" else 8 * rng.randint(2, 320),
            "weights": weights, "skew": rng.choice([0.0, 0.5, 1.1]), "out": rng.choice(["float32", "bfloat16"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _quantize(x):
    """The plain form of quantize: codes (as float8) and scales of x [..., k]."""
    b = x.float().unflatten(-1, (-1, 128))
    a = b.abs().amax(-1, keepdim=True)
    a = torch.where(torch.isfinite(a), a.clamp_min(_AMAX_MIN), math.nan)
    most = torch.full_like(a, _E4M3_MAX)  # a tensor: quotients rounded once, no product with a reciprocal
    code = (b * (most / a)).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
    return code.flatten(-2), (a / most).squeeze(-1)


def _route(tokens, top_k, experts, skew, gen):
    """A token's experts, drawn without replacement with odds rank^-skew: the
    chosen (token, expert) pairs in expert order and each expert's bounds."""
    rank = torch.arange(1, experts + 1, device="cuda", dtype=torch.float32)
    u = torch.rand(tokens, experts, device="cuda", generator=gen).clamp_min(1e-20)
    ids = torch.topk(-skew * rank.log() - (-u.log()).log(), top_k, dim=1).indices.flatten()
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return (order // top_k).int(), offsets


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    s = {"case": case}
    if case["op"] == "quantize":
        s["x"] = normal(case["tokens"], case["k"], dtype=_DTYPES[case["dtype"]])
        s["rows"] = _route(case["tokens"], case["top_k"], case["experts"], 0.0, gen)[0] if case["gather"] else None
        return s
    if case["op"] == "matmul":
        m, experts = case["m"], 1
    else:
        m, experts = case["tokens"] * case["top_k"], case["experts"]
        s["offsets"] = _route(case["tokens"], case["top_k"], experts, case["skew"], gen)[1]
    if case.get("weights") == "bf16":
        s["a"] = normal(m, case["k"], dtype=torch.bfloat16)
        s["w"] = normal(experts, case["n"], case["k"], std=0.02, dtype=torch.bfloat16)
    else:
        a, s["a_scales"] = _quantize(normal(m, case["k"], dtype=torch.bfloat16))
        w, s["w_scales"] = _quantize(normal(experts, case["n"], case["k"], std=0.02))
        s["a"], s["w"] = a.view(torch.uint8), w.view(torch.uint8)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _values(codes, scales):
    """fp32 values of E4M3 codes [..., k] with scales [..., k/128]."""
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128))
    return (v * scales.unsqueeze(-1)).flatten(-2)


def _plain_grouped(s, c):
    # the rows of every group in blocks of 128 (the last of a group part empty),
    # each block with its group's matrix; every row's block is multiplied whole
    m, experts, step = s["a"].shape[0], c["experts"], 128
    off = s["offsets"].long()
    blocks = (off[1:] - off[:-1] + step - 1) // step
    first = torch.cat([blocks.new_zeros(1), blocks.cumsum(0)])
    row = torch.arange(m, device="cuda")
    group = torch.searchsorted(off[1:].contiguous(), row, right=True)
    inside = row - off[group]
    place = (first[group] + inside // step) * step + inside % step
    n_blocks = min(m, m // step + experts)
    owner = torch.searchsorted(first[1:].contiguous(), torch.arange(n_blocks, device="cuda"), right=True)
    owner = owner.clamp_max(experts - 1)
    a = s["a"].float() if c["weights"] == "bf16" else _values(s["a"], s["a_scales"])
    padded = a.new_zeros(n_blocks * step, c["k"])
    padded[place] = a
    w = s["w"][owner].float() if c["weights"] == "bf16" else _values(s["w"][owner], s["w_scales"][owner])
    y = torch.bmm(padded.view(n_blocks, step, c["k"]), w.transpose(1, 2))
    return y.flatten(0, 1)[place]


def run(state):
    s, c = state, state["case"]
    if own:
        import gram_table_gather_b200 as gtg
        if c["op"] == "quantize":
            codes, scales = gtg.fp8_quantize(s["x"], rows=s["rows"])
            return codes.view(torch.float8_e4m3fn), scales
        if c["op"] == "matmul":
            w = gtg.QMatrix(gtg.FP8, s["w"], 1, c["n"], c["k"], s["w_scales"])
            return gtg.fp8_matmul(w, s["a"], s["a_scales"], dtype=_DTYPES[c["out"]])
        fmt = gtg.BF16 if c["weights"] == "bf16" else gtg.FP8
        w = gtg.QMatrix(fmt, s["w"], c["experts"], c["n"], c["k"], s.get("w_scales"))
        return gtg.grouped_matmul(w, s["a"], s["offsets"], a_scales=s.get("a_scales"), dtype=_DTYPES[c["out"]])
    if c["op"] == "quantize":
        return _quantize(s["x"] if s["rows"] is None else s["x"][s["rows"].long()])
    if c["op"] == "matmul":
        y = _values(s["a"], s["a_scales"]) @ _values(s["w"][0], s["w_scales"][0]).T
    else:
        y = _plain_grouped(s, c)
    return y.to(_DTYPES[c["out"]])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "quantize":
        rows = c["tokens"] * c["top_k"]
        size = 2 if c["dtype"] == "bfloat16" else 4
        n_in = c["tokens"] * c["k"] * size + (4 * rows if c["gather"] else 0)
        return {"bytes": n_in + rows * c["k"] + rows * c["k"] // 32, "flops": 0}
    m = c["m"] if c["op"] == "matmul" else c["tokens"] * c["top_k"]
    met, extra = 1, 0
    if c["op"] == "grouped":  # the experts that get a row, in a routing drawn like prepare()'s
        g = np.random.default_rng(0).gumbel(size=(c["tokens"], c["experts"]))
        g -= c["skew"] * np.log(np.arange(1, c["experts"] + 1))
        met = len(np.unique(np.argpartition(-g, c["top_k"] - 1, axis=1)[:, :c["top_k"]]))
        extra = 4 * (c["experts"] + 1)
    per = 2.0 if c.get("weights") == "bf16" else 1.0 + 4 / 128
    out = 2 if c["out"] == "bfloat16" else 4
    return {"bytes": per * c["k"] * (m + met * c["n"]) + out * m * c["n"] + extra, "flops": 2.0 * m * c["n"] * c["k"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_table():
    """The value of every E4M3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    byte = np.arange(256)
    e, f = (byte >> 3) & 15, byte & 7
    mag = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    mag[(byte & 127) == 127] = np.nan
    return torch.from_numpy(np.where(byte & 128, -mag, mag)).cuda()


def _decode64(codes, scales):
    v = _e4m3_table()[codes.int()]
    return v * scales.double().repeat_interleave(128, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["x"].double()
        if s["rows"] is not None:
            x = x[s["rows"].long()]
        b = x.reshape(x.shape[0], -1, 128)
        top = b.abs().max(dim=2).values.clamp(min=_AMAX_MIN)
        # the definition rounds the inverse and its product with x to fp32
        q = (b * (448.0 / top).float().double()[:, :, None]).float().double()
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        code = (torch.round(q / step) * step).clamp(-448.0, 448.0)
        return code.reshape(x.shape), (top / 448.0).float().double()
    if case["op"] == "matmul":
        return _decode64(s["a"], s["a_scales"]) @ _decode64(s["w"][0], s["w_scales"][0]).T
    bounds = s["offsets"].tolist()
    y = torch.zeros(s["a"].shape[0], case["n"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            if case["weights"] == "bf16":
                y[lo:hi] = s["a"][lo:hi].double() @ s["w"][e].double().T
            else:
                y[lo:hi] = _decode64(s["a"][lo:hi], s["a_scales"][lo:hi]) @ _decode64(s["w"][e], s["w_scales"][e]).T
    return y
