"""The operators of a training step of the n-gram memory, and the 8-bit product that also serves
its projection: which calls of them are measured, on what inputs, and their plain forms.

  embed      out[t][c * seg + d] = scale * table[ids[t][c]][d]; id -1 gives zeros
  embed_grad its gradient: grad[r] = scale * sum of dout over the places that looked row r up,
             dense (every row of the table is written) or sparse (one row for each distinct id)
  quantize   blocks of 1 x 128 to e4m3 with one scale each, along the rows and / or, transposed,
             along the columns
  linear     v = x W^T: x quantised in the call, W held in 8 bits with a scale for each 128 x 128
  linear_bwd its gradients: dx = dv W and dW = dv^T x, all operands in 8 bits with block scales
  gate_bwd   the backward pass of streams <- streams + sigmoid(<streams, v> / sqrt(hidden)) v

Scales are float32 (amax / 448), or powers of two held as e8m0 bytes where the case says so.
"""
import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
DEV = "cuda"
VOCAB = 129_280
TINY = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def up(n, m):
    return -(-n // m) * m


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step's lookup: 256 slots, 24 hash columns of 256 elements, a bf16 training table
        {"name": "embed_step", "op": "embed", "T": 256, "cols": 24, "dim": 256, "seg": 256, "rows": 1_048_576,
         "ids": "zipf", "pad": 0.0, "scale": 1.0, "table": "bf16", "out": "bf16"},
        # a training batch of 8 x 8,192 tokens on a site of the released shape (24 x 256), scaled
        {"name": "embed_batch", "op": "embed", "T": 65_536, "cols": 24, "dim": 256, "seg": 256, "rows": 4_194_304,
         "ids": "zipf", "pad": 0.02, "scale": 16.0, "table": "bf16", "out": "bf16"},
        # the smallest training call: 512 tokens, 6 columns of 128, three small tables back to back
        {"name": "grad_small", "op": "embed_grad", "T": 512, "cols": 6, "dim": 128, "seg": 128, "rows": 12_288,
         "ids": "uniform", "pad": 0.0, "scale": 1.0, "dout": "bf16", "grad": "f32", "mode": "dense"},
        # the memory's gradient for 4 x 4,096 tokens: 384M rows, so one row per distinct id
        {"name": "grad_memory", "op": "embed_grad", "T": 16_384, "cols": 24, "dim": 256, "seg": 256,
         "rows": 384_006_168, "ids": "zipf", "pad": 0.02, "scale": 1.0, "dout": "bf16", "grad": "f32", "mode": "sparse"},
        # the token embedding's gradient: whole vocabulary, Zipf tokens (one row takes a tenth of them)
        {"name": "grad_tokens", "op": "embed_grad", "T": 16_384, "cols": 1, "dim": 4096, "seg": 4096, "rows": VOCAB,
         "ids": "zipf", "pad": 0.0, "scale": 64.0, "dout": "bf16", "grad": "f32", "mode": "dense"},
        # the activations of one decode step, quantised ahead of the projection
        {"name": "quantize_step", "op": "quantize", "M": 256, "K": 6144, "x": "bf16", "rows": True, "cols": False,
         "scales": "f32"},
        # the projection's incoming gradient, quantised for both backward products; an odd token count
        {"name": "quantize_both", "op": "quantize", "M": 16_381, "K": 4096, "x": "f32", "rows": True, "cols": True,
         "scales": "f32"},
        # the projection of a few decoded tokens: the weight's bytes are the work
        {"name": "linear_step", "op": "linear", "T": 16, "K": 6144, "N": 4096, "x": "bf16", "out": "f32",
         "scales": "f32"},
        # the projection of a full batch at the released widths
        {"name": "linear_batch", "op": "linear", "T": 65_536, "K": 6144, "N": 4096, "x": "bf16", "out": "f32",
         "scales": "f32"},
        # the projection's backward pass; a ragged batch, so the weight's gradient sums over an odd length
        {"name": "linear_back", "op": "linear_bwd", "T": 16_381, "K": 6144, "N": 4096, "scales": "e8m0"},
        # the gate's backward pass for one small batch and for 4 x 4,096 tokens with image spans
        {"name": "gate_small", "op": "gate_bwd", "T": 256, "hidden": 4096, "dead": 0.0},
        {"name": "gate_batch", "op": "gate_bwd", "T": 16_384, "hidden": 4096, "dead": 0.06},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "quantize", "linear", "linear", "linear_bwd", "gate_bwd"])
    if op in ("embed", "embed_grad"):
        cols = rng.choice([1, 3, 6, 24])
        dim = rng.choice([64, 128, 256, 512, 1024, _log(rng, 1, 1500)]) if cols > 1 else _log(rng, 32, 4096)
        seg = up(dim, 64)
        most = 24 * 256 * (65_536 if op == "embed" else 16_384)
        T = _log(rng, 1, min(65_536, most // (cols * seg)))
        case = {"op": op, "T": T, "cols": cols, "dim": dim, "seg": seg, "ids": rng.choice(["zipf", "uniform"]),
                "pad": rng.choice([0.0, 0.05, 0.5]), "scale": rng.choice([1.0, 0.5, 22.627416])}
        if op == "embed":
            return {**case, "rows": _log(rng, 1, min(4_194_304, 2 ** 30 // dim)), "table": rng.choice(["bf16", "f32"]),
                    "out": rng.choice(["bf16", "f32"])}
        mode = rng.choice(["dense", "sparse"])
        most = 384_006_168 if mode == "sparse" else min(1_000_000, 129_280 * 4096 // dim)
        return {**case, "rows": _log(rng, 1, most), "dout": rng.choice(["bf16", "f32"]),
                "grad": rng.choice(["bf16", "f32"]), "mode": mode}
    scales = rng.choice(["f32", "e8m0"])
    if op == "quantize":
        K = rng.choice([768, 4096, 6144, _log(rng, 8, 19_584)])
        way = rng.choice(["rows", "cols", "both"])
        return {"op": op, "M": _log(rng, 1, min(65_536, 16_381 * 4096 // K)), "K": K, "x": rng.choice(["bf16", "f32"]),
                "rows": way != "cols", "cols": way != "rows", "scales": scales}
    if op in ("linear", "linear_bwd"):
        K = rng.choice([768, 1536, 6144, 19_584, 8 * _log(rng, 16, 1024)])
        N = rng.choice([256, 1024, 4096, 8 * _log(rng, 8, 640)])
        most = (65_536 * 6144 * 4096 if op == "linear" else 16_381 * 6144 * 4096) // (K * N)
        case = {"op": op, "T": _log(rng, 1, min(65_536 if op == "linear" else 16_384, most)), "K": K, "N": N,
                "scales": scales}
        return {**case, "x": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"])} if op == "linear" else case
    return {"op": op, "T": _log(rng, 1, 16_384), "hidden": rng.choice([256, 1024, 4096, 8 * _log(rng, 8, 512)]),
            "dead": rng.choice([0.0, 0.06, 0.5])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ids(case, g):
    """int32 [T][cols] row ids: uniform, or Zipf(1.1) ranks spread over the rows by a multiplier;
    a share `pad` of them -1."""
    n, rows = case["T"] * case["cols"], case["rows"]
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    if case["ids"] == "zipf":
        rank = (1.0 - u * (1.0 - float(rows) ** -0.1)) ** -10.0
        ids = ((rank.floor().long().clamp_(1, rows) - 1) * 2_654_435_761) % rows
    else:
        ids = (u * rows).long().clamp_(0, rows - 1)
    pad = torch.rand(n, generator=g, device=DEV) < case["pad"]
    return torch.where(pad, -1, ids).int().view(case["T"], case["cols"])


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)


def _codes(rows, k):
    """The buffer a quantised operand lives in: whole blocks of 128 along the row."""
    return torch.empty((rows, up(k, 128)), dtype=F8, device=DEV)


def _scales(case, kb, n):
    return torch.empty((kb, n), dtype=torch.uint8 if case["scales"] == "e8m0" else torch.float32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "embed":
        s["ids"] = _ids(case, g)
        s["table"] = torch.empty((case["rows"], case["dim"]), dtype=TYPES[case["table"]], device=DEV).normal_(generator=g)
        s["out"] = torch.empty((case["T"], case["cols"] * case["seg"]), dtype=TYPES[case["out"]], device=DEV)
    elif op == "embed_grad":
        n = case["T"] * case["cols"]
        s["ids"] = _ids(case, g)
        s["dout"] = _randn(g, case["T"], case["cols"] * case["seg"], dtype=TYPES[case["dout"]], std=1e-2)
        lines = case["rows"] if case["mode"] == "dense" else n
        s["grad"] = torch.zeros((lines, case["dim"]), dtype=TYPES[case["grad"]], device=DEV)
        if case["mode"] == "sparse":
            s["unique"] = torch.empty(n, dtype=torch.int32, device=DEV)
            s["count"] = torch.empty(1, dtype=torch.int32, device=DEV)
    elif op == "quantize":
        M, K = case["M"], case["K"]
        # rows of very different size, as gradients and activations have
        s["x"] = _randn(g, M, K).mul_(torch.exp(_randn(g, M, 1, std=2.0))).to(TYPES[case["x"]])
        if case["rows"]:
            s["q"], s["s"] = _codes(M, K), _scales(case, up(K, 128) // 128, M)
        if case["cols"]:
            s["qt"], s["st"] = _codes(K, M), _scales(case, up(M, 128) // 128, K)
    elif op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        s["x"] = _randn(g, T, K, dtype=TYPES[case["x"]])
        s["wq"], s["ws"] = _weight(case, _randn(g, N, K, std=0.02))
        s["xq"], s["xs"] = _codes(T, K), _scales(case, up(K, 128) // 128, T)
        s["out"] = torch.empty((T, N), dtype=TYPES[case["out"]], device=DEV)
    elif op == "linear_bwd":
        T, K, N = case["T"], case["K"], case["N"]
        s["x"] = _randn(g, T, K, dtype=torch.bfloat16)
        s["dv"] = _randn(g, T, N, std=1e-3)
        # the weight as dx = dv W reads it: W^T, [K][N]
        s["wt"], s["wts"] = _weight(case, _randn(g, K, N, std=0.02))
        s["dvq"], s["dvs"] = _codes(T, N), _scales(case, up(N, 128) // 128, T)
        s["dvt"], s["dvts"] = _codes(N, T), _scales(case, up(T, 128) // 128, N)
        s["xt"], s["xts"] = _codes(K, T), _scales(case, up(T, 128) // 128, K)
        s["dx"] = torch.empty((T, K), dtype=torch.bfloat16, device=DEV)
        s["dw"] = torch.empty((N, K), dtype=torch.float32, device=DEV)
    else:
        T, h = case["T"], case["hidden"]
        s["v"] = _randn(g, T, h)
        s["x"] = _randn(g, T, 4, h, dtype=torch.bfloat16)
        s["dy"] = _randn(g, T, 4, h, dtype=torch.bfloat16, std=1e-2)
        s["keep"] = (torch.rand(T, generator=g, device=DEV) >= case["dead"]).to(torch.uint8)
        s["dx"] = torch.empty_like(s["dy"])
        s["dv"] = torch.empty_like(s["v"])
    return s


def _weight(case, w):
    """A weight as a checkpoint holds it: e4m3 codes [N][K up to 128s], one scale per 128 x 128,
    laid out [K / 128][N / 128]."""
    N, K = w.shape
    nb, kb = up(N, 128) // 128, up(K, 128) // 128
    blocks = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, nb * 128 - N)).view(nb, 128, kb, 128)
    scale = _scale_of(case, blocks.abs().amax(dim=(1, 3)))
    codes = (blocks / scale[:, None, :, None]).to(F8).view(nb * 128, kb * 128)[:N].contiguous()
    return codes, _held(case, scale).t().contiguous()


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _scale_of(case, amax):
    """The scale of blocks whose largest magnitude is amax, float32."""
    s = (amax / torch.full_like(amax, 448.0)).clamp_min(TINY)  # a quotient of tensors is rounded once
    if case["scales"] == "e8m0":
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return s


def _held(case, s):
    """A scale as it is held: the float32 itself, or its e8m0 byte (the exponent's bits)."""
    return (s.contiguous().view(torch.int32) >> 23).to(torch.uint8) if case["scales"] == "e8m0" else s


def _stands_for(s):
    """The float32 that a held scale stands for."""
    return (s.to(torch.int32) << 23).view(torch.float32) if s.dtype == torch.uint8 else s


def _quantize(case, x):
    """Codes [M][K up to 128s] and float32 scales [K / 128][M] of x [M][K]."""
    M, K = x.shape
    kb = up(K, 128) // 128
    b = torch.nn.functional.pad(x.float(), (0, kb * 128 - K)).view(M, kb, 128)
    s = _scale_of(case, b.abs().amax(dim=2))
    return (b / s[:, :, None]).to(F8).view(M, kb * 128), s.t().contiguous()


def _dequantize(q, s, block):
    """float32 [M][K] of codes and scales [K / 128][M] (block 1) or [K / 128][M / 128] (block 128)."""
    M, kb = q.shape[0], q.shape[1] // 128
    rows = _stands_for(s).t().repeat_interleave(block, dim=0)[:M]
    return (q.float().view(M, kb, 128) * rows[:, :, None]).view(M, kb * 128)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "embed":
        T, cols, dim, seg = case["T"], case["cols"], case["dim"], case["seg"]
        ids = s["ids"].long()
        rows = s["table"][ids.clamp_min(0)].float() * case["scale"]
        rows = torch.where(ids[..., None] < 0, 0.0, rows)
        return torch.nn.functional.pad(rows, (0, seg - dim)).to(TYPES[case["out"]]).view(T, cols * seg)
    if op == "embed_grad":
        T, cols, dim, seg, rows = case["T"], case["cols"], case["dim"], case["seg"], case["rows"]
        ids = s["ids"].long().view(-1)
        g = s["dout"].view(T * cols, seg)[:, :dim].float()
        g = torch.where(ids[:, None] < 0, 0.0, g)
        if case["mode"] == "dense":
            grad = torch.zeros((rows, dim), device=DEV).index_add_(0, ids.clamp_min(0), g)
            return (grad * case["scale"]).to(TYPES[case["grad"]])
        key, order = torch.sort(torch.where(ids < 0, rows, ids))
        first = torch.ones_like(key)
        first[1:] = key[1:] != key[:-1]
        line = torch.cumsum(first, 0) - 1
        grad = torch.zeros((T * cols, dim), device=DEV).index_add_(0, line, g[order])
        unique = torch.full_like(key, -1).scatter_(0, line, torch.where(key == rows, -1, key))
        count = (first * (key < rows)).sum().view(1)
        return [(grad * case["scale"]).to(TYPES[case["grad"]]), unique.int(), count.int()]
    if op == "quantize":
        out = []
        if case["rows"]:
            out += _quantize(case, s["x"])
        if case["cols"]:
            out += _quantize(case, s["x"].t())
        return out
    if op == "linear":
        x = _dequantize(*_quantize(case, s["x"]), 1)
        return (x @ _dequantize(s["wq"], s["ws"], 128).t()).to(TYPES[case["out"]])
    if op == "linear_bwd":
        T, K, N = case["T"], case["K"], case["N"]
        dv = _dequantize(*_quantize(case, s["dv"]), 1)
        dx = dv @ _dequantize(s["wt"], s["wts"], 128).t()
        dvt = _dequantize(*_quantize(case, s["dv"].t()), 1)
        xt = _dequantize(*_quantize(case, s["x"].t()), 1)
        return [dx.to(torch.bfloat16), dvt @ xt.t()]
    v, x, dy = s["v"][:, None, :], s["x"].float(), s["dy"].float()
    root = 1.0 / math.sqrt(case["hidden"])
    keep = s["keep"].float()[:, None]
    gate = torch.sigmoid((x * v).sum(-1) * root)
    e = keep * (dy * v).sum(-1) * gate * (1.0 - gate) * root
    dx = dy + e[..., None] * v
    dv = ((keep * gate)[..., None] * dy + e[..., None] * x).sum(1)
    return [dx.to(torch.bfloat16), dv]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own(s):
    import hashed_gram_memory_tid2eid_amd as eng
    case = s["case"]
    op = case["op"]
    if op == "embed":
        eng.engram_embed(s["table"], s["ids"], s["out"], scale=case["scale"], seg_pitch=case["seg"])
        return s["out"]
    if op == "embed_grad":
        if "work" not in s:
            s["work"] = torch.empty(eng.engram_embed_grad_workspace(case["T"] * case["cols"], case["rows"], case["dim"]),
                                    dtype=torch.uint8, device=DEV)
        eng.engram_embed_grad(s["ids"], s["dout"], s["grad"], rows=case["rows"], scale=case["scale"], mode=case["mode"],
                              seg_pitch=case["seg"], unique=s.get("unique"), count=s.get("count"), workspace=s["work"])
        return s["grad"] if case["mode"] == "dense" else [s["grad"], s["unique"], s["count"]]
    if op == "quantize":
        eng.engram_fp8_quantize(s["x"], s.get("q"), s.get("s"), q_t=s.get("qt"), scales_t=s.get("st"))
        return [s[k] if k[0] == "q" else _stands_for(s[k]) for k in ("q", "s", "qt", "st") if k in s]
    if op == "linear":
        if "work" not in s:
            s["work"] = _space(eng, (case["T"], case["N"], case["K"]))
        eng.engram_fp8_quantize(s["x"], s["xq"], s["xs"])
        eng.engram_fp8_matmul(s["xq"], s["xs"], s["wq"], s["ws"], s["out"], workspace=s["work"])
        return s["out"]
    if op == "linear_bwd":
        if "work" not in s:
            T, K, N = case["T"], case["K"], case["N"]
            s["work"] = _space(eng, (T, K, N), (N, K, T))
        eng.engram_fp8_quantize(s["dv"], s["dvq"], s["dvs"], q_t=s["dvt"], scales_t=s["dvts"])
        eng.engram_fp8_quantize(s["x"], None, None, q_t=s["xt"], scales_t=s["xts"])
        eng.engram_fp8_matmul(s["dvq"], s["dvs"], s["wt"], s["wts"], s["dx"], workspace=s["work"])
        eng.engram_fp8_matmul(s["dvt"], s["dvts"], s["xt"], s["xts"], s["dw"], workspace=s["work"])
        return [s["dx"], s["dw"]]
    eng.engram_gate_add_backward(s["v"], s["x"], s["dy"], s["dx"], s["dv"], keep=s["keep"])
    return [s["dx"], s["dv"]]


def _space(eng, *shapes):
    """The workspace that products of these (M, N, K) share."""
    return torch.empty(max(eng.engram_fp8_matmul_workspace(*shape) for shape in shapes), dtype=torch.uint8, device=DEV)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the work of one pass
# ---------------------------------------------------------------------------

def _distinct(case):
    """Distinct rows among the ids that a case draws, as expected from their distribution."""
    n, rows = case["T"] * case["cols"] * (1.0 - case["pad"]), case["rows"]
    if case["ids"] == "uniform" or rows == 1:
        return rows * -math.expm1(n * math.log1p(-1.0 / rows)) if rows > 1 else min(1.0, n)
    edge = np.unique(np.floor(np.geomspace(1.0, rows + 1.0, 4000)))  # ranks in groups: P(rank <= k) as they are drawn
    below = (1.0 - edge ** -0.1) / (1.0 - float(rows) ** -0.1)
    many = np.diff(edge)
    p = np.clip(np.diff(np.minimum(below, 1.0)) / many, 0.0, 1.0 - 1e-12)
    return float((many * -np.expm1(n * np.log1p(-p))).sum())


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    scale = 1 if case.get("scales") == "e8m0" else 4
    if op == "embed":
        n = case["T"] * case["cols"]
        return {"bytes": 4 * n + _distinct(case) * case["dim"] * size[case["table"]] + n * case["seg"] * size[case["out"]],
                "flops": n * case["dim"]}
    if op == "embed_grad":
        n = case["T"] * case["cols"]
        lines = case["rows"] if case["mode"] == "dense" else _distinct(case)
        held = 0 if case["mode"] == "dense" else 4 * n + 4
        return {"bytes": 4 * n + n * (1.0 - case["pad"]) * case["dim"] * size[case["dout"]]
                + lines * case["dim"] * size[case["grad"]] + held, "flops": n * case["dim"]}
    if op == "quantize":
        M, K = case["M"], case["K"]
        total = M * K * size[case["x"]]
        if case["rows"]:
            total += up(K, 128) * M + up(K, 128) // 128 * M * scale
        if case["cols"]:
            total += up(M, 128) * K + up(M, 128) // 128 * K * scale
        return {"bytes": total, "flops": 3 * M * K * (case["rows"] + case["cols"])}
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": T * K * size[case["x"]] + N * up(K, 128) + up(N, 128) // 128 * (up(K, 128) // 128) * scale
                + T * N * size[case["out"]], "flops": 2 * T * N * K}
    if op == "linear_bwd":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": T * K * 2 + T * N * 4 + K * up(N, 128) + up(N, 128) // 128 * (up(K, 128) // 128) * scale
                + T * K * 2 + N * K * 4, "flops": 4 * T * N * K}
    T, h = case["T"], case["hidden"]
    return {"bytes": T * (h * 4 + 8 * h * 3 + h * 4 + 1), "flops": T * h * 4 * 8}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_codes(case, x):
    """(codes as float64 [M][K / 128][128], scales as float64 [M][K / 128]) of x [M][K], whose scale is a
    float32 and whose quotient is rounded to float32 before the code is."""
    M, K = x.shape
    wide = torch.zeros((M, up(K, 128)), dtype=torch.float64, device=DEV)
    wide[:, :K] = x
    wide = wide.view(M, -1, 128)
    s = (wide.abs().max(dim=2).values / 448.0).float().double().clamp(min=TINY)
    if case["scales"] == "e8m0":
        s = torch.exp2(torch.ceil(torch.log2(s)))
    q = (wide / s.unsqueeze(2)).float().double()
    # e4m3: 3 bits behind the leading one down to 2^-6, steps of 2^-9 below
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(q / step) * step, s


def _exact_values(case, x):
    q, s = _exact_codes(case, x)
    return (q * s.unsqueeze(2)).flatten(1)


def _exact_weight(codes, scales):
    """float64 values of a weight: codes [N][K], scales [K / 128][N / 128]."""
    s = scales.double() if scales.dtype == torch.float32 else torch.exp2(scales.double() - 127.0)
    n, k = torch.arange(codes.shape[0], device=DEV) // 128, torch.arange(codes.shape[1], device=DEV) // 128
    return codes.double() * s.t()[n][:, k]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        ids = s["ids"].long()
        out = torch.zeros((case["T"], case["cols"], case["seg"]), dtype=torch.float64, device=DEV)
        out[..., :case["dim"]] = s["table"][ids.clamp(min=0)].double() * case["scale"]
        out[ids < 0] = 0.0
        return out.flatten(1)
    if op == "embed_grad":
        n, dim = case["T"] * case["cols"], case["dim"]
        ids = s["ids"].long().flatten()
        live = ids >= 0
        g = s["dout"].view(n, case["seg"])[live][:, :dim].double() * case["scale"]
        if case["mode"] == "dense":
            out = torch.zeros((case["rows"], dim), dtype=torch.float64, device=DEV)
            out.index_add_(0, ids[live], g)
            return out
        names, line = torch.unique(ids[live], return_inverse=True)
        out = torch.zeros((n, dim), dtype=torch.float64, device=DEV)
        out.index_add_(0, line, g)
        unique = torch.full((n,), -1, dtype=torch.int32, device=DEV)
        unique[:names.numel()] = names.int()
        return [out, unique, torch.tensor([names.numel()], dtype=torch.int32, device=DEV)]
    if op == "quantize":
        out = []
        for x in ([s["x"]] if case["rows"] else []) + ([s["x"].t()] if case["cols"] else []):
            q, scale = _exact_codes(case, x)
            out += [q.flatten(1), scale.t().contiguous()]
        return out
    if op == "linear":
        return _exact_values(case, s["x"]) @ _exact_weight(s["wq"], s["ws"]).t()
    if op == "linear_bwd":
        dx = _exact_values(case, s["dv"]) @ _exact_weight(s["wt"], s["wts"]).t()
        return [dx, _exact_values(case, s["dv"].t()) @ _exact_values(case, s["x"].t()).t()]
    v, x, dy = s["v"].double().unsqueeze(1), s["x"].double(), s["dy"].double()
    keep = s["keep"].double().view(-1, 1, 1)
    root = math.sqrt(case["hidden"])
    gate = 1.0 / (1.0 + torch.exp(-(x * v).sum(2, keepdim=True) / root))
    e = (dy * v).sum(2, keepdim=True) * gate * (1.0 - gate) / root * keep
    return [dy + e * v, (keep * gate * dy + e * x).sum(1)]
