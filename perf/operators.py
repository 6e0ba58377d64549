"""The 8-bit operators around the routed FFN: what is measured, and their plain forms.

Four operators of a layer whose weights are E4M3 with one float32 scale per
128 x 128 block and whose activations are E4M3 with one float32 scale per row
and 128 values:

  norm     residual addition, root-mean-square norm, E4M3 output with scales
  gemm     out[T, N] = dequantised A [T, K] times dequantised W [N, K] transposed
  swiglu   rows grouped by expert: h = silu(A Wg^T) * (A Wu^T), E4M3 with scales
  grouped  rows grouped by expert: A We^T, written in the rows' original order

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is set, with the library's entry points.  ``exact`` computes them in 64
bits.  8-bit outputs are float8_e4m3fn tensors beside their scales.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
MIN_SCALE = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 128


# ------------------------------------------------------------------- cases ---
def listed():
    """Hidden size 4096 with 256 experts of 2048 (8 chosen) or 64 of 1408 (2
    chosen): the shapes of this repository's benchmark workloads."""
    return [
        # one decoded token's norm in front of the layer: pure latency
        {"name": "norm decode T1", "op": "norm", "T": 1, "H": 4096, "type": "bf16", "residual": True, "y": True},
        # a long prefill chunk's norm: memory traffic
        {"name": "norm prefill T4096", "op": "norm", "T": 4096, "H": 4096, "type": "bf16", "residual": True, "y": True},
        # half-precision rows of a width that ends inside a block of 128, codes only
        {"name": "norm ragged T777", "op": "norm", "T": 777, "H": 7088, "type": "f16", "residual": False, "y": False},
        # one token through a dense projection (shared expert, gate): weight streaming
        {"name": "gemm decode T1", "op": "gemm", "T": 1, "N": 2048, "K": 4096, "out": "bf16"},
        # a dense projection of a prefill chunk: tensor throughput
        {"name": "gemm prefill T4096", "op": "gemm", "T": 4096, "N": 8192, "K": 4096, "out": "bf16"},
        # odd row and column counts, K ending inside a block, float32 result
        {"name": "gemm odd T300", "op": "gemm", "T": 300, "N": 1000, "K": 1424, "out": "f32"},
        # one decoded token: eight experts' gate and up matrices are read
        {"name": "swiglu decode T1", "op": "swiglu", "T": 1, "H": 4096, "I": 2048, "E": 256, "k": 8},
        # a draft-verify batch of 1 + 4 tokens on the 64-expert shape
        {"name": "swiglu verify T5", "op": "swiglu", "T": 5, "H": 4096, "I": 1408, "E": 64, "k": 2},
        # a prefill chunk: every expert active, buckets of very different sizes
        {"name": "swiglu prefill T2048", "op": "swiglu", "T": 2048, "H": 4096, "I": 2048, "E": 256, "k": 8},
        # the down projection of a draft-verify batch, float32 rows for the combine
        {"name": "down verify T5", "op": "grouped", "T": 5, "N": 4096, "K": 2048, "E": 256, "k": 8, "out": "f32"},
        # the down projection of a prefill chunk
        {"name": "down prefill T2048", "op": "grouped", "T": 2048, "N": 4096, "K": 2048, "E": 256, "k": 8, "out": "bf16"},
        # a middle batch of odd sizes, some buckets empty
        {"name": "grouped odd T77", "op": "grouped", "T": 77, "N": 1000, "K": 1424, "E": 64, "k": 2, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log16(rng, lo, hi):
    return 16 * _log(rng, lo // 16, hi // 16)


def draw(rng):
    """One more case: token counts from one up, widths in steps of 16 (rows of
    codes are 16-byte multiples), output widths of any size."""
    op = rng.choice(("norm", "gemm", "swiglu", "grouped"))
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 4096), "H": _log16(rng, 256, 8192), "type": rng.choice(sorted(TYPES)),
                "residual": rng.random() < 0.5, "y": rng.random() < 0.5}
    if op == "gemm":
        return {"op": op, "T": _log(rng, 1, 4096), "N": _log(rng, 16, 8192), "K": _log16(rng, 256, 4096),
                "out": rng.choice(sorted(TYPES))}
    E = _log(rng, 8, 256)
    k = rng.randint(1, min(8, E))
    if op == "swiglu":
        return {"op": op, "T": _log(rng, 1, 2048), "H": _log16(rng, 256, 4096), "I": _log16(rng, 128, 2048), "E": E, "k": k}
    return {"op": op, "T": _log(rng, 1, 2048), "N": _log(rng, 128, 4096), "K": _log16(rng, 128, 2048), "E": E, "k": k,
            "out": rng.choice(sorted(TYPES))}


# ------------------------------------------------------------------ inputs ---
def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _activations(g, rows, K):
    """E4M3 rows with a float32 scale per 128 values: what a quantised layer
    input looks like (N(0, 1) with a few strong channels)."""
    v = torch.randn(rows, K, generator=g, device="cuda")
    v *= 1.0 + 7.0 * (torch.rand(K, generator=g, device="cuda") < 0.01)
    pad = torch.nn.functional.pad(v, (0, _blocks(K) * BLOCK - K)).view(rows, -1, BLOCK)
    s = (pad.abs().amax(2) / FP8_MAX).clamp_min(MIN_SCALE)
    return (pad / s[..., None]).view(rows, -1)[:, :K].contiguous().to(FP8), s


def _weights(g, n, rows, K):
    """n matrices N(0, 0.02), E4M3 with a float32 scale per 128 x 128 block."""
    q = torch.empty(n, rows, K, dtype=FP8, device="cuda")
    s = torch.empty(n, _blocks(rows), _blocks(K), device="cuda")
    step = max(1, (1 << 27) // (rows * K))
    for a in range(0, n, step):
        m = min(step, n - a)
        v = torch.randn(m, rows, K, generator=g, device="cuda") * 0.02
        p = torch.nn.functional.pad(v, (0, _blocks(K) * BLOCK - K, 0, _blocks(rows) * BLOCK - rows))
        p = p.view(m, _blocks(rows), BLOCK, _blocks(K), BLOCK)
        s[a:a + m] = p.abs().amax((2, 4)) / FP8_MAX
        p = p / s[a:a + m, :, None, :, None]
        q[a:a + m] = p.view(m, _blocks(rows) * BLOCK, -1)[:, :rows, :K].to(FP8)
    return q, s


def _routing(g, T, E, k):
    """Pairs (token, slot) sorted by expert, logits spread and popularity falling
    off like the benchmark's router: offsets [E + 1], entries [T k]."""
    rank = torch.randperm(E, generator=g, device="cuda").float() + 1
    logits = torch.randn(T, E, generator=g, device="cuda") * 1.28 - 0.156 * torch.log(rank)
    idx = torch.topk(logits, k, dim=1).indices.reshape(-1)
    entries = torch.argsort(idx, stable=True).int()
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(idx, minlength=E), 0)
    return offsets, entries


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    op, T = case["op"], case["T"]
    if op == "norm":
        dt, H = TYPES[case["type"]], case["H"]
        st["x"] = torch.randn(T, H, generator=g, device="cuda").to(dt)
        channel = 1.0 + 15.0 * (torch.rand(H, generator=g, device="cuda") < 0.01)
        st["res"] = (3.0 * torch.randn(T, H, generator=g, device="cuda") * channel).to(dt) if case["residual"] else None
        st["weight"] = 1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")
        st["res_out"] = torch.empty_like(st["x"]) if case["residual"] else None
        st["y"] = torch.empty_like(st["x"]) if case["y"] else None
        st["q"] = torch.empty(T, H, dtype=FP8, device="cuda")
        st["s"] = torch.empty(T, _blocks(H), device="cuda")
        return st
    if op == "gemm":
        st["a_q"], st["a_s"] = _activations(g, T, case["K"])
        w_q, w_s = _weights(g, 1, case["N"], case["K"])
        st["w_q"], st["w_s"] = w_q[0], w_s[0]
        st["y"] = torch.empty(T, case["N"], dtype=TYPES[case["out"]], device="cuda")
    else:
        E, k = case["E"], case["k"]
        st["offsets"], st["entries"] = _routing(g, T, E, k)
        if op == "swiglu":
            st["a_q"], st["a_s"] = _activations(g, T, case["H"])
            st["gate_q"], st["gate_s"] = _weights(g, E, case["I"], case["H"])
            st["up_q"], st["up_s"] = _weights(g, E, case["I"], case["H"])
            st["q"] = torch.empty(T * k, case["I"], dtype=FP8, device="cuda")
            st["s"] = torch.empty(T * k, _blocks(case["I"]), device="cuda")
        else:
            st["a_q"], st["a_s"] = _activations(g, T * k, case["K"])  # bucket order
            st["w_q"], st["w_s"] = _weights(g, E, case["N"], case["K"])
            st["y"] = torch.empty(T * k, case["N"], dtype=TYPES[case["out"]], device="cuda")
    st["ws"] = torch.zeros(1024, dtype=torch.uint8, device="cuda")  # a zeroed workspace
    return st


# ------------------------------------------------------------- plain forms ---
def _quantise(v):
    """Rows of float32 -> E4M3 codes and a scale per 128 values."""
    rows, n = v.shape
    p = torch.nn.functional.pad(v, (0, _blocks(n) * BLOCK - n)).view(rows, -1, BLOCK)
    s = (p.abs().amax(2) / FP8_MAX).clamp_min(MIN_SCALE)
    return (p / s[..., None]).view(rows, -1)[:, :n].contiguous().to(FP8), s


def _dequant_rows(q, s):
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _dequant_blocks(q, s):
    s = s.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :]
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _slots(offsets, rows):
    """The active experts, and their rows padded to the largest bucket: row
    numbers [active, most] and which of them are rows."""
    counts = offsets[1:] - offsets[:-1]
    active = torch.nonzero(counts).reshape(-1)
    most = int(counts.max())
    row = offsets[active][:, None] + torch.arange(most, device=offsets.device)[None]
    valid = torch.arange(most, device=offsets.device)[None] < counts[active][:, None]
    return active, row.clamp_max(rows - 1).long(), valid


def _norm(st):
    v = st["x"].float()
    if st["res"] is not None:
        v = v + st["res"].float()
    n = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * st["weight"]
    q, s = _quantise(n)
    out = {"q": q, "s": s}
    if st["res"] is not None:
        out["res"] = v.to(st["x"].dtype)
    if st["y"] is not None:
        out["y"] = n.to(st["x"].dtype)
    return out


def _gemm(st):
    return {"y": (_dequant_rows(st["a_q"], st["a_s"]) @ _dequant_blocks(st["w_q"], st["w_s"]).T).to(st["y"].dtype)}


def _swiglu(st):
    active, row, valid = _slots(st["offsets"], st["entries"].shape[0])
    a = _dequant_rows(st["a_q"], st["a_s"])[st["entries"][row].long() // st["k"]]
    gate = torch.bmm(a, _dequant_blocks(st["gate_q"][active], st["gate_s"][active]).transpose(1, 2))
    up = torch.bmm(a, _dequant_blocks(st["up_q"][active], st["up_s"][active]).transpose(1, 2))
    h = gate / (1.0 + torch.exp(-gate)) * up
    q, s = _quantise(h[valid])  # buckets are consecutive: bucket order
    return {"q": q, "s": s}


def _grouped(st):
    active, row, valid = _slots(st["offsets"], st["entries"].shape[0])
    a = _dequant_rows(st["a_q"], st["a_s"])[row]
    o = torch.bmm(a, _dequant_blocks(st["w_q"][active], st["w_s"][active]).transpose(1, 2))[valid]
    y = torch.empty_like(st["y"])
    y[st["entries"].long()] = o.to(y.dtype)
    return {"y": y}


def run(st):
    if own:
        from routed_expert_ffn_fp32_b200 import moe
        if st["op"] == "norm":
            moe.moe_rmsnorm_quant_fp8(st["x"], st["weight"], 1e-6, st["q"], st["s"], residual=st["res"],
                                      residual_out=st["res_out"], y_out=st["y"])
            out = {"q": st["q"], "s": st["s"]}
            if st["res"] is not None:
                out["res"] = st["res_out"]
            if st["y"] is not None:
                out["y"] = st["y"]
            return out
        if st["op"] == "gemm":
            moe.moe_gemm_fp8(st["a_q"], st["a_s"], st["w_q"], st["w_s"], st["y"], st["ws"])
            return {"y": st["y"]}
        if st["op"] == "swiglu":
            moe.moe_grouped_swiglu_fp8(st["a_q"], st["a_s"], st["gate_q"], st["gate_s"], st["up_q"], st["up_s"],
                                       st["offsets"], st["entries"], st["q"], st["s"], st["ws"], a_div=st["k"])
            return {"q": st["q"], "s": st["s"]}
        moe.moe_grouped_gemm_fp8(st["a_q"], st["a_s"], st["w_q"], st["w_s"], st["offsets"], st["entries"], st["y"],
                                 st["ws"], scatter=True)
        return {"y": st["y"]}
    return {"norm": _norm, "gemm": _gemm, "swiglu": _swiglu, "grouped": _grouped}[st["op"]](st)


# -------------------------------------------------------------------- work ---
def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        H, n = case["H"], TYPES[case["type"]].itemsize
        per = n * (1 + 2 * case["residual"] + case["y"]) + 1
        return {"bytes": T * (H * per + 4 * _blocks(H)) + 4 * H, "flops": 8 * T * H}
    if op == "gemm":
        N, K = case["N"], case["K"]
        moved = T * (K + 4 * _blocks(K)) + N * K + 4 * _blocks(N) * _blocks(K) + T * N * TYPES[case["out"]].itemsize
        return {"bytes": moved, "flops": 2 * T * N * K}
    E, k = case["E"], case["k"]
    P = T * k
    index = 4 * (P + E + 1)
    # experts that P picks reach, taken as even: k distinct ones for each token
    active = E * (1.0 - (1.0 - k / E) ** T)
    if op == "swiglu":
        H, I = case["H"], case["I"]
        w = 2 * (I * H + 4 * _blocks(I) * _blocks(H))
        return {"bytes": index + active * w + T * (H + 4 * _blocks(H)) + P * (I + 4 * _blocks(I)), "flops": 4 * P * H * I}
    N, K = case["N"], case["K"]
    w = N * K + 4 * _blocks(N) * _blocks(K)
    return {"bytes": index + active * w + P * (K + 4 * _blocks(K) + N * TYPES[case["out"]].itemsize), "flops": 2 * P * N * K}


# ------------------------------------------------------------------- exact ---
def _wide(q, s, *axes):
    """Codes times block scales in 64 bits: element i of an axis takes scale i // 128."""
    s = s.double()
    for ax in axes:
        s = s.index_select(ax, torch.arange(q.shape[ax], device=q.device) // BLOCK)
    return q.double() * s


def _codes(v):
    """Values before the rounding to 8 bits, and their scales."""
    n = v.shape[1]
    s = torch.stack([v[:, a:a + BLOCK].abs().max(1).values for a in range(0, n, BLOCK)], 1) / FP8_MAX
    s = torch.clamp(s, min=MIN_SCALE)
    return v / s[:, torch.arange(n, device=v.device) // BLOCK], s


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = st["x"].double() if st["res"] is None else st["x"].double() + st["res"].double()
        n = v / torch.sqrt(v.square().sum(1, keepdim=True) / case["H"] + 1e-6) * st["weight"].double()
        q, s = _codes(n)
        out = {"q": q, "s": s}
        if st["res"] is not None:
            out["res"] = v
        if st["y"] is not None:
            out["y"] = n
        return out
    if op == "gemm":
        return {"y": torch.mm(_wide(st["a_q"], st["a_s"], 1), _wide(st["w_q"], st["w_s"], 0, 1).t())}
    a = _wide(st["a_q"], st["a_s"], 1)
    at, pairs = st["offsets"].tolist(), st["entries"].long()
    width = case["I"] if op == "swiglu" else case["N"]
    out = torch.empty(pairs.shape[0], width, dtype=torch.float64, device=a.device)
    for e in range(case["E"]):
        b, c = at[e], at[e + 1]
        if b == c:
            continue
        if op == "swiglu":
            t = a[torch.div(pairs[b:c], case["k"], rounding_mode="floor")]
            u = t.mm(_wide(st["gate_q"][e], st["gate_s"][e], 0, 1).t())
            out[b:c] = u * torch.sigmoid(u) * t.mm(_wide(st["up_q"][e], st["up_s"][e], 0, 1).t())
        else:
            out[pairs[b:c]] = a[b:c].mm(_wide(st["w_q"][e], st["w_s"][e], 0, 1).t())
    if op == "swiglu":
        q, s = _codes(out)
        return {"q": q, "s": s}
    return {"y": out}
