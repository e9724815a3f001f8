"""The measured cases of the expert-product operators, with their plain forms.

Three operators: the product of ragged expert groups with 16-bit weights
(``grouped``) and its two gradients (``grads``), the quantisation to E4M3 with
one fp32 scale per block of 128 (``quant``), and the product of such operands,
dense or per expert (``fp8``).

``run`` computes a case in elementary torch operations in fp32, or, with
``own`` set, through the package's entry points.  Rows of all experts are
sorted by expert; ``offsets`` [E + 1] bounds each expert's rows; rows at and
after ``offsets[E]`` (``spare`` rows: slots of experts held elsewhere) belong
to none and give zeros.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128          # elements of one scale
E4M3_MAX = 448.0
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decode step of a small layer (the "tiny" workload's FC1): pure latency
        dict(name="grouped tiny", op="grouped", S=32, spare=0, E=8, N=256, K=256, skew=0.0, dtype="bf16", out="bf16"),
        # FC1 of a decode step, 64 tokens x top-16 over 896 experts (the "decode" workload), 16-bit weights
        dict(name="grouped decode", op="grouped", S=1024, spare=0, E=896, N=768, K=3584, skew=0.0, dtype="bf16",
             out="bf16"),
        # FC1 of an expert-parallel shard's prefill: 112 of 896 experts, some slots held elsewhere
        dict(name="grouped prefill", op="grouped", S=8357, spare=299, E=112, N=6144, K=3584, skew=0.3, dtype="bf16",
             out="bf16"),
        # a fine-tuning step on short ragged batches: odd rows, skewed experts, some empty, fp32 weight gradients
        dict(name="grads ragged", op="grads", S=1003, spare=21, E=12, N=1000, K=2056, skew=1.2, dtype="f16", out="f32"),
        # a training step's backward products: about 1,024 rows per expert, skewed
        dict(name="grads train", op="grads", S=32768, spare=0, E=32, N=4096, K=3584, skew=0.3, dtype="bf16", out="bf16"),
        # activations of a decode step
        dict(name="quant decode", op="quant", E=1, R=64, K=3584, rows=1, dtype="bf16"),
        # activations of a prefill, a scale per row and 128 columns
        dict(name="quant prefill", op="quant", E=1, R=8192, K=3584, rows=1, dtype="bf16"),
        # weights at load time, a scale per 128 x 128 block, the last blocks partial
        dict(name="quant weights", op="quant", E=16, R=2000, K=3600, rows=128, dtype="bf16"),
        # a shared expert's projection while decoding a few sequences
        dict(name="fp8 decode", op="fp8", S=5, spare=0, E=1, N=6144, K=3584, skew=0.0, out="bf16"),
        # the same projection in a prefill
        dict(name="fp8 prefill", op="fp8", S=8192, spare=0, E=1, N=6144, K=3584, skew=0.0, out="bf16"),
        # the routed experts of a shard while decoding 64 tokens
        dict(name="fp8 experts decode", op="fp8", S=128, spare=0, E=112, N=6144, K=3584, skew=0.0, out="bf16"),
        # the routed experts' down projection in a ragged prefill; the last block of K is partial
        dict(name="fp8 experts prefill", op="fp8", S=16411, spare=117, E=64, N=3584, K=2000, skew=0.5, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grads", "grads", "quant", "quant", "fp8", "fp8", "fp8"])
    if op == "quant":
        rows = rng.choice([1, 128])
        K, R = 8 * _log(rng, 16, 768), _log(rng, 1, 16384)
        E = min(_log(rng, 1, 64) if rows == 128 else 1, max(1, (1 << 27) // (R * K)))
        return dict(op=op, E=E, R=R, K=K, rows=rows, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    step = 16 if op == "fp8" else 8
    K, N = step * _log(rng, 128 // step, 6144 // step), 8 * _log(rng, 16, 768)
    E = _log(rng, 1, 256) if op != "fp8" or rng.random() < 0.6 else 1
    E = max(1, min(E, int(1.6e9 / (N * K))))
    S = _log(rng, 1, 32768)
    S = max(1, min(S, int(1.5e12 / (2.0 * N * K * (2 if op == "grads" else 1)))))
    case = dict(op=op, S=S, spare=rng.choice([0, 0, min(S // 8, rng.randrange(512))]), E=E, N=N, K=K,
                skew=rng.choice([0.0, 0.0, round(rng.uniform(0.1, 1.2), 2)]) if E > 1 else 0.0,
                out=rng.choice(["bf16", "f32"]))
    if op != "fp8":
        case["dtype"] = rng.choice(["bf16", "f16"])
        if case["out"] == "bf16":
            case["out"] = case["dtype"]
    return case


def _shares(c):
    p = np.arange(1, c["E"] + 1, dtype=np.float64) ** -c["skew"]
    return p / p.sum()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * int(seed) + 17)

    def normal(shape, std, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

    def uniform(shape, lo, hi):
        return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(lo, hi, generator=g)

    if c["op"] == "quant":
        # activations with a few strong channels, or weights; in either case rows of different size
        x = normal((c["E"], c["R"], c["K"]), 1.0 if c["rows"] == 1 else 0.02, torch.float32)
        x *= torch.where(uniform((c["K"],), 0, 1) < 0.01, 12.0, 1.0)
        x *= torch.exp2(uniform((c["E"], c["R"], 1), -2, 2))
        c["x"] = x.to(DT[c["dtype"]]).contiguous()
        if c["rows"] == 1:
            c["x"] = c["x"][0]
        return c

    rng = np.random.RandomState((int(seed) * 7919 + 31) % (1 << 31))
    S, E, N, K = c["S"], c["E"], c["N"], c["K"]
    kept = S - c["spare"]
    counts = rng.permutation(rng.multinomial(kept, _shares(c))) if E > 1 else np.array([kept])
    c["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    c["kept"], c["longest"] = int(kept), int(counts.max())
    if c["op"] == "fp8":
        nkb = -(-K // BLOCK)
        # the codes that the block scaling leaves: the largest of 128 (16,384) normal values at 448
        c["x_q"] = normal((S, K), 165.0, torch.bfloat16).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        c["x_scale"] = torch.exp2(uniform((S, nkb), -8.4, -6.4))
        c["w_q"] = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        for e in range(E):
            c["w_q"][e] = normal((N, K), 105.0, torch.bfloat16).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        c["w_scale"] = torch.exp2(uniform((E, -(-N // BLOCK), nkb), -13.4, -11.4))
        if E == 1:
            c["w_q"], c["w_scale"] = c["w_q"][0], c["w_scale"][0]
        return c
    dt = DT[c["dtype"]]
    c["x"] = normal((S, K), 1.0, dt)
    c["w"] = normal((E, N, K), 0.02, dt)
    if c["op"] == "grads":
        c["dy"] = normal((S, N), 0.05, dt)
    return c


# ---------------------------------------------------------------------------
# the plain forms: fp32 throughout, one rounding at the end
# ---------------------------------------------------------------------------

def _groups(s):
    """(expert, place within the expert) of each kept row."""
    row = torch.arange(s["kept"], device=s["offsets"].device)
    e = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    return e, row - s["offsets"].long()[e]


def _pad(s, rows, e, at):
    """Rows [kept, C] as [E, longest, C], zeros after each expert's last."""
    p = rows.new_zeros((s["E"], max(1, s["longest"]), rows.shape[1]))
    p[e, at] = rows
    return p


def _unpad(s, y, e, at, dtype):
    out = y.new_zeros((s["S"], y.shape[2]))
    out[: s["kept"]] = y[e, at]
    return out.to(dtype)


def _spread(scale, rows, cols, n_rows):
    """A scale per (n_rows x 128) block as one factor per element of [..., rows, cols]."""
    f = scale.repeat_interleave(BLOCK, -1)[..., :cols]
    return f if n_rows == 1 else f.repeat_interleave(n_rows, -2)[..., :rows, :]


def _plain_quant(s):
    x, n = s["x"].float(), s["rows"]
    R, K = x.shape[-2:]
    nr, nk = -(-R // n), -(-K // BLOCK)
    a = torch.nn.functional.pad(x.abs(), (0, nk * BLOCK - K, 0, nr * n - R))
    amax = a.reshape(*x.shape[:-2], nr, n, nk, BLOCK).amax((-3, -1))
    scale = (amax / E4M3_MAX).clamp(min=2.0 ** -126)
    q = (x / _spread(scale, R, K, n)).to(torch.float8_e4m3fn)
    return {"q": q, "scale": scale}


def _plain_fp8(s):
    out = DT[s["out"]]
    x = s["x_q"].float() * _spread(s["x_scale"], s["S"], s["K"], 1)
    w = s["w_q"].float() * _spread(s["w_scale"], s["N"], s["K"], BLOCK)
    if s["E"] == 1:
        y = x @ w.T
        y[s["kept"]:] = 0
        return y.to(out)
    e, at = _groups(s)
    y = torch.bmm(_pad(s, x[: s["kept"]], e, at), w.transpose(1, 2))
    return _unpad(s, y, e, at, out)


def _plain_grouped(s):
    e, at = _groups(s)
    y = torch.bmm(_pad(s, s["x"][: s["kept"]].float(), e, at), s["w"].float().transpose(1, 2))
    return _unpad(s, y, e, at, DT[s["out"]])


def _plain_grads(s):
    e, at = _groups(s)
    dy = _pad(s, s["dy"][: s["kept"]].float(), e, at)
    dx = torch.bmm(dy, s["w"].float())
    dw = torch.bmm(dy.transpose(1, 2), _pad(s, s["x"][: s["kept"]].float(), e, at))
    return {"dx": _unpad(s, dx, e, at, DT[s["dtype"]]), "dw": dw.to(DT[s["out"]])}


def run(s):
    if not own:
        return {"quant": _plain_quant, "fp8": _plain_fp8, "grouped": _plain_grouped, "grads": _plain_grads}[s["op"]](s)
    from block_scaled_fp4_permute_gb300 import binding as b
    if s["op"] == "quant":
        q, scale = b.situ_moe_quant_fp8(s["x"], s["rows"])
        return {"q": q.view(torch.float8_e4m3fn), "scale": scale}
    if s["op"] == "fp8":
        if s["E"] == 1 and not s["spare"]:
            return b.situ_moe_fp8_gemm(s["x_q"], s["x_scale"], s["w_q"], s["w_scale"], out_dtype=DT[s["out"]])
        return b.situ_moe_fp8_grouped_gemm(s["x_q"], s["x_scale"], s["w_q"], s["w_scale"], s["offsets"],
                                           out_dtype=DT[s["out"]])
    if s["op"] == "grouped":
        return b.situ_moe_grouped_gemm(s["x"], s["w"], s["offsets"], out_dtype=DT[s["out"]])
    return {"dx": b.situ_moe_grouped_gemm_dgrad(s["dy"], s["w"], s["offsets"]),
            "dw": b.situ_moe_grouped_gemm_wgrad(s["dy"], s["x"], s["offsets"], out_dtype=DT[s["out"]])}


def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if c["op"] == "quant":
        n, blocks = c["E"] * c["R"] * c["K"], c["E"] * -(-c["R"] // c["rows"]) * -(-c["K"] // BLOCK)
        return {"bytes": n * (size[c["dtype"]] + 1) + 4 * blocks, "flops": 2 * n}
    S, E, N, K = c["S"], c["E"], c["N"], c["K"]
    kept = S - c["spare"]
    held = float(np.sum(1.0 - (1.0 - _shares(c)) ** kept))    # experts that have rows, on average
    flops = 2 * kept * N * K
    if c["op"] == "fp8":
        nkb = -(-K // BLOCK)
        read = held * (N * K + 4 * -(-N // BLOCK) * nkb) + kept * (K + 4 * nkb)
        return {"bytes": int(read + S * N * size[c["out"]]), "flops": flops}
    el = size[c["dtype"]]
    if c["op"] == "grouped":
        return {"bytes": int(held * N * K * el + kept * K * el + S * N * size[c["out"]]), "flops": flops}
    return {"bytes": int(held * N * K * el + kept * (N + K) * el + S * K * el + E * N * K * size[c["out"]]),
            "flops": 2 * flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _nearest_e4m3(v):
    """The E4M3 value nearest to v (|v| <= 448), ties to the even mantissa."""
    _, p = torch.frexp(v)                          # |v| in [2^(p-1), 2^p)
    step = torch.ldexp(torch.ones_like(v), (p - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "quant":
        x = s["x"].reshape(-1, *s["x"].shape[-2:])
        n, (E, R, K) = s["rows"], x.shape
        q = torch.empty(x.shape, dtype=f64, device=x.device)
        scale = torch.empty((E, -(-R // n), -(-K // BLOCK)), dtype=f64, device=x.device)
        for k in range(scale.shape[2]):
            cols = slice(k * BLOCK, min(K, (k + 1) * BLOCK))
            if n == 1:
                scale[:, :, k] = x[:, :, cols].to(f64).abs().amax(2) / E4M3_MAX
                q[:, :, cols] = _nearest_e4m3(x[:, :, cols].to(f64) / scale[:, :, k, None].clamp(min=2.0 ** -126))
                continue
            for r in range(scale.shape[1]):
                rows = slice(r * n, min(R, (r + 1) * n))
                block = x[:, rows, cols].to(f64)
                scale[:, r, k] = block.abs().amax((1, 2)) / E4M3_MAX
                q[:, rows, cols] = _nearest_e4m3(block / scale[:, r, k, None, None].clamp(min=2.0 ** -126))
        scale.clamp_(min=2.0 ** -126)
        return {"q": q.reshape(s["x"].shape), "scale": scale.reshape(*s["x"].shape[:-2], *scale.shape[1:])}
    off = s["offsets"].cpu().tolist()
    groups = [(e, slice(off[e], off[e + 1])) for e in range(s["E"]) if off[e + 1] > off[e]]
    if s["op"] == "fp8":
        w_q, w_scale = s["w_q"].reshape(s["E"], s["N"], s["K"]), s["w_scale"].reshape(s["E"], -1, s["x_scale"].shape[1])
        y = torch.zeros((s["S"], s["N"]), dtype=f64, device="cuda")
        col = torch.arange(s["K"], device="cuda") // BLOCK
        blk = torch.arange(s["N"], device="cuda") // BLOCK
        for e, rows in groups:
            w = w_q[e].to(f64) * w_scale[e].to(f64)[blk][:, col]
            y[rows] = (s["x_q"][rows].to(f64) * s["x_scale"][rows].to(f64)[:, col]) @ w.T
        return y
    if s["op"] == "grouped":
        y = torch.zeros((s["S"], s["N"]), dtype=f64, device="cuda")
        for e, rows in groups:
            y[rows] = s["x"][rows].to(f64) @ s["w"][e].to(f64).T
        return y
    dx = torch.zeros((s["S"], s["K"]), dtype=f64, device="cuda")
    dw = torch.zeros((s["E"], s["N"], s["K"]), dtype=f64, device="cuda")
    for e, rows in groups:
        dy = s["dy"][rows].to(f64)
        dx[rows] = dy @ s["w"][e].to(f64)
        dw[e] = dy.T @ s["x"][rows].to(f64)
    return {"dx": dx, "dw": dw}
