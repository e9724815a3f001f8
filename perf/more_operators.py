"""The measured cases of the fine-tuning operators, with their plain forms.

Four operators: the router's balance loss with per-expert counts and the
gradient that reaches the router's logits (``router``), the gated activation
with its input kept in 8 bits and its backward pass from those (``gated``,
``gated_back``), 16-bit activations kept in 8 bits and given back
(``checkpoint``), and low-rank adapters of many requests beside a shared
projection, for serving (``lora``) and with their gradients (``lora_grads``).

``run`` computes a case in elementary torch operations in fp32, or, with
``own`` set, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32           # elements of one 8-bit scale
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one short sequence through a small layer's router: pure latency
        dict(name="router tiny", op="router", T=32, E=8, k=2, masked=0.0, renorm=True),
        # a padded batch of odd sizes; the weights are probabilities over all experts
        dict(name="router padded", op="router", T=5003, E=130, k=6, masked=0.2, renorm=False),
        # a training step's micro-batches over 896 experts, top-16: beyond the L2
        dict(name="router step", op="router", T=65536, E=896, k=16, masked=0.0, renorm=True),
        # a short ragged batch over the experts' gate/up rows, some experts empty
        dict(name="gated ragged", op="gated", S=1003, spare=21, E=12, I=200, act="swiglu_bias", dtype="f16"),
        # a training step's gate/up rows: activation and 8-bit copy
        dict(name="gated step", op="gated", S=32768, spare=0, E=32, I=2048, act="situ", dtype="bf16"),
        # the same rows in the backward pass, from the 8-bit copy
        dict(name="gated back step", op="gated_back", S=32768, spare=0, E=32, I=2048, act="situ", dtype="bf16"),
        # a layer's input kept for its weight gradient: one short odd batch, one training step's
        dict(name="checkpoint ragged", op="checkpoint", S=517, K=1000, dtype="f16"),
        dict(name="checkpoint step", op="checkpoint", S=32768, K=3584, dtype="bf16"),
        # one request's token beside the gate/up projection
        dict(name="lora one token", op="lora", S=1, n=4, r=16, K=3584, N=6144, order="mixed", bare=0.0, dtype="bf16",
             out="bf16"),
        # a decode step of 64 requests, each with an adapter of its own choice, some without
        dict(name="lora decode", op="lora", S=64, n=112, r=16, K=3584, N=6144, order="mixed", bare=0.1, dtype="bf16",
             out="bf16"),
        # prompts of several requests in one batch, fp32 sums to add to
        dict(name="lora prefill", op="lora", S=8211, n=9, r=32, K=3584, N=2048, order="runs", bare=0.05, dtype="f16",
             out="f32"),
        # a fine-tuning step: rows sorted by adapter, every gradient
        dict(name="lora grads", op="lora_grads", S=16384, n=4, r=64, K=3584, N=6144, bare=0.0, dtype="bf16",
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "router", "gated", "gated_back", "checkpoint", "lora", "lora", "lora_grads"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "router":
        E = _log(rng, 4, 4096)
        T = min(_log(rng, 1, 65536), 65536 * 896 // E)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(16, E)), masked=rng.choice([0.0, 0.0, 0.3]),
                    renorm=rng.random() < 0.6)
    if op in ("gated", "gated_back"):
        I = 8 * _log(rng, 1, 768)
        S = min(_log(rng, 1, 65536), 32768 * 2048 // I)
        return dict(op=op, S=S, spare=rng.choice([0, 0, min(S // 8, rng.randrange(300))]), E=_log(rng, 1, 512), I=I,
                    act=rng.choice(["situ", "situ", "swiglu_bias"]), dtype=dtype)
    if op == "checkpoint":
        K = 8 * _log(rng, 1, 2048)
        return dict(op=op, S=min(_log(rng, 1, 65536), 32768 * 3584 // K), K=K, dtype=dtype)
    K, N, r = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024), 8 * rng.choice([1, 1, 2, 2, 3, 4, 6, 8])
    S = max(1, min(_log(rng, 1, 16384), 16384 * 9728 // (K + N)))
    case = dict(op=op, S=S, r=r, K=K, N=N, bare=rng.choice([0.0, 0.0, 0.2]), dtype=dtype,
                out=rng.choice([dtype, "f32"]))
    if op == "lora_grads":
        case["n"] = _log(rng, 1, 16)
    else:
        case["n"], case["order"] = max(1, min(_log(rng, 1, 256), (1 << 26) // (r * (K + N)))), rng.choice(["mixed", "runs"])
    return case


def _counts(rng, total, groups, skew):
    p = np.arange(1, groups + 1, dtype=np.float64) ** -skew
    return rng.permutation(rng.multinomial(total, p / p.sum()))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * int(seed) + 29)
    rng = np.random.RandomState((int(seed) * 7919 + 47) % (1 << 31))

    def normal(shape, std, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

    def uniform(shape, lo, hi):
        return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(lo, hi, generator=g)

    if c["op"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        # logits of a router that favours some experts
        c["logits"] = normal((T, E), 1.5) + normal((E,), 0.7)
        top, ids = c["logits"].topk(k, dim=1)
        c["ids"] = ids.int()
        c["weights"] = torch.softmax(top, 1) if c["renorm"] else torch.softmax(c["logits"], 1).gather(1, ids)
        c["dweights"] = normal((T, k), 0.05)
        c["dloss"] = uniform((), 0.5, 1.5)
        c["mask"] = uniform((T,), 0, 1) >= c["masked"] if c["masked"] else None
        c["coef"] = 0.01
        return c

    dt = DT[c["dtype"]]
    if c["op"] == "checkpoint":
        # activations with a few strong channels, rows of different size
        x = normal((c["S"], c["K"]), 1.0)
        x *= torch.where(uniform((c["K"],), 0, 1) < 0.01, 12.0, 1.0)
        c["x"] = (x * torch.exp2(uniform((c["S"], 1), -2, 2))).to(dt)
        return c

    if c["op"] in ("gated", "gated_back"):
        S, E, I = c["S"], c["E"], c["I"]
        counts = _counts(rng, S - c["spare"], E, 0.5) if E > 1 else np.array([S - c["spare"]])
        c["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        if c["act"] == "situ":
            # caps of the gate and of the up half; the up half of some experts has none
            c["p0"], c["p1"] = uniform((E,), 0.5, 3.0), uniform((E,), 0.5, 3.0)
            c["p1"] = torch.where(uniform((E,), 0, 1) < 0.1, 0.0, c["p1"])
        else:
            c["p0"], c["p1"] = uniform((E,), 1.0, 2.0), uniform((E,), 0.0, 1.0)
        x = normal((S, 2 * I), 1.0) * torch.exp2(uniform((S, 1), -2, 1))
        x[S - c["spare"]:] = 0          # as the products leave rows of no expert
        if c["op"] == "gated":
            c["x"] = x.to(dt)
            return c
        # what a forward pass of this step has kept: E4M3 codes and power-of-two scales
        blocks = torch.nn.functional.pad(x.reshape(S, 2, I), (0, -I % BLOCK)).reshape(S, 2, -1, BLOCK)
        e = torch.ceil(torch.log2(blocks.abs().amax(-1) / 448.0).clamp(min=-120.0))
        q = (blocks * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn).reshape(S, 2, -1)[:, :, :I]
        c["q"] = q.reshape(S, 2 * I).contiguous().view(torch.uint8)
        c["scale"] = (e + 127.0).reshape(S, -1).to(torch.uint8)
        c["dh"] = normal((S, I), 0.05, dt)
        return c

    S, n, r, K, N = c["S"], c["n"], c["r"], c["K"], c["N"]
    kept = S - int(S * c["bare"])
    counts = _counts(rng, kept, n, 0.5 if n <= 16 else 0.0)
    ids = np.concatenate([np.repeat(rng.permutation(n) if c["op"] == "lora" else np.arange(n), counts),
                          np.full(S - kept, -1)])
    if c.get("order") == "mixed":
        ids = rng.permutation(ids)
    c["ids"] = torch.from_numpy(ids.astype(np.int32)).cuda()
    c["kept"], c["longest"] = int(kept), max(1, int(counts.max()))
    c["x"] = normal((S, K), 1.0, dt)
    c["a"] = normal((n, r, K), K ** -0.5, dt)
    c["b"] = normal((n, N, r), 0.3 * r ** -0.5, dt)
    c["scale"] = uniform((n,), 0.5, 2.0)
    c["base"] = normal((S, N), 1.0, DT[c["out"]])
    if c["op"] == "lora_grads":
        c["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        c["dy"] = normal((S, N), 0.05, dt)
        c["dx0"] = normal((S, K), 0.05, dt)
    return c


# ---------------------------------------------------------------------------
# the plain forms: fp32 throughout, one rounding at the end
# ---------------------------------------------------------------------------

def _plain_router(s):
    l, ids, T, E, k = s["logits"], s["ids"].long(), s["T"], s["E"], s["k"]
    p = torch.softmax(l, 1)
    m = torch.ones(T, device=l.device) if s["mask"] is None else s["mask"].float()
    n = m.sum().clamp(min=1.0)
    chosen = torch.zeros_like(l).scatter_(1, ids, 1.0)
    counts = (chosen * m[:, None]).sum(0, dtype=torch.float64)
    f = (counts / (n.double() * k)).float()
    mean_p = ((p * m[:, None]).sum(0, dtype=torch.float64) / n).float()
    loss = s["coef"] * E * (f * mean_p).sum()
    # the balance loss's part: p (f - <f, p>); the routing weights' part: a softmax's
    d = p * (f - (p * f).sum(1, keepdim=True)) * (s["dloss"] * s["coef"] * E / n * m)[:, None]
    wd = s["weights"] * s["dweights"]
    if s["renorm"]:
        d.scatter_add_(1, ids, wd - s["weights"] * wd.sum(1, keepdim=True))
    else:
        d.scatter_add_(1, ids, wd)
        d -= p * wd.sum(1, keepdim=True)
    return {"loss": loss, "counts": counts.int(), "dlogits": d}


def _pow2(n):
    """2^n in fp32 for int32 n in [-149, 127], by its bits: exp2 and ldexp may be off in the last one."""
    return torch.where(n >= -126, (n + 127) << 23, torch.bitwise_left_shift(torch.ones_like(n), (n + 149).clamp(0, 23))).view(
        torch.float32)


def _save(x):
    """16-bit [S, K] as E4M3 codes and the bytes of one power of two per 32 columns."""
    S, K = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).reshape(S, -1, BLOCK)
    amax = b.abs().amax(-1)
    m, p = torch.frexp(amax)                                     # amax = m 2^p, m in [0.5, 1)
    e = torch.where(amax > 0, torch.where(m > 0.875, p - 8, p - 9), torch.full_like(p, -127)).clamp(min=-127)
    q = (b * _pow2(-e)[..., None]).to(torch.float8_e4m3fn).reshape(S, -1)[:, :K].contiguous()
    return q, (e + 127).to(torch.uint8)


def _restore(q, scale):
    """fp32 [S, K] of codes with a scale byte per 32 columns."""
    return q.float() * _pow2(scale.int() - 127).repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _plain_checkpoint(s):
    q, scale = _save(s["x"])
    return {"q": q, "scale": scale, "x": _restore(q, scale).to(s["x"].dtype)}


def _params(s):
    """(p0, p1) of each row as columns, and whether it belongs to an expert."""
    row = torch.arange(s["S"], device=s["offsets"].device)
    e = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    kept = (e < s["E"])[:, None]
    e = e.clamp(max=s["E"] - 1)
    return s["p0"][e][:, None], s["p1"][e][:, None], kept


def _plain_gated(s):
    p0, p1, kept = _params(s)
    x = s["x"].float() * kept
    g, u = x.chunk(2, 1)
    if s["act"] == "situ":
        h = p0 * torch.tanh(g / p0) * torch.sigmoid(g) * torch.where(p1 > 0, p1 * torch.tanh(u / p1.clamp(min=1e-3)), u)
    else:
        h = g * torch.sigmoid(p0 * g) * (u + p1)
    q, scale = _save(x.reshape(-1, s["I"]))
    return {"h": torch.where(kept, h, 0.0).to(s["x"].dtype), "q": q.reshape(x.shape), "scale": scale.reshape(s["S"], -1)}


def _plain_gated_back(s):
    p0, p1, kept = _params(s)
    S, I, dt = s["S"], s["I"], s["dh"].dtype
    x = _restore(s["q"].view(torch.float8_e4m3fn).reshape(2 * S, I), s["scale"].reshape(2 * S, -1)).reshape(S, 2 * I)
    g, u = x.chunk(2, 1)
    dh = s["dh"].float()
    if s["act"] == "situ":
        sg, t = torch.sigmoid(g), torch.tanh(g / p0)
        tu = torch.tanh(u / p1.clamp(min=1e-3))
        gate, up = p0 * t * sg, torch.where(p1 > 0, p1 * tu, u)
        dgate = (1 - t * t) * sg + gate * (1 - sg)
        dup = torch.where(p1 > 0, 1 - tu * tu, 1.0)
    else:
        sg = torch.sigmoid(p0 * g)
        gate, up = g * sg, u + p1
        dgate, dup = sg + p0 * gate * (1 - sg), 1.0
    dx = torch.cat((dh * dgate * up, dh * gate * dup), 1)
    return {"dx": torch.where(kept, dx, 0.0).to(dt), "h": torch.where(kept, gate * up, 0.0).to(dt)}


def _by_adapter(s):
    """(rows, adapter, place) of the rows that have an adapter, sorted by it."""
    ids = s["ids"].long()
    key = torch.where(ids < 0, s["n"], ids)
    rows = torch.argsort(key, stable=True)[: s["kept"]]
    e = key[rows]
    first = torch.searchsorted(e, torch.arange(s["n"], device=e.device))
    return rows, e, torch.arange(s["kept"], device=e.device) - first[e]


def _pad(s, t, where):
    rows, e, at = where
    p = torch.zeros((s["n"], s["longest"], t.shape[1]), device=t.device)
    p[e, at] = t[rows].float()
    return p


def _added(base, delta, where, dtype):
    rows, e, at = where
    y = base.float().clone()
    y[rows] += delta[e, at]
    return y.to(dtype)


def _plain_lora(s):
    where = _by_adapter(s)
    u = torch.bmm(_pad(s, s["x"], where), s["a"].float().transpose(1, 2)) * s["scale"][:, None, None]
    return _added(s["base"], torch.bmm(u, s["b"].float().transpose(1, 2)), where, DT[s["out"]])


def _plain_lora_grads(s):
    where = _by_adapter(s)
    a, b, f = s["a"].float(), s["b"].float(), s["scale"][:, None, None]
    x, dy = _pad(s, s["x"], where), _pad(s, s["dy"], where)
    u, v = torch.bmm(x, a.transpose(1, 2)) * f, torch.bmm(dy, b) * f
    return {"y": _added(s["base"], torch.bmm(u, b.transpose(1, 2)), where, DT[s["out"]]),
            "dx": _added(s["dx0"], torch.bmm(v, a), where, DT[s["dtype"]]),
            "da": torch.bmm(v.transpose(1, 2), x).to(DT[s["dtype"]]),
            "db": torch.bmm(dy.transpose(1, 2), u).to(DT[s["dtype"]])}


def run(s):
    if not own:
        return {"router": _plain_router, "gated": _plain_gated, "gated_back": _plain_gated_back,
                "checkpoint": _plain_checkpoint, "lora": _plain_lora, "lora_grads": _plain_lora_grads}[s["op"]](s)
    from block_scaled_fp4_permute_gb300 import binding as b
    if s["op"] == "router":
        loss, counts, tokens, stats = b.situ_moe_balance_loss(s["logits"], s["ids"], mask=s["mask"], coef=s["coef"])
        d = b.situ_moe_router_backward(s["logits"], s["ids"], counts, tokens, stats, dloss=s["dloss"], coef=s["coef"],
                                       mask=s["mask"], topk_weights=s["weights"], dweights=s["dweights"],
                                       renormalize=s["renorm"])
        return {"loss": loss, "counts": counts, "dlogits": d}
    if s["op"] == "checkpoint":
        q, scale = b.situ_moe_save_mxfp8(s["x"])
        return {"q": q.view(torch.float8_e4m3fn), "scale": scale,
                "x": b.situ_moe_restore_mxfp8(q, scale, s["x"].dtype)}
    if s["op"] in ("gated", "gated_back"):
        act = b.SITU_ACT_FN_SITU if s["act"] == "situ" else b.SITU_ACT_FN_SWIGLU_BIAS
        if s["op"] == "gated":
            h, q, scale = b.situ_moe_gated(s["x"], s["p0"], s["p1"], s["offsets"], activation=act, save=True)
            return {"h": h, "q": q.view(torch.float8_e4m3fn), "scale": scale}
        dx, h = b.situ_moe_gated_backward(s["dh"], s["q"], s["scale"], s["p0"], s["p1"], s["offsets"], activation=act,
                                          want_h=True)
        return {"dx": dx, "h": h}
    if s["op"] == "lora":
        return b.situ_moe_lora(s["base"], s["x"], s["a"], s["b"], ids=s["ids"], scale=s["scale"])
    y, u = b.situ_moe_lora(s["base"], s["x"], s["a"], s["b"], offsets=s["offsets"], scale=s["scale"], keep=True)
    dx, da, db = b.situ_moe_lora_backward(s["dy"], s["x"], s["a"], s["b"], s["offsets"], u, scale=s["scale"],
                                          dx=s["dx0"])
    return {"y": y, "dx": dx, "da": da, "db": db}


def work(case):
    c = case
    if c["op"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 8 * T * E + 12 * T * k + 4 * E, "flops": 8 * T * E}
    if c["op"] == "checkpoint":
        n, blocks = c["S"] * c["K"], c["S"] * -(-c["K"] // BLOCK)
        return {"bytes": n * 5 + blocks, "flops": 2 * n}
    if c["op"] in ("gated", "gated_back"):
        n, blocks = c["S"] * c["I"], c["S"] * 2 * -(-c["I"] // BLOCK)
        # two 16-bit inputs, one 16-bit and two 8-bit results; or two 8-bit inputs, one 16-bit, three 16-bit results
        return {"bytes": n * (8 if c["op"] == "gated" else 10) + blocks, "flops": (12 if c["op"] == "gated" else 24) * n}
    S, n, r, K, N, el = c["S"], c["n"], c["r"], c["K"], c["N"], SIZE[c["dtype"]]
    kept = S - int(S * c["bare"])
    held = n * (1.0 - (1.0 - 1.0 / n) ** kept)                   # adapters in use, on average
    adapters = held * r * (K + N) * el
    rows = kept * K * el + 2 * S * N * SIZE[c["out"]]
    flops = 2 * kept * r * (K + N)
    if c["op"] == "lora":
        return {"bytes": int(adapters + rows + 4 * S), "flops": flops}
    return {"bytes": int(adapters + rows + kept * N * el + 2 * S * K * el + n * r * (K + N) * el), "flops": 3 * flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _nearest_e4m3(v):
    """The E4M3 value nearest to v (|v| <= 448), ties to the even mantissa."""
    _, p = torch.frexp(v)                          # |v| in [2^(p-1), 2^p)
    step = _two_to((p - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _two_to(n):
    """2^n in fp64 for whole n in [-1000, 1000]."""
    return ((n.long() + 1023) * (1 << 52)).view(torch.float64)


def _exact_saved(x):
    """(values of the codes, scales' exponents + 127) of x [S, K], in 64 bits."""
    q, scale = torch.empty_like(x), torch.empty((x.shape[0], -(-x.shape[1] // BLOCK)), device=x.device, dtype=x.dtype)
    for k in range(scale.shape[1]):
        block = x[:, k * BLOCK:(k + 1) * BLOCK]
        amax = block.abs().amax(1)
        e = torch.floor(torch.log2(amax / 448.0).clamp(min=-127.0))
        e = torch.where(amax > 448.0 * _two_to(e), e + 1, e)             # the smallest with amax 2^-e <= 448
        e = torch.where(amax <= 448.0 * _two_to(e - 1), e - 1, e).clamp(min=-127.0)
        q[:, k * BLOCK:(k + 1) * BLOCK] = _nearest_e4m3(block * _two_to(-e)[:, None])
        scale[:, k] = e + 127
    return q, scale


def _exact_restored(q, scale):
    x = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    for k in range(scale.shape[1]):
        x[:, k * BLOCK:(k + 1) * BLOCK] = q[:, k * BLOCK:(k + 1) * BLOCK].double() * _two_to(scale[:, k, None].double() - 127)
    return x


def _exact_situ(v, cap):
    """cap tanh(v / cap) and its derivative; v and 1 without a cap."""
    if cap <= 0:
        return v, torch.ones_like(v)
    return cap * torch.tanh(v / cap), 1 / torch.cosh(v / cap) ** 2


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "router":
        l, ids, k, E = s["logits"].to(f64), s["ids"].long(), s["k"], s["E"]
        z = torch.exp(l - l.amax(1, keepdim=True))
        p = z / z.sum(1, keepdim=True)
        keep = torch.ones(s["T"], dtype=torch.bool, device=l.device) if s["mask"] is None else s["mask"]
        n = max(1, int(keep.sum()))
        counts = torch.bincount(ids[keep].reshape(-1), minlength=E)
        f = counts.to(f64) / (n * k)
        factor = s["coef"] * E
        d = factor * float(s["dloss"]) / n * p * (f - (p @ f)[:, None]) * keep.to(f64)[:, None]
        # the weights are a softmax of the chosen logits, or of all
        dw = s["dweights"].to(f64)
        if s["renorm"]:
            w = torch.softmax(l.gather(1, ids), 1)
            d.scatter_add_(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
        else:
            full = torch.zeros_like(l).scatter_(1, ids, dw)
            d += p * (full - (p * full).sum(1, keepdim=True))
        return {"loss": factor * (f * p[keep].sum(0) / n).sum(), "counts": counts.int(), "dlogits": d}
    if s["op"] == "checkpoint":
        q, scale = _exact_saved(s["x"].to(f64))
        return {"q": q, "scale": scale.to(torch.uint8), "x": _exact_restored(q, scale)}
    if s["op"] in ("gated", "gated_back"):
        S, I, off = s["S"], s["I"], s["offsets"].tolist()
        if s["op"] == "gated":
            x = s["x"].to(f64)
            x[off[-1]:] = 0
        else:
            x = _exact_restored(s["q"].view(torch.float8_e4m3fn).reshape(2 * S, I).to(f64),
                                s["scale"].reshape(2 * S, -1)).reshape(S, 2 * I)
            dh, dx = s["dh"].to(f64), torch.zeros((S, 2 * I), dtype=f64, device="cuda")
        h = torch.zeros((S, I), dtype=f64, device="cuda")
        p0, p1 = s["p0"].tolist(), s["p1"].tolist()
        for e in range(s["E"]):
            rows = slice(off[e], off[e + 1])
            g, u = x[rows, :I], x[rows, I:]
            if s["act"] == "situ":
                sg = 1 / (1 + torch.exp(-g))
                (t, dt), (up, dup) = _exact_situ(g, p0[e]), _exact_situ(u, p1[e])
                gate, dgate = t * sg, dt * sg + t * sg * (1 - sg)
            else:
                sg = 1 / (1 + torch.exp(-p0[e] * g))
                gate, dgate = g * sg, sg + p0[e] * g * sg * (1 - sg)
                up, dup = u + p1[e], torch.ones_like(u)
            h[rows] = gate * up
            if s["op"] == "gated_back":
                dx[rows, :I], dx[rows, I:] = dh[rows] * dgate * up, dh[rows] * gate * dup
        if s["op"] == "gated_back":
            return {"dx": dx, "h": h}
        q, scale = _exact_saved(x.reshape(2 * S, I))
        return {"h": h, "q": q.reshape(S, 2 * I), "scale": scale.reshape(S, -1).to(torch.uint8)}
    ids = s["ids"].tolist()
    rows_of = [[] for _ in range(s["n"])]
    for i, e in enumerate(ids):
        if e >= 0:
            rows_of[e].append(i)
    y, grads = s["base"].to(f64), s["op"] == "lora_grads"
    if grads:
        dx, da, db = s["dx0"].to(f64), torch.zeros(s["a"].shape, dtype=f64, device="cuda"), torch.zeros(
            s["b"].shape, dtype=f64, device="cuda")
    for e, rows in enumerate(rows_of):
        if not rows:
            continue
        rows = torch.tensor(rows, device="cuda")
        a, b, x, f = s["a"][e].to(f64), s["b"][e].to(f64), s["x"][rows].to(f64), float(s["scale"][e])
        y[rows] += f * ((x @ a.T) @ b.T)
        if grads:
            dy = s["dy"][rows].to(f64)
            dx[rows] += f * ((dy @ b) @ a)
            da[e], db[e] = f * ((dy @ b).T @ x), f * (dy.T @ (x @ a.T))
    return {"y": y, "dx": dx, "da": da, "db": db} if grads else y
