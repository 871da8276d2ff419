"""Timing cases of the many-adapter linear layer and the many-tensor AdamW step.

Three operators: the forward of Y_i = X_i W' + s[a_i] X_i L1[a_i] L2[a_i] over
one frozen NF4 weight and a bank of adapters (token i uses adapter a_i, or none
where a_i = -1), its backward, and an AdamW step over the adapters' tensors
with states in 32 or 8 bits.  ``run`` computes them in plain torch operations,
or, with ``own`` set, through the framework's entry points.
"""
from __future__ import annotations

import math
import statistics

import numpy as np
import torch

own = False

BLOCK = 64        # weights per first-level constant
DQ_BLOCK = 256    # first-level constants per second-level constant
STATE_BLOCK = 256  # optimizer state elements per scale
E4M3_MAX = 448.0
BETA1, BETA2, EPS, LR, DECAY, MAX_NORM = 0.9, 0.999, 1e-8, 2e-4, 0.01, 0.3
STEPS_DONE = 10   # optimizer steps before the timed one


# ---------------------------------------------------------------- cases

def _linear(name, op, M, h, o, n, r, ids, out, none=0.0):
    return {"name": name, "op": op, "M": M, "h": h, "o": o, "n": n, "r": r, "ids": ids, "out": out, "none": none}


def listed():
    return [
        # one token of one request, an attention projection of a 7B-shaped model: latency
        _linear("fwd_1_token", "fwd", 1, 4096, 4096, 8, 64, "requests", "bf16"),
        # 16 requests, each with an adapter of its own, one decode step of a 65B-shaped up projection
        _linear("fwd_16_decode", "fwd", 16, 8192, 22016, 16, 64, "each", "bf16"),
        # 29 requests over 12 adapters, some without, an 8192-wide projection, fp32 out
        _linear("fwd_29_decode", "fwd", 29, 8192, 8192, 12, 16, "mixed", "f32", 0.1),
        # a chunk of prompts mixed with decode tokens, 13B-shaped down projection, odd token count
        _linear("fwd_333_mixed", "fwd", 333, 13824, 5120, 24, 32, "mixed", "bf16", 0.05),
        # prompts of 8 adapters, 7B-shaped up projection
        _linear("fwd_4096_prompts", "fwd", 4096, 4096, 11008, 8, 64, "requests", "bf16"),
        # a small layer's training step, fp32 gradient of the input
        _linear("bwd_200_small", "bwd", 200, 1024, 768, 3, 8, "requests", "f32"),
        # four adapters trained side by side, 7B-shaped attention projection
        _linear("bwd_4096", "bwd", 4096, 4096, 4096, 4, 64, "requests", "bf16"),
        # eight adapters, samples shuffled in the batch, 13B-shaped up projection
        _linear("bwd_8190_shuffled", "bwd", 8190, 5120, 13824, 8, 64, "shuffled", "bf16", 0.02),
        # the factors of one small linear, and of one 7B-shaped layer (7 linears): few launches
        {"name": "adamw32_pair", "op": "adamw", "layers": 1, "h": 1024, "o": 1000, "linears": 1, "r": 8, "bits": 32, "grad": "f32"},
        {"name": "adamw8_layer", "op": "adamw", "layers": 1, "h": 4096, "o": 11008, "linears": 7, "r": 64, "bits": 8, "grad": "f32"},
        # every linear of a 7B-shaped model, 448 tensors
        {"name": "adamw32_model", "op": "adamw", "layers": 32, "h": 4096, "o": 11008, "linears": 7, "r": 64, "bits": 32, "grad": "f32"},
        {"name": "adamw8_model", "op": "adamw", "layers": 32, "h": 4096, "o": 11008, "linears": 7, "r": 64, "bits": 8, "grad": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "adamw"])
    if op == "adamw":
        return {"op": "adamw", "layers": rng.randint(1, 16), "h": _log(rng, 64, 8192), "o": _log(rng, 64, 14000),
                "linears": rng.choice([1, 2, 4, 7]), "r": 8 * _log(rng, 1, 8), "bits": rng.choice([8, 32]),
                "grad": rng.choice(["f32", "bf16"])}
    h, o = 128 * _log(rng, 2, 64), 128 * _log(rng, 2, 108)
    # no more products than the largest listed case
    M = min(_log(rng, 1, 8192), 8190 * 5120 * 13824 // (h * o))
    return {"op": op, "M": M, "h": h, "o": o, "n": _log(rng, 1, 32), "r": 8 * _log(rng, 1, 16),
            "ids": rng.choice(["requests", "mixed", "shuffled", "each"]), "out": rng.choice(["bf16", "f32"]),
            "none": rng.choice([0.0, 0.0, 0.1, 0.4])}


def _tensor_sizes(c):
    """Element counts of the factors L1 [h][r], L2 [r][o] of a model's linears: seven have the
    q, k, v, o, gate, up, down shapes; fewer are h x o."""
    h, o, r = c["h"], c["o"], c["r"]
    shapes = [(h, h)] * 4 + [(h, o), (h, o), (o, h)] if c["linears"] == 7 else [(h, o)] * c["linears"]
    return [r * d for _ in range(c["layers"]) for pair in shapes for d in pair]


def work(case):
    c = case
    if c["op"] == "adamw":
        n = sum(_tensor_sizes(c))
        state = 16 if c["bits"] == 32 else 4 + 16 / STATE_BLOCK
        return {"bytes": n * (8 + (4 if c["grad"] == "f32" else 2) + 2 + state), "flops": 16 * n}
    M, h, o, r = c["M"], c["h"], c["o"], c["r"]
    used = min(c["n"], M)
    out = 2 if c["out"] == "bf16" else 4
    weight = h * o * (0.5 + 1 / BLOCK + 4 / (BLOCK * DQ_BLOCK))
    factors = 2 * used * r * (h + o)
    if c["op"] == "fwd":
        return {"bytes": weight + factors + 2 * M * h + out * M * o + 4 * M * r + 4 * M,
                "flops": 2 * M * h * o + 2 * M * r * (h + o)}
    grads = 4 * c["n"] * r * (h + o)
    return {"bytes": weight + factors + 2 * M * (h + o) + out * M * h + 4 * M * r + 4 * M + grads,
            "flops": 2 * M * h * o + 6 * M * r * (h + o)}


# ---------------------------------------------------------------- inputs

def _nf4():
    """Normal-quantile code values of the NF4 type (8 positive, 7 negative, an exact zero)."""
    d = statistics.NormalDist()
    top = ((1 - 1 / 30) + (1 - 1 / 32)) / 2
    pos = [d.inv_cdf(top + (0.5 - top) * i / 8) for i in range(8)]
    neg = [-d.inv_cdf(top + (0.5 - top) * i / 7) for i in range(7)]
    v = np.array(sorted(neg + [0.0] + pos))
    return torch.tensor((v / np.abs(v).max()).astype(np.float32))


def _quantized(h, o, g):
    """A frozen weight W^T[o][h] ~ N(0, 0.02) as packed codes and double-quantized constants."""
    q = _nf4().cuda()
    w = (torch.randn(o, h, device="cuda", generator=g) * 0.02).bfloat16().float().view(-1, BLOCK)
    c = w.abs().amax(1)
    code = torch.bucketize(w / c[:, None], (q[1:] + q[:-1]) / 2).to(torch.uint8).view(-1, 2)
    packed = (code[:, 0] << 4) | code[:, 1]
    mean = c.double().mean().float().view(1)
    d = (c - mean).view(-1, DQ_BLOCK)
    scale = d.abs().amax(1)
    fp8 = (d * (E4M3_MAX / scale)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)
    return {"codes": packed, "fp8": fp8, "scale": scale, "mean": mean, "codebook": q}


def _ids(c, seed):
    """The adapter of each token: `requests` are contiguous runs of ragged lengths, one or more to an
    adapter; `each` gives neighbouring tokens different adapters; `mixed` and `shuffled` have no order."""
    rng = np.random.default_rng(seed)
    M, n = c["M"], c["n"]
    if c["ids"] == "each":
        a = rng.permutation(n)[np.arange(M) % n]
    elif c["ids"] == "requests":
        cuts = np.sort(rng.choice(np.arange(1, M), size=min(n, M) - 1, replace=False)) if M > 1 else np.zeros(0, int)
        a = rng.permutation(n)[np.searchsorted(cuts, np.arange(M), side="right")]
    else:
        a = rng.integers(0, n, M)
    a = np.where(rng.random(M) < c["none"], -1, a)
    return torch.from_numpy(a.astype(np.int32)).cuda()


def _linear_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, h, o, n, r = c["M"], c["h"], c["o"], c["n"], c["r"]
    s = {"W": _quantized(h, o, g), "ids": _ids(c, seed),
         "X": torch.randn(M, h, device="cuda", generator=g).bfloat16(),
         "L1": (torch.randn(n, h, r, device="cuda", generator=g) * 0.01).bfloat16(),
         "L2": (torch.randn(n, r, o, device="cuda", generator=g) * 0.01).bfloat16(),
         "s": 16.0 / r * (0.5 + torch.rand(n, device="cuda", generator=g))}
    if c["op"] == "bwd":
        s["dY"] = torch.randn(M, o, device="cuda", generator=g).bfloat16()
        # T = X L1 of each token, kept by the forward
        T = torch.zeros(M, r, device="cuda")
        for a in range(n):
            rows = (s["ids"] == a).nonzero().view(-1)
            T[rows] = s["X"][rows].float() @ s["L1"][a].float()
        s["T"] = T
    return s


def _offsets(c):
    """Where each tensor starts in the flat state: every tensor starts a new block."""
    sizes = _tensor_sizes(c)
    starts = np.concatenate([[0], np.cumsum([-(-k // STATE_BLOCK) * STATE_BLOCK for k in sizes])])
    return sizes, [int(v) for v in starts]


def _adamw_inputs(c, seed):
    """Flat buffers whose views are the tensors; between two tensors up to a block of zeros."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    sizes, starts = _offsets(c)
    total = starts[-1]
    live = torch.zeros(total, device="cuda", dtype=torch.bool)
    for k, a in zip(sizes, starts):
        live[a:a + k] = True

    def normal(std):
        return torch.randn(total, device="cuda", generator=g).mul_(std).mul_(live)
    s = {"p": normal(0.02), "g": normal(1e-3)}
    s["copy"] = s["p"].bfloat16()
    if c["grad"] == "bf16":
        s["g"] = s["g"].bfloat16()
    m, v = normal(3e-4), normal(1e-3).square_().mul_(0.01)
    if c["bits"] == 32:
        return {**s, "m": m, "v": v}
    for name, x in (("m", m), ("v", v.sqrt_())):
        top = x.view(-1, STATE_BLOCK).abs().amax(1)
        s[name] = (x.view(-1, STATE_BLOCK) * (E4M3_MAX / top)[:, None]).to(torch.float8_e4m3fn).view(-1)
        s[name + "_scale"] = top / E4M3_MAX
    return s


def prepare(case, seed):
    c = case
    if c["op"] == "adamw":
        s = _adamw_inputs(c, seed)
        sizes, starts = _offsets(c)
        if own:
            from bit_nf4_quantized_blockwise_b200.multi_adamw import MultiAdamW
            from bit_nf4_quantized_blockwise_b200.paged import AdamWConfig

            def views(name):
                return [s[name][a:a + k] for k, a in zip(sizes, starts)]
            cfg = AdamWConfig(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, max_grad_norm=MAX_NORM)
            s["opt"] = MultiAdamW(views("p"), cfg, copies=views("copy"), state_bits=c["bits"])
            s["opt"].load_state({k: s[k] for k in ("m", "v", "m_scale", "v_scale") if k in s}, steps=STEPS_DONE)
            s["grads"] = views("g")
        else:
            s["steps"] = STEPS_DONE
        return {**s, "case": c}
    s = _linear_inputs(c, seed)
    if own:
        import bit_nf4_quantized_blockwise_b200 as q
        w = s["W"]
        s["Wq"] = q.NF4Weight(w["codes"], w["fp8"], w["scale"], w["mean"], c["o"], c["h"], tuple(w["codebook"].tolist()))
        s["bank"] = q.AdapterBank(s["L1"], s["L2"], s["s"])
        s["plan"] = q.qlora_adapter_plan(s["ids"], c["n"])
    return {**s, "case": c}


# ---------------------------------------------------------------- the operators, plain

def _weight(w, h, o):
    """W'^T[o][h] = bf16(q[code] c') as fp32 values."""
    c = w["fp8"].view(torch.float8_e4m3fn).float() * (w["scale"] / torch.full_like(w["scale"], E4M3_MAX)).repeat_interleave(DQ_BLOCK) + w["mean"]
    codes = torch.stack([w["codes"] >> 4, w["codes"] & 15], 1).view(-1).int()
    return (w["codebook"][codes].view(-1, BLOCK) * c[:, None]).bfloat16().float().view(o, h)


def _owner(s, c):
    """[M][n r]: s[a_i] in the columns of token i's adapter, 0 elsewhere."""
    hot = (s["ids"][:, None] == torch.arange(c["n"], device="cuda", dtype=torch.int32)) * s["s"]
    return hot.repeat_interleave(c["r"], 1)


def _wide(s, c):
    """The bank's factors side by side: L1 [h][n r], L2 [n r][o]."""
    return s["L1"].float().transpose(0, 1).reshape(c["h"], -1), s["L2"].float().reshape(-1, c["o"])


def _out(x, c):
    return x.bfloat16() if c["out"] == "bf16" else x


def _fwd(s, c):
    L1, L2 = _wide(s, c)
    X, hot = s["X"].float(), _owner(s, c)
    T = X @ L1
    Y = X @ _weight(s["W"], c["h"], c["o"]).t() + (T * hot) @ L2
    return {"Y": _out(Y, c), "T": (T * (hot != 0)).view(c["M"], c["n"], c["r"]).sum(1)}


def _bwd(s, c):
    L1, L2 = _wide(s, c)
    X, dY, hot = s["X"].float(), s["dY"].float(), _owner(s, c)
    U = (dY @ L2.t()) * hot
    dX = dY @ _weight(s["W"], c["h"], c["o"]) + U @ L1.t()
    dL2 = (s["T"].repeat(1, c["n"]) * hot).t() @ dY
    return {"dX": _out(dX, c), "dL1": (X.t() @ U).view(c["h"], c["n"], c["r"]).transpose(0, 1).contiguous(),
            "dL2": dL2.view(c["n"], c["r"], c["o"])}


def _encode(x, floor):
    """E4M3 codes and the scale of each block; floor: nothing above 0 becomes 0."""
    b = x.view(-1, STATE_BLOCK)
    top = b.abs().amax(1)
    live = top >= 2.0 ** -100
    inv = torch.where(live, torch.full_like(top, E4M3_MAX) / top, torch.zeros_like(top))
    y = b * inv[:, None]
    if floor:
        y = torch.where((y > 0) & (y < 2.0 ** -9), torch.full_like(y, 2.0 ** -9), y)
    scale = torch.where(live, top / torch.full_like(top, E4M3_MAX), torch.zeros_like(top))
    return y.to(torch.float8_e4m3fn).view(-1), scale


def _decode(code, scale):
    return (code.float().view(-1, STATE_BLOCK) * scale[:, None]).view(-1)


def _adamw(s, c):
    f = np.float32
    s["steps"] += 1
    t = s["steps"]
    step = float(f(float(f(LR)) / (1 - float(f(BETA1)) ** t)))
    root = torch.full((), float(f(math.sqrt(1 - float(f(BETA2)) ** t))), device="cuda")
    g = s["g"].float()
    norm = g.double().square_().sum().sqrt()
    g = g * (float(f(MAX_NORM)) / (norm + 1e-6)).float().clamp(max=1.0)
    eight = c["bits"] == 8
    m = _decode(s["m"], s["m_scale"]) if eight else s["m"]
    v = _decode(s["v"], s["v_scale"]).square() if eight else s["v"]
    m = m + (g - m) * float(f(1) - f(BETA1))
    v = v * float(f(BETA2)) + (g * g) * float(f(1) - f(BETA2))
    r = v.sqrt()
    p = s["p"] * float(f(1) - f(LR) * f(DECAY)) - (m / (r / root + float(f(EPS)))) * step
    s["p"], s["copy"] = p, p.bfloat16()
    if eight:
        (s["m"], s["m_scale"]), (s["v"], s["v_scale"]) = _encode(m, False), _encode(r, True)
    else:
        s["m"], s["v"] = m, v
    return {k: s[k] for k in ("p", "copy", "m", "v", "m_scale", "v_scale") if k in s}


# ---------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"fwd": _fwd, "bwd": _bwd, "adamw": _adamw}[c["op"]](s, c)
    if c["op"] == "adamw":
        opt = s["opt"]
        opt.step(s["grads"])
        out = {"p": s["p"], "copy": s["copy"], "m": opt.m, "v": opt.v}
        if c["bits"] == 8:
            out.update(m_scale=opt.m_scale, v_scale=opt.v_scale)
        return out
    import bit_nf4_quantized_blockwise_b200 as q
    dt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
    if c["op"] == "fwd":
        Y, T = q.qlora_multi_linear_fwd(s["Wq"], s["X"], s["bank"], s["plan"], y_dtype=dt)
        return {"Y": Y, "T": T}
    dX, dL1, dL2 = q.qlora_multi_linear_bwd(s["Wq"], s["X"], s["dY"], s["bank"], s["plan"], T_saved=s["T"], dx_dtype=dt)
    return {"dX": dX, "dL1": dL1, "dL2": dL2}


# ---------------------------------------------------------------- 64 bits

def _exact_weight(w, h, o):
    """The bf16 weights that the codes stand for: the product q c' is rounded to fp32 and then to
    bf16 by definition (c' likewise has fp32 steps), so these are whole steps, not sums."""
    nb = h * o // BLOCK
    e = w["fp8"].view(torch.float8_e4m3fn).double()
    step = (w["scale"].double() / E4M3_MAX).float().double()
    c = ((e * step[torch.arange(nb, device="cuda") // DQ_BLOCK]).float().double() + w["mean"].double()).float().double()
    out = torch.empty(o * h, device="cuda", dtype=torch.float64)
    for half, code in ((0, w["codes"] // 16), (1, w["codes"] % 16)):
        at = torch.arange(half, o * h, 2, device="cuda")
        out[at] = (w["codebook"].double()[code.long()] * c[at // BLOCK]).float().bfloat16().double()
    return out.view(o, h)


def exact(case, seed):
    c = case
    if c["op"] == "adamw":
        return _exact_adamw(c, seed)
    s = _linear_inputs(c, seed)
    W = _exact_weight(s["W"], c["h"], c["o"])
    X, ids = s["X"].double(), s["ids"]
    if c["op"] == "fwd":
        Y, T = X @ W.t(), torch.zeros(c["M"], c["r"], device="cuda", dtype=torch.float64)
        for a in ids.unique().tolist():
            if a >= 0:
                at = (ids == a).nonzero().view(-1)
                T[at] = X[at] @ s["L1"][a].double()
                Y[at] += float(s["s"][a]) * (T[at] @ s["L2"][a].double())
        return {"Y": Y, "T": T}
    dY = s["dY"].double()
    dX = dY @ W
    dL1 = torch.zeros(c["n"], c["h"], c["r"], device="cuda", dtype=torch.float64)
    dL2 = torch.zeros(c["n"], c["r"], c["o"], device="cuda", dtype=torch.float64)
    for a in ids.unique().tolist():
        if a >= 0:
            at = (ids == a).nonzero().view(-1)
            U = float(s["s"][a]) * (dY[at] @ s["L2"][a].double().t())
            dX[at] += U @ s["L1"][a].double().t()
            dL1[a] = X[at].t() @ U
            dL2[a] = float(s["s"][a]) * (s["T"][at].double().t() @ dY[at])
    return {"dX": dX, "dL1": dL1, "dL2": dL2}


def _exact_adamw(c, seed):
    """Codes have no value in 64 bits (a code next to a border goes by the last bit of the fp32
    value that is stored), so only the scales, the parameters and 32-bit states are given."""
    s = _adamw_inputs(c, seed)
    f = lambda x: float(np.float32(x))  # noqa: E731  the hyper-parameters are fp32 values
    t = STEPS_DONE + 1
    g = s["g"].double()
    g = g * min(1.0, f(MAX_NORM) / (float(g.norm()) + 1e-6))
    if c["bits"] == 8:
        m = s["m"].double() * s["m_scale"].double().repeat_interleave(STATE_BLOCK)
        v = (s["v"].double() * s["v_scale"].double().repeat_interleave(STATE_BLOCK)) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = f(BETA1) * m + (1 - f(BETA1)) * g
    v = f(BETA2) * v + (1 - f(BETA2)) * g ** 2
    p = s["p"].double() * (1 - f(LR) * f(DECAY))
    p -= f(LR) / (1 - f(BETA1) ** t) * m / (v.sqrt() / math.sqrt(1 - f(BETA2) ** t) + f(EPS))
    out = {"p": p, "copy": p}
    if c["bits"] == 32:
        return {**out, "m": m, "v": v}
    peaks = [x.view(-1, STATE_BLOCK).abs().amax(1) / E4M3_MAX for x in (m, v.sqrt())]
    return {**out, "m": None, "v": None, "m_scale": peaks[0], "v_scale": peaks[1]}
