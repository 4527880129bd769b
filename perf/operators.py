"""The operators at the two ends of a language model whose token table this
library holds, each as a user calls it and in a plain form of elementary torch
operations:

  lookup   rows of a dense table for token ids, scaled, and the gradient of
           the table summed by sorted tokens
  norm     layer norm over the last axis, forward and backward
  xent     softmax cross entropy of hidden rows against a large vocabulary,
           without keeping the logits: scores, or scores with both gradients
  adamw    one AdamW step over many tensors, states in 32 or in 8 bits

A case names its operator in "op".  ``own`` selects the library's kernels.
"""

import math

import torch

own = False
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
IGNORE = -100
BLOCK = 256       # elements that share one scale of an 8-bit state
M_TOP, V_TOP = 448.0, 57344.0  # largest values of e4m3 and e5m2
TINY = 2.0 ** -100             # least block maximum that a scale is made from
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
LN_EPS = 1e-5


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of sixteen sequences: a launch and sixteen rows
        {"name": "lookup_decode", "op": "lookup", "train": False, "n": 16, "V": 131072, "D": 4096, "type": "bf16",
         "scale": 64.0, "pad": -1, "add": False, "gap": 0, "zipf": 1.05},
        # the 10^6-row, 64-column table with 32768 Zipf(1.05) lookups, kept
        # dense; its gradient is added to the one the output layer left
        {"name": "lookup_rows", "op": "lookup", "train": True, "n": 32768, "V": 1000000, "D": 64, "type": "f32",
         "scale": 8.0, "pad": -1, "add": True, "gap": 0, "zipf": 1.05},
        # a training batch of 65536 tokens, every row of the gradient written
        {"name": "lookup_tokens", "op": "lookup", "train": True, "n": 65536, "V": 131072, "D": 1024, "type": "bf16",
         "scale": 32.0, "pad": 0, "add": False, "gap": 0, "zipf": 1.05},
        # the norm before the output layer while decoding
        {"name": "norm_decode", "op": "norm", "train": False, "n": 4, "D": 4096, "type": "bf16", "beta": True, "gap": 0},
        # pooled 128-column bags of a batch of 32768, in the library's own fp32
        {"name": "norm_bags", "op": "norm", "train": True, "n": 32768, "D": 128, "type": "f32", "beta": True, "gap": 0},
        # a training batch of 16384 tokens of a wide model
        {"name": "norm_tokens", "op": "norm", "train": True, "n": 16384, "D": 4096, "type": "bf16", "beta": True, "gap": 0},
        # scoring the next token of a few sequences: the table is read once
        {"name": "xent_score", "op": "xent", "train": False, "n": 5, "V": 131072, "D": 4096, "type": "bf16",
         "ignored": 0.0, "gap": 0},
        # next-item loss over a catalogue of 10^6 rows of 128 columns, fp32
        {"name": "xent_catalogue", "op": "xent", "train": True, "n": 2048, "V": 1000000, "D": 128, "type": "f32",
         "ignored": 0.0, "gap": 0},
        # the loss of a training batch of 8192 tokens, prompt tokens ignored
        {"name": "xent_tokens", "op": "xent", "train": True, "n": 8192, "V": 131072, "D": 4096, "type": "bf16",
         "ignored": 0.1, "gap": 0},
        # the three cores of the 1000-row table: the launch is what counts
        {"name": "adamw_table", "op": "adamw", "bits": 32, "kind": "table", "copy": False, "step": 1},
        # all 78 cores of 26 tables of ranks 16, 32 and 64
        {"name": "adamw_cores", "op": "adamw", "bits": 32, "kind": "cores", "copy": False, "step": 100},
        # a dense 131072 x 1024 table beside the cores, bf16 gradients, states
        # in 8 bits, and the bf16 copy that the next forward reads
        {"name": "adamw_bytes", "op": "adamw", "bits": 8, "kind": "model", "copy": True, "step": 1000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "norm", "xent", "adamw"])
    t = rng.choice(["f32", "bf16", "f16"])
    if op == "lookup":
        n, V, D = _log(rng, 1, 65536), _log(rng, 500, 1000000), _log(rng, 8, 4096)
        V = max(16, min(V, 134217728 // D))
        n = max(1, min(n, 67108864 // D))
        return {"op": op, "train": rng.random() < 0.7, "n": n, "V": V, "D": D, "type": t,
                "scale": rng.choice([1.0, math.sqrt(D)]), "pad": rng.choice([-1, 0]), "add": rng.random() < 0.5,
                "gap": rng.choice([0, 0, 5, 64]), "zipf": round(rng.uniform(0.8, 1.3), 3)}
    if op == "norm":
        D = _log(rng, 16, 8192)
        return {"op": op, "train": rng.random() < 0.7, "n": _log(rng, 1, min(65536, 67108864 // D)), "D": D, "type": t,
                "beta": rng.random() < 0.7, "gap": rng.choice([0, 0, 3, 32])}
    if op == "xent":
        n, V, D = _log(rng, 1, 8192), _log(rng, 1000, 1000000), _log(rng, 16, 4096)
        V = max(500, min(V, 536870912 // D, 1073741824 // n))
        return {"op": op, "train": rng.random() < 0.7, "n": n, "V": V, "D": D, "type": rng.choice(["f32", "bf16"]),
                "ignored": rng.choice([0.0, 0.1]), "gap": rng.choice([0, 0, 1, 64])}
    return {"op": op, "bits": rng.choice([32, 8]), "kind": "drawn", "count": _log(rng, 1, 150),
            "largest": _log(rng, 300, 1000000), "sizes": rng.randrange(1 << 30), "copy": rng.random() < 0.5,
            "step": _log(rng, 1, 10000)}


def _shapes(case):
    """Shapes of the tensors of an adamw case."""
    import numpy as np

    def core(n, R):
        return [(n, 1, 4, R), (n, R, 4, R), (n, R, 4, 1)]

    if case["kind"] == "table":
        return [(10, 1, 2, 8), (10, 8, 2, 8), (10, 8, 4, 1)]
    g = np.random.default_rng(case.get("sizes", 20264))
    if case["kind"] == "drawn":
        s = np.exp(g.uniform(0.0, math.log(case["largest"]), case["count"])).astype(int)
        return [(max(1, int(x)),) for x in s]
    out = []
    for _ in range(26):
        out += core(int(math.ceil(math.exp(g.uniform(math.log(1e3), math.log(4e7))) ** (1 / 3))),
                    int((16, 32, 64)[int(g.integers(0, 3))]))
    return out + [(131072, 1024), (1024,), (1024,)] if case["kind"] == "model" else out


def _numel(shape):
    return int(math.prod(shape))


def _places(case):
    """(shape, first element) of every tensor in a flat buffer where each one
    begins at a multiple of BLOCK elements, and the buffer's length."""
    at, got = 0, []
    for s in _shapes(case):
        got.append((s, at))
        at += -(-_numel(s) // BLOCK) * BLOCK
    return got, at


# ------------------------------------------------------------------ inputs

def _rows(g, n, D, dtype, gap, std=1.0):
    """[n, D] values, the rows `gap` elements further apart than D."""
    x = torch.empty((n, D + gap), device=DEV, dtype=torch.float32).normal_(0.0, std, generator=g)
    return x.to(dtype)[:, :D]


def _zipf(g, n, V, alpha):
    """n ids of 0..V-1, the k-th most frequent with weight k^-alpha, frequent
    ids scattered over the range."""
    w = torch.arange(1, V + 1, device=DEV, dtype=torch.float64).pow_(-alpha).cumsum_(0)
    u = torch.rand(n, device=DEV, dtype=torch.float64, generator=g) * w[-1]
    k = torch.searchsorted(w, u).clamp_(max=V - 1)
    return (k * 7919 + 12345) % V


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    tt = None
    if own:
        import tensor_train_compressed_gather_amd as tt
    if op == "lookup":
        t = TYPES[case["type"]]
        n, V, D = case["n"], case["V"], case["D"]
        s["weight"] = _rows(g, V, D, t, 0, 0.02)
        s["tokens"] = _zipf(g, n, V, case["zipf"])
        if case["pad"] >= 0:
            s["tokens"][torch.rand(n, device=DEV, generator=g) < 0.1] = case["pad"]
        if case["train"]:
            s["grad"] = _rows(g, n, D, t, case["gap"])
            s["grad_weight"] = _rows(g, V, D, t, 0) if case["add"] else None
        if own:
            s["call"] = tt.TokenEmbedding(V, D, scale=case["scale"], padding_idx=case["pad"], device=DEV)
    elif op == "norm":
        t = TYPES[case["type"]]
        n, D = case["n"], case["D"]
        s["x"] = _rows(g, n, D, t, case["gap"], 2.0)
        s["x"] += torch.randn((n, 1), device=DEV, generator=g).to(t)
        s["gamma"] = 1 + 0.1 * torch.randn(D, device=DEV, generator=g)
        s["beta"] = 0.1 * torch.randn(D, device=DEV, generator=g) if case["beta"] else None
        if case["train"]:
            s["grad"] = _rows(g, n, D, t, case["gap"])
        if own:
            s["call"] = tt.LayerNorm(D, eps=LN_EPS, device=DEV)
    elif op == "xent":
        t = TYPES[case["type"]]
        n, V, D = case["n"], case["V"], case["D"]
        w = torch.empty((V, D), device=DEV).normal_(0.0, 1.5 / math.sqrt(D), generator=g)
        target = _zipf(g, n, V, 1.05)
        wt = w[target]
        # hidden rows after a norm; the target's logit is raised by up to 12
        h = torch.randn((n, D + case["gap"]), device=DEV, generator=g)
        h[:, :D] += wt * (12 * torch.rand((n, 1), device=DEV, generator=g) / wt.square().sum(1, keepdim=True))
        s["hidden"], s["weight"] = h.to(t)[:, :D], w.to(t)
        if case["ignored"]:
            target[torch.rand(n, device=DEV, generator=g) < case["ignored"]] = IGNORE
        s["target"] = target
        if case["train"]:  # the mean over the rows that count
            s["grad"] = torch.ones(n, device=DEV) / (target != IGNORE).sum().clamp(min=1)
        if own:
            s["call"] = tt.VocabCrossEntropy(V, D, ignore_index=IGNORE, device=DEV)
    else:
        places, length = _places(case)
        real = torch.zeros(length, dtype=torch.bool, device=DEV)
        for shape, at in places:
            real[at:at + _numel(shape)] = True
        flat = lambda std: torch.empty(length, device=DEV).normal_(0.0, std, generator=g) * real  # noqa: E731
        size = torch.exp2(torch.empty(length, device=DEV).uniform_(-12.0, 0.0, generator=g))
        s["p"], s["g"] = flat(0.05), (flat(1e-2) * size).to(torch.bfloat16 if case["copy"] else torch.float32)
        s["m"], s["v"] = flat(4e-3) * size, (flat(1e-2) * size).square()
        s["copy"] = s["p"].to(torch.bfloat16) if case["copy"] else None
        s["step"], s["seed"] = case["step"], int(seed) % 65521
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _pack(s["m"], 0, torch.float8_e4m3fn)
            s["v"], s["v_scale"] = _pack(s["v"], 0, torch.float8_e5m2)
        if own:
            cut = lambda b: None if b is None else [b[at:at + _numel(sh)].view(sh) for sh, at in places]  # noqa: E731
            s["call"] = tt.AdamW(cut(s["p"]), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                                 state_bits=case["bits"], copies=cut(s["copy"]), seed=s["seed"])
            s["grads"] = cut(s["g"])
            if case["bits"] == 8:
                s["call"].load_state(s["m"], s["v"], s["step"] - 1, s["m_scale"], s["v_scale"])
            else:
                s["call"].load_state(s["m"], s["v"], s["step"] - 1)
    return s


# --------------------------------------------------------- 8-bit AdamW states

def _noise(length, key):
    """16 + 16 random bits of every element: a 32-bit finaliser (two rounds of
    multiply and shift) of the element's number and the step's key."""
    m32 = 0xFFFFFFFF
    h = torch.arange(length, device=DEV, dtype=torch.int64)
    h = ((h & m32) ^ key) & m32
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & m32
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & m32
    h = h ^ (h >> 16)
    return h & 0xFFFF, h >> 16


def _key(seed, step):
    return ((seed * 0x9E3779B1) ^ (step * 0x85EBCA77)) & 0xFFFFFFFF


def _pack(x, noise, kind):
    """8-bit codes and the scale of every block of BLOCK elements.  `noise`:
    16 bits that decide which of the two neighbours a value goes to, in
    proportion to its distance (0: always towards zero)."""
    e4 = kind == torch.float8_e4m3fn
    top, drop, low, bias, last = (M_TOP, 20, -6, 120 << 3, 0x7E) if e4 else (V_TOP, 21, -14, 112 << 2, 0x7B)
    step = low - (23 - drop)  # log2 of the distance of the smallest values
    b = x.view(-1, BLOCK)
    scale = torch.maximum(b.abs().amax(1), torch.tensor(TINY, dtype=x.dtype, device=DEV)) / top
    a = (b.abs() * (1.0 / scale)[:, None]).reshape(-1)
    small = torch.floor(a * 2.0 ** -step + noise * 2.0 ** -16)
    bits = a.float().view(torch.int32).to(torch.int64)
    if a.dtype == torch.float64:  # the fraction that 32 bits do not hold
        bits = bits + torch.where(a.float() > a, -1, 0)
    code = ((bits + noise * (1 << (drop - 16))) >> drop) - bias
    code = torch.where(a < 2.0 ** low, torch.nan_to_num(small).to(torch.int64), code).clamp(max=last)
    if not e4:  # a second moment that is not zero is not stored as zero
        code = torch.where((code == 0) & (a > 0), 1, code)
    code = torch.where(a.isnan(), 0x7F, code)
    code = code + 128 * (x < 0)
    return code.to(torch.uint8).view(kind), scale


def _unpack(code, scale):
    return (code.to(scale.dtype).view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw(p, g, m, v, step):
    """One step of AdamW in the type of its inputs."""
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * (1.0 - BETA2)) * g
    root = 1.0 / math.sqrt(1.0 - BETA2 ** step)
    size = LR / (1.0 - BETA1 ** step)
    p = p * (1.0 - LR * DECAY) - (m * size) / (v.sqrt() * root + EPS)
    return p, m, v


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        call = s["call"]
        if op == "lookup":
            out = call.forward(s["weight"], s["tokens"])
            if not case["train"]:
                return out
            return out, call.backward(s["grad"], s["tokens"], grad_weight=s["grad_weight"], accumulate=case["add"])
        if op == "norm":
            y, mean, rstd = call.forward(s["x"], s["gamma"], s["beta"])
            if not case["train"]:
                return y, mean, rstd
            dx, dgamma, dbeta = call.backward(s["grad"], s["x"], s["gamma"], mean, rstd)
            return y, dx, dgamma, dbeta
        if op == "xent":
            if not case["train"]:
                return call.forward(s["hidden"], s["weight"], s["target"])
            return call.loss_and_grad(s["hidden"], s["weight"], s["target"], s["grad"])
        call.step(s["grads"])
        got = {"p": s["p"], "m": call.exp_avg, "v": call.exp_avg_sq}
        if case["bits"] == 8:
            got["m_scale"], got["v_scale"] = call.exp_avg_scale, call.exp_avg_sq_scale
        if case["copy"]:
            got["copy"] = s["copy"]
        return got
    if op == "lookup":
        t = s["weight"].dtype
        out = (s["weight"][s["tokens"]].float() * case["scale"]).to(t)
        if not case["train"]:
            return out
        dw = torch.zeros(s["weight"].shape, dtype=torch.float32, device=DEV)
        counts = (s["tokens"] != case["pad"])[:, None]
        dw.index_add_(0, s["tokens"], s["grad"].float() * counts)
        dw = dw * case["scale"]
        if case["add"]:
            return out, s["grad_weight"].copy_(s["grad_weight"].float() + dw)
        return out, dw.to(t)
    if op == "norm":
        t = s["x"].dtype
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        c = x - mean
        rstd = (c.square().mean(1, keepdim=True) + LN_EPS).rsqrt()
        xhat = c * rstd
        y = xhat * s["gamma"]
        if s["beta"] is not None:
            y = y + s["beta"]
        if not case["train"]:
            return y.to(t), mean[:, 0], rstd[:, 0]
        dy = s["grad"].float()
        a = dy * s["gamma"]
        dx = (a - a.mean(1, keepdim=True) - xhat * (a * xhat).mean(1, keepdim=True)) * rstd
        return y.to(t), dx.to(t), (dy * xhat).sum(0), dy.sum(0)
    if op == "xent":
        h, w, target = s["hidden"].float(), s["weight"].float(), s["target"]
        counts = target != IGNORE
        at = torch.where(counts, target, 0)[:, None]
        logits = h @ w.t()
        top = logits.amax(1, keepdim=True)
        lse = ((logits - top).exp().sum(1, keepdim=True)).log() + top
        loss = torch.where(counts, (lse - logits.gather(1, at))[:, 0], 0.0)
        if not case["train"]:
            return loss, lse[:, 0]
        d = (logits - lse).exp_()
        d.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
        d *= torch.where(counts, s["grad"], 0.0)[:, None]
        dw = (d.t() @ h).to(s["weight"].dtype)
        if case["type"] == "f32":  # a sum over up to 10^6 rows: 32 bits would lose 2e-5 of it
            d, w = d.double(), w.double()
        return loss, lse[:, 0], (d @ w).to(s["hidden"].dtype), dw
    step = s["step"]
    s["step"] += 1
    if case["bits"] == 8:
        m, v = _unpack(s["m"], s["m_scale"]), _unpack(s["v"], s["v_scale"])
    else:
        m, v = s["m"], s["v"]
    p, m, v = _adamw(s["p"], s["g"].float(), m, v, step)
    s["p"].copy_(p)
    got = {"p": s["p"]}
    if case["copy"]:
        got["copy"] = s["copy"].copy_(p)
    if case["bits"] == 8:
        low, high = _noise(p.numel(), _key(s["seed"], step))
        s["m"], s["m_scale"] = _pack(m, low, torch.float8_e4m3fn)
        s["v"], s["v_scale"] = _pack(v, high, torch.float8_e5m2)
        got["m_scale"], got["v_scale"] = s["m_scale"], s["v_scale"]
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    got["m"], got["v"] = s["m"], s["v"]
    return got


# -------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "lookup":
        tok = s["tokens"]
        out = s["weight"][tok].to(f64).mul_(case["scale"])
        if not case["train"]:
            return out
        total = torch.zeros(s["weight"].shape, dtype=f64, device=DEV)
        keep = tok != case["pad"]
        total.index_put_((tok[keep],), s["grad"][keep].to(f64).mul_(case["scale"]), accumulate=True)
        return out, total.add_(s["grad_weight"].to(f64)) if case["add"] else total
    if op == "norm":
        x = s["x"].to(f64)
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1.0 / torch.sqrt(var + LN_EPS)
        xhat = (x - mean[:, None]) * rstd[:, None]
        y = xhat * s["gamma"].to(f64) + (0.0 if s["beta"] is None else s["beta"].to(f64))
        if not case["train"]:
            return y, mean, rstd
        dy = s["grad"].to(f64)
        n, D = x.shape
        along = dy * s["gamma"].to(f64)
        # the norm's Jacobian: rstd (I - 1 1'/D - xhat xhat'/D)
        dx = rstd[:, None] * (along - along.sum(1, keepdim=True) / D
                              - xhat * torch.einsum("nd,nd->n", along, xhat)[:, None] / D)
        return y, dx, torch.einsum("nd,nd->d", dy, xhat), torch.einsum("nd->d", dy)
    if op == "xent":
        n, V = case["n"], case["V"]
        w, h = s["weight"].to(f64), s["hidden"].to(f64)
        loss, lse = torch.zeros(n, dtype=f64, device=DEV), torch.zeros(n, dtype=f64, device=DEV)
        dh = torch.zeros_like(h)
        dw = torch.zeros_like(w) if case["train"] else None
        rows = max(1, 268435456 // V)
        for i in range(0, n, rows):
            z = h[i:i + rows] @ w.t()
            lse[i:i + rows] = torch.logsumexp(z, 1)
            t = s["target"][i:i + rows]
            j = torch.nonzero(t != IGNORE)[:, 0]
            loss[i + j] = lse[i + j] - z[j, t[j]]
            if case["train"]:
                z = torch.softmax(z, 1)
                z[j, t[j]] -= 1.0
                z *= (s["grad"][i:i + rows].to(f64) * (t != IGNORE))[:, None]
                dh[i:i + rows] = z @ w
                dw += z.t() @ h[i:i + rows]
            del z
        return (loss, lse, dh, dw) if case["train"] else (loss, lse)
    p, g, step = s["p"].to(f64), s["g"].to(f64), s["step"]
    if case["bits"] == 8:
        m, v = _unpack(s["m"], s["m_scale"].to(f64)), _unpack(s["v"], s["v_scale"].to(f64))
    else:
        m, v = s["m"].to(f64), s["v"].to(f64)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    mhat, vhat = m / (1 - BETA1 ** step), v / (1 - BETA2 ** step)
    p = p - LR * (mhat / (torch.sqrt(vhat) + EPS) + DECAY * p)
    got = {"p": p}
    if case["copy"]:
        got["copy"] = p
    if case["bits"] == 8:
        low, high = _noise(p.numel(), _key(s["seed"], step))
        (qm, got["m_scale"]), (qv, got["v_scale"]) = _pack(m, low, torch.float8_e4m3fn), _pack(v, high, torch.float8_e5m2)
        got["m"], got["v"] = qm.to(f64), qv.to(f64)
    else:
        got["m"], got["v"] = m, v
    return got


# -------------------------------------------------------------------- work

def work(case):
    """Bytes that have to be read and written once, and operations."""
    op = case["op"]
    size = 2 if case.get("type") in ("bf16", "f16") else 4
    if op == "lookup":
        n, V, D = case["n"], case["V"], case["D"]
        rows = min(n, V)
        b = 8 * n + (rows + n) * D * size
        if case["train"]:
            b += 8 * n + n * D * size + (2 * rows if case["add"] else V) * D * size
        return {"bytes": b, "flops": n * D * (3 if case["train"] else 1)}
    if op == "norm":
        e = case["n"] * case["D"]
        b = 2 * e * size + 8 * case["n"] + 8 * case["D"]
        if case["train"]:
            b += 3 * e * size + 8 * case["n"] + 12 * case["D"]
        return {"bytes": b, "flops": e * (20 if case["train"] else 8)}
    if op == "xent":
        n, V, D = case["n"], case["V"], case["D"]
        b = (n + V) * D * size + 16 * n
        if case["train"]:
            b += (n + V) * D * size + 4 * n
        return {"bytes": b, "flops": 2.0 * n * V * D * (3 if case["train"] else 1)}
    count = sum(_numel(x) for x in _shapes(case))
    b = 8 + (2 if case["copy"] else 4) + (2 if case["copy"] else 0) + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
    return {"bytes": count * b, "flops": count * 14}
