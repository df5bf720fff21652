"""Workloads of the expert-path operators, with their plain forms.

Five operators: FP4 quantisation of rows (with the values read back), the
grouped product of two FP4 operands, tokens sorted by expert (sort, gather and
the gather's gradient), and tokens brought back with their gates (weighted sum
and its gradients).  ``run`` makes one pass through an operator: the plain form
in elementary torch operations where ``own`` is false, the library's calls
where it is true.  ``exact`` gives the same outputs from the definitions in
64 bits, written apart from the plain forms.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's activations before an FP4 product: 8 tokens of a 2048-wide layer
        dict(name="quantise decode", op="quantise", fmt="mxfp4", dtype="bf16", groups=8, rows=1, K=2048),
        # prefill activations, one fp32 scale per token
        dict(name="quantise prefill", op="quantise", fmt="nvfp4", dtype="bf16", groups=8192, rows=1, K=4096),
        # checkpoint conversion: the gate matrices of 64 experts, one fp32 scale per matrix
        dict(name="quantise experts", op="quantise", fmt="nvfp4", dtype="bf16", groups=64, rows=1024, K=2048),
        # one token through a dense FP4 projection (weights streamed once)
        dict(name="product dense decode", op="product", fmt="mxfp4", out="bf16", E=1, rows=1, tail=0, N=4096, K=4096),
        # 32 tokens x 8 experts of 64: gate and up in one matrix, a few rows per expert
        dict(name="product grouped decode", op="product", fmt="nvfp4", out="bf16", E=64, rows=256, tail=0, N=2048,
             K=2048),
        # 2048 tokens x 8 experts of 128, ragged segments of about 128 rows
        dict(name="product grouped prefill", op="product", fmt="nvfp4", out="bf16", E=128, rows=16384, tail=0,
             N=1536, K=2048),
        # a dense FP4 projection of a prefill batch, fp32 result
        dict(name="product dense prefill", op="product", fmt="mxfp4", out="f32", E=1, rows=8192, tail=0, N=4096,
             K=4096),
        # decode: 8 tokens, 8 experts each
        dict(name="dispatch decode", op="dispatch", train=False, dtype="bf16", T=8, k=8, E=64, sinks=0, H=2048),
        # prefill with 512 experts and two sink targets, whose pairs are dropped
        dict(name="dispatch prefill", op="dispatch", train=False, dtype="bf16", T=8192, k=10, E=512, sinks=2, H=4096),
        # a training step's gather and its gradient, odd token count and width
        dict(name="dispatch train", op="dispatch", train=True, dtype="f32", T=2047, k=6, E=256, sinks=0, H=2047),
        # decode: 33 tokens (a ragged batch) brought back with their gates
        dict(name="combine decode", op="combine", train=False, dtype="bf16", T=33, k=8, E=64, sinks=0, H=2048),
        # a training step's weighted sum and its gradients
        dict(name="combine train", op="combine", train=True, dtype="bf16", T=8192, k=8, E=128, sinks=0, H=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "product", "dispatch", "combine"])
    if op == "quantise":
        K = 32 * _log(rng, 1, 224)
        if rng.random() < 0.5:                              # activations: a scale per row
            groups, rows = _log(rng, 1, 16384), 1
        else:                                               # weights: a scale per matrix
            groups, rows = _log(rng, 1, 64), _log(rng, 1, 2048)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        while groups * rows * K * BYTES[dtype] > 64 * 1024 * 2048 * 2:
            groups = (groups + 1) // 2
        return dict(op=op, fmt=rng.choice(["mxfp4", "nvfp4"]), dtype=dtype, groups=groups, rows=rows, K=K)
    if op == "product":
        E = 1 if rng.random() < 0.4 else _log(rng, 2, 256)
        N, K, rows = _log(rng, 64, 4096), 32 * _log(rng, 4, 128), _log(rng, 1, 8192)
        while E * N * K > 128 * 1536 * 2048:
            E = (E + 1) // 2
        return dict(op=op, fmt=rng.choice(["mxfp4", "nvfp4"]), out=rng.choice(["bf16", "bf16", "f16", "f32"]), E=E,
                    rows=rows, tail=rng.choice([0, 0, 1, 7]) if rows > 8 else 0, N=N, K=K)
    T, k, E = _log(rng, 1, 8192), rng.randint(1, 10), _log(rng, 10, 512)
    H = _log(rng, 64, 4096)
    H = H if rng.random() < 0.25 else -(-H // 64) * 64
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    while T * k * H * BYTES[dtype] > 8192 * 8 * 2048 * 2:
        T = (T + 1) // 2
    return dict(op=op, train=rng.random() < 0.5, dtype=dtype, T=T, k=k, E=E,
                sinks=rng.choice([0, 0, 1, 2]) if T > 8 else 0, H=H)


def work(case):
    c = case
    if c["op"] == "quantise":
        n = c["groups"] * c["rows"] * c["K"]
        q = n / 2 + n / BLOCK[c["fmt"]] + (4 * c["groups"] if c["fmt"] == "nvfp4" else 0)
        return {"bytes": n * BYTES[c["dtype"]] + q + n * BYTES[c["dtype"]], "flops": 0}
    if c["op"] == "product":
        per = 0.5 + 1 / BLOCK[c["fmt"]]
        active = c["E"] * (1 - (1 - 1 / c["E"]) ** c["rows"]) if c["E"] > 1 else 1
        return {"bytes": c["rows"] * c["K"] * per + active * c["N"] * c["K"] * per
                + c["rows"] * c["N"] * BYTES[c["out"]], "flops": 2 * c["rows"] * c["N"] * c["K"]}
    pairs, row = c["T"] * c["k"], c["H"] * BYTES[c["dtype"]]
    if c["op"] == "dispatch":
        b = pairs * 4 * 3 + (c["T"] + pairs) * row
        return {"bytes": b + ((c["T"] + pairs) * row if c["train"] else 0), "flops": 0}
    b = pairs * 8 + (c["T"] + pairs) * row
    return {"bytes": b + (c["T"] * row + 2 * pairs * row + pairs * 4 if c["train"] else 0),
            "flops": 2 * pairs * c["H"] * (3 if c["train"] else 1)}


# -------------------------------------------------------------------- inputs
def _activations(shape, g):
    """Hidden states: a normal bulk with a few channels that are much larger."""
    x = torch.randn(shape, generator=g, device="cuda")
    c = torch.rand(shape[-1], generator=g, device="cuda")
    return x * torch.where(c > 0.99, 20.0, 1.0)


def _ids(T, k, n, g):
    """k different targets of n for each token, the lower ones a little more often."""
    score = torch.rand((T, n), generator=g, device="cuda") - 0.2 * torch.arange(n, device="cuda") / n
    return score.topk(k, dim=1).indices.to(torch.int32)


def _quantised(x, fmt, rows):
    """Codes, block scales and matrix scales of x [n, K] in the checkpoint layout (plain form)."""
    n, K = x.shape
    v = x.float().view(n, K // BLOCK[fmt], BLOCK[fmt])
    amax = v.abs().amax(2)
    if fmt == "mxfp4":
        e = (amax.view(torch.int32) >> 23) - 127 - 2
        code = torch.where(amax > 0, (e + 127).clamp(1, 254), torch.ones_like(e))
        q = v * ((254 - code) << 23).view(torch.float32).unsqueeze(2)
        scales, G = code.to(torch.uint8), None
    else:
        top = amax.view(n // rows, -1).amax(1)
        m, e = torch.frexp(top.double() / 2688)
        e = (e - (m == 0.5).int()).clamp(min=-100)
        G = torch.where(top > 0, ((e + 127) << 23).view(torch.float32), torch.ones_like(top))
        per_row = G.repeat_interleave(rows).unsqueeze(1)
        s8 = (amax / (6 * per_row)).to(torch.float8_e4m3fn)
        d = s8.float() * per_row
        q = torch.where(d.unsqueeze(2) > 0, v / d.unsqueeze(2), torch.zeros_like(v))
        scales = s8.view(torch.uint8)
    a = q.abs()
    idx = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    idx = (idx + 8 * (q < 0)).to(torch.uint8).view(n, K // 2, 2)
    return idx[..., 0] | (idx[..., 1] << 4), scales, G


def _values(codes, scales, G, fmt, rows):
    """What the codes stand for, fp32 [n, K] (plain form)."""
    codes, scales = codes.flatten(0, -2), scales.flatten(0, -2)
    n, half = codes.shape
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], 2).int()].view(n, -1, BLOCK[fmt])
    if fmt == "mxfp4":
        s = (scales.to(torch.int32) << 23).view(torch.float32)
    else:
        s = scales.view(torch.float8_e4m3fn).float() * G.repeat_interleave(rows).unsqueeze(1)
    return (v * s.unsqueeze(2)).view(n, 2 * half)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "quantise":
        x = _activations((c["groups"] * c["rows"], c["K"]), g)
        if c["rows"] > 1:
            x = x * 0.02
        s["x"] = x.to(DTYPES[c["dtype"]])
    elif c["op"] == "product":
        n, E = c["rows"], c["E"]
        s["x"] = _quantised(_activations((n, c["K"]), g), c["fmt"], 1)
        w = [torch.randn((c["N"], c["K"]), generator=g, device="cuda") * 0.02 for _ in range(E)]
        parts = [_quantised(m, c["fmt"], c["N"]) for m in w]
        codes, scales, G = (None if p[0] is None else torch.cat(p) for p in zip(*parts))
        s["w"] = codes.view(E, c["N"], -1), scales.view(E, c["N"], -1), G
        s["y"] = torch.zeros((n, c["N"]), dtype=DTYPES[c["out"]], device="cuda")
        if E > 1 or c["tail"]:
            used = max(0, n - c["tail"])                    # rows behind the last segment stay as they are
            e = (E * torch.rand(used, generator=g, device="cuda") ** 1.1).long().clamp(max=E - 1)
            counts = torch.bincount(e, minlength=E)
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            s["cap"] = int(counts.max())
        else:
            s["offsets"], s["cap"] = None, n
    else:
        T, k, E, H, dt = c["T"], c["k"], c["E"], c["H"], DTYPES[c["dtype"]]
        s["ids"] = _ids(T, k, E + c["sinks"], g)
        s["gates"] = torch.rand((T, k), generator=g, device="cuda") / k
        if c["op"] == "dispatch":
            s["x"] = _activations((T, H), g).to(dt)
            s["xs"] = torch.zeros((T * k, H), dtype=dt, device="cuda")
            if c["train"]:
                s["dxs"] = torch.randn((T * k, H), generator=g, device="cuda").to(dt)
        else:
            flat = s["ids"].view(-1).long()
            kept = flat < E
            order = torch.where(kept, flat, E).argsort(stable=True)
            inv = torch.empty_like(order)
            inv[order] = torch.arange(T * k, device="cuda")
            s["inv"] = torch.where(kept, inv, -1).to(torch.int32).view(T, k)
            s["ys"] = torch.randn((T * k, H), generator=g, device="cuda").to(dt)
            if c["train"]:
                s["dy"] = torch.randn((T, H), generator=g, device="cuda").to(dt)
                s["dys"] = torch.zeros((T * k, H), dtype=dt, device="cuda")
    return s


# -------------------------------------------------------------- plain forms
def _sorted_pairs(ids, E):
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < E)
    order = torch.where(kept, flat, E).argsort(stable=True)
    counts = torch.bincount(torch.where(kept, flat, E), minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.arange(flat.numel(), device=flat.device)
    inv = torch.empty_like(order)
    inv[order] = place
    inv = torch.where(kept, inv, -1).view(ids.shape)
    perm = torch.where(place < offsets[E], order, -1)
    return {"counts": counts.int(), "offsets": offsets.int(), "perm": perm.int(), "inv": inv.int()}


def _gathered(rows, inv):
    """rows[inv] in fp32 [T, k, H], zero where a pair was dropped."""
    r = rows[inv.clamp(min=0).long()].float()
    return torch.where((inv >= 0).unsqueeze(2), r, torch.zeros_like(r))


def _plain(s):
    c = s["case"]
    if c["op"] == "quantise":
        codes, scales, G = _quantised(s["x"], c["fmt"], c["rows"])
        return {"values": _values(codes, scales, G, c["fmt"], c["rows"]).to(DTYPES[c["dtype"]]), "global": G}
    if c["op"] == "product":
        x = _values(*s["x"], c["fmt"], 1)
        w = _values(*s["w"], c["fmt"], c["N"])
        y, off = s["y"], s["offsets"]
        if off is None:
            return (x @ w.t()).to(y.dtype)
        E, cap = c["E"], s["cap"]
        r = torch.arange(c["rows"], device=x.device, dtype=torch.int32)
        e = torch.searchsorted(off, r, right=True) - 1       # the segment of each row; E behind the last one
        at = torch.where(e < E, e * cap + r - off[e.clamp(max=E)], E * cap)
        xp = x.new_zeros((E * cap + 1, c["K"])).index_copy_(0, at, x)
        yp = torch.bmm(xp[:E * cap].view(E, cap, c["K"]), w.view(E, c["N"], -1).transpose(1, 2)).view(E * cap, c["N"])
        got = yp[at.clamp(max=max(0, E * cap - 1))].to(y.dtype) if cap else y
        return torch.where((e < E).unsqueeze(1), got, y)
    if c["op"] == "dispatch":
        r = _sorted_pairs(s["ids"], c["E"])
        perm = r["perm"].long()
        kept = (perm >= 0).unsqueeze(1)
        out = dict(r, xs=torch.where(kept, s["x"][perm.clamp(min=0) // c["k"]], s["xs"]))
        if c["train"]:
            out["dx"] = _gathered(s["dxs"], r["inv"]).sum(1).to(s["x"].dtype)
        return out
    ys, inv, gates = s["ys"], s["inv"], s["gates"]
    v = _gathered(ys, inv)
    out = {"y": (v * gates.unsqueeze(2)).sum(1).to(ys.dtype)}
    if c["train"]:
        dy = s["dy"].float()
        out["dgates"] = (v * dy.unsqueeze(1)).sum(2)
        at = torch.where(inv >= 0, inv.long(), ys.shape[0]).view(-1)
        rows = (gates.unsqueeze(2) * dy.unsqueeze(1)).to(ys.dtype).view(-1, c["H"])
        full = torch.cat([s["dys"], s["dys"].new_zeros(1, c["H"])])
        out["dys"] = full.index_copy(0, at[at < ys.shape[0]], rows[at < ys.shape[0]])[:-1] if c["sinks"] else \
            s["dys"].index_copy(0, at, rows)
    return out


def run(state):
    if not own:
        return _plain(state)
    import fp4_expert_layer_b200 as F
    s, c = state, state["case"]
    if c["op"] == "quantise":
        q = F.fp4_quantize(s["x"], c["fmt"], rows_per_scale=c["rows"])
        return {"values": F.fp4_dequantize(q, dtype=s["x"].dtype), "global": q.global_scale}
    if c["op"] == "product":
        x, w = F.FP4Tensor(*s["x"], c["fmt"]), F.FP4Tensor(*s["w"], c["fmt"])
        return F.fp4_matmul(x, w, offsets=s["offsets"], out=s["y"])
    if c["op"] == "dispatch":
        r = F.sort_tokens(s["ids"], c["E"])
        r["xs"] = F.dispatch(s["x"], r["inv"], out=s["xs"])
        if c["train"]:
            r["dx"] = F.dispatch_backward(s["dxs"], r["inv"])
        return r
    out = {"y": F.combine(s["ys"], s["inv"], s["gates"])}
    if c["train"]:
        out["dys"], out["dgates"] = F.combine_backward(s["dy"], s["ys"], s["inv"], s["gates"], out=s["dys"])
    return out


# -------------------------------------------------- the definitions, 64 bits
def _two(e):
    """2^e in 64 bits, put together from its exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(a, low, bits):
    """|a| to the nearest value with `bits` digits behind the leading one and no exponent under `low`, ties to even."""
    e = torch.frexp(a)[1] - 1
    step = _two(e.clamp(min=low) - bits)
    return torch.round(a / step) * step


def _exact_quantise(x, fmt, rows):
    n, K = x.shape
    v = x.double().reshape(n, -1, BLOCK[fmt])
    top = v.abs().max(dim=2).values
    G = None
    if fmt == "mxfp4":
        X = torch.where(top > 0, torch.frexp(top)[1] - 3, -126).clamp(-126, 127)
        d = _two(X)
    else:
        most = top.reshape(n // rows, -1).max(dim=1).values
        e = torch.frexp(most / 2688)[1]
        e = torch.where(2688 * _two(e - 1) >= most, e - 1, e).clamp(min=-100)
        G = torch.where(most > 0, _two(e), 1.0)
        Gr = G.repeat_interleave(rows)[:, None]
        d = _nearest(top / (6 * Gr), -6, 3).clamp(max=448.0) * Gr
    q = torch.where(d[..., None] > 0, v.abs() / torch.where(d > 0, d, 1.0)[..., None], 0.0)
    return (torch.sign(v) * _nearest(q, 0, 1).clamp(max=6.0) * d[..., None]).reshape(n, K), G


def _exact_read(q, fmt, rows):
    """The reals that codes stand for: sign, exponent and fraction fields taken apart."""
    codes, scales, G = q[0].flatten(0, -2), q[1].flatten(0, -2), q[2]
    nib = torch.stack([codes.long() % 16, codes.long() // 16], -1).reshape(codes.shape[0], -1)
    e, f = (nib // 2) % 4, nib % 2
    v = torch.where(e > 0, (1 + f / 2.0).double() * _two(e - 1), f.double() / 2)
    v = torch.where(nib >= 8, -v, v)
    sc = scales.long()
    if fmt == "mxfp4":
        d = _two(sc - 127)
    else:
        e, f = sc // 8, (sc % 8).double()
        d = torch.where(e > 0, (1 + f / 8) * _two(e - 7), f * 2.0 ** -9)
        d = d * G.double().repeat_interleave(rows)[:, None]
    return v * d.repeat_interleave(BLOCK[fmt], dim=1)


def exact(case, seed):
    c = case
    if c["op"] == "quantise" and c["groups"] * c["rows"] * c["K"] > 1 << 28:
        return None
    s = prepare(c, seed)
    if c["op"] == "quantise":
        v, G = _exact_quantise(s["x"], c["fmt"], c["rows"])
        return {"values": v, "global": G}
    if c["op"] == "product":
        x = _exact_read(s["x"], c["fmt"], 1)
        w = _exact_read(s["w"], c["fmt"], c["N"]).reshape(c["E"], c["N"], -1)
        y = s["y"].double()
        off = [0, c["rows"]] if s["offsets"] is None else s["offsets"].tolist()
        for e in range(c["E"]):
            y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w[e].T
        return y
    T, k, E = c["T"], c["k"], c["E"]
    if c["op"] == "dispatch":
        flat = s["ids"].reshape(-1).tolist()
        lists = [[] for _ in range(E)]
        for p, e in enumerate(flat):
            if 0 <= e < E:
                lists[e].append(p)
        perm = [p for one in lists for p in one]
        xs = s["xs"].double()
        if perm:
            xs[:len(perm)] = s["x"].double()[torch.tensor(perm, device="cuda") // k]
        counts = torch.tensor([len(one) for one in lists], dtype=torch.int32)
        inv = torch.full((T * k,), -1, dtype=torch.int64)
        inv[torch.tensor(perm, dtype=torch.int64)] = torch.arange(len(perm))
        out = {"counts": counts, "offsets": torch.cat([torch.zeros(1), counts.cumsum(0)]).to(torch.int32),
               "perm": torch.tensor(perm + [-1] * (T * k - len(perm)), dtype=torch.int32),
               "inv": inv.to(torch.int32).view(T, k), "xs": xs}
        if c["train"]:
            dx = torch.zeros((T, c["H"]), dtype=torch.float64, device="cuda")
            if perm:
                dx.index_add_(0, torch.tensor(perm, device="cuda") // k, s["dxs"][:len(perm)].double())
            out["dx"] = dx
        return out
    H = c["H"]
    out = {"y": torch.zeros((T, H), dtype=torch.float64, device="cuda")}
    if c["train"]:
        dy, dys = s["dy"].double(), s["dys"].double()
        dg = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(s["inv"][:, j] >= 0).reshape(-1)
        r = s["inv"][t, j].long()
        w = s["gates"][t, j].double()[:, None]
        v = s["ys"][r].double()
        out["y"][t] += w * v
        if c["train"]:
            dg[t, j] = (v * dy[t]).sum(1)
            dys[r] = w * dy[t]
    if c["train"]:
        out.update(dgates=dg, dys=dys)
    return out
