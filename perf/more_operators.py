"""More operators around the MoE layer in a training step, measured: routing by scores (softmax or sigmoid, a balance
bias, groups of experts), the AdamW step over many tensors with states in 32 or 8 bits, and the matrix product with
bias, activation and residual.

`own` false: the operators in plain torch, in 32 bits (the selection of experts, whose borders 32 bits would move, in
64), rounded once at the end; `own` true: the calls that a user makes of the library."""
import math

import torch
import torch.nn.functional as F

own = False

F32, BF16, F64, I64 = torch.float32, torch.bfloat16, torch.float64, torch.int64
E4M3 = torch.float8_e4m3fn
DTYPES = {"f32": F32, "bf16": BF16}
MX = 32            # elements that share a scale of an 8-bit state
LOW = 0xFFFFFFFF


# ---- cases ----
def listed():
    gate = dict(op="gate", train=True, score="sigmoid", bias=True, groups=1, topk_groups=1, group_top=1, renorm=1, scale=1.0, pad=0.0)
    adamw = dict(op="adamw", state="f32", dtype="bf16", g_dtype="bf16", master=False, stochastic=False)
    linear = dict(op="linear", train=True, act="none", dtype="bf16", bias=True, res=True)
    return [
        # one token of a decode step through a sigmoid router of 128 experts: latency
        dict(gate, name="gate_fwd_one_token", train=False, T=1, E=128, k=8),
        # the 30B-A3B layer's router with softmax scores and a balance bias, a training step
        dict(gate, name="gate_train_4096x128", score="softmax", T=4096, E=128, k=8),
        # 256 experts in 8 groups of which a token takes 4, by the sum of a group's two best
        dict(gate, name="gate_train_16384x256_groups", groups=8, topk_groups=4, group_top=2, scale=2.5, T=16384, E=256, k=8),
        # an odd batch with padding, 84 experts in 7 groups, whole softmax weights, no bias
        dict(gate, name="gate_train_1021x84_padded", score="softmax", bias=False, groups=7, topk_groups=3, renorm=0, pad=0.2, T=1021, E=84, k=5),
        # the small tensors of a block (norms, biases, a router of 8 experts), fp32 states: latency
        dict(adamw, name="adamw_24_small_f32", dtype="f32", g_dtype="f32", sizes="many", n=24, size=1024),
        # tensors of odd sizes, fp32 gradients, 8-bit states
        dict(adamw, name="adamw_9_odd_8bit", state="8bit", g_dtype="f32", stochastic=True, sizes="odd", n=9, size=333 * 1000),
        # all W_down of the 235B-A22B share, bf16 with fp32 copies and fp32 states
        dict(adamw, name="adamw_16x1536x4096_f32", master=True, sizes="one", n=1, size=16 * 1536 * 4096),
        # all W_gate of the 30B-A3B layer, bf16 rounded stochastically, 8-bit states
        dict(adamw, name="adamw_128x2048x768_8bit", state="8bit", stochastic=True, sizes="one", n=1, size=128 * 2048 * 768),
        # one token of a decode step through a projection: latency
        dict(linear, name="linear_fwd_one_token", train=False, act="silu", T=1, K=2048, N=768),
        # a dense expert's first product at the 30B-A3B layer's sizes, a training step
        dict(linear, name="linear_train_4096x2048x768", act="gelu", res=False, T=4096, K=2048, N=768),
        # the 235B-A22B share's sizes with the residual sum
        dict(linear, name="linear_train_16384x1536x4096", act="silu", T=16384, K=1536, N=4096),
        # odd sizes in fp32, that no wide load divides
        dict(linear, name="linear_train_1003x769x333_f32", act="relu", dtype="f32", T=1003, K=769, N=333),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "adamw", "linear"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 7, 8])
        per = max(2, _log(rng, 4, 512) // groups)
        E = groups * per
        topk_groups = rng.randint(1, groups)
        group_top = rng.choice([1, 2]) if groups > 1 else 1
        return dict(op=op, train=rng.random() < 0.7, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups, topk_groups=topk_groups,
                    group_top=group_top, renorm=rng.choice([0, 1, 1]), scale=rng.choice([1.0, 2.5]), pad=rng.choice([0.0, 0.0, 0.2, 0.5]),
                    T=min(_log(rng, 1, 16384), 16384 * 256 // E), E=E, k=rng.randint(1, min(16, topk_groups * per)))
    if op == "adamw":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        sizes = rng.choice(["one", "odd", "many"])
        return dict(op=op, state=rng.choice(["f32", "8bit"]), dtype=dtype, g_dtype=rng.choice(["bf16", "f32"]), master=dtype == "bf16" and rng.random() < 0.5,
                    stochastic=rng.random() < 0.5, sizes=sizes, n=1 if sizes == "one" else rng.randint(2, 40), size=_log(rng, 64, 1 << 26 if sizes == "one" else 1 << 20))
    T, K, N = _log(rng, 1, 16384), _log(rng, 32, 4096), _log(rng, 32, 4096)
    if rng.random() < 0.6:
        K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    T = max(1, min(T, 16384 * 1536 * 4096 // (K * N) // (16 if dtype == "f32" else 1)))
    return dict(op=op, train=rng.random() < 0.7, act=rng.choice(["none", "relu", "silu", "gelu"]), dtype=dtype, bias=rng.random() < 0.6, res=rng.random() < 0.5,
                T=T, K=K, N=N)


def _sizes(case):
    """Elements of an optimizer's tensors."""
    n, size = case["n"], case["size"]
    if case["sizes"] == "many":   # vectors and small matrices
        return [size * (1, 1, 16, 1, 8, 2)[i % 6] for i in range(n)]
    if case["sizes"] == "odd":    # single values, vectors, a ragged matrix
        return [(1, 31, 33, 1021 * 37, 769, 257)[i] if i < 6 else max(1, size // (i - 5) - i) for i in range(n)]
    return [size]


def _rooms(sizes):
    """Places of the tensors in the states' buffers: each starts a block of a shared scale."""
    return [-(-s // MX) * MX for s in sizes]


# ---- inputs ----
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape, dtype=F32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    st = dict(case=case)
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = randn(T, E) + 0.7 * randn(E)   # a router that prefers some experts
        st["bias"] = (0.1 if case["score"] == "sigmoid" else 0.5 / E) * randn(E) if case["bias"] else None
        st["mask"] = (rand(T) >= case["pad"]).to(torch.uint8) if case["pad"] else None
        st["rate"] = 1e-3
        st["d_topk_w"] = randn(T, k)
        st["new_bias"] = torch.empty(E, device="cuda")
    elif case["op"] == "adamw":
        sizes = _sizes(case)
        N, dt = sum(_rooms(sizes)), DTYPES[case["dtype"]]
        st["p"] = [(0.02 * randn(s)).to(dt) for s in sizes]
        st["g"] = [(1e-3 * (0.3 + rand(1)) * randn(s)).to(DTYPES[case["g_dtype"]]) for s in sizes]
        st["master"] = [p.float() + 1e-5 * randn(p.numel()) for p in st["p"]] if case["master"] else None
        # moments of some steps ago: the mean far below the root of the mean square
        v = torch.square(1e-3 * (0.3 + rand(N)))
        m = 3e-4 * randn(N)
        on = _flat([torch.ones(s, device="cuda") for s in sizes], sizes)
        v, m = v * on, m * on
        if case["state"] == "8bit":
            st["m"], st["m_scale"] = _code(m, None)
            st["v"], st["v_scale"] = _code(torch.sqrt(v), None)
        else:
            st["m"], st["v"] = m, v
        st["t"], st["seed"] = 10, int(seed) & 0x7FFFFFFF
        st["hyper"] = dict(lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, wd=0.1)
    else:
        T, K, N, dt = case["T"], case["K"], case["N"], DTYPES[case["dtype"]]
        st["x"], st["w"] = randn(T, K).to(dt), (randn(K, N) / math.sqrt(K)).to(dt)
        st["b"] = (0.1 * randn(N)).to(dt) if case["bias"] else None
        st["res"] = randn(T, N).to(dt) if case["res"] else None
        if case["train"]:
            st["dy"] = randn(T, N).to(dt)
    if own:
        st["op"] = _handle(case, st)
    return st


def _handle(case, st):
    import combine_top_router_amd as moe
    code = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16}
    if case["op"] == "gate":
        score = {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}[case["score"]]
        return moe.Gate(case["T"], case["E"], case["k"], score=score, groups=case["groups"], topk_groups=case["topk_groups"], group_top=case["group_top"],
                        renorm=case["renorm"], scale=case["scale"])
    if case["op"] == "adamw":
        h = st["hyper"]
        op = moe.AdamW(st["p"], state=moe.MOE_STATE_8BIT if case["state"] == "8bit" else moe.MOE_STATE_F32, betas=(h["b1"], h["b2"]), eps=h["eps"],
                       weight_decay=h["wd"], master=case["master"], stochastic=case["stochastic"], seed=st["seed"])
        op.t = st["t"]
        if case["state"] == "8bit":
            for mine, given in ((op.m, "m"), (op.v, "v"), (op.m_scale, "m_scale"), (op.v_scale, "v_scale")):
                mine.copy_(st[given].view(torch.uint8))
        else:
            op.m.copy_(st["m"])
            op.v.copy_(st["v"])
        if case["master"]:
            for mine, given in zip(op.master, st["master"]):
                mine.copy_(given)
        return op
    act = {"none": moe.MOE_ACT_NONE, "relu": moe.MOE_ACT_RELU, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU}[case["act"]]
    return moe.Linear(case["T"], case["K"], case["N"], act=act, dtype=code[case["dtype"]], train=case["train"])


# ---- one pass ----
def run(st):
    if own:
        return _run_own(st)
    return {"gate": _gate, "adamw": _adamw, "linear": _linear}[st["case"]["op"]](st)


def _run_own(st):
    op, case = st["op"], st["case"]
    if case["op"] == "gate":
        idx, w = op.forward(st["logits"], bias=st["bias"], mask=st["mask"], count=case["train"])
        out = {"topk_idx": idx, "topk_w": w}
        if case["train"]:
            out["d_logits"] = op.backward(st["d_topk_w"])
            out["counts"] = op.counts
            if case["bias"]:
                out["bias"] = op.update_bias(st["bias"], st["rate"], out=st["new_bias"])
        return out
    if case["op"] == "adamw":
        op.step(st["g"], st["hyper"]["lr"])
        out = {"p": st["p"], "m": op.m, "v": op.v}
        if case["master"]:
            out["master"] = op.master
        if case["state"] == "8bit":   # the codes and the scales as the values that they stand for
            out["m"], out["v"] = op.m.view(E4M3), op.v.view(E4M3)
            out["m_scale"], out["v_scale"] = _power(op.m_scale), _power(op.v_scale)
        return out
    out = {"y": op.forward(st["x"], st["w"], st["b"], res=st["res"])}
    if case["train"]:
        grads = op.backward(st["dy"])
        out["dx"], out["dw"] = grads["dx"], grads["dw"]
        if case["bias"]:
            out["db"] = grads["db"]
    return out


# ---- routing by scores ----
def _gate(st):
    case, logits, mask = st["case"], st["logits"], st["mask"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = logits.double()
    if case["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    by_score = s if st["bias"] is None else s + st["bias"].double()
    choice = l if st["bias"] is None else by_score   # the scores rise with the logits
    if G > 1:
        per = choice.view(T, G, E // G)
        if case["group_top"] == 1:
            of_group = per.amax(2)
        else:
            of_group = by_score.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        best = of_group.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, best, True)
        choice = torch.where(open_[:, :, None], per, -math.inf).reshape(T, E)
    idx = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    q = s.gather(1, idx)
    if case["renorm"]:
        q = q / q.sum(1, keepdim=True)
    w = case["scale"] * q
    on = None if mask is None else (mask != 0)[:, None]
    ids = idx.to(torch.int32)
    if on is not None:
        ids, w = torch.where(on, ids, -1), torch.where(on, w, 0.0)
    out = {"topk_idx": ids, "topk_w": w.float()}
    if case["train"]:
        d = case["scale"] * st["d_topk_w"].double()
        if case["renorm"]:
            d = q * (d - (q * d).sum(1, keepdim=True))
            if case["score"] == "sigmoid":
                d = d * (1.0 - s.gather(1, idx))
            dl = torch.zeros_like(s).scatter_(1, idx, d)
        elif case["score"] == "sigmoid":
            dl = torch.zeros_like(s).scatter_(1, idx, d * q * (1.0 - q))
        else:
            dl = s * (torch.zeros_like(s).scatter_(1, idx, d) - (q * d).sum(1, keepdim=True))
        hits = torch.ones(T, k, dtype=torch.int32, device=l.device)
        if on is not None:
            dl, hits = torch.where(on, dl, 0.0), hits * on.to(torch.int32)
        out["d_logits"] = dl.float()
        counts = torch.zeros(E, dtype=torch.int32, device=l.device)
        out["counts"] = counts.index_add_(0, idx.reshape(-1), hits.reshape(-1))
        if st["bias"] is not None:
            out["bias"] = st["bias"] + st["rate"] * torch.sign(counts.sum() - E * counts.long()).float()
    return out


# ---- the AdamW step ----
def _flat(tensors, sizes):
    """The tensors one behind the other, each filled up with zeros to its room."""
    return torch.cat([F.pad(t.float(), (0, r - s)) for t, r, s in zip(tensors, _rooms(sizes), sizes)])


def _mix(v):
    """32 bits mixed (the output permutation of PCG, O'Neill 2014), on whole numbers below 2^32."""
    s = (v * 747796405 + 2891336453) & LOW
    w = (((s >> ((s >> 28) + 4)) ^ s) * 277803737) & LOW
    return (w >> 22) ^ w


def _bits(st, n):
    """32 random bits for each place of the states' buffers at this step, from the seed."""
    seed = st["seed"]
    k = _mix(((st["t"] & LOW) + _mix(((seed & LOW) + _mix(seed >> 32)) & LOW)) & LOW)
    i = torch.arange(n, device="cuda")
    return _mix((i & LOW) ^ _mix(((i >> 32) + k) & LOW))


def _power(scale):
    """2^(scale - 127) of e8m0 codes, the values that they stand for."""
    return scale.view(torch.float8_e8m0fnu)


def _values(code, scale):
    x = code.float().view(-1, MX)
    return torch.ldexp(x, (scale.view(torch.uint8).to(torch.int32) - 127)[:, None]).reshape(-1)


def _code(x, r16, keep=False):
    """E4M3 codes of x, blocks of 32 sharing a power of two (the smallest that takes the block's largest to 448 at
    most), to nearest or, with 16 random bits each, stochastically; keep: what is above 0 stays above 0."""
    b = x.view(-1, MX)
    amax = b.abs().amax(1)
    mant, e = torch.frexp(amax)   # in [0.5, 1), and 448 = 0.875 * 2^9
    e = torch.where(amax > 0, (e - 9 + (mant > 0.875).to(e.dtype)).clamp(-127, 127), 0)
    y = torch.ldexp(b.abs(), -e[:, None])
    if r16 is not None:
        step = torch.exp2((torch.frexp(y).exponent - 1).clamp(min=-6).to(x.dtype) - 3.0)
        n = y / step
        low = torch.floor(n)
        y = (low + (r16.view(-1, MX).to(x.dtype) < (n - low) * 65536.0)) * step
    y = y.float().to(E4M3).float()
    if keep:
        y = torch.where((b > 0) & (y == 0), 2.0 ** -9, y)
    return torch.copysign(y, b.float()).to(E4M3).reshape(-1), (e + 127).to(torch.uint8)


def _moments(st):
    if st["case"]["state"] == "8bit":
        return _values(st["m"], st["m_scale"]), torch.square(_values(st["v"], st["v_scale"]))
    return st["m"], st["v"]


def _adamw(st):
    case, h = st["case"], st["hyper"]
    sizes = [p.numel() for p in st["p"]]
    st["t"] += 1
    g = _flat(st["g"], sizes)
    p = _flat(st["master"] or st["p"], sizes)
    m, v = _moments(st)
    m = h["b1"] * m + (1.0 - h["b1"]) * g
    v = h["b2"] * v + (1.0 - h["b2"]) * (g * g)
    to_m, to_v = 1.0 - h["b1"] ** st["t"], 1.0 - h["b2"] ** st["t"]
    p = p * (1.0 - h["lr"] * h["wd"]) - h["lr"] * (m / to_m) / (torch.sqrt(v / to_v) + h["eps"])
    r = _bits(st, g.numel()) if case["stochastic"] else None
    out = {"p": st["p"]}
    if case["state"] == "8bit":
        st["m"], st["m_scale"] = _code(m, None if r is None else r & 0xFFFF)
        st["v"], st["v_scale"] = _code(torch.sqrt(v), None if r is None else r >> 16, keep=True)
        out["m_scale"], out["v_scale"] = _power(st["m_scale"]), _power(st["v_scale"])
    else:
        st["m"], st["v"] = m, v
    out["m"], out["v"] = st["m"], st["v"]
    new = [t[:s] for t, s in zip(torch.split(p, _rooms(sizes)), sizes)]
    if case["master"]:
        torch._foreach_copy_(st["master"], new)
        out["master"] = st["master"]
    elif case["dtype"] == "bf16" and r is not None:
        bits = (p.view(torch.int32).to(I64) & LOW) + (_mix(r) & 0xFFFF)
        bf = ((bits >> 16) & 0xFFFF).to(torch.int32)
        p = (bf << 16).view(F32)
        new = [t[:s] for t, s in zip(torch.split(p, _rooms(sizes)), sizes)]
    torch._foreach_copy_(st["p"], new)
    return out


# ---- the matrix product ----
def _act(z, act):
    """The activation and its slope."""
    if act == "relu":
        return torch.clamp(z, min=0), (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return z, None


def _linear(st):
    case, dt = st["case"], DTYPES[st["case"]["dtype"]]
    x, w = st["x"].float(), st["w"].float()
    z = x @ w
    if case["bias"]:
        z = z + st["b"].float()
    y, slope = _act(z, case["act"])
    if case["res"]:
        y = y + st["res"].float()
    out = {"y": y.to(dt)}
    if case["train"]:
        dz = st["dy"].float()
        if slope is not None:
            dz = dz * slope
        out["dx"], out["dw"] = (dz @ w.t().contiguous()).to(dt), (x.t().contiguous() @ dz).to(dt)
        if case["bias"]:
            out["db"] = dz.sum(0).to(dt)
    return out


# ---- what a pass cannot do without ----
def work(case):
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        fwd = T * E * 4 + T * k * 8 + (E * 4 if case["bias"] else 0) + (T if case["pad"] else 0)
        bwd = T * E * 4 + T * k * 4 + E * 4 if case["train"] else 0
        return {"bytes": fwd + bwd, "flops": T * E * (10 + 4 * case["train"])}
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        p, g = (2 if case[d] == "bf16" else 4 for d in ("dtype", "g_dtype"))
        state = 16 if case["state"] == "f32" else 4 * (1 + 1 / MX)
        return {"bytes": n * ((p + 8 if case["master"] else 2 * p) + g + state), "flops": n * 16}
    T, K, N, b = case["T"], case["K"], case["N"], 2 if case["dtype"] == "bf16" else 4
    fwd = T * K + K * N + T * N * (1 + case["res"])
    bwd = (T * N + T * K + K * N) if case["train"] else 0
    return {"bytes": (fwd + bwd) * b, "flops": (6.0 if case["train"] else 2.0) * T * K * N}


# ---- the definitions in 64 bits ----
def exact(case, seed):
    st = prepare(case, seed)
    return {"gate": _exact_gate, "adamw": _exact_adamw, "linear": _exact_linear}[case["op"]](case, st)


def _exact_gate(case, st):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = st["logits"].double().requires_grad_(True)
    s = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
    with torch.no_grad():
        c = s if st["bias"] is None else s + st["bias"].double()
        # where there is no bias the logits order the experts
        c = c.detach().clone()
        order = l.detach().clone() if st["bias"] is None else c
        if G > 1:
            grouped = torch.topk(c.view(T, G, -1), case["group_top"], dim=2).values.sum(2) if case["group_top"] > 1 else order.view(T, G, -1).amax(2)
            shut = torch.ones(T, G, device=l.device).scatter(1, torch.argsort(grouped, dim=1, descending=True, stable=True)[:, :case["topk_groups"]], 0.0)
            order = order.masked_fill(shut.repeat_interleave(E // G, dim=1) > 0, -math.inf)
        idx = torch.argsort(order, dim=1, descending=True, stable=True)[:, :k]
    w = s.gather(1, idx)
    w = w / w.sum(1, keepdim=True) if case["renorm"] else w
    w = w * case["scale"]
    live = torch.ones(T, 1, dtype=F64, device=l.device) if st["mask"] is None else (st["mask"] != 0).double()[:, None]
    w = w * live
    out = {"topk_idx": torch.where(live > 0, idx, -1).to(torch.int32), "topk_w": w.detach()}
    if case["train"]:
        (w * st["d_topk_w"].double()).sum().backward()
        counts = torch.bincount(idx[live[:, 0] > 0].reshape(-1), minlength=E)
        out["d_logits"], out["counts"] = l.grad, counts.to(torch.int32)
        if st["bias"] is not None:
            mean = counts.sum().double() / E
            out["bias"] = st["bias"].double() + st["rate"] * ((counts < mean).double() - (counts > mean).double())
    return out


def _exact_adamw(case, st):
    h, sizes, t = st["hyper"], _sizes(case), st["t"] + 1
    rooms = _rooms(sizes)
    flat = lambda ts: torch.cat([F.pad(x.double(), (0, r - x.numel())) for x, r in zip(ts, rooms)])  # noqa: E731
    if case["state"] == "8bit":
        held = lambda c, s: c.double() * torch.pow(2.0, s.double() - 127).repeat_interleave(MX)  # noqa: E731
        m, v = held(st["m"], st["m_scale"]), held(st["v"], st["v_scale"]) ** 2
    else:
        m, v = st["m"].double(), st["v"].double()
    g, p = flat(st["g"]), flat(st["master"] or st["p"])
    m = torch.lerp(g, m, h["b1"])
    v = torch.lerp(g * g, v, h["b2"])
    p = p - h["lr"] * (h["wd"] * p + (m / (1 - h["b1"] ** t)) / ((v / (1 - h["b2"] ** t)).sqrt() + h["eps"]))
    st["t"] = t
    out, r = {}, _bits(st, g.numel()) if case["stochastic"] else None
    if case["state"] == "8bit":
        for name, x, shift in (("m", m, 0), ("v", v.sqrt(), 16)):
            blocks = x.abs().view(-1, MX)
            top = blocks.amax(1, keepdim=True)
            power = torch.pow(2.0, torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0)))
            y = (blocks / power).reshape(-1)
            # the grid's step at y: an eighth of the power of two below it, 2^-9 at least
            step = torch.pow(2.0, torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
            if r is None:
                y = torch.round(y / step) * step   # ties to even
            else:
                low = torch.floor(y / step)
                y = (low + (((r >> shift) & 0xFFFF).double() / 65536.0 < y / step - low).double()) * step
            if name == "v":
                y = torch.where((x > 0) & (y == 0), 2.0 ** -9, y)
            out[name], out[name + "_scale"] = torch.copysign(y, x), power[:, 0]
    else:
        out["m"], out["v"] = m, v
    of = lambda x: [t[:s] for t, s in zip(torch.split(x, rooms), sizes)]  # noqa: E731
    if case["master"]:
        out["master"] = of(p)
    elif case["dtype"] == "bf16" and r is not None:   # up by the bits' share of the step between two bf16 numbers
        step = torch.pow(2.0, torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
        low = torch.floor(p.abs() / step)
        rest = torch.floor((p.abs() / step - low) * 65536.0)
        p = torch.copysign((low + (rest + (_mix(r) & 0xFFFF) >= 65536).double()) * step, p)
    out["p"] = of(p)
    return out


def _exact_linear(case, st):
    x, w = (st[n].double().requires_grad_(True) for n in ("x", "w"))
    b = st["b"].double().requires_grad_(True) if case["bias"] else None
    z = F.linear(x, w.t(), b)
    y = {"none": lambda v: v, "relu": torch.relu, "silu": F.silu, "gelu": F.gelu}[case["act"]](z)
    if case["res"]:
        y = y + st["res"].double()
    out = {"y": y.detach()}
    if case["train"]:
        y.backward(st["dy"].double())
        out["dx"], out["dw"] = x.grad, w.grad
        if case["bias"]:
            out["db"] = b.grad
    return out
