"""Cases of the dense half of a decode step: the operators between a layer
stack's output and the next token.

* ``norm``   - residual addition, root-mean-square norm with a gain, and the
  normalised row in 8 bits with scales (one per row, or one per group of
  columns): the operand of an 8-bit product.
* ``linear`` - out = act(a w^T scaled + bias) + residual, with bf16 operands or
  with 8-bit operands and scales: projections, a shared dense FFN, and the
  product with the vocabulary that gives the logits.
* ``sample`` - one token per row from its logits: temperature, top-k, min-p,
  top-p, and given uniform random numbers.

Sizes are the library's own (hidden 2048, intermediate 768, vocabulary 2^17,
1 and 8 decode tokens, 4096-token chunks, chunks of up to 8192) and odd ones
beside them.

``run`` computes an operator in elementary torch operations, or with ``own``
set by the library's calls. ``exact`` gives the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu")


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one decoded token at the end of the layer stack (fp32 activations), ready for an 8-bit product
        dict(name="norm_decode1", op="norm", T=1, H=2048, dtype="f32", group=0, residual=True, gain=True, norm=False),
        # a ragged batch of a wider model, one scale per 128 columns
        dict(name="norm_ragged1003", op="norm", T=1003, H=5248, dtype="f32", group=128, residual=True, gain=True, norm=False),
        # the largest prefill chunk, bf16 stream, 8-bit rows and the bf16 rows beside them
        dict(name="norm_chunk8192", op="norm", T=8192, H=2048, dtype="bf16", group=0, residual=True, gain=True, norm=True),
        # one token through a square 8-bit projection back onto the residual stream
        dict(name="linear_decode1_i8", op="linear", M=1, N=2048, K=2048, dtype="i8", out="f32", act="none", bias=False, residual=True),
        # logits of a verify batch of 8 tokens over the vocabulary
        dict(name="linear_logits8", op="linear", M=8, N=131072, K=2048, dtype="bf16", out="f32", act="none", bias=False, residual=False),
        # a small odd batch: every size ends inside a tile
        dict(name="linear_odd77", op="linear", M=77, N=1000, K=1501, dtype="bf16", out="f32", act="gelu", bias=True, residual=False),
        # down projection of a shared dense FFN over a prefill chunk, 8-bit, added onto the residual stream
        dict(name="linear_down4096_i8", op="linear", M=4096, N=2048, K=768, dtype="i8", out="bf16", act="none", bias=True, residual=True),
        # up projection of a dense FFN over the largest prefill chunk
        dict(name="linear_up8192", op="linear", M=8192, N=4096, K=2048, dtype="bf16", out="bf16", act="silu", bias=True, residual=False),
        # the next token of one sequence: everything on
        dict(name="sample_decode1", op="sample", T=1, V=131072, dtype="f32", top_k=50, top_p=0.9, min_p=0.02, greedy=False, masked=False),
        # a verify batch, bf16 logits, nucleus only
        dict(name="sample_verify8", op="sample", T=8, V=131072, dtype="bf16", top_k=0, top_p=0.95, min_p=0.0, greedy=False, masked=False),
        # a served batch of a smaller odd vocabulary, some rows greedy, some tokens masked out, min-p
        dict(name="sample_odd61", op="sample", T=61, V=32003, dtype="f32", top_k=0, top_p=1.0, min_p=0.05, greedy=True, masked=True),
        # a large served batch
        dict(name="sample_batch256", op="sample", T=256, V=131072, dtype="f32", top_k=0, top_p=0.9, min_p=0.0, greedy=False, masked=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "linear", "sample"))
    if op == "norm":
        H = 128 * _log(rng, 2, 64)
        group = rng.choice((0, 0, 32, 64, 128))
        if not group:
            H += 16 * rng.randrange(8)
        T = max(1, min(_log(rng, 1, 8192), 8192 * 2048 // H))
        return dict(op="norm", T=T, H=H, dtype=rng.choice(("f32", "bf16")), group=group,
                    residual=rng.random() < 0.8, gain=rng.random() < 0.8, norm=rng.random() < 0.4)
    if op == "linear":
        head = rng.random() < 0.3
        M = _log(rng, 1, 64) if head else _log(rng, 1, 8192)
        N = _log(rng, 16384, 131072) if head else _log(rng, 64, 8192)
        K = _log(rng, 512, 2048) if head else _log(rng, 64, 8192)
        while M * N * K > 8192 * 4096 * 2048:
            M = max(1, M // 2)
        return dict(op="linear", M=M, N=N, K=K, dtype=rng.choice(("bf16", "i8")), out=rng.choice(("f32", "bf16")),
                    act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.4)
    V = _log(rng, 1000, 131072)
    T = _log(rng, 1, 256)
    return dict(op="sample", T=T, V=V, dtype=rng.choice(("f32", "bf16")), top_k=rng.choice((0, 0, 1, 20, 50, 200, 1000)),
                top_p=rng.choice((1.0, 0.95, 0.9, 0.5)), min_p=rng.choice((0.0, 0.0, 0.02, 0.1)),
                greedy=rng.random() < 0.3, masked=rng.random() < 0.4)


def work(case):
    c = case
    if c["op"] == "norm":
        e = c["T"] * c["H"]
        b = 4 if c["dtype"] == "f32" else 2
        nbytes = e * (b * (2 if c["residual"] else 1)) + e + 4 * c["T"] * (c["H"] // c["group"] if c["group"] else 1)
        nbytes += e * b if c["residual"] else 0        # the residual stream written back
        nbytes += 4 * c["H"] if c["gain"] else 0
        nbytes += 2 * e if c["norm"] else 0
        return {"bytes": nbytes, "flops": 8 * e}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        b, o = (2 if c["dtype"] == "bf16" else 1), (4 if c["out"] == "f32" else 2)
        nbytes = (M + N) * K * b + M * N * o + (4 * N if c["bias"] else 0) + (M * N * o if c["residual"] else 0)
        nbytes += 4 * (M + N) if c["dtype"] == "i8" else 0
        return {"bytes": nbytes, "flops": 2 * M * N * K}
    e = c["T"] * c["V"]
    return {"bytes": e * (4 if c["dtype"] == "f32" else 2) + 28 * c["T"], "flops": 8 * e}


# ------------------------------------------------------------------ inputs --
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _ld(n, align):
    """Row stride of a buffer whose rows start on 16 bytes."""
    return (n + align - 1) // align * align


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": dict(c), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if c["op"] == "norm":
        T, H, dt = c["T"], c["H"], _DT[c["dtype"]]
        # a residual stream with a few outlying columns, and a block's output
        col = torch.exp(0.5 * normal(H))
        s["x"] = (normal(T, H) * col * 2.0).to(dt)
        s["y"] = (normal(T, H) * 0.7).to(dt) if c["residual"] else None
        s["gain"] = 1.0 + 0.2 * normal(H) if c["gain"] else None
        s["z"] = torch.empty((T, H), dtype=dt, device="cuda") if c["residual"] else None
        s["norm"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda") if c["norm"] else None
        s["codes"] = torch.empty((T, H), dtype=torch.int8, device="cuda")
        s["scales"] = torch.empty((T, H // c["group"] if c["group"] else 1), dtype=torch.float32, device="cuda")
    elif c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        if c["dtype"] == "bf16":
            ld = _ld(K, 8)
            s["a"] = normal(M, ld).to(torch.bfloat16)[:, :K]
            s["w"] = (normal(N, ld) / math.sqrt(K)).to(torch.bfloat16)[:, :K]
            s["as"] = s["ws"] = None
        else:
            ld = _ld(K, 16)
            s["a"] = (normal(M, ld) * 36.0).round().clamp(-127, 127).to(torch.int8)[:, :K]
            s["w"] = (normal(N, ld) * 36.0).round().clamp(-127, 127).to(torch.int8)[:, :K]
            s["as"] = (0.5 + uniform(M)) / 36.0
            s["ws"] = (0.5 + uniform(N)) / (36.0 * math.sqrt(K))
        s["bias"] = 0.5 * normal(N) if c["bias"] else None
        s["res"] = normal(M, N).to(_DT[c["out"]]) if c["residual"] else None
        s["out"] = torch.empty((M, N), dtype=_DT[c["out"]], device="cuda")
    else:
        T, V = c["T"], c["V"]
        # logits of a language model: a broad bulk and a few hundred likely tokens
        l = 2.2 * normal(T, V)
        head = torch.randint(0, V, (T, min(V, 300)), generator=g, device="cuda")
        l.scatter_add_(1, head, 4.0 + 3.0 * normal(*head.shape))
        if c["masked"]:
            l.masked_fill_(uniform(T, V) < 0.3, float("-inf"))
        s["logits"] = l.to(_DT[c["dtype"]])
        temp = 0.6 + 0.6 * uniform(T)
        if c["greedy"]:
            temp[::4] = 0.0
        s["temperature"] = temp
        s["top_k"] = torch.randint(max(1, c["top_k"] // 2), c["top_k"] + 1, (T,), generator=g, device="cuda",
                                   dtype=torch.int32) if c["top_k"] else None
        s["top_p"] = c["top_p"] - 0.1 * uniform(T) if c["top_p"] < 1 else None
        s["min_p"] = c["min_p"] * (0.5 + uniform(T)) if c["min_p"] > 0 else None
        s["u"] = uniform(T)
        s["token"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["prob"] = torch.empty(T, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------- framework calls --
_ACT_CODE = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}


def _own(s):
    import quantised_expert_decode_b200 as q
    c = s["case"]
    if c["op"] == "norm":
        q.qmoe_rmsnorm_residual_q8(s["x"], s["y"], q.F32 if c["dtype"] == "f32" else q.BF16, s["gain"], 1e-6, c["T"], c["H"],
                                   c["group"], s["z"], s["norm"], s["codes"], s["scales"])
        G = s["scales"].shape[1]
        return [s["z"], s["norm"], s["codes"].view(c["T"], G, -1) * s["scales"].unsqueeze(-1), s["scales"]]
    if c["op"] == "linear":
        q.qmoe_linear(s["a"], q.BF16 if c["dtype"] == "bf16" else q.I8, s["w"], c["M"], c["N"], c["K"], s["as"], s["ws"],
                      s["bias"], _ACT_CODE[c["act"]], s["res"], s["out"], q.F32 if c["out"] == "f32" else q.BF16,
                      s["status"], lda=s["a"].stride(0), ldw=s["w"].stride(0))
        return s["out"]
    q.qmoe_sample(s["logits"], q.F32 if c["dtype"] == "f32" else q.BF16, c["T"], c["V"], s["temperature"], s["top_k"],
                  s["top_p"], s["min_p"], s["u"], s["token"], s["prob"], s["status"])
    return [s["token"], s["prob"]]


# -------------------------------------------------------------- plain forms --
def _plain_norm(s):
    c = s["case"]
    T, H = c["T"], c["H"]
    z = s["x"].float() + s["y"].float() if c["residual"] else s["x"].float()
    p = z.double() * s["gain"].double() if c["gain"] else z.double()   # 64 bits: codes next to a rounding border
    inv = 1.0 / torch.sqrt((z.double() * z.double()).mean(-1, keepdim=True) + 1e-6)
    G = H // c["group"] if c["group"] else 1
    pg = p.view(T, G, -1)
    top = pg.abs().amax(-1, keepdim=True)
    codes = torch.round((pg * 127.0) / top)
    codes = torch.where(top > 0, codes, torch.zeros_like(codes))
    scales = (top * inv.unsqueeze(-1) / 127.0).float()
    out = z.to(s["x"].dtype) if c["residual"] else None
    norm = (p * inv).to(torch.bfloat16) if c["norm"] else None
    return [out, norm, codes.float() * scales, scales.squeeze(-1)]


def _act(v, name):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(v * -math.sqrt(0.5))
    return v


def _plain_linear(s):
    c = s["case"]
    v = s["a"].float() @ s["w"].float().t()
    if s["as"] is not None:
        v = v * s["as"].unsqueeze(1) * s["ws"]
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _act(v, c["act"])
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(_DT[c["out"]])


def _plain_sample(s):
    V = s["case"]["V"]
    l = s["logits"].double()                                   # 64 bits: the sums decide between neighbours
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l)
    order = torch.argsort(l, dim=-1, descending=True, stable=True)
    top = l.gather(-1, order[:, :1])
    rank0 = order[:, :1]                                       # the lowest index of the largest logit
    t = s["temperature"].double().unsqueeze(-1)
    d = torch.where(l == top, torch.zeros_like(l), (l - top) / t)
    w = torch.exp(d)
    w = torch.where(w < 2.0 ** -64, torch.zeros_like(w), w)
    first = torch.arange(V, device=l.device).unsqueeze(0) == rank0
    w = torch.where((t == 0) & ~first, torch.zeros_like(w), w)
    w = torch.where(top == -math.inf, torch.zeros_like(w), w)  # a row that the mask leaves empty
    ws = w.gather(-1, order)
    rank = torch.arange(V, device=l.device).unsqueeze(0)
    keep = ws > 0
    if s["top_k"] is not None:
        k = s["top_k"].long().unsqueeze(-1)
        keep = keep & ((rank < k) | (k <= 0))
    if s["min_p"] is not None:
        keep = keep & (ws >= s["min_p"].double().unsqueeze(-1))
    if s["top_p"] is not None:
        mass = torch.where(keep, ws, torch.zeros_like(ws))
        before = mass.cumsum(-1) - mass
        keep = keep & ((before < s["top_p"].double().unsqueeze(-1) * mass.sum(-1, keepdim=True)) | (rank == 0))
    kept = torch.zeros_like(w).scatter(-1, order, torch.where(keep, ws, torch.zeros_like(ws)))
    cum = kept.cumsum(-1)
    total = cum[:, -1:]
    hit = (cum > s["u"].double().unsqueeze(-1) * total) & (kept > 0)
    token = torch.where(hit, rank.expand_as(hit), V).amin(-1)
    empty = token == V
    at = torch.where(empty, torch.zeros_like(token), token).unsqueeze(-1)
    prob = torch.where(empty, torch.zeros_like(total[:, 0]), (kept.gather(-1, at) / total)[:, 0])
    return [torch.where(empty, torch.full_like(token, -1), token).int(), prob.float()]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "linear": _plain_linear, "sample": _plain_sample}[state["case"]["op"]](state)


# ------------------------------------------------------------ 64-bit values --
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "norm":
        # z is the stream's sum rounded to 32 bits; everything after it in 64
        z = (s["x"].float() + s["y"].float() if s["y"] is not None else s["x"].float()).double()
        n = z * torch.rsqrt(z.square().sum(1, keepdim=True) / c["H"] + 1e-6)
        gain = s["gain"].double() if s["gain"] is not None else torch.ones(c["H"], dtype=torch.float64, device="cuda")
        group = c["group"] or c["H"]
        blocks = (z * gain).reshape(-1, group)
        peak = blocks.abs().max(1, keepdim=True).values
        codes = (blocks * 127.0 / peak).round()
        peak_n = (n * gain).reshape(-1, group).abs().max(1, keepdim=True).values
        values = (codes * (peak_n / 127.0)).reshape(c["T"], -1, group)
        return [z if s["y"] is not None else None, n * gain if c["norm"] else None, values, (peak_n / 127.0).reshape(c["T"], -1)]
    if c["op"] == "linear":
        a, w = s["a"].double(), s["w"].double()
        if s["as"] is not None:
            a, w = a * s["as"].double()[:, None], w * s["ws"].double()[:, None]
        v = torch.mm(a, w.T)
        if s["bias"] is not None:
            v += s["bias"].double()
        if c["act"] == "relu":
            v.clamp_(min=0)
        elif c["act"] == "silu":
            v *= torch.sigmoid(v)
        elif c["act"] == "gelu":
            v *= torch.special.ndtr(v)
        if s["res"] is not None:
            v += s["res"].double()
        return v
    # one row at a time, on the row's own sorted list
    tokens, probs = [], []
    for t in range(c["T"]):
        l = s["logits"][t].double()
        live = torch.nonzero(l > -math.inf)[:, 0]
        if live.numel() == 0:
            tokens.append(-1)
            probs.append(0.0)
            continue
        temp = float(s["temperature"][t])
        v, at = torch.sort(l[live], descending=True, stable=True)
        at = live[at]
        if temp == 0:
            tokens.append(int(at[0]))
            probs.append(1.0)
            continue
        e = torch.exp((v - v[0]) / temp)
        n = int((e >= 2.0 ** -64).sum())
        if s["top_k"] is not None and int(s["top_k"][t]) > 0:
            n = min(n, int(s["top_k"][t]))
        if s["min_p"] is not None:
            n = min(n, int((e >= float(s["min_p"][t])).sum()))
        if s["top_p"] is not None:
            c_ = torch.cumsum(e[:n], 0)
            n = int(torch.searchsorted(c_, float(s["top_p"][t]) * c_[-1])) + 1
        at, by = torch.sort(at[:n])
        cum = torch.cumsum(e[:n][by], 0)
        i = min(int(torch.searchsorted(cum, float(s["u"][t]) * cum[-1], right=True)), n - 1)
        tokens.append(int(at[i]))
        probs.append(float(e[:n][by][i] / cum[-1]))
    return [torch.tensor(tokens, dtype=torch.int32, device="cuda"), torch.tensor(probs, dtype=torch.float64, device="cuda")]


if __name__ == "__main__":
    rng = random.Random(0)
    for case in listed() + [draw(rng) for _ in range(6)]:
        print(case, work(case))
