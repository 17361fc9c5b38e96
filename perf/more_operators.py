"""Cases, plain forms and 64-bit definitions of the operators of a sampling decode head with 4-bit weights.

What a decode or verify step does at its end when its dense matrices are kept in 4 bits and its tokens are drawn:

* ``linear``  a few tokens times a matrix of 4-bit codes with a scale (and, optionally, a zero point) per group of
  32, 64 or 128 values of a row: fp32, bf16 or fp16 activations, or int8 codes with a scale per token;
* ``sample``  a token per row from the row's logits, with a temperature, top-k, top-p and min-p of its own and one given
  random number.

``run`` computes them with elementary torch operations, or, where ``own`` is true, with the library's calls.
``exact`` computes the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
SIZES = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # a small projection for a single token: pure latency
        dict(name="linear one token", op="linear", T=1, N=2048, K=2048, group=32, zeros=False, x="bf16", out="bf16", bias=False),
        # the vocabulary head for a single token, behind the int8 norm: the weights' way from memory
        dict(name="linear head of 1", op="linear", T=1, N=129280, K=4096, group=128, zeros=False, x="i8", out="f32", bias=False),
        # the same over the verify step's columns, an odd vocabulary, fp32 activations, codes with zero points
        dict(name="linear odd head of 5", op="linear", T=5, N=129279, K=4096, group=64, zeros=True, x="f32", out="f32", bias=False),
        # a small batch of decoding sequences through a projection; K that is no multiple of a whole chunk
        dict(name="linear batch of 16", op="linear", T=16, N=8192, K=4144, group=128, zeros=True, x="bf16", out="bf16", bias=True),
        # a larger batch, ragged, through a long contraction
        dict(name="linear batch of 61", op="linear", T=61, N=4096, K=14336, group=128, zeros=False, x="f16", out="f16", bias=False),
        # a prompt's rest through a projection of the same weights
        dict(name="linear chunk of 300", op="linear", T=300, N=8192, K=4096, group=64, zeros=False, x="bf16", out="bf16", bias=False),
        # one sequence with every filter: latency
        dict(name="sample one row", op="sample", R=1, V=129280, dtype="f32", top_k=50, top_p=0.95, min_p=0.02),
        # the verify step's columns by temperature alone, odd vocabulary
        dict(name="sample five rows", op="sample", R=5, V=129279, dtype="f32", top_k=0, top_p=1.0, min_p=0.0),
        # a middling batch over a small vocabulary, rows of many parameters
        dict(name="sample 64 short rows", op="sample", R=64, V=32000, dtype="f16", top_k=-1, top_p=-1.0, min_p=-1.0),
        # a serving batch: top-k, then top-p
        dict(name="sample batch of 256", op="sample", R=256, V=129280, dtype="bf16", top_k=64, top_p=0.9, min_p=0.0),
        # a serving batch whose rows keep what top-p leaves of the whole vocabulary
        dict(name="sample top-p of 128 rows", op="sample", R=128, V=151936, dtype="f32", top_k=0, top_p=0.9, min_p=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    if rng.random() < 0.5:
        K = 16 * _log(rng, 4, 1024)
        N = _log(rng, 16, min(129280, 129280 * 4096 // K))
        T = _log(rng, 1, max(1, min(300, 300 * 8192 * 4096 // (N * K))))
        return dict(op="linear", T=T, N=N, K=K, group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.4,
                    x=rng.choice(["f32", "bf16", "f16", "i8"]), out=rng.choice(["f32", "bf16", "f16"]),
                    bias=rng.random() < 0.3)
    R = _log(rng, 1, 256)
    V = _log(rng, 500, min(160000, 128 * 151936 // R))
    return dict(op="sample", R=R, V=V, dtype=rng.choice(["f32", "bf16", "f16"]),
                top_k=rng.choice([0, 0, -1, 1, _log(rng, 2, V), _log(rng, 2, 100)]),
                top_p=rng.choice([1.0, 1.0, -1.0, rng.uniform(0.05, 0.99), 0.95]),
                min_p=rng.choice([0.0, 0.0, -1.0, rng.uniform(0.001, 0.3)]))


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1013 + 29)


# A row of codes is kept in chunks of 128 values, 16 words of 32 bits: word 4 t + j holds the values 32 j + 8 t .. + 7
# of the chunk, and value i of a word its bits SHIFTS[i] .. + 3.
SHIFTS = [0, 16, 4, 20, 8, 24, 12, 28]


def _pack(q):
    """Codes [n, 128 C] (uint8, 0 .. 15) as the library keeps them: [n, 64 C] bytes."""
    n = q.shape[0]
    v = q.view(n, -1, 4, 4, 8).transpose(2, 3)  # chunk, t, j, value
    w = torch.zeros(v.shape[:-1], dtype=torch.int32, device=q.device)
    for i, s in enumerate(SHIFTS):
        w |= v[..., i].to(torch.int32) << s
    return w.reshape(n, -1).view(torch.uint8)


def _unpack(wq, K):
    """The codes [n, K] (int32) of packed rows."""
    n = wq.shape[0]
    w = wq.view(torch.int32).view(n, -1, 4, 4)
    v = torch.stack([(w >> s) & 15 for s in SHIFTS], dim=-1)
    return v.transpose(2, 3).reshape(n, -1)[:, :K]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=dict(case))
    if case["op"] == "linear":
        T, N, K, G = case["T"], case["N"], case["K"], -(-case["K"] // case["group"])
        C = -(-K // 128)
        s["wq"] = torch.empty((N, 64 * C), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (128 * C))
        for n in range(0, N, step):
            m = min(step, N - n)
            # bell-shaped codes, as rounding a trained matrix's groups leaves them
            q = (torch.randn((m, 128 * C), generator=g, device="cuda") * 3.2 + 8.0).round_().clamp_(0, 15)
            s["wq"][n:n + m] = _pack(q.to(torch.uint8))
        s["ws"] = ((torch.rand((N, G), generator=g, device="cuda") + 0.5) * 4e-3).to(torch.float16)
        s["zeros"] = None
        if case["zeros"]:
            s["zeros"] = torch.randint(5, 12, (N, G), generator=g, device="cuda").to(torch.uint8)
        x = torch.randn((T, K), generator=g, device="cuda")
        hot = torch.randint(0, K, (max(1, K // 512),), generator=g, device="cuda")
        s["xs"] = None
        if case["x"] == "i8":
            s["x"] = (x * 20.0).round_().clamp_(-127, 127).to(torch.int8)
            s["xs"] = (torch.rand(T, generator=g, device="cuda") + 0.5) * 0.03
        else:
            x[:, hot] *= 12.0  # a few channels run much larger than the rest
            s["x"] = x.to(DTYPES[case["x"]])
        s["bias"] = torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["out"] = torch.empty((T, N), dtype=DTYPES[case["out"]], device="cuda")
        return s
    R, V = case["R"], case["V"]
    l = torch.randn((R, V), generator=g, device="cuda") * 2.0
    # the plausible continuations stand out of the rest, as in a trained model's logits
    n = min(40, V // 4)
    ids = torch.randint(0, V, (R, n), generator=g, device="cuda")
    l.scatter_(1, ids, 14.0 - torch.rand((R, n), generator=g, device="cuda").pow_(0.5) * 8.0)
    l[:, 7::13] = -math.inf  # what a grammar has masked
    s["logits"] = l.to(DTYPES[case["dtype"]])
    s["u"] = torch.rand(R, generator=g, device="cuda")
    row = torch.arange(R, device="cuda")
    s["temperature"] = torch.rand(R, generator=g, device="cuda") * 0.9 + 0.4
    if R >= 8:
        s["temperature"][5::8] = 0.0  # greedy rows

    def per_row(value, off, values):
        """None where the filter is off, one value for all, or (value < 0) each row's own."""
        if value == off:
            return None
        if value >= 0:
            return torch.full((R,), value, dtype=values.dtype, device="cuda")
        return values[row % len(values)].contiguous()

    s["top_k"] = per_row(case["top_k"], 0, torch.tensor([0, 1, 40, 7, 1000, 0, 20000, 64], dtype=torch.int32, device="cuda"))
    s["top_p"] = per_row(case["top_p"], 1.0, torch.tensor([0.9, 1.0, 0.5, 0.99, 0.95], device="cuda"))
    s["min_p"] = per_row(case["min_p"], 0.0, torch.tensor([0.0, 0.05, 0.001], device="cuda"))
    s["idx"] = torch.empty(R, dtype=torch.int32, device="cuda")
    s["prob"] = torch.empty(R, dtype=torch.float32, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms
def _plain_linear(s):
    c = s["case"]
    K, g = c["K"], c["group"]
    q = _unpack(s["wq"], K).float()
    of = torch.arange(K, device=q.device) // g
    q -= 8.0 if s["zeros"] is None else s["zeros"].float()[:, of]
    q *= s["ws"].float()[:, of]
    y = s["x"].float() @ q.t()
    if s["xs"] is not None:
        y = y * s["xs"][:, None]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["out"].dtype)


def _column(t, like, off):
    return torch.full((like.shape[0], 1), off, dtype=torch.float64, device=like.device) if t is None else t.double()[:, None]


def _plain_sample(s):
    # (64 bits: a cumulative sum over the vocabulary decides the token)
    l, by = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    R, V = l.shape
    temp = s["temperature"].double()[:, None]
    greedy = temp == 0
    w = torch.exp((l - l[:, :1]) / torch.where(greedy, torch.ones_like(temp), temp))
    place = torch.arange(V, device=l.device)
    k = _column(s["top_k"], l, 0.0)
    k = torch.where(k > 0, k, torch.full_like(k, V))
    k = torch.where(greedy, torch.ones_like(k), k)
    w = torch.where(place < k, w, torch.zeros_like(w))
    p = _column(s["top_p"], l, 1.0)
    before = torch.cumsum(w, dim=1)
    total = before[:, -1:].clone()
    before -= w
    w = torch.where((before < p * total) | (p >= 1.0), w, torch.zeros_like(w))
    w = torch.where(w >= _column(s["min_p"], l, 0.0), w, torch.zeros_like(w))
    kept = torch.zeros_like(w).scatter_(1, by, w)  # in the vocabulary's order
    upto = torch.cumsum(kept, dim=1)
    total = upto[:, -1:].clone()
    idx = ((upto <= s["u"].double()[:, None] * total) | (kept == 0)).to(torch.int8).argmin(dim=1)
    prob = kept.gather(1, idx[:, None]) / total
    return dict(idx=idx.to(torch.int32), prob=prob[:, 0].float())


def run(s):
    op = s["case"]["op"]
    if not own:
        return _plain_linear(s) if op == "linear" else _plain_sample(s)
    from quantized_moe_decode_luce_gb300 import binding as B
    if op == "linear":
        B.luce_linear_w4(s["x"], s["xs"], s["wq"], s["ws"], s["zeros"], s["case"]["group"], s["bias"], s["out"])
        return s["out"]
    B.luce_sample(s["logits"], s["u"], s["idx"], s["prob"], temperature=s["temperature"], top_k=s["top_k"],
                  top_p=s["top_p"], min_p=s["min_p"])
    return dict(idx=s["idx"], prob=s["prob"])


# ----------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "linear":
        T, N, K, G = case["T"], case["N"], case["K"], -(-case["K"] // case["group"])
        b = N * K // 2 + 2 * N * G + T * K * SIZES[case["x"]] + T * N * SIZES[case["out"]]
        b += (N * G if case["zeros"] else 0) + (4 * N if case["bias"] else 0) + (4 * T if case["x"] == "i8" else 0)
        return {"bytes": b, "flops": 2 * T * N * K}
    R, V = case["R"], case["V"]
    per_row = 4 * (2 + 2 + (case["top_k"] != 0) + (case["top_p"] != 1.0) + (case["min_p"] != 0.0))
    return {"bytes": R * V * SIZES[case["dtype"]] + R * per_row, "flops": 4 * R * V}


# ----------------------------------------------------------------------------- definitions in 64 bits
def _exact_linear(s):
    c = s["case"]
    T, N, K, g = c["T"], c["N"], c["K"], c["group"]
    x = s["x"].double() if s["xs"] is None else s["x"].double() * s["xs"].double()[:, None]
    y = torch.empty((T, N), dtype=torch.float64, device="cuda")
    k = torch.arange(K, device="cuda")
    i = k % 8
    byte = 64 * (k // 128) + 16 * (k % 32 // 8) + 4 * (k % 128 // 32) + 2 * (i % 2) + i // 4
    high = (i // 2) % 2 == 1
    step = max(1, (1 << 26) // K)
    for n in range(0, N, step):  # (a slice of the channels at a time: the weights in 64 bits take sixteen times their room)
        b = s["wq"][n:n + step][:, byte]
        v = torch.where(high, b // 16, b % 16).double()
        for m in range(0, K, g):
            z = 8.0 if s["zeros"] is None else s["zeros"][n:n + step, m // g, None].double()
            v[:, m:m + g] = (v[:, m:m + g] - z) * s["ws"][n:n + step, m // g, None].double()
        y[:, n:n + step] = torch.einsum("tk,nk->tn", x, v)
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_row(l, t, k, p, m, u):
    """(token, probability) of one row: the vocabulary's tokens struck off one rule after the other."""
    V = l.numel()
    top = l.max()
    if t == 0:
        return int((l == top).nonzero()[0]), 1.0
    w = torch.exp((l - top) / t)
    order = torch.argsort(l, descending=True, stable=True)
    if 0 < k < V:
        order = order[:k]
    if p < 1.0:
        sums = torch.cat([torch.zeros(1, dtype=w.dtype, device=w.device), w[order].cumsum(0)])
        order = order[:max(1, int((sums[:-1] < p * sums[-1]).sum()))]
    order = order[w[order] >= m]
    ids = torch.sort(order).values
    ids = ids[w[ids] > 0]
    sums = w[ids].cumsum(0)
    at = min(int((sums <= u * sums[-1]).sum()), ids.numel() - 1)
    return int(ids[at]), float(w[ids[at]] / sums[-1])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(s)
    R = case["R"]

    def column(name, off):
        return [off] * R if s[name] is None else s[name].double().tolist()
    rows = zip(s["logits"], column("temperature", 1.0), column("top_k", 0), column("top_p", 1.0), column("min_p", 0.0),
               column("u", 0.0))
    out = [_exact_row(l.double(), t, int(k), p, m, u) for l, t, k, p, m, u in rows]
    return dict(idx=torch.tensor([i for i, _ in out], dtype=torch.int32, device="cuda"),
                prob=torch.tensor([q for _, q in out], dtype=torch.float64, device="cuda"))
