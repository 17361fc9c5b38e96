"""Cases, plain forms and 64-bit definitions of the int8 decode-head operators.

The operators around the routed-MoE step of a decoder that keeps its dense matrices in int8:

* ``quantize``  rows of activations (or weights) to int8 codes with one scale per row;
* ``norm``      the residual's addition, the root-mean-square norm of the sum, int8 codes with one scale per row;
* ``linear``    the product of int8 activations with int8 weights, scales per token and per channel, optional bias;
* ``logits``    penalties for repeated tokens, per-token biases and grammar masks on a batch of logits.

``run`` computes them with elementary torch operations, or, where ``own`` is true, with the library's calls.
``exact`` computes the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one token between two layers of the decode stack: pure latency
        dict(name="norm, one token", op="norm", T=1, H=2048, dtype="f32", residual=True),
        # a long prompt's rows in the residual stream's type: bandwidth, a ragged token count
        dict(name="norm, 8191 rows f32", op="norm", T=8191, H=4096, dtype="f32", residual=True),
        # the verify step's five columns before a dense projection
        dict(name="quantize, five rows", op="quantize", T=5, H=4096, dtype="bf16"),
        # a prompt's attention outputs before the output projection; rows that are no multiple of 16 bytes
        dict(name="quantize, 4095 odd rows", op="quantize", T=4095, H=4099, dtype="bf16"),
        # a small projection for a single token: latency
        dict(name="linear, one token", op="linear", T=1, N=2048, K=2048, out="f32", bias=False),
        # the vocabulary head over the verify step's columns: every weight read once from memory
        dict(name="linear, head of 5", op="linear", T=5, N=129280, K=4096, out="f32", bias=False),
        # a batch of decoding sequences through one projection: weights still bound it, the products no longer fit one column
        dict(name="linear, batch of 61", op="linear", T=61, N=4096, K=4096, out="bf16", bias=True),
        # a prompt chunk through a projection of the prefill layer
        dict(name="linear, chunk of 512", op="linear", T=512, N=8192, K=4096, out="bf16", bias=False),
        # long prompts together: bound by the products; ragged tokens
        dict(name="linear, 4093 tokens", op="linear", T=4093, N=4096, K=4096, out="bf16", bias=False),
        # one sequence, its history and a grammar: latency
        dict(name="logits, one row", op="logits", R=1, V=129280, dtype="f32", hist=4096, prompt=1024, bias=0, mask=True),
        # the verify step's columns with penalties and biases, odd vocabulary
        dict(name="logits, five rows", op="logits", R=5, V=129279, dtype="f32", hist=2000, prompt=500, bias=300, mask=True),
        # a serving batch with long histories, half precision logits
        dict(name="logits, batch of 256", op="logits", R=256, V=129280, dtype="bf16", hist=32768, prompt=16384, bias=32, mask=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear", "linear", "logits", "logits"])
    if op in ("norm", "quantize"):
        H = _log(rng, 64, 16384)
        T = _log(rng, 1, max(1, min(8191, 8191 * 4096 // H)))
        c = dict(op=op, T=T, H=H, dtype=rng.choice(["f32", "bf16", "f16"]))
        if op == "norm":
            c["residual"] = rng.random() < 0.7
        return c
    if op == "linear":
        K = 16 * _log(rng, 4, 1024)
        N = _log(rng, 16, min(129280, 129280 * 4096 // K))
        T = _log(rng, 1, max(1, min(4093, 4093 * 4096 * 4096 // (N * K))))
        return dict(op=op, T=T, N=N, K=K, out=rng.choice(["f32", "bf16", "f16"]), bias=rng.random() < 0.3)
    R = _log(rng, 1, 256)
    V = _log(rng, 1000, min(160000, 256 * 129280 // R))
    hist = _log(rng, 16, 32768)
    return dict(op=op, R=R, V=V, dtype=rng.choice(["f32", "bf16", "f16"]), hist=hist,
                prompt=rng.randrange(0, hist), bias=rng.choice([0, 0, 1, 30, 300]), mask=rng.random() < 0.6)


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1009 + 17)


def _codes(rows, cols, sigma, g):
    """int8 codes as the row quantizer leaves them: bell-shaped, each within [-127, 127]."""
    q = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        q[r:r + n] = (torch.randn((n, cols), generator=g, device="cuda") * sigma).round_().clamp_(-127, 127).to(torch.int8)
    return q


def _hist_lens(case):
    """Tokens in each row's history: between half of the longest and all of it."""
    L = case["hist"]
    return [L - (r * 7919) % (L // 2 + 1) for r in range(case["R"])]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=dict(case))
    if case["op"] in ("norm", "quantize"):
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        x = torch.randn((T, H), generator=g, device="cuda")
        # a few channels run much larger than the rest, as in the residual stream of a trained model
        hot = torch.randint(0, H, (max(1, H // 512),), generator=g, device="cuda")
        x[:, hot] *= 20.0
        if T > 4:
            x[T - 1] = 0.0  # a padding row
        s["x"] = x.to(dt)
        s["q"] = torch.empty((T, H), dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(T, dtype=torch.float32, device="cuda")
        if case["op"] == "norm":
            s["gamma"] = torch.rand(H, generator=g, device="cuda") + 0.5
            if case["residual"]:
                r = torch.randn((T, H), generator=g, device="cuda") * 0.5
                if T > 4:
                    r[T - 1] = 0.0
                s["residual"] = r.to(dt)
                s["x_sum"] = torch.empty((T, H), dtype=dt, device="cuda")
        return s
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        s["xq"] = _codes(T, K, 20.0, g)
        s["xs"] = (torch.rand(T, generator=g, device="cuda") + 0.5) * 0.03
        s["wq"] = _codes(N, K, 31.0, g)
        s["ws"] = (torch.rand(N, generator=g, device="cuda") + 0.5) * 1e-3
        s["bias"] = torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["out"] = torch.empty((T, N), dtype=DTYPES[case["out"]], device="cuda")
        return s
    R, V, L = case["R"], case["V"], case["hist"]
    s["logits"] = (torch.randn((R, V), generator=g, device="cuda") * 3.0).to(DTYPES[case["dtype"]])
    lens = _hist_lens(case)
    # frequent tokens come back often: cubes of uniform numbers crowd the low ids
    ids = (torch.rand((R, L), generator=g, device="cuda").pow_(3) * V).to(torch.int32).clamp_(0, V - 1)
    s["hist"] = ids
    s["hist_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["prompt_len"] = torch.tensor([min(case["prompt"], n) for n in lens], dtype=torch.int32, device="cuda")
    s["rep"] = torch.rand(R, generator=g, device="cuda") * 0.3 + 1.0
    s["freq"] = torch.rand(R, generator=g, device="cuda") * 0.5
    s["pres"] = torch.rand(R, generator=g, device="cuda") * 0.5
    s["bias_ids"] = s["bias_vals"] = s["mask"] = s["mask_rows"] = None
    if case["bias"]:
        b = case["bias"]
        # distinct ids in each row: one of each of b equal stretches of the vocabulary
        first = torch.arange(b, device="cuda") * V // b
        s["bias_ids"] = (first + torch.randint(0, V // b, (R, b), generator=g, device="cuda")).to(torch.int32)
        s["bias_vals"] = torch.randn((R, b), generator=g, device="cuda") * 4.0
    if case["mask"]:
        m, words = max(1, R // 2), (V + 31) // 32
        full = torch.randint(-2**31, 2**31, (m, words), generator=g, device="cuda", dtype=torch.int64)
        rare = torch.rand((m, words), generator=g, device="cuda") < 0.05
        full[0::2] *= rare[0::2]  # every second grammar state allows few tokens
        if m > 3:
            full[m - 1] = 0  # a dead end: nothing is allowed
        s["mask"] = full.to(torch.int32)
        rows = torch.arange(R, dtype=torch.int32, device="cuda") % m
        if R >= 4:
            rows[3::4] = -1  # rows without a grammar
        s["mask_rows"] = rows
    s["out"] = torch.empty((R, V), dtype=torch.float32, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms
def _half_away(v):
    """Nearest whole number, halves away from zero (exact in 32 bits for |v| < 2^22)."""
    t = torch.trunc(v)
    return t + torch.sign(v) * ((v - t).abs() >= 0.5)


def _row_codes(p):
    """(codes, step) of rows p in 32 bits: step = max|p| / 127, codes = round(p / step)."""
    m = p.abs().amax(dim=1, keepdim=True)
    d = m / torch.full_like(m, 127.0)
    q = _half_away(p / torch.where(d > 0, d, torch.ones_like(d))).clamp(-127.0, 127.0)
    return q.to(torch.int8), d[:, 0]


def _plain_quantize(s):
    q, d = _row_codes(s["x"].float())
    return dict(q=q, scale=d)


def _plain_norm(s):
    x = s["x"]
    out = {}
    if "residual" in s:
        x = (x.float() + s["residual"].float()).to(x.dtype)
        out["x_sum"] = x
    v = x.float()
    r = 1.0 / torch.sqrt(v.square().mean(dim=1) + EPS)
    out["q"], d = _row_codes(v * s["gamma"])
    out["scale"] = d * r
    return out


def _plain_linear(s):
    y = s["xq"].float() @ s["wq"].float().t()
    y = y * (s["xs"][:, None] * s["ws"][None, :])
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["out"].dtype)


def _plain_logits(s):
    l = s["logits"].float()
    R, V = l.shape
    hist = s["hist"].long()
    pos = torch.arange(hist.shape[1], device=hist.device)
    live = pos < s["hist_len"][:, None]
    new = live & (pos >= s["prompt_len"][:, None])
    seen = torch.zeros((R, V), dtype=torch.int32, device=l.device).scatter_add_(1, hist, live.to(torch.int32))
    count = torch.zeros((R, V), dtype=torch.int32, device=l.device).scatter_add_(1, hist, new.to(torch.int32))
    rep = s["rep"][:, None]
    l = torch.where(seen > 0, torch.where(l > 0, l / rep, l * rep), l)
    l = torch.where(count > 0, l - (count * s["freq"][:, None] + s["pres"][:, None]), l)
    if s["bias_ids"] is not None:
        ids = s["bias_ids"].long()
        l.scatter_(1, ids, l.gather(1, ids) + s["bias_vals"])
    if s["mask"] is not None:
        m = s["mask"][s["mask_rows"].clamp(min=0).long()]
        bits = (m[:, :, None] >> torch.arange(32, dtype=torch.int32, device=l.device)) & 1
        allowed = (bits.reshape(R, -1)[:, :V] == 1) | (s["mask_rows"] < 0)[:, None]
        l = torch.where(allowed, l, torch.full_like(l, -math.inf))
    return l


def run(s):
    op = s["case"]["op"]
    if not own:
        return dict(norm=_plain_norm, quantize=_plain_quantize, linear=_plain_linear, logits=_plain_logits)[op](s)
    from quantized_moe_decode_luce_gb300 import binding as B
    if op == "quantize":
        B.luce_quantize_i8(s["x"], s["q"], s["scale"])
        return dict(q=s["q"], scale=s["scale"])
    if op == "norm":
        if "residual" in s:
            B.luce_add_rmsnorm_i8(s["x"], s["residual"], s["x_sum"], s["gamma"], EPS, s["q"], s["scale"])
            return dict(x_sum=s["x_sum"], q=s["q"], scale=s["scale"])
        B.luce_rmsnorm_i8(s["x"], s["gamma"], EPS, s["q"], s["scale"])
        return dict(q=s["q"], scale=s["scale"])
    if op == "linear":
        B.luce_linear_i8(s["xq"], s["xs"], s["wq"], s["ws"], s["bias"], s["out"])
        return s["out"]
    B.luce_logits_process(s["logits"], s["out"], hist=s["hist"], hist_len=s["hist_len"], prompt_len=s["prompt_len"],
                          repetition=s["rep"], frequency=s["freq"], presence=s["pres"], bias_ids=s["bias_ids"],
                          bias_vals=s["bias_vals"], mask=s["mask"], mask_rows=s["mask_rows"])
    return s["out"]


# ----------------------------------------------------------------------------- work
def work(case):
    if case["op"] in ("norm", "quantize"):
        T, H, e = case["T"], case["H"], SIZES[case["dtype"]]
        moved = 1
        if case["op"] == "norm":
            moved = 3 if case["residual"] else 1
        gamma = 4 * H if case["op"] == "norm" else 0
        return {"bytes": T * H * (e * moved + 1) + 4 * T + gamma, "flops": 8 * T * H}
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": N * K + T * K + 4 * (N + T) + T * N * SIZES[case["out"]] + (4 * N if case["bias"] else 0),
                "flops": 2 * T * N * K}
    R, V = case["R"], case["V"]
    b = R * V * (SIZES[case["dtype"]] + 4) + 4 * sum(_hist_lens(case)) + 20 * R + 8 * R * case["bias"]
    if case["mask"]:
        b += 4 * ((V + 31) // 32) * max(1, R // 2) + 4 * R
    return {"bytes": b, "flops": 6 * R * V}


# ----------------------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        # the codes are whole numbers: they are compared as such
        return dict(q=None, scale=s["x"].double().abs().max(dim=1).values / 127.0)
    if case["op"] == "norm":
        out, x = {}, s["x"].double()
        if "residual" in s:
            # the norm reads the sum that is stored, in the type of the stream
            x = (x + s["residual"].double()).to(DTYPES[case["dtype"]]).double()
            out["x_sum"] = x
        rms = torch.linalg.vector_norm(x, dim=1).square() / case["H"] + EPS
        out["q"] = None
        out["scale"] = (x * s["gamma"].double()).abs().max(dim=1).values / (127.0 * rms.sqrt())
        return out
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        if 2.0 * T * N * K > 3e12:
            return None
        y = torch.empty((T, N), dtype=torch.float64, device="cuda")
        x = s["xq"].double()
        step = max(1, (1 << 27) // K)
        for n in range(0, N, step):  # (a slice of the channels at a time: the weights in 64 bits take eight times their room)
            y[:, n:n + step] = torch.mm(x, s["wq"][n:n + step].double().T) * s["ws"][n:n + step].double()
        y *= s["xs"].double()[:, None]
        return y if s["bias"] is None else y + s["bias"].double()
    R, V = case["R"], case["V"]
    out = s["logits"].double()
    hist, hl, pl = s["hist"].long(), s["hist_len"].tolist(), s["prompt_len"].tolist()
    mrows = s["mask_rows"].tolist() if s["mask"] is not None else [-1] * R
    word, bit = torch.arange(V, device="cuda") // 32, torch.arange(V, device="cuda") % 32
    for r in range(R):
        row = out[r]
        rep, freq, pres = (float(s[k][r]) for k in ("rep", "freq", "pres"))
        once = torch.unique(hist[r, :hl[r]])
        v = row[once]
        row[once] = torch.maximum(v, torch.zeros_like(v)) / rep + torch.minimum(v, torch.zeros_like(v)) * rep
        ids, times = torch.unique(hist[r, pl[r]:hl[r]], return_counts=True)
        row[ids] -= times.double() * freq + pres
        if s["bias_ids"] is not None:
            row[s["bias_ids"][r].long()] += s["bias_vals"][r].double()
        if mrows[r] >= 0:
            words = s["mask"][mrows[r]].long() & 0xFFFFFFFF
            row[((words[word] >> bit) & 1) == 0] = -math.inf
    return out
