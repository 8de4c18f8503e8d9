"""The routed layer's operators, each in plain torch and as the library's calls.

Four operators that belong together in a mixture-of-experts layer:

* the router: top-k experts and their weights from a token's logits, and its
  backward;
* microscaled 4-bit floating point (e2m1 elements, one e8m0 scale for every 32
  along the contraction): quantizing activation rows and expert weights, and
  reading them back;
* the grouped product with 4-bit weights, its rows in e4m3 with a float scale a
  row or in the same 4-bit format;
* a whole gated expert layer for a few tokens.

``own`` chooses between the plain form (False) and the library (True).
``listed`` and ``draw`` give cases, ``prepare`` their inputs, ``run`` one pass,
``work`` the bytes and operations a pass cannot do without, ``exact`` the
outputs in 64 bits from the definition, written apart from the plain form.
"""

import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
# e2m1 magnitudes by code; bit 3 of a code is the sign
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decoding step of one sequence: a single row of logits, sigmoid scores with the load-balancing
        # bias that only the choice sees; latency is all that counts
        dict(name="router, one token", op="router", T=1, E=256, k=8, dtype="f32", score="sigmoid", bias=True, renorm=True,
             scale=2.5),
        # a prompt's or a training step's tokens over many experts, logits in the layer's own bfloat16 (many ties)
        dict(name="router, a step's tokens", op="router", T=8192, E=256, k=8, dtype="bf16", score="softmax", bias=False,
             renorm=False, scale=1.0),
        # the router's gradient in a training step: the weights' gradients come from the combine's backward
        dict(name="router backward", op="router_bwd", T=32768, E=64, k=8, dtype="f32", score="softmax", renorm=True, scale=1.0),
        # a few rows of an odd width, as a short prompt's tail gives
        dict(name="4-bit rows, few and odd", op="mx4_rows", R=37, C=2080),
        # a step's activations on their way into a 4-bit by 4-bit product
        dict(name="4-bit rows, a step's tokens", op="mx4_rows", R=8192, C=7168),
        # expert weights being converted when a checkpoint is loaded
        dict(name="4-bit weights", op="mx4_weights", E=8, K=7168, N=2048),
        # a small, skewed batch at odd sizes: some experts get nothing, some a single row
        dict(name="product, small and ragged", op="gmm", lhs="e4m3", T=256, k=2, E=8, K=2080, N=1040, skew=2.0),
        # both input projections of one device's experts, activations in 4 bits too
        dict(name="product, 4-bit by 4-bit slice", op="gmm", lhs="mx4", T=1024, k=8, E=32, K=7168, N=4096, skew=0.0),
        # both input projections of a layer with many small experts, e4m3 activations
        dict(name="product, e4m3 by 4-bit layer", op="gmm", lhs="e4m3", T=4096, k=8, E=64, K=2048, N=1536, skew=0.0),
        # decoding one sequence: eight experts' weights stream past one row
        dict(name="layer, one token e4m3", op="ffn", T=1, k=8, E=32, H=7168, I=2048, weights="e4m3", block=128),
        # decoding a small batch with 4-bit weights
        dict(name="layer, 16 tokens 4-bit", op="ffn", T=16, k=8, E=64, H=2048, I=768, weights="mx4", block=0),
        # decoding a larger batch: every expert is met, by a few tokens each
        dict(name="layer, 64 tokens e4m3", op="ffn", T=64, k=8, E=64, H=2048, I=768, weights="e4m3", block=0),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("router", "router_bwd", "mx4_rows", "mx4_weights", "gmm", "gmm", "ffn", "ffn"))
    if op in ("router", "router_bwd"):
        E = rng.choice((8, 13, 32, 64, 72, 128, 160, 256))
        least = 2 if op == "router_bwd" else 1         # the only weight of one, made to sum to 1, is constant: no gradient
        c = dict(op=op, T=_span(rng, 1, 32768), E=E, k=rng.randint(least, min(8, E)), dtype=rng.choice(("f32", "bf16")),
                 score=rng.choice(("softmax", "sigmoid")), renorm=rng.random() < 0.5, scale=rng.choice((1.0, 2.5)))
        if op == "router":
            c["bias"] = rng.random() < 0.5
        return c
    if op == "mx4_rows":
        R = _span(rng, 1, 16384)
        return dict(op=op, R=R, C=32 * _span(rng, 8, max(8, min(256, 58 * (1 << 20) // (32 * R)))))
    if op == "mx4_weights":
        E = rng.randint(1, 8)
        return dict(op=op, E=E, K=32 * _span(rng, 8, 224), N=16 * _span(rng, 4, 128))
    if op == "gmm":
        k = rng.choice((1, 2, 4, 8))
        E = rng.choice((8, 16, 32, 64))
        aligned = rng.random() < 0.5                   # whole tiles, or any size the call takes
        return dict(op=op, lhs=rng.choice(("e4m3", "mx4")), T=_span(rng, 1, 8192 // k), k=k, E=E,
                    K=128 * _span(rng, 2, 32) if aligned else 32 * _span(rng, 8, 128),
                    N=128 * _span(rng, 2, 20) if aligned else 16 * _span(rng, 16, 160), skew=rng.choice((0.0, 0.0, 1.0)))
    weights = rng.choice(("e4m3", "mx4"))
    block = rng.choice((0, 128)) if weights == "e4m3" else 0
    E = rng.choice((8, 16, 32, 64))
    step = 128 if block else 32
    return dict(op=op, T=_span(rng, 1, 64), k=rng.choice((1, 2, 4, 8)), E=E, H=step * _span(rng, 512 // step, 4096 // step),
                I=step * _span(rng, 256 // step, 1024 // step), weights=weights, block=block)


# ----------------------------------------------------------------- the inputs
def _mx4_codes(x):
    """e2m1 codes (0..15) and e8m0 scale codes of rows in float32, blocks of 32 along the last axis: the block's
    scale is the power of two that brings its largest magnitude into [4, 8), 1 for a block of zeros."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    scale = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)
    scale = torch.where(amax == 0, torch.full_like(scale, 127), scale)
    y = b * ((254 - scale) << 23).view(torch.float32).unsqueeze(-1)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + torch.signbit(y).to(torch.uint8) * 8
    return code.reshape(x.shape), scale.to(torch.uint8)


def _mx4_packed(x):
    code, scale = _mx4_codes(x)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _rows_e4m3(x):
    """Per-row absmax quantization: e4m3 bytes and float32 scales."""
    amax = x.abs().amax(-1)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    return (x / s[:, None]).clamp(-448.0, 448.0).to(F8).view(torch.uint8), s


def _routing(gen, T, E, k, skew):
    """Experts of every token without repetition, and their softmax weights."""
    z = torch.randn(T, E, generator=gen, device=DEV)
    if skew:
        z = z - 2.0 * skew * torch.log(1.0 + torch.randperm(E, generator=gen, device=DEV))
    w, ids = torch.softmax(z, -1).sort(dim=-1, descending=True, stable=True)
    return ids[:, :k].to(torch.int32).contiguous(), w[:, :k].contiguous()


def _expert_weights(gen, fmt, E, N, K, block):
    """One weight stack [E, N, K] (contraction last): codes and scales."""
    codes, scales = [], []
    for _ in range(E):
        w = (torch.randn(N, K, generator=gen, device=DEV) * 0.02).bfloat16().float()
        if fmt == "mx4":
            q, s = _mx4_packed(w)
        elif block:
            t = w.view(N // block, block, K // block, block)
            s = t.abs().amax((1, 3)) / 448.0
            q = (t / s[:, None, :, None]).to(F8).view(torch.uint8).view(N, K)
            s = s.t()                                   # [K blocks, N blocks]
        else:
            q, s = _rows_e4m3(w)
            s = s[None, :]                              # [1, N]
        codes.append(q)
        scales.append(s)
    q, s = torch.stack(codes), torch.stack(scales).contiguous()
    return q, s if fmt == "mx4" else s.unsqueeze(2)     # mx4 [E, N, K/32]; e4m3 [E, K blocks, 1, N blocks]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, st = case["op"], {"case": case}
    if op in ("router", "router_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        z = torch.randn(T, E, generator=gen, device=DEV) * 1.5
        if T > 1:
            # experts out of service for some tokens, and padded rows of the batch: no expert is left there
            z.masked_fill_(torch.rand(T, E, generator=gen, device=DEV) < 0.01, -math.inf)
            z.masked_fill_(torch.rand(T, 1, generator=gen, device=DEV) < 0.01, -math.inf)
        st["logits"] = z.to(torch.bfloat16) if case["dtype"] == "bf16" else z
        st["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        st["weights"] = torch.empty(T, k, device=DEV)
        st["bias"] = torch.randn(E, generator=gen, device=DEV) * 0.05 if case.get("bias") else None
        if op == "router_bwd":
            st["ids"] = st["logits"].float().sort(dim=-1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
            st["dweights"] = torch.randn(T, k, generator=gen, device=DEV)
            st["dlogits"] = torch.empty_like(st["logits"])
    elif op == "mx4_rows":
        R, C = case["R"], case["C"]
        x = torch.randn(R, C, generator=gen, device=DEV)
        x *= torch.where(torch.rand(R, 1, generator=gen, device=DEV) < 0.01, 50.0, 1.0)      # outlier tokens
        st["x"] = x.to(torch.bfloat16)
        st["q"] = torch.empty(R, C // 2, dtype=torch.uint8, device=DEV)
        st["s"] = torch.empty(R, C // 32, dtype=torch.uint8, device=DEV)
        st["out"] = torch.empty(R, C, dtype=torch.bfloat16, device=DEV)
    elif op == "mx4_weights":
        E, K, N = case["E"], case["K"], case["N"]
        st["w"] = (torch.randn(E, K, N, generator=gen, device=DEV) * 0.02).to(torch.bfloat16)
        st["q"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
        st["s"] = torch.empty(E, N, K // 32, dtype=torch.uint8, device=DEV)
        st["out"] = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    elif op == "gmm":
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        ids, _ = _routing(gen, T, E, k, case["skew"])
        st["sizes"] = torch.bincount(ids.flatten().long(), minlength=E).to(torch.int32)
        st["longest"] = int(st["sizes"].max())          # the plain form's padding
        x = torch.randn(T * k, K, generator=gen, device=DEV).bfloat16().float()
        st["x"], st["xs"] = _rows_e4m3(x) if case["lhs"] == "e4m3" else _mx4_packed(x)
        st["w"], st["ws"] = _expert_weights(gen, "mx4", E, N, K, 0)
        st["out"] = torch.empty(T * k, N, dtype=torch.bfloat16, device=DEV)
    else:
        T, k, E, H, I = (case[n] for n in ("T", "k", "E", "H", "I"))
        st["ids"], st["weights"] = _routing(gen, T, E, k, 0.0)
        st["x"] = torch.randn(T, H, generator=gen, device=DEV).to(torch.bfloat16)
        st["w01"], st["w01s"] = _expert_weights(gen, case["weights"], E, 2 * I, H, case["block"])
        st["wo"], st["wos"] = _expert_weights(gen, case["weights"], E, H, I, case["block"])
        st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    return st


# ----------------------------------------------------------------- the plain forms
def _unpack(q):
    return torch.stack((q & 15, q >> 4), -1).flatten(-2)


def _mx4_values(code, scale):
    """float32 values of e2m1 codes [..., C] and e8m0 scale codes [..., C/32]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    p = torch.exp2(scale.double() - 127.0).float()
    return (lut[code.long()].unflatten(-1, (-1, 32)) * p.unsqueeze(-1)).flatten(-2)


def _weight_values(q, s, fmt, block):
    """float32 values of a weight stack, contraction last."""
    if fmt == "mx4":
        return _mx4_values(_unpack(q), s)
    w = q.view(F8).float()
    if not block:
        return w * s[:, 0, 0, :, None]
    E, N, K = w.shape
    w = w.view(E, N // block, block, K // block, block)
    return (w * s[:, :, 0, :].transpose(1, 2)[:, :, None, :, None]).view(E, N, K)


def _scores(z, score, dtype):
    """Scores of logits; a row without a finite logit scores nothing."""
    z = z.to(dtype)
    if score == "sigmoid":
        return torch.sigmoid(z)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _router(st):
    c, z = st["case"], st["logits"]
    if st["bias"] is None:              # scores rise with the logits: the logits themselves are in order
        p, key = _scores(z, c["score"], torch.float32), z.float()
    else:                               # in 64 bits: two sums next to each other decide which expert it is
        p = _scores(z, c["score"], torch.float64)
        key = torch.where(z == -math.inf, -math.inf, p + st["bias"].double())
    ids = key.sort(dim=-1, descending=True, stable=True)[1][:, :c["k"]]
    w = p.gather(-1, ids)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _router_bwd(st):
    c, z, ids = st["case"], st["logits"], st["ids"].long()
    p = _scores(z, c["score"], torch.float32)
    g = st["dweights"] * c["scale"]
    pk = p.gather(-1, ids)
    if c["renorm"]:
        total = pk.sum(-1, keepdim=True)
        total = torch.where(total == 0, torch.ones_like(total), total)
        g = (g - (g * pk).sum(-1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_add_(-1, ids, g)
    dz = dp * p * (1 - p) if c["score"] == "sigmoid" else p * (dp - (dp * p).sum(-1, keepdim=True))
    return dz.to(z.dtype)


def _gmm(st):
    c = st["case"]
    x = st["x"].view(F8).float() * st["xs"][:, None] if c["lhs"] == "e4m3" else _mx4_values(_unpack(st["x"]), st["xs"])
    w = _mx4_values(_unpack(st["w"]), st["ws"])
    # the ragged groups as one padded batch: row i of expert e is sorted row start[e] + i
    sizes = st["sizes"].long()
    start = sizes.cumsum(0) - sizes
    i = torch.arange(st["longest"], device=DEV)
    rows = torch.where(i < sizes[:, None], start[:, None] + i, x.shape[0])
    xp = torch.cat((x, x.new_zeros(1, x.shape[1])))[rows]
    y = torch.bmm(xp, w.transpose(1, 2))
    out = x.new_zeros(x.shape[0] + 1, y.shape[2])
    out[rows.flatten()] = y.flatten(0, 1)
    return out[:-1].to(torch.bfloat16)


def _ffn(st):
    c = st["case"]
    T, k, E, H, I = (c[n] for n in ("T", "k", "E", "H", "I"))
    x, ids = st["x"].float(), st["ids"].long()
    if T * k <= E:                      # the chosen experts' weights, one copy a slot
        pick = ids.flatten()
        xe, share = x.repeat_interleave(k, 0).unsqueeze(1), None
    else:                               # every expert over every token; a token's other experts have no weight
        pick = torch.arange(E, device=DEV)
        xe, share = x.expand(E, T, H), torch.zeros(T, E, device=DEV).scatter_add_(1, ids, st["weights"])
    w01 = _weight_values(st["w01"][pick], st["w01s"][pick], c["weights"], c["block"])
    wo = _weight_values(st["wo"][pick], st["wos"][pick], c["weights"], c["block"])
    ab = torch.bmm(xe, w01.transpose(1, 2))
    a, b = ab[..., :I], ab[..., I:]
    y = torch.bmm(a / (1 + torch.exp(-a)) * b, wo.transpose(1, 2))
    y = y.view(T, k, H) * st["weights"][..., None] if share is None else (y * share.t()[..., None]).transpose(0, 1)
    return y.sum(1).to(torch.bfloat16)


# ----------------------------------------------------------------- one pass
_kept = {}


def _workspace(m, op, d0, d1, d2, E):
    """The workspace that a program keeps from call to call."""
    key = (op, d0, d1, d2, E)
    if key not in _kept:
        _kept[key] = m.workspace(op, d0, d1, d2, E)
    return _kept[key]


def _own(st):
    import moe_fp8_grouped_amd as m
    c, op = st["case"], st["case"]["op"]
    if op in ("router", "router_bwd"):
        T, E, k, z = c["T"], c["E"], c["k"], st["logits"]
        dt = m.MOE_BF16 if c["dtype"] == "bf16" else m.MOE_F32
        score = m.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else m.MOE_SCORE_SOFTMAX
        if op == "router":
            m.moe_router_topk(z, dt, E, T, E, k, score, st["bias"], int(c["renorm"]), c["scale"], st["ids"], st["weights"])
            return st["ids"], st["weights"]
        m.moe_router_topk_backward(z, dt, E, st["ids"], st["dweights"], T, E, k, score, int(c["renorm"]), c["scale"],
                                   st["dlogits"], E)
        return st["dlogits"]
    if op == "mx4_rows":
        R, C = c["R"], c["C"]
        m.moe_quantize_rows_mx4(st["x"], None, C, m.MOE_ACT_NONE, R, C, st["q"], C // 2, st["s"], C // 32)
        m.moe_dequantize_rows_mx4(st["q"], C // 2, st["s"], C // 32, R, C, m.MOE_BF16, st["out"], C)
        return st["out"]
    if op == "mx4_weights":
        E, K, N = c["E"], c["K"], c["N"]
        m.moe_quantize_weights_mx4(st["w"], E, K, N, st["q"], st["s"])
        m.moe_dequantize_rows_mx4(st["q"].view(E * N, -1), K // 2, st["s"].view(E * N, -1), K // 32, E * N, K, m.MOE_BF16,
                                  st["out"].view(E * N, K), K)
        return st["out"]
    if op == "gmm":
        M, E, K, N = c["T"] * c["k"], c["E"], c["K"], c["N"]
        a8 = c["lhs"] == "e4m3"
        m.moe_gmm_mx4(st["x"], K if a8 else K // 2, st["xs"], 0 if a8 else K // 32, m.MOE_E4M3FN if a8 else m.MOE_MX4,
                      m.MOE_SCALE_ROW_DYNAMIC, st["w"], st["ws"], st["sizes"], E, 0, E, M, K, N, m.MOE_BF16, st["out"],
                      _workspace(m, m.MOE_OP_GMM_MX4, M, K, N, E))
        return st["out"]
    T, k, E, H, I = (c[n] for n in ("T", "k", "E", "H", "I"))
    f8 = c["weights"] == "e4m3"
    s01, so = st["w01s"], st["wos"]
    m.moe_ffn_tokens(st["x"], H, st["ids"], st["weights"], T, k, H, I, E, 0, E, m.MOE_E4M3FN if f8 else m.MOE_MX4,
                     st["w01"], s01, s01.shape[1] if f8 else 0, s01.shape[3] if f8 else 0, st["wo"], so,
                     so.shape[1] if f8 else 0, so.shape[3] if f8 else 0, m.MOE_BF16, st["out"],
                     _workspace(m, m.MOE_OP_FFN_TOKENS, T * k, H, I, E))
    return st["out"]


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    if op == "router":
        return _router(st)
    if op == "router_bwd":
        return _router_bwd(st)
    if op == "mx4_rows":
        return _mx4_values(*_mx4_codes(st["x"].float())).to(torch.bfloat16)
    if op == "mx4_weights":
        return _mx4_values(*_mx4_codes(st["w"].float().transpose(1, 2).contiguous())).to(torch.bfloat16)
    return _gmm(st) if op == "gmm" else _ffn(st)


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("router", "router_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * E * size * (1 if op == "router" else 2) + T * k * 8, "flops": 6 * T * E}
    if op in ("mx4_rows", "mx4_weights"):
        n = case["R"] * case["C"] if op == "mx4_rows" else case["E"] * case["K"] * case["N"]
        return {"bytes": 2 * n + n * 17 // 32 + 2 * n, "flops": 4 * n}    # values in, codes and scales out, values read back
    if op == "gmm":
        M, E, K, N = case["T"] * case["k"], case["E"], case["K"], case["N"]
        met = E * (1 - (1 - case["k"] / E) ** case["T"])                   # experts that get a row, where none is preferred
        lhs = M * (K + 4) if case["lhs"] == "e4m3" else M * K * 17 // 32
        return {"bytes": int(lhs + met * N * K * 17 / 32 + 2 * M * N), "flops": 2 * M * K * N}
    T, k, E, H, I = (case[n] for n in ("T", "k", "E", "H", "I"))
    met = E * (1 - (1 - k / E) ** T)
    a_weight = 1.0 if case["weights"] == "e4m3" else 17 / 32
    return {"bytes": int(met * 3 * H * I * a_weight + 4 * T * H + 8 * T * k), "flops": 6 * T * k * H * I}


# ----------------------------------------------------------------- in 64 bits, from the definitions
def _nearest4(x):
    """The nearest value of the block format to each of float64 rows [R, C], ties to the even code."""
    out = torch.empty_like(x)
    even_first = torch.tensor([E2M1[i] for i in (0, 2, 4, 6, 1, 3, 5, 7)], dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // x.shape[1])
    for r in range(0, x.shape[0], step):
        b = x[r:r + step].reshape(-1, 32)
        top = b.abs().amax(1, keepdim=True)
        p = torch.exp2(torch.floor(torch.log2(torch.where(top == 0, 4.0, top))).clamp(min=-125.0) - 2)
        v = b / p
        best = (v.abs().unsqueeze(-1) - even_first).abs().argmin(-1)
        out[r:r + step] = (torch.copysign(even_first[best], v) * p).reshape(-1, x.shape[1])
    return out


def _read4(q, s):
    """float64 values of packed codes [N, C/2] and scales [N, C/32]."""
    N, C = q.shape[0], 2 * q.shape[1]
    v = torch.empty(N, C, dtype=torch.float64, device=q.device)
    for half, c in ((0, q & 15), (1, q >> 4)):
        e, f, sign = (c >> 1) & 3, (c & 1).double(), 1.0 - 2.0 * (c >> 3).double()
        v[:, half::2] = sign * torch.where(e == 0, f / 2, (1 + f / 2) * torch.exp2(e.double() - 1))
    return v * torch.exp2(s.double() - 127.0).repeat_interleave(32, 1)


def _read8(q, s, block):
    """float64 values of one expert's e4m3 weight [N, K] with scales [K blocks, 1, N blocks]."""
    w, s = q.view(F8).double(), s[:, 0, :].double().t()
    return w * (s.repeat_interleave(block, 0).repeat_interleave(block, 1) if block else s)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("router", "router_bwd"):
        z, k = st["logits"].double(), case["k"]
        if case["score"] == "softmax":
            p = torch.nan_to_num(torch.exp(z - torch.logsumexp(z, -1, keepdim=True)), nan=0.0)
        else:
            p = 0.5 + 0.5 * torch.tanh(z / 2)
        if op == "router":
            choice = z if st["bias"] is None else torch.where(torch.isinf(z), z, p + st["bias"].double())
            ids = torch.argsort(choice, dim=-1, descending=True, stable=True)[:, :k]
        else:
            ids = st["ids"].long()
        one = torch.nn.functional.one_hot(ids, case["E"]).double()                     # [T, k, E]
        w = (one * p[:, None]).sum(-1)
        total = w.sum(-1, keepdim=True).clamp(min=1e-300) if case["renorm"] else torch.ones_like(w[:, :1])
        if op == "router":
            return ids.to(torch.int32), w / total * case["scale"]
        r, g = w / total, st["dweights"].double() * case["scale"]
        if case["renorm"] and case["score"] == "softmax":        # a softmax over the chosen logits
            d = r * (g - (g * r).sum(-1, keepdim=True))
            return (one * d[..., None]).sum(1)
        if case["renorm"]:
            g = (g - (g * r).sum(-1, keepdim=True)) / total
        d = g * w
        if case["score"] == "sigmoid":
            return (one * (d * (1 - w))[..., None]).sum(1)
        return (one * d[..., None]).sum(1) - p * d.sum(-1, keepdim=True)
    if op == "mx4_rows":
        return _nearest4(st["x"].double())
    if op == "mx4_weights":
        E, K, N = case["E"], case["K"], case["N"]
        return torch.stack([_nearest4(st["w"][e].double().t().contiguous()) for e in range(E)])
    if op == "gmm":
        x = st["x"].view(F8).double() * st["xs"].double()[:, None] if case["lhs"] == "e4m3" else _read4(st["x"], st["xs"])
        out, r = torch.zeros(x.shape[0], case["N"], dtype=torch.float64, device=DEV), 0
        for e, n in enumerate(st["sizes"].tolist()):
            if n:
                out[r:r + n] = x[r:r + n] @ _read4(st["w"][e], st["ws"][e]).t()
            r += n
        return out
    out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
    ids, x = st["ids"].tolist(), st["x"].double()
    for e in sorted({e for row in ids for e in row}):
        t = [i for i, row in enumerate(ids) if e in row]
        j = [ids[i].index(e) for i in t]
        w01, wo = ((_read4(st[n][e], st[n + "s"][e]) if case["weights"] == "mx4" else _read8(st[n][e], st[n + "s"][e], case["block"]))
                   for n in ("w01", "wo"))
        a, b = (x[t] @ w01.t()).chunk(2, -1)
        out[t] += st["weights"].double()[t, j][:, None] * ((a * torch.sigmoid(a) * b) @ wo.t())
    return out
