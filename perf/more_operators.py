"""The block-scaled expert layer's operators and the router's balance loss, each in plain torch and as the library's calls.

Five operators that belong together in training and serving a mixture-of-experts layer in 8-bit floating point
with a scale for every block of 128 (e4m3 elements, power-of-two scales):

* the quantizers: activation rows (plain, or silu(a) * b), and expert weights in
  blocks of 128 by 128, both orientations in one pass;
* the grouped product of such rows and weights (one group: a linear layer; one
  row: decoding), the weights' scales e8m0 or float32;
* the weight gradient: both operands quantized along the rows of each group,
  straight from bfloat16, and their product per group;
* the router's balance loss with the experts' counts, and its gradient.

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
E8 = torch.float8_e8m0fnu
B = 128                                     # elements that share a scale
OUT_OF_SERVICE = -1e30                      # logits at or below it (and NaN) take their expert out


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # a few rows of an odd width, as a short prompt's tail gives; the last block of a row is a quarter full
        dict(name="rows, few and odd", op="rows", R=37, C=2080, gated=False),
        # a step's activations on their way into a product
        dict(name="rows, a step's tokens", op="rows", R=8192, C=7168, gated=False),
        # expert weights after an optimizer step: the forward's and the input gradient's orientation
        dict(name="weights, both orientations", op="weights", E=8, K=7168, N=2048),
        # decoding one sequence through a linear layer, float scales as checkpoints hold them; latency is what counts
        dict(name="product, one token", op="product", T=1, k=1, E=1, K=7168, N=4096, skew=0.0, scales="f32"),
        # decoding a small batch: most experts are met, by a row or two each
        dict(name="product, 16 tokens of 64 experts", op="product", T=16, k=8, E=64, K=2048, N=1536, skew=0.0, scales="e8m0"),
        # a small, skewed batch at odd sizes: some experts get nothing, some a single row
        dict(name="product, small and ragged", op="product", T=256, k=2, E=8, K=2080, N=1040, skew=2.0, scales="e8m0"),
        # a prompt through a layer of many small experts, float scales as checkpoints hold them
        dict(name="product, layer of 64 experts", op="product", T=4096, k=8, E=64, K=2048, N=1536, skew=0.0, scales="f32"),
        # both input projections of one device's experts in a training step
        dict(name="product, slice of 32 experts", op="product", T=1024, k=8, E=32, K=7168, N=4096, skew=0.0, scales="e8m0"),
        # the weight gradient of a small, skewed batch at odd sizes
        dict(name="weight gradient, small and ragged", op="wgrad", T=256, k=2, E=8, K=2080, N=1040, skew=2.0, gated=False),
        # an input projection's weight gradient in a training step: tokens gathered by the routing, many experts
        dict(name="weight gradient, 64 experts", op="wgrad", T=8192, k=4, E=64, K=4096, N=1536, skew=0.0, gated=False),
        # a step's tokens over many experts, logits in the layer's own bfloat16, a few packed sequences
        dict(name="balance loss, a step's tokens", op="balance", T=8192, E=256, k=8, dtype="bf16", score="softmax", S=5),
        # the gradient in a training step, over packed sequences of ragged length
        dict(name="balance loss backward", op="balance_bwd", T=32768, E=64, k=8, dtype="f32", score="sigmoid", S=24),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rows", "weights", "product", "product", "product", "wgrad", "wgrad", "balance", "balance_bwd"))
    if op in ("balance", "balance_bwd"):
        E, T = rng.choice((8, 13, 32, 64, 72, 128, 160, 256)), _span(rng, 1, 32768)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E - 1)), dtype=rng.choice(("f32", "bf16")),
                    score=rng.choice(("softmax", "sigmoid")), S=_span(rng, 1, max(1, min(T, 64))))
    if op == "rows":
        R = _span(rng, 1, 16384)
        return dict(op=op, R=R, C=16 * _span(rng, 8, max(8, min(512, 56 * (1 << 20) // (16 * R)))), gated=rng.random() < 0.5)
    if op == "weights":
        return dict(op=op, E=rng.randint(1, 8), K=16 * _span(rng, 8, 448), N=16 * _span(rng, 4, 128))
    k = rng.choice((1, 2, 4, 8))
    E = rng.choice((1, 8, 16, 32, 64)) if op == "product" else rng.choice((1, 8, 16, 32))
    k = min(k, E)
    aligned = rng.random() < 0.5                       # whole tiles, or any size the call takes
    K = 128 * _span(rng, 2, 32) if aligned else 16 * _span(rng, 8, 256)
    N = 128 * _span(rng, 2, 20) if aligned else 16 * _span(rng, 16, 160)
    T = _span(rng, 1, 8192 // k)
    c = dict(op=op, T=T, k=k, E=E, K=K, N=N, skew=rng.choice((0.0, 0.0, 1.0)))
    if op == "product":
        c["scales"] = rng.choice(("e8m0", "f32"))
    else:
        c["gated"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------- the inputs
def _pad(x, dim, m=B):
    """x with zeros up to a whole number of blocks along dim."""
    n = -x.shape[dim] % m
    if not n:
        return x
    shape = list(x.shape)
    shape[dim] = n
    return torch.cat((x, x.new_zeros(shape)), dim)


def _scale_code(amax):
    """e8m0 code of the smallest power of two, at least 2^-127, with amax <= 448 times it; 127 for zero."""
    bits = amax.view(torch.int32)
    code = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=0)
    return torch.where(amax == 0, torch.full_like(code, 127), code)


def _power(code):
    """float32 of e8m0 codes."""
    return torch.exp2(code.double() - 127.0).float()


def _block_rows(x):
    """e4m3 elements [..., C] and e8m0 codes [..., C / 128 rounded up] of float32 rows."""
    C = x.shape[-1]
    b = _pad(x, -1).unflatten(-1, (-1, B))
    code = _scale_code(b.abs().amax(-1))
    q = (b * _power(254 - code).unsqueeze(-1)).to(F8)
    return q.flatten(-2)[..., :C].contiguous(), code.to(torch.uint8)


def _tiles(w):
    """Blocks of 128 by 128 of the last two dimensions, padded: [..., a, 128, b, 128]."""
    return _pad(_pad(w, -1), -2).unflatten(-1, (-1, B)).unflatten(-3, (-1, B))


def _block_weights(w, scales):
    """One weight [N, K] float32: e4m3 elements and scales [K blocks, N blocks], e8m0 codes or float32."""
    N, K = w.shape
    t = _tiles(w)
    amax = t.abs().amax((1, 3))
    if scales == "e8m0":
        code = _scale_code(amax)
        q, s = t * _power(254 - code)[:, None, :, None], code.to(torch.uint8)
    else:
        s = amax / 448.0
        q = t / s[:, None, :, None]
    return q.to(F8).flatten(2, 3).flatten(0, 1)[:N, :K], s.t()


def _routing(gen, T, E, k, skew):
    """Experts of every token, without repetition."""
    z = torch.randn(T, E, generator=gen, device=DEV)
    if skew:
        z = z - 2.0 * skew * torch.log(1.0 + torch.randperm(E, generator=gen, device=DEV))
    return z.sort(dim=-1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()


def _bf16(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def _with_outliers(gen, x):
    x.mul_(torch.where(torch.rand(x.shape[0], 1, generator=gen, device=DEV) < 0.01, 50.0, 1.0).to(x.dtype))
    return x


def _wide(C):
    """Bytes from one quantized row to the next: elements, scales, up to a multiple of 16."""
    return C + -(-(-(-C // B)) // 16) * 16


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, st = case["op"], {"case": case}
    if op == "rows":
        R, C = case["R"], case["C"]
        st["x"] = _with_outliers(gen, _bf16(gen, R, C))
        st["up"] = _bf16(gen, R, C) if case["gated"] else None
        st["rows"] = torch.empty(R, _wide(C), dtype=torch.uint8, device=DEV)
    elif op == "weights":
        E, K, N = case["E"], case["K"], case["N"]
        kb, nb = -(-K // B), -(-N // B)
        st["w"] = _bf16(gen, E, K, N, scale=0.02)
        st["q"], st["qt"] = (torch.empty(E, *s, dtype=torch.uint8, device=DEV) for s in ((N, K), (K, N)))
        st["s"], st["s_t"] = (torch.empty(E, a, 1, b, dtype=torch.uint8, device=DEV) for a, b in ((kb, nb), (nb, kb)))
    elif op in ("product", "wgrad"):
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        ids = _routing(gen, T, E, k, case["skew"])
        M = T * k
        st["sizes"] = torch.bincount(ids.flatten().long(), minlength=E).to(torch.int32)
        st["perm"] = ids.flatten().argsort(stable=True).to(torch.int32)
        st["longest"] = int(st["sizes"].max())          # the plain form's padding
        if op == "product":
            # sorted rows as the quantizer leaves them: elements and scales side by side
            q, s = _block_rows(_with_outliers(gen, _bf16(gen, M, K)).float())
            st["rows"] = torch.zeros(M, _wide(K), dtype=torch.uint8, device=DEV)
            st["rows"][:, :K] = q.view(torch.uint8)
            st["rows"][:, K:K + s.shape[1]] = s
            w = [_block_weights(_bf16(gen, N, K, scale=0.02).float(), case["scales"]) for _ in range(E)]
            st["w"] = torch.stack([q.view(torch.uint8) for q, _ in w])
            st["ws"] = torch.stack([s for _, s in w]).unsqueeze(2).contiguous()            # [E, K blocks, 1, N blocks]
            st["out"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        else:
            # tokens that the routing gathers, or the two halves of the input projections' output, in sorted order
            st["x"] = _bf16(gen, M, 2 * K) if case["gated"] else _with_outliers(gen, _bf16(gen, T, K))
            st["dy"] = _bf16(gen, M, N, scale=1e-3)
            st["cols"] = 256 * -(-(M + B * E) // 256)
            for n, c in (("xt", K), ("dyt", N)):
                st[n] = torch.empty(c, st["cols"], dtype=torch.uint8, device=DEV)
                st[n + "_s"] = torch.empty(st["cols"] // B, c, dtype=torch.uint8, device=DEV)
            st["dw"] = torch.empty(E, K, N, dtype=torch.bfloat16, device=DEV)
    else:
        T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
        z = torch.randn(T, E, generator=gen, device=DEV) * 1.5 + torch.randn(E, generator=gen, device=DEV) * 0.5
        if T > 1:
            # experts out of service for some tokens, and padded rows of the batch: no expert is left there
            z.masked_fill_(torch.rand(T, E, generator=gen, device=DEV) < 0.01, -math.inf)
            z.masked_fill_(torch.rand(T, 1, generator=gen, device=DEV) < 0.01, -math.inf)
        st["logits"] = z = z.to(torch.bfloat16) if case["dtype"] == "bf16" else z
        # the choice is made with the selection bias on
        key = z.float() + torch.randn(E, generator=gen, device=DEV) * 0.1
        st["ids"] = key.sort(dim=-1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
        # packed sequences of ragged length, empty ones among them; some rows behind the last one
        cuts = (torch.rand(S + 1, generator=gen, device=DEV).sort()[0] * (T + 1)).floor().clamp(max=T)
        cuts[0], cuts[S] = 0, T - T // 16
        st["offsets"] = cuts.clamp(max=T - T // 16).to(torch.int32)
        seg = torch.searchsorted(st["offsets"].long(), torch.arange(T, device=DEV), right=True) - 1
        st["seg"] = torch.where(seg < S, seg, S)         # the plain form's: row S is nobody's
        st["loss"] = torch.empty(S, device=DEV)
        st["counts"] = torch.empty(S, E, dtype=torch.int32, device=DEV)
        st["tokens"] = torch.empty(S, dtype=torch.int32, device=DEV)
        if op == "balance_bwd":
            st["dloss"] = torch.rand(S, generator=gen, device=DEV) + 0.5
            st["counts"], st["tokens"] = _counts(st)
            st["dlogits"] = torch.zeros_like(z)
    if own:
        st["workspace"] = _workspace(case)
    return st


# ----------------------------------------------------------------- the plain forms
def _silu_mul(a, b):
    return a / (1 + torch.exp(-a)) * b


def _values(q, code):
    """float32 values of e4m3 elements [..., C] with e8m0 codes [..., C / 128 rounded up]."""
    C = q.shape[-1]
    return (_pad(q.float(), -1).unflatten(-1, (-1, B)) * _power(code).unsqueeze(-1)).flatten(-2)[..., :C]


def _padded(x, sizes, longest):
    """The ragged groups [M, C] as one padded batch [E, longest, C], and each slot's row (M: none)."""
    sizes = sizes.long()
    i = torch.arange(longest, device=DEV)
    rows = torch.where(i < sizes[:, None], (sizes.cumsum(0) - sizes)[:, None] + i, x.shape[0])
    return torch.cat((x, x.new_zeros(1, x.shape[1])))[rows], rows


def _weights(st):
    w = st["w"].float()                                 # [E, K, N]
    E, K, N = w.shape
    t = _tiles(w)                                       # [E, K blocks, 128, N blocks, 128]
    code = _scale_code(t.abs().amax((2, 4)))
    q = (t * _power(254 - code)[:, :, None, :, None]).to(F8).view(torch.uint8)
    q = q.flatten(3, 4).flatten(1, 2)[:, :K, :N].contiguous()
    code = code.to(torch.uint8)
    return (q.transpose(1, 2).contiguous().view(F8), code.unsqueeze(2).view(E8), q.view(F8),
            code.transpose(1, 2).contiguous().unsqueeze(2).view(E8))


def _product(st):
    c = st["case"]
    K, N = c["K"], c["N"]
    x = _values(st["rows"][:, :K].view(F8), st["rows"][:, K:K + -(-K // B)])
    s = st["ws"][:, :, 0].transpose(1, 2)               # [E, N blocks, K blocks]
    s = _power(s) if c["scales"] == "e8m0" else s
    w = (_tiles(st["w"].view(F8).float()) * s[:, :, None, :, None]).flatten(3, 4).flatten(1, 2)[:, :N, :K]
    xp, rows = _padded(x, st["sizes"], st["longest"])
    y = torch.bmm(xp, w.transpose(1, 2))
    out = x.new_zeros(x.shape[0] + 1, N)
    out[rows.flatten()] = y.flatten(0, 1)
    return out[:-1].to(torch.bfloat16)


def _along_rows(x, st):
    """Rows [M, C], quantized in blocks of 128 of each group's rows: the values, [E, longest up to a block, C]."""
    t = _pad(_padded(x, st["sizes"], st["longest"])[0], 1).unflatten(1, (-1, B))
    code = _scale_code(t.abs().amax(2, keepdim=True))
    return ((t * _power(254 - code)).to(F8).float() * _power(code)).flatten(1, 2)


def _wgrad(st):
    c = st["case"]
    K = c["K"]
    if c["gated"]:
        x = _silu_mul(st["x"][:, :K].float(), st["x"][:, K:].float())
    else:
        x = st["x"][st["perm"].long() // c["k"]].float()
    return torch.bmm(_along_rows(x, st).transpose(1, 2), _along_rows(st["dy"].float(), st)).to(torch.bfloat16)


def _counts(st):
    """Choices of each expert and rows that have an expert, per sequence."""
    c, z, ids = st["case"], st["logits"], st["ids"].long()
    here = z > OUT_OF_SERVICE
    hit = torch.zeros(c["T"], c["E"], device=DEV).scatter_(1, ids, 1.0) * here
    member = _member(st, torch.float32)                 # (whole numbers below 2^24: exact)
    return (member @ hit).to(torch.int32), (member @ here.any(-1, keepdim=True).float())[:, 0].to(torch.int32)


def _member(st, dtype):
    """[S, T]: 1 where the token is the sequence's."""
    return (st["seg"] == torch.arange(st["case"]["S"], device=DEV)[:, None]).to(dtype)


def _shares(z, score):
    """A row's scores as shares that sum to 1 (0 for a row without an expert), in 64 bits, and 1 - sigmoid."""
    z = torch.where(z > OUT_OF_SERVICE, z.double(), -math.inf)
    v, rest = z, None
    if score == "sigmoid":
        e = torch.exp(-z.abs())
        v, rest = z.clamp(max=0.0) - torch.log1p(e), torch.where(z < 0, 1 / (1 + e), e / (1 + e))
    top = v.amax(-1, keepdim=True)
    e = torch.exp(v - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total), rest


def _balance(st):
    c = st["case"]
    counts, tokens = _counts(st)
    p, _ = _shares(st["logits"], c["score"])
    P = _member(st, torch.float64) @ p
    n = tokens.double().clamp(min=1)
    return ((P * counts).sum(-1) * c["E"] / (c["k"] * n * n)).float(), counts, tokens


def _balance_bwd(st):
    c = st["case"]
    p, rest = _shares(st["logits"], c["score"])
    n = st["tokens"].double().clamp(min=1)
    factor = torch.cat((st["dloss"].double() * c["E"] / (c["k"] * n * n), n.new_zeros(1)))[st["seg"]]
    counts = torch.cat((st["counts"].double(), p.new_zeros(1, c["E"])))[st["seg"]]
    d = factor[:, None] * p * (counts - (counts * p).sum(-1, keepdim=True))
    return (d if rest is None else d * rest).to(st["logits"].dtype)


# ----------------------------------------------------------------- one pass
def _workspace(case):
    """The workspace that a program keeps beside its buffers (and a pass on another stream has one of its own)."""
    import moe_fp8_grouped_amd as m
    if case["op"] in ("product", "wgrad"):
        op = m.MOE_OP_GMM_B128 if case["op"] == "product" else m.MOE_OP_TGMM_B128
        return m.workspace(op, case["T"] * case["k"], case["K"], case["N"], case["E"])
    return m.workspace(m.MOE_OP_BALANCE, case["T"], case["S"], 0, case["E"]) if case["op"] == "balance" else None


def _own(st):
    import moe_fp8_grouped_amd as m
    c, op = st["case"], st["case"]["op"]
    if "workspace" not in st:
        st["workspace"] = _workspace(c)
    if op == "rows":
        R, C, rows, up = c["R"], c["C"], st["rows"], st["up"]
        ld, kb = rows.shape[1], -(-C // B)
        q, s = rows[:, :C], rows[:, C:C + kb]
        m.moe_quantize_rows_b128(st["x"], up, C, m.MOE_ACT_NONE if up is None else m.MOE_ACT_SILU_MUL, R, C, q, ld, s, ld)
        return q.view(F8), s.view(E8)
    if op == "weights":
        m.moe_quantize_weights_b128(st["w"], c["E"], c["K"], c["N"], st["q"], st["s"], st["qt"], st["s_t"])
        return st["q"].view(F8), st["s"].view(E8), st["qt"].view(F8), st["s_t"].view(E8)
    if op == "product":
        M, E, K, N, rows = c["T"] * c["k"], c["E"], c["K"], c["N"], st["rows"]
        ld, kb = rows.shape[1], -(-K // B)
        m.moe_gmm_b128(rows[:, :K], ld, rows[:, K:K + kb], ld, st["w"], st["ws"],
                       m.MOE_E8M0 if c["scales"] == "e8m0" else m.MOE_F32, st["sizes"], E, 0, E, M, K, N, m.MOE_BF16,
                       st["out"], st["workspace"])
        return st["out"]
    if op == "wgrad":
        T, k, E, K, N = (c[n] for n in ("T", "k", "E", "K", "N"))
        M, x, sizes = T * k, st["x"], st["sizes"]
        ws = st["workspace"]
        if c["gated"]:
            m.moe_quantize_cols_b128(x[:, :K], x[:, K:], 2 * K, m.MOE_ACT_SILU_MUL, M, 1, None, sizes, E, 0, E, M, K,
                                     st["xt"], st["xt_s"], ws)
        else:
            m.moe_quantize_cols_b128(x, None, K, m.MOE_ACT_NONE, T, k, st["perm"], sizes, E, 0, E, M, K, st["xt"],
                                     st["xt_s"], ws)
        m.moe_quantize_cols_b128(st["dy"], None, N, m.MOE_ACT_NONE, M, 1, None, sizes, E, 0, E, M, N, st["dyt"],
                                 st["dyt_s"], ws)
        m.moe_tgmm_b128(st["xt"], st["xt_s"], st["dyt"], st["dyt_s"], sizes, E, 0, E, M, K, N, m.MOE_BF16, st["dw"], ws)
        return st["dw"]
    T, E, k, S, z = c["T"], c["E"], c["k"], c["S"], st["logits"]
    dt = m.MOE_BF16 if c["dtype"] == "bf16" else m.MOE_F32
    score = m.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else m.MOE_SCORE_SOFTMAX
    if op == "balance":
        m.moe_balance_loss(z, dt, E, st["ids"], T, E, k, score, st["offsets"], S, st["loss"], st["counts"], st["tokens"],
                           st["workspace"])
        return st["loss"], st["counts"], st["tokens"]
    m.moe_balance_loss_backward(z, dt, E, st["counts"], st["tokens"], st["dloss"], T, E, k, score, st["offsets"], S, 0,
                                st["dlogits"], E)
    return st["dlogits"]


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    if op == "rows":
        x = st["x"].float()
        q, s = _block_rows(x if st["up"] is None else _silu_mul(x, st["up"].float()))
        return q, s.view(E8)
    return {"weights": _weights, "product": _product, "wgrad": _wgrad, "balance": _balance, "balance_bwd": _balance_bwd}[op](st)


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "rows":
        n = case["R"] * case["C"]
        inputs = 2 if case["gated"] else 1
        return {"bytes": 2 * n * inputs + n + case["R"] * -(-case["C"] // B), "flops": (8 if case["gated"] else 3) * n}
    if op == "weights":
        n = case["E"] * case["K"] * case["N"]
        return {"bytes": 2 * n + 2 * n, "flops": 3 * n}
    if op in ("product", "wgrad"):
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        M = T * k
        if op == "product":
            met = E * (1 - (1 - k / E) ** T)                               # experts that get a row, where none is preferred
            return {"bytes": int(M * (K + -(-K // B)) + met * N * K + 2 * M * N), "flops": 2 * M * K * N}
        x = 2 * M * 2 * K if case["gated"] else 2 * T * K
        return {"bytes": x + 2 * M * N + 2 * E * K * N, "flops": 2 * M * K * N}
    T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
    z = T * E * (2 if case["dtype"] == "bf16" else 4)
    return {"bytes": z + 4 * T * k + 4 * S * E if op == "balance" else 2 * z + 4 * S * E, "flops": 6 * T * E}


# ----------------------------------------------------------------- in 64 bits, from the definitions
def _table():
    """The finite e4m3 magnitudes, even codes first, so that the first of two nearest is the even one."""
    c = torch.arange(127, device=DEV)
    e, f = (c >> 3).double(), (c & 7).double()
    v = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2(e - 7))
    return torch.cat((v[0::2], v[1::2]))


def _exact_scale(top):
    """The smallest power of two, at least 2^-127, that brings top to 448 at most; 1 for zero."""
    p = torch.ceil(torch.log2(torch.where(top == 0, 1.0, top) / 448.0)).clamp(min=-127.0)
    p = torch.where(top > 448.0 * torch.exp2(p), p + 1, p)
    p = torch.where((top <= 448.0 * torch.exp2(p - 1)) & (p > -127.0), p - 1, p)
    return torch.where(top == 0, 1.0, torch.exp2(p))


def _nearest8(v):
    """The e4m3 value nearest to each of v (at most 448 in magnitude), ties to the even code."""
    flat, table = v.reshape(-1), _table()
    order = table.sort()[0]
    out = torch.empty_like(flat)
    for i in range(0, flat.numel(), 1 << 24):
        a = flat[i:i + (1 << 24)].abs()
        hi = torch.searchsorted(order, a).clamp(max=126)                    # the value at or above, and the one below
        lo = (hi - 1).clamp(min=0)
        below, above = a - order[lo], order[hi] - a
        up = (above < below) | ((above == below) & (hi % 2 == 0))
        out[i:i + (1 << 24)] = torch.copysign(torch.where(up, order[hi], order[lo]), flat[i:i + (1 << 24)])
    return out.view_as(v)


def _exact_rows(x):
    """Elements and scales of float64 rows [R, C], block by block."""
    q, s = torch.empty_like(x), x.new_empty(x.shape[0], -(-x.shape[1] // B))
    for b in range(s.shape[1]):
        v = x[:, b * B:(b + 1) * B]
        s[:, b] = _exact_scale(v.abs().amax(1))
        q[:, b * B:(b + 1) * B] = _nearest8(v / s[:, b:b + 1])
    return q, s


def _spread(s, n0, n1):
    """Block scales [a, b] over the [n0, n1] elements they belong to."""
    return s.repeat_interleave(B, 0)[:n0].repeat_interleave(B, 1)[:, :n1]


def _exact_share(z, score):
    z = torch.where(torch.isnan(z) | (z <= OUT_OF_SERVICE), -math.inf, z)
    if score == "softmax":
        return torch.nan_to_num(torch.exp(z - torch.logsumexp(z, -1, keepdim=True)), nan=0.0), None
    sigma = 0.5 + 0.5 * torch.tanh(z / 2)
    return sigma / sigma.sum(-1, keepdim=True).clamp(min=1e-300), sigma


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "rows":
        x = st["x"].double()
        return _exact_rows(x if st["up"] is None else x * torch.sigmoid(x) * st["up"].double())
    if op == "weights":
        K, N = case["K"], case["N"]
        q, s = torch.empty(st["w"].shape, dtype=torch.float64, device=DEV), []
        for e in range(case["E"]):
            w = st["w"][e].double()
            top = torch.nn.functional.max_pool2d(w.abs()[None, None], B, ceil_mode=True)[0, 0]
            s.append(_exact_scale(top))
            q[e] = _nearest8(w / _spread(s[-1], K, N))
        s = torch.stack(s)
        return q.transpose(1, 2).contiguous(), s.unsqueeze(2), q, s.transpose(1, 2).contiguous().unsqueeze(2)
    if op == "product":
        K, N, r = case["K"], case["N"], 0
        kb = -(-K // B)
        x = st["rows"][:, :K].contiguous().view(F8).double()
        x *= torch.exp2(st["rows"][:, K:K + kb].double() - 127.0).repeat_interleave(B, 1)[:, :K]
        out = torch.zeros(x.shape[0], N, dtype=torch.float64, device=DEV)
        for e, n in enumerate(st["sizes"].tolist()):
            if n:
                s = st["ws"][e, :, 0].t().double()
                s = torch.exp2(s - 127.0) if case["scales"] == "e8m0" else s
                out[r:r + n] = x[r:r + n] @ (st["w"][e].view(F8).double() * _spread(s, N, K)).t()
            r += n
        return out
    if op == "wgrad":
        K, N, r = case["K"], case["N"], 0
        out = torch.zeros(case["E"], K, N, dtype=torch.float64, device=DEV)
        for e, n in enumerate(st["sizes"].tolist()):
            x, dy = st["x"][r:r + n].double(), st["dy"][r:r + n].double()
            if case["gated"]:
                x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
            else:
                x = st["x"][st["perm"][r:r + n].long() // case["k"]].double()
            if n:                                       # blocks along the rows: rows of the transpose
                (xq, xs), (dq, ds) = _exact_rows(x.t().contiguous()), _exact_rows(dy.t().contiguous())
                out[e] = (xq * xs.repeat_interleave(B, 1)[:, :n]) @ (dq * ds.repeat_interleave(B, 1)[:, :n]).t()
            r += n
        return out
    T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
    z, ids, off = st["logits"].double(), st["ids"].long(), st["offsets"].tolist()
    p, sigma = _exact_share(z, case["score"])
    there = (z > OUT_OF_SERVICE)
    loss, counts, tokens = [], [], []
    d = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    for s in range(S):
        a, b = off[s], off[s + 1]
        n = int(there[a:b].any(1).sum())
        one = torch.nn.functional.one_hot(ids[a:b].flatten(), E).view(b - a, k, E).sum(1) * there[a:b]
        c = one.sum(0)
        factor = E / (k * n * n) if n else 0.0
        loss.append(factor * float((c * p[a:b].sum(0)).sum()))
        counts.append(c)
        tokens.append(n)
        if op == "balance_bwd":
            g = c - (p[a:b] * c).sum(1, keepdim=True)
            d[a:b] = float(st["dloss"][s]) * factor * p[a:b] * g * (1 if sigma is None else 1 - sigma[a:b])
    if op == "balance_bwd":
        return d
    return (torch.tensor(loss, dtype=torch.float64, device=DEV), torch.stack(counts).to(torch.int32),
            torch.tensor(tokens, dtype=torch.int32, device=DEV))
