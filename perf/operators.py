"""The language-model operators beside the scoring core, as measurable cases.

Four operators of a head and its training step, in the sizes a scoring,
training or serving program meets:

* ``quantize``: e4m3 codes with one fp32 scale per 128 values of a row
  (activations and gradients, as they lie or transposed) or per 128 x 128 tile
  (weights);
* ``matmul``: the product of two such operands, each 128-block of the
  reduction scaled by its own pair of scales;
* ``logprobs``: log probabilities of given tokens under rows of logits, the
  rows' log-sum-exp and entropy, and their top alternatives;
* ``logprobs_grad``: the gradient of those log probabilities, log-sum-exps and
  entropies with respect to the logits.

With ``own`` false ``run`` computes the plain form in 32 bits with elementary
torch operations; with ``own`` true it calls this package.  ``exact`` is the
definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
IGNORE = -100


def listed():
    return [
        # one new token's hidden state, quantized before the head
        dict(name="quantize_one_row", op="quantize", R=1, C=5120, dtype="bf16", block="row", transpose=False),
        # a micro-batch's hidden states, quantized along the tokens for a weight gradient
        dict(name="quantize_columns", op="quantize", R=16384, C=5120, dtype="bf16", block="row", transpose=True),
        # an fp32 master weight after an optimizer step
        dict(name="quantize_weight", op="quantize", R=32000, C=2048, dtype="fp32", block="tile", transpose=False),
        # the head on one new token: every weight byte is read for one row
        dict(name="matmul_one_token", op="matmul", M=1, N=151936, K=5120, out="bf16", b_block="tile"),
        # a ragged serving batch with fp32 logits
        dict(name="matmul_33_tokens", op="matmul", M=33, N=32000, K=2048, out="fp32", b_block="tile"),
        # the head on a training batch
        dict(name="matmul_head", op="matmul", M=8192, N=128256, K=4096, out="bf16", b_block="tile"),
        # a weight gradient: both operands scaled per row and 128 tokens
        dict(name="matmul_weight_gradient", op="matmul", M=32000, N=2048, K=4096, out="fp32", b_block="row"),
        # one generated token with its 20 top alternatives
        dict(name="logprobs_one_row", op="logprobs", T=1, V=151936, pad=0, dtype="bf16", K=1, top=20,
             temperature=True, mask=False),
        # a ragged batch under a grammar mask, odd vocabulary and row stride
        dict(name="logprobs_masked_odd", op="logprobs", T=301, V=32001, pad=2, dtype="fp16", K=5, top=5,
             temperature=True, mask=True),
        # replayed tokens of a training batch with their alternatives
        dict(name="logprobs_batch", op="logprobs", T=8192, V=128256, pad=0, dtype="bf16", K=1, top=20,
             temperature=False, mask=False),
        # a small distillation batch, 64 tokens a row, some of them given twice
        dict(name="logprobs_grad_distill", op="logprobs_grad", T=257, V=32001, pad=2, dtype="fp32", K=64,
             temperature=True, mask=True),
        # the logits' gradient of a training batch
        dict(name="logprobs_grad_batch", op="logprobs_grad", T=8192, V=128256, pad=0, dtype="bf16", K=1,
             temperature=False, mask=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("quantize", "matmul", "logprobs", "logprobs_grad"))
    if op == "quantize":
        C = _log_int(rng, 1, 8192)
        R = _log_int(rng, 1, min(32768, 80_000_000 // C))
        return dict(op=op, R=R, C=C, dtype=rng.choice(("bf16", "fp16", "fp32")), block=rng.choice(("row", "tile")),
                    transpose=rng.choice((False, True)))
    if op == "matmul":
        K = 16 * _log_int(rng, 1, 512)
        N = _log_int(rng, 1, 150_000)
        M = _log_int(rng, 1, max(1, min(16384, int(4e12 / (N * K)), 10**9 // N)))
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(("bf16", "fp16", "fp32")),
                    b_block=rng.choice(("tile", "row")))
    V = _log_int(rng, 2, 200_000)
    T = _log_int(rng, 1, min(8192, 10**9 // V))
    c = dict(op=op, T=T, V=V, pad=rng.choice((0, 0, 1, 7, 64)), dtype=rng.choice(("bf16", "fp16", "fp32")),
             K=_log_int(rng, 1, 100), temperature=rng.choice((False, True)), mask=rng.choice((False, True)))
    if op == "logprobs":
        c["top"] = rng.choice((0, 1, _log_int(rng, 1, 128)))
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _codes(gen, rows, cols):
    """e4m3 codes of normal values whose blocks reach 448 or nearly."""
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(0.0, 120.0, generator=gen)
    return x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _logits(gen, c):
    """Logits of a trained head: a broad bulk and a few likely tokens a row;
    with a mask, a grammar that allows one token in eight, and some rows
    nothing at all."""
    T, V = c["T"], c["V"]
    buf = torch.empty(T, V + c["pad"], dtype=DTYPES[c["dtype"]], device="cuda").normal_(0.0, 2.0, generator=gen)
    z = buf[:, :V]
    top = torch.randint(0, V, (T, min(8, V)), generator=gen, device="cuda")
    z.scatter_(1, top, (torch.rand(top.shape, generator=gen, device="cuda") * 8 + 4).to(z.dtype))
    if c["mask"]:
        z.masked_fill_(torch.rand(T, V, generator=gen, device="cuda") >= 0.125, -math.inf)
        z[3::97] = -math.inf
    tokens = torch.randint(0, V, (T, c["K"]), generator=gen, device="cuda")
    k = min(c["K"], top.shape[1])
    tokens[:, :k] = top[:, :k]
    if c["K"] > 2:
        tokens[:, -1] = tokens[:, 0]        # the same token twice
    tokens[1::7, c["K"] // 2] = IGNORE      # places without a token
    temperature = torch.rand(T, generator=gen, device="cuda") + 0.5 if c["temperature"] else None
    return z, tokens, temperature


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] == "quantize":
        # hidden states or weights with a few large channels
        s["x"] = torch.empty(c["R"], c["C"], dtype=DTYPES[c["dtype"]], device="cuda").normal_(generator=gen)
        s["x"][:, 5::509] *= 30
        if c["R"] > 4:
            s["x"][4, : 2 * BLOCK] = 0      # blocks of zeros (padding tokens)
    elif c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        kb = -(-K // BLOCK)
        nb = -(-N // BLOCK) if c["b_block"] == "tile" else N
        s["a"], s["b"] = _codes(gen, M, K), _codes(gen, N, K)
        # one scale per block; the block index runs slowest in memory
        s["a_scale"] = torch.rand(kb, M, generator=gen, device="cuda").add_(0.5).mul_(8e-3).t()
        s["b_scale"] = torch.rand(kb, nb, generator=gen, device="cuda").add_(0.5).mul_(2e-4).t()
    else:
        s["z"], s["tokens"], s["temperature"] = _logits(gen, c)
        if c["op"] == "logprobs_grad":
            T, K = s["tokens"].shape
            # what the forward left: the row's largest logit, the log of the
            # sum of exponentials over it, and the entropy
            t = torch.ones(T, device="cuda") if s["temperature"] is None else s["temperature"]
            m, log_sum, entropy, _ = _row_statistics(s["z"], t)
            s["stats"] = torch.stack((m, log_sum, entropy, torch.zeros_like(m)), 1)
            s["g_logprob"] = torch.randn(T, K, generator=gen, device="cuda") / T
            s["g_entropy"] = torch.full((T,), -1e-2 / T, device="cuda")
            s["g_lse"] = torch.randn(T, generator=gen, device="cuda") * (1e-2 / T)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _quantize_rows(x):
    """codes and scales of the 128-blocks of x's rows, the row padded to a
    multiple of 16 with zeros"""
    R, C = x.shape
    kb = -(-C // BLOCK)
    p = torch.zeros(R, kb * BLOCK, device=x.device)
    p[:, :C] = x
    p = p.view(R, kb, BLOCK)
    scale = p.abs().amax(2) / E4M3_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = (p / scale[:, :, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(R, kb * BLOCK)
    return q[:, : -(-C // 16) * 16].contiguous(), scale


def _quantize_tiles(x):
    R, C = x.shape
    rb, kb = -(-R // BLOCK), -(-C // BLOCK)
    p = torch.zeros(rb * BLOCK, kb * BLOCK, device=x.device)
    p[:R, :C] = x
    p = p.view(rb, BLOCK, kb, BLOCK)
    scale = p.abs().amax((1, 3)) / E4M3_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = (p / scale[:, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(rb * BLOCK, kb * BLOCK)[:R, : -(-C // 16) * 16].contiguous(), scale


def _dequantize(q, scale, rows_per_scale):
    K = q.shape[1]
    s = scale.repeat_interleave(BLOCK, 1)[:, :K]
    if rows_per_scale > 1:
        s = s.repeat_interleave(rows_per_scale, 0)[: q.shape[0]]
    return q.float() * s


def _row_statistics(z, t):
    """(largest logit, log sum of exp((z - largest) / t), entropy, exponents)"""
    z = z.float()
    m = z.amax(1)
    d = (z - torch.where(m == -math.inf, 0.0, m)[:, None]) / t[:, None]
    e = d.exp()
    total = e.sum(1)
    log_sum = total.log()
    mean = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1) / total
    entropy = torch.where(m == -math.inf, torch.zeros_like(m), log_sum - mean)
    return m, log_sum, entropy, d


def _top(z, n):
    """values and ids of the n largest logits above -inf, the lower id first
    among equal ones; id -1 where a row has no more"""
    V = z.shape[1]
    k = min(n, V)
    bits = (z.float() + 0.0).view(torch.int32).to(torch.int64)     # (+ 0.0: one zero)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    order = order * 2**32 + (V - 1 - torch.arange(V, device=z.device))
    ids = V - 1 - (order.topk(k, 1).values & 0xFFFFFFFF)
    values = z.gather(1, ids).float()
    ids = torch.where(values == -math.inf, torch.full_like(ids, -1), ids)
    if k < n:
        values = torch.cat((values, values.new_full((len(z), n - k), -math.inf)), 1)
        ids = torch.cat((ids, ids.new_full((len(z), n - k), -1)), 1)
    return values, ids


def _plain_logprobs(c, z, tokens, temperature):
    t = torch.ones(len(z), device=z.device) if temperature is None else temperature
    m, log_sum, entropy, d = _row_statistics(z, t)
    empty = (m == -math.inf)[:, None]
    given = tokens != IGNORE
    logprob = d.gather(1, tokens.clamp(min=0)) - log_sum[:, None]
    logprob = torch.where(empty, torch.full_like(logprob, -math.inf), logprob)
    logprob = torch.where(given, logprob, torch.zeros_like(logprob))
    out = dict(logprob=logprob, lse=m / t + log_sum, entropy=entropy)
    if c["top"]:
        values, ids = _top(z, c["top"])
        lp = (values - torch.where(empty, 0.0, m[:, None])) / t[:, None] - log_sum[:, None]
        out["top_logprob"] = torch.where(ids < 0, torch.full_like(lp, -math.inf), lp)
        out["top_id"] = ids
    return out


def _plain_logprobs_grad(s):
    z, tokens, g, stats = s["z"], s["tokens"], s["g_logprob"], s["stats"]
    t = torch.ones(len(z), device=z.device) if s["temperature"] is None else s["temperature"]
    m, log_sum, entropy = stats[:, 0], stats[:, 1], stats[:, 2]
    empty = m == -math.inf
    logp = (z.float() - torch.where(empty, 0.0, m)[:, None]) / t[:, None] - log_sum[:, None]
    p = logp.exp()
    # a masked token scores -inf and passes no gradient
    given = (tokens != IGNORE) & (z.gather(1, tokens.clamp(min=0)) > -math.inf)
    g = torch.where(given, g, torch.zeros_like(g))
    slope = s["g_lse"] - g.sum(1)
    dz = p * (slope[:, None] - s["g_entropy"][:, None] * (logp + entropy[:, None]))
    dz = torch.where(p > 0, dz, torch.zeros_like(dz))
    dz.scatter_add_(1, tokens.clamp(min=0), g)
    dz = dz / t[:, None]
    dz = torch.where(empty[:, None], torch.zeros_like(dz), dz)
    return dz.to(z.dtype)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from sampling_transform_logprob_amd import binding
        if op == "quantize":
            codes, scale = binding.fp8_quantize_blocks(s["x"], block=c["block"], transpose=c["transpose"])
            return dict(codes=codes, scale=scale)
        if op == "matmul":
            return binding.fp8_block_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=DTYPES[c["out"]])
        if op == "logprobs":
            out = binding.token_logprobs(s["z"], s["tokens"], s["temperature"], top_n=c["top"], ignore_index=IGNORE,
                                         check=False)
            return {k: out[k] for k in ("logprob", "lse", "entropy", "top_logprob", "top_id") if k in out}
        return binding.token_logprobs_backward(s["z"], s["tokens"], s["stats"], s["g_logprob"], s["g_entropy"],
                                               s["g_lse"], temperature=s["temperature"], ignore_index=IGNORE)
    if op == "quantize":
        x = s["x"].t() if c["transpose"] else s["x"]
        codes, scale = (_quantize_rows if c["block"] == "row" else _quantize_tiles)(x)
        return dict(codes=codes, scale=scale)
    if op == "matmul":
        a = _dequantize(s["a"], s["a_scale"], 1)
        b = _dequantize(s["b"], s["b_scale"], BLOCK if c["b_block"] == "tile" else 1)
        return (a @ b.t()).to(DTYPES[c["out"]])
    if op == "logprobs":
        return _plain_logprobs(c, s["z"], s["tokens"], s["temperature"])
    return _plain_logprobs_grad(s)


def work(case):
    c = case
    if c["op"] == "quantize":
        R, C = (c["C"], c["R"]) if c["transpose"] else (c["R"], c["C"])
        rows = R if c["block"] == "row" else -(-R // BLOCK)
        return dict(bytes=R * C * BYTES[c["dtype"]] + R * (-(-C // 16) * 16) + 4 * rows * -(-C // BLOCK),
                    flops=2 * R * C)
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        nb = -(-N // BLOCK) if c["b_block"] == "tile" else N
        return dict(bytes=M * K + N * K + 4 * -(-K // BLOCK) * (M + nb) + M * N * BYTES[c["out"]],
                    flops=2 * M * N * K)
    T, V, K = c["T"], c["V"], c["K"]
    size = T * V * BYTES[c["dtype"]]
    if c["op"] == "logprobs":
        return dict(bytes=size + T * (12 * K + 8 + 12 * c["top"]) + 4 * T * c["temperature"], flops=6 * T * V)
    return dict(bytes=2 * size + T * (12 * K + 24) + 4 * T * c["temperature"], flops=8 * T * V)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e4m3(v):
    """The nearest e4m3 value of every |v| <= 448, ties to the even mantissa."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0**-6))) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantize":
        x = s["x"].double()
        x = x.t() if c["transpose"] else x
        rows = 1 if c["block"] == "row" else BLOCK
        R, C = x.shape
        x = torch.nn.functional.pad(x, (0, -C % BLOCK, 0, -R % rows))
        t = x.reshape(x.shape[0] // rows, rows, x.shape[1] // BLOCK, BLOCK)
        scale = t.abs().amax((1, 3), keepdim=True) / E4M3_MAX
        scale[scale == 0] = 1
        codes = _e4m3(t / scale).reshape(x.shape)[:R, : C + -C % 16]
        return dict(codes=codes.contiguous(), scale=scale[:, 0, :, 0].contiguous())
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        col = torch.arange(K, device="cuda") // BLOCK
        a = s["a"].double() * s["a_scale"].double()[:, col]
        out = torch.empty(M, N, dtype=torch.float64, device="cuda")
        for n0 in range(0, N, 16384):
            n = torch.arange(n0, min(N, n0 + 16384), device="cuda")
            row = n // BLOCK if c["b_block"] == "tile" else n
            b = s["b"].view(torch.uint8)[n].view(torch.float8_e4m3fn).double() * s["b_scale"].double()[row][:, col]
            out[:, n] = a @ b.t()
        return out
    T, V = c["T"], c["V"]
    parts = []
    step = max(1, 2**27 // V)
    for r in range(0, T, step):
        z = s["z"][r:r + step].double().requires_grad_(c["op"] == "logprobs_grad")
        n = len(z)
        t = torch.ones(n, dtype=torch.float64, device="cuda")
        if s["temperature"] is not None:
            t = s["temperature"][r:r + step].double()
        tok = s["tokens"][r:r + step]
        dead = (z == -math.inf).all(1)
        x = torch.where(dead[:, None], torch.zeros_like(z), z) / t[:, None]
        lse = torch.logsumexp(x, 1)
        logp = x - lse[:, None]
        entropy = -(logp.exp() * logp.masked_fill(logp == -math.inf, 0.0)).sum(1)
        picked = logp.gather(1, tok.clamp(min=0))
        if c["op"] == "logprobs_grad":
            w = s["g_logprob"][r:r + step].double().masked_fill((tok == IGNORE) | (picked == -math.inf), 0.0)
            loss = (w * picked.masked_fill(picked == -math.inf, 0.0)).sum(1)
            loss = loss + s["g_entropy"][r:r + step].double() * entropy + s["g_lse"][r:r + step].double() * lse
            g, = torch.autograd.grad(torch.where(dead, 0.0, loss).sum(), z)
            parts.append((torch.where(dead[:, None], 0.0, g),))
            continue
        inf = torch.full_like(picked, -math.inf)
        picked = torch.where(dead[:, None], inf, picked)
        row = [torch.where(tok == IGNORE, 0.0, picked), lse.masked_fill(dead, -math.inf),
               entropy.masked_fill(dead, 0.0)]
        if c["top"]:
            top = logp.masked_fill(dead[:, None], -math.inf).topk(min(c["top"], V), 1).values
            row.append(torch.nn.functional.pad(top, (0, c["top"] - top.shape[1]), value=-math.inf))
        parts.append(tuple(row))
    joined = [torch.cat(p) for p in zip(*parts)]
    if c["op"] == "logprobs_grad":
        return joined[0]
    out = dict(zip(("logprob", "lse", "entropy", "top_logprob"), joined))
    return dict(out, top_id=None) if c["top"] else out
