"""Block-scaled e4m3 quantization (bit for bit) and product against the fp64
oracle.

The product's tolerance: a product of two e4m3 values is exact in fp32; an fp32
output's sum over one block of 128 is held to 128 roundings of 2^-23 (the matrix
instruction may truncate), the scale pair and its application to three of 2^-24,
the sum over blocks to one per block: |error| <= (2 * 128 + 4 + blocks) 2^-24 sum
|a b| (scaled).  A 16-bit output may come from the fp8 matrix instructions, which
align the eight products of a group to the largest and keep 13 binary places
below it: at most 8 * 2^-13 of the group's largest product, so 2^-10 of sum |a b|
more.  Half a step of the output's type on top."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, say
from oracle import head_ops_oracle as ref
from sampling_transform_logprob_amd import binding

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


def check_quantized(x, codes, scales, block, transpose):
    q, s = ref.quantize_blocks(x.float().numpy(), block, transpose)
    assert codes.dtype == torch.float8_e4m3fn and tuple(codes.shape) == q.shape and tuple(scales.shape) == s.shape
    got = scales.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(s))
    ok = ~np.isnan(s)
    assert np.array_equal(got[ok].view(np.int32), s[ok].view(np.int32)), "scales differ"
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), q), "codes differ"


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("R,C,pad", [(1, 1, 0), (1, 16, 0), (1, 5120, 0), (3, 129, 1), (16, 128, 0), (127, 130, 2),
                                     (130, 257, 0), (129, 1, 0), (260, 300, 5), (515, 640, 0)])
def test_quantize(rng, dtype, block, transpose, R, C, pad):
    say(f"quantize {dtype} {block} transpose={transpose} {R}x{C} pad={pad}")
    x = torch.from_numpy((rng.standard_normal((R, C)) * 2.0 ** rng.integers(-12, 4, (R, 1))).astype(np.float32))
    x = x.to(DT[dtype])
    if R > 2:
        x[1] = 0
        x[2, 0] = -0.0
    buf = torch.full((R, C + pad), 100.0, dtype=x.dtype, device=dev())
    buf[:, :C] = x.to(dev())
    codes, scales = binding.fp8_quantize_blocks(buf[:, :C], block=block, transpose=transpose)
    check_quantized(x, codes, scales, block, transpose)


@pytest.mark.parametrize("block", ["row", "tile"])
def test_quantize_extremes(rng, block):
    """Zeros, subnormals, the largest values, ties between codes, NaN and infinities."""
    x = torch.zeros(200, 512)
    x[0, :128] = torch.from_numpy(rng.standard_normal(128).astype(np.float32)) * 1e-44
    x[1, :128] = torch.from_numpy(rng.standard_normal(128).astype(np.float32)) * 1e-37
    x[2, 128:256] = torch.finfo(torch.float32).max * torch.linspace(-1, 1, 128)
    v = ref.e4m3_values()[:127]
    x[3, 256:256 + 126] = torch.from_numpy(((v[:-1] + v[1:]) / 2).astype(np.float32))   # halfway between codes
    x[3, 383] = 448.0
    x[4, 5] = float("nan")
    x[130, 400] = float("-inf")
    for tr in (False, True):
        codes, scales = binding.fp8_quantize_blocks(x.to(dev()), block=block, transpose=tr)
        check_quantized(x, codes, scales, block, tr)
        assert torch.isnan(scales).sum().item() > 0


def operands(rng, M, N, K, b_block):
    a = ref.e4m3_nearest(np.clip(rng.standard_normal((M, K)) * 120, -448, 448))
    b = ref.e4m3_nearest(np.clip(rng.standard_normal((N, K)) * 120, -448, 448))
    kb = -(-K // 128)
    sa = rng.uniform(1e-3, 2e-2, (M, kb)).astype(np.float32)
    sb = rng.uniform(1e-4, 4e-4, (N if b_block == "row" else -(-N // 128), kb)).astype(np.float32)
    return a, sa, b, sb


def run(a, sa, b, sb, dtype, layout, **kw):
    g = lambda x: torch.from_numpy(x).to(dev())  # noqa: E731
    place = (lambda s: g(np.ascontiguousarray(s.T)).t()) if layout == "block" else g
    return binding.fp8_block_matmul(g(a).view(torch.float8_e4m3fn), place(sa), g(b), place(sb), out_dtype=DT[dtype], **kw)


def check_product(got, a, sa, b, sb, out, extra=0.0):
    want, mag = ref.block_matmul(a, sa, b, sb)
    want = want + extra
    d = np.abs(got.double().cpu().numpy() - want)
    tol = (260 + sa.shape[1]) * 2.0 ** -24 * (mag + np.abs(extra)) + np.abs(want) * torch.finfo(DT[out]).eps / 2
    if out != "fp32":
        tol = tol + 2.0 ** -10 * mag
    if out == "fp16":
        tol = tol + 2.0 ** -25
    assert np.linalg.norm(d) <= (2.0 ** -14 * (out != "fp32") + torch.finfo(DT[out]).eps) * np.linalg.norm(want) + 1e-30
    assert np.all(d <= tol), (float((d / tol).max()), np.argwhere(d > tol)[:5])


@pytest.mark.parametrize("b_block", ["tile", "row"])
@pytest.mark.parametrize("out,layout", [("bf16", "block"), ("fp32", "row"), ("fp16", "block")])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 200, 128), (1, 4096, 1040), (2, 129, 144), (15, 130, 272), (16, 64, 2048), (17, 1000, 512),
    (33, 513, 640), (64, 300, 4112), (65, 256, 128), (100, 700, 1296), (127, 129, 384), (200, 1, 256),
    (256, 256, 256), (257, 255, 1024), (300, 777, 400), (1100, 530, 912),
])
def test_product(rng, b_block, out, layout, M, N, K):
    say(f"block matmul M={M} N={N} K={K} {b_block} out={out}")
    a, sa, b, sb = operands(rng, M, N, K, b_block)
    check_product(run(a, sa, b, sb, out, layout), a, sa, b, sb, out)


def test_one_large_scale_does_not_reach_its_neighbours(rng):
    """Scales over many binades: each block must take its own pair."""
    a, sa, b, sb = operands(rng, 70, 300, 640, "row")
    sa *= 2.0 ** rng.integers(-20, 20, sa.shape)
    sb *= 2.0 ** rng.integers(-20, 20, sb.shape)
    check_product(run(a, sa, b, sb, "fp32", "row"), a, sa, b, sb, "fp32")
    check_product(run(b, sb, a, sa, "fp32", "block"), b, sb, a, sa, "fp32")


@pytest.mark.parametrize("M", [1, 40, 300])
def test_nan_scale_reaches_its_row_or_tile_only(rng, M):
    a, sa, b, sb = operands(rng, M, 400, 512, "tile")
    sa[M // 2, 1] = np.nan
    got = run(a, sa, b, sb, "fp32", "block")
    rows = torch.isnan(got).all(1).cpu()
    assert rows[M // 2] and rows.sum() == 1 and torch.isnan(got).sum().item() == 400
    a, sa, b, sb = operands(rng, M, 400, 512, "tile")
    sb[2, 3] = np.nan
    got = torch.isnan(run(a, sa, b, sb, "fp32", "block")).cpu()
    assert got[:, 256:384].all() and not got[:, :256].any() and not got[:, 384:].any()


@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (50, 129, 256), (300, 300, 272), (500, 260, 4096)])
def test_out_strides_and_accumulate(rng, M, N, K):
    a, sa, b, sb = operands(rng, M, N, K, "tile")
    c = rng.standard_normal((M, N)).astype(np.float32)
    buf = torch.full((M + 1, N + 5), 9.0, device=dev())
    buf[:M, 2:2 + N] = torch.from_numpy(c).to(dev())
    out = run(a, sa, b, sb, "fp32", "row", out=buf[:M, 2:2 + N], accumulate=True)
    assert out.data_ptr() == buf[:, 2:].data_ptr()
    check_product(out, a, sa, b, sb, "fp32", c.astype(np.float64))
    assert torch.all(buf[M] == 9) and torch.all(buf[:, :2] == 9) and torch.all(buf[:, 2 + N:] == 9)
    half = torch.full((M, N + 3), 9.0, dtype=torch.bfloat16, device=dev())
    check_product(run(a, sa, b, sb, "bf16", "row", out=half[:, 1:1 + N]), a, sa, b, sb, "bf16")
    assert torch.all(half[:, 0] == 9) and torch.all(half[:, 1 + N:] == 9)


@pytest.mark.parametrize("M", [3, 270])
def test_strided_operands(rng, M):
    a, sa, b, sb = operands(rng, M, 260, 256, "tile")
    wide_a = np.full((M, 256 + 32), 0x7F, np.uint8)     # NaN codes beside the operand
    wide_b = np.full((260, 256 + 48), 0x7F, np.uint8)
    wide_a[:, 16:272], wide_b[:, 32:288] = a, b
    g = lambda x: torch.from_numpy(x).to(dev())  # noqa: E731
    got = binding.fp8_block_matmul(g(wide_a)[:, 16:272], g(sa), g(wide_b)[:, 32:288], g(sb), out_dtype=torch.float32)
    check_product(got, a, sa, b, sb, "fp32")


def test_empty_products():
    e = lambda *s: torch.empty(*s, dtype=torch.float8_e4m3fn, device=dev())  # noqa: E731
    f = lambda *s: torch.ones(*s, device=dev())  # noqa: E731
    assert binding.fp8_block_matmul(e(0, 64), f(0, 1), e(5, 64), f(5, 1)).shape == (0, 5)
    assert binding.fp8_block_matmul(e(4, 64), f(4, 1), e(0, 64), f(0, 1)).shape == (4, 0)
    z = binding.fp8_block_matmul(e(4, 0), f(4, 0), e(5, 0), f(5, 0), out_dtype=torch.float32)
    assert torch.equal(z, torch.zeros(4, 5, device=dev()))
    acc = torch.full((4, 5), 2.0, device=dev())
    binding.fp8_block_matmul(e(4, 0), f(4, 0), e(5, 0), f(5, 0), out=acc, accumulate=True)
    assert torch.all(acc == 2)
    q, s = binding.fp8_quantize_blocks(torch.empty(0, 40, device=dev()))
    assert q.shape == (0, 48) and s.shape == (0, 1)


def test_deterministic_and_captured(rng):
    made = []
    for M, N, K in ((1, 3000, 4096), (40, 700, 5120), (600, 520, 1024)):
        a, sa, b, sb = operands(rng, M, N, K, "tile")
        ts = [torch.from_numpy(x).to(dev()) for x in (a, sa, b, sb)]
        eager = binding.fp8_block_matmul(*ts, out_dtype=torch.float32)
        assert torch.equal(eager, binding.fp8_block_matmul(*ts, out_dtype=torch.float32))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = binding.fp8_block_matmul(*ts, out_dtype=torch.float32)
        made.append((graph, held, eager, ts))
    for _ in range(3):
        for graph, held, *_ in made:
            held.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, held, eager, _ in made:
            assert torch.equal(held, eager)


def test_linear_layer_and_its_gradients(rng):
    """Fp8BlockLinearFunction against the oracle's quantized products."""
    T, H, V = 150, 272, 400
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dev()).requires_grad_()
    w = torch.from_numpy((rng.standard_normal((V, H)) * 0.05).astype(np.float32)).to(dev()).requires_grad_()
    g = torch.from_numpy(rng.standard_normal((T, V)).astype(np.float32)).to(dev())
    y = binding.Fp8BlockLinearFunction.apply(x, w)
    y.backward(g)
    xn, wn, gn = (t.detach().cpu().numpy() for t in (x, w, g))
    q = ref.quantize_blocks
    for got, (a, sa), (b, sb) in [(y.detach(), q(xn), q(wn, "tile")), (x.grad, q(gn), q(wn, "tile", True)),
                                  (w.grad, q(gn, "row", True), q(xn, "row", True))]:
        check_product(got, a, sa, b, sb, "fp32")
    # and near the unquantized layer: each e4m3 value is off by at most 2^-4
    # of itself, so a product by 2^-3 + 2^-8 of the magnitudes' product
    exact, mag = xn.astype(np.float64) @ wn.T.astype(np.float64), np.abs(xn) @ np.abs(wn).T
    assert np.all(np.abs(y.detach().cpu().numpy() - exact) <= mag * (2.0 ** -3 + 2.0 ** -8) + 1e-3)


@pytest.mark.parametrize("T,H,V", [(37, 100, 77), (1, 33, 200), (5, 1, 1), (0, 64, 40)])
def test_linear_layer_at_odd_sizes(rng, T, H, V):
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dev()).requires_grad_()
    w = torch.from_numpy(rng.standard_normal((V, H)).astype(np.float32)).to(dev()).requires_grad_()
    y = binding.Fp8BlockLinearFunction.apply(x, w)
    assert y.shape == (T, V)
    y.sum().backward()                                  # (an expanded gradient: no strides of its own)
    assert x.grad.shape == x.shape and w.grad.shape == w.shape
    if T == 0:
        assert torch.all(w.grad == 0)
        return
    xn, wn, gn = x.detach().cpu().numpy(), w.detach().cpu().numpy(), np.ones((T, V), np.float32)
    q = ref.quantize_blocks
    for got, (a, sa), (b, sb) in [(y.detach(), q(xn), q(wn, "tile")), (x.grad, q(gn), q(wn, "tile", True)),
                                  (w.grad, q(gn, "row", True), q(xn, "row", True))]:
        check_product(got, a, sa, b, sb, "fp32")


def test_two_streams_at_once(rng):
    """The same calls on two streams at the same time: workspaces of their own."""
    a, sa, b, sb = (torch.from_numpy(x).to(dev()) for x in operands(rng, 20, 500, 4096, "tile"))
    z = torch.from_numpy(rng.standard_normal((3, 90000)).astype(np.float32)).to(dev())
    want = binding.fp8_block_matmul(a, sa, b, sb, torch.float32)
    lse = binding.token_logprobs(z, top_n=30)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    held = [[], []]
    for _ in range(10):
        for s, h in zip(streams, held):
            with torch.cuda.stream(s):
                h.append((binding.fp8_block_matmul(a, sa, b, sb, torch.float32),
                          binding.token_logprobs(z, top_n=30, check=False)))
    torch.cuda.synchronize()
    for h in held:
        for o, t in h:
            assert torch.equal(o, want)
            assert all(torch.equal(t[k], lse[k]) for k in lse)


def test_head_and_token_logprobs_together(rng):
    """hidden -> fp8 head -> log probabilities and entropy -> loss -> gradients,
    as a training step runs them, against fp64 on the same quantized operands."""
    T, H, V = 96, 256, 1500
    h = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dev()).requires_grad_()
    w = torch.from_numpy((rng.standard_normal((V, H)) * 0.08).astype(np.float32)).to(dev()).requires_grad_()
    tok = torch.from_numpy(rng.integers(0, V, (T, 2))).to(dev())
    adv = torch.from_numpy(rng.standard_normal((T, 2)).astype(np.float32)).to(dev())
    logits = binding.Fp8BlockLinearFunction.apply(h, w)
    logits.retain_grad()
    lp, lse, ent, _, ids = binding.TokenLogprobFunction.apply(logits, tok, None, None, 4)
    ((adv * lp).sum() / T - 0.01 * ent.mean() + 1e-4 * (lse ** 2).mean()).backward()
    q = ref.quantize_blocks
    hn, wn = h.detach().cpu().numpy(), w.detach().cpu().numpy()
    z, mag = ref.block_matmul(*q(hn), *q(wn, "tile"))
    r = ref.token_logprobs(z, tok.cpu().numpy(), top_n=4)
    assert np.abs(lp.detach().cpu().numpy() - r["logprob"]).max() < 1e-3
    dz = ref.token_logprobs_backward(z, tok.cpu().numpy(), (adv / T).cpu().numpy(), np.full(T, -0.01 / T),
                                     2e-4 * r["lse"] / T)
    got = logits.grad.double().cpu().numpy()
    assert np.linalg.norm(got - dz) <= 1e-4 * np.linalg.norm(dz)
    gn = logits.grad.cpu().numpy()
    check_product(h.grad, *q(gn), *q(wn, "tile", True), "fp32")
    check_product(w.grad, *q(gn, "row", True), *q(hn, "row", True), "fp32")


def test_serving_step(rng):
    """One token's hidden state through a kept fp8 head to its alternatives."""
    H, V = 512, 5000
    w = torch.from_numpy((rng.standard_normal((V, H)) * 0.1).astype(np.float32))
    h = torch.from_numpy(rng.standard_normal((1, H)).astype(np.float32)).to(torch.bfloat16)
    wq, ws = binding.fp8_quantize_blocks(w.to(dev()), block="tile")
    hq, hs = binding.fp8_quantize_blocks(h.to(dev()))
    out = binding.token_logprobs(binding.fp8_block_matmul(hq, hs, wq, ws, torch.float32), top_n=10)
    z, _ = ref.block_matmul(*ref.quantize_blocks(h.float().numpy()), *ref.quantize_blocks(w.numpy(), "tile"))
    r = ref.token_logprobs(z, None, top_n=10)
    assert np.array_equal(out["top_id"].cpu().numpy(), r["top_id"])
    assert np.abs(out["top_logprob"].cpu().numpy() - r["top_logprob"]).max() < 1e-4


def test_refusals(rng):
    a, sa, b, sb = (torch.from_numpy(x).to(dev()) for x in operands(rng, 4, 300, 64, "tile"))
    mm = binding.fp8_block_matmul
    with pytest.raises(ValueError, match="a_scale must have shape"):
        mm(a, sa[:3], b, sb)
    with pytest.raises(ValueError, match="b_scale must have shape"):
        mm(a, sa, b, sb[:2])
    with pytest.raises(TypeError, match="b_scale must be fp32"):
        mm(a, sa, b, sb.double())
    with pytest.raises(ValueError, match="share K"):
        mm(a[:, :48], sa, b, sb)
    with pytest.raises(ValueError, match="multiple of 16"):
        mm(a[:, :40], sa, b[:, :40], sb)
    with pytest.raises(ValueError, match="multiple of 16"):
        mm(a[:, 8:24], sa, b[:, :16], sb)
    with pytest.raises(TypeError, match="out_dtype"):
        mm(a, sa, b, sb, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="accumulate needs out"):
        mm(a, sa, b, sb, accumulate=True)
    with pytest.raises(binding.StceError, match="accumulate"):
        mm(a, sa, b, sb, out=torch.empty(4, 300, dtype=torch.bfloat16, device=dev()), accumulate=True)
    with pytest.raises(ValueError, match="out must be"):
        mm(a, sa, b, sb, out=torch.empty(4, 301, device=dev()))
    both = torch.zeros(4 * 300 * 4, dtype=torch.uint8, device=dev())
    with pytest.raises(binding.StceError, match="overlaps"):
        mm(both[1024:1280].view(4, 64), sa, b, sb, out=both.view(torch.float32).view(4, 300))


def test_both_marshalling_paths_agree(rng, monkeypatch):
    """The marshalling module and the ctypes calls make the same call."""
    def run_all():
        x = torch.from_numpy(rng.standard_normal((70, 200)).astype(np.float32)).to(dev())
        out = list(binding.fp8_quantize_blocks(x)) + list(binding.fp8_quantize_blocks(x, block="tile", transpose=True))
        q, s = binding.fp8_quantize_blocks(x[:, ::2])                   # a copy is needed
        w, ws = binding.fp8_quantize_blocks(torch.from_numpy(rng.standard_normal((300, 100)).astype(np.float32)).to(dev()),
                                            block="tile")
        out += [q, s, w, ws] + [binding.fp8_block_matmul(q, s, w, ws, d) for d in DT.values()]
        z = torch.from_numpy(rng.standard_normal((9, 300)).astype(np.float32)).to(dev())
        tok = torch.from_numpy(rng.integers(0, 300, (9, 3))).to(dev())
        temp = torch.full((9,), 0.7, device=dev())
        for zz, tt in ((z, tok), (z[:, 3:290], tok.clamp(max=200)[:, 0])):
            for n in (0, 4):
                o = binding.token_logprobs(zz, tt, temp, top_n=n, ignore_index=-100)
                out += [o[k] for k in sorted(o)]
            out.append(binding.token_logprobs_backward(zz, tt, o["stats"], torch.ones(tt.shape, device=dev()), temp, None,
                                                       temperature=temp, ignore_index=-100))
        out.append(binding.token_logprobs(z)["lse"])
        return out
    assert binding._load_fast() is not False, "the marshalling module is not built"
    state = rng.bit_generator.state
    a = run_all()
    monkeypatch.setattr(binding, "_fast", False)
    rng.bit_generator.state = state
    b = run_all()
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.shape == y.shape and x.dtype == y.dtype and x.stride() == y.stride()
        xb, yb = (t.contiguous().reshape(-1).view(torch.uint8) for t in (x, y))
        assert torch.equal(xb, yb)
