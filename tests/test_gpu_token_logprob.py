"""Token log probabilities with entropy and alternatives, and the gradient of
the logits, against the fp64 oracle.

Tolerances, fixed by the arithmetic (u = 2^-24): every exponential carries at
most two roundings of its argument x (|x| u each, in units of ln 2) and one ulp
of the exponential; a thread adds at most V / 256 + 64 terms one after another,
so a relative error of (V / 256 + 64) u bounds each sum; the entropy's sum of
e^x x is bounded by ln V + 1 times the mass.  Alternatives must be equal."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, say
from oracle import head_ops_oracle as ref
from sampling_transform_logprob_amd import binding

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    binding.load()


def sums(V):
    return V / 256 + 64


def make(rng, T, V, K, dtype, mask, scale=3.0):
    """(logits on the CPU in dtype, tokens, temperature)"""
    z = torch.from_numpy((rng.standard_normal((T, V)) * scale).astype(np.float32))
    if mask == "ties":
        z = torch.round(z)
    elif mask == "equal":
        z[:] = 1.5
    elif mask == "sorted":                      # every element a new maximum
        z = z.sort(1).values
    elif mask == "lowest":                      # rows and places at the type's lowest finite value
        lo = torch.finfo(DT[dtype]).min
        z[:, ::3] = lo
        z[0] = lo
    elif mask == "masked":
        z[torch.from_numpy(rng.random((T, V)) < 0.7)] = -np.inf
        z[T // 2] = -np.inf
        z[T - 1] = -np.inf
        z[T - 1, V - 1] = -2.0                  # one token left
    elif mask == "late":                        # nothing before the last tenth
        z[:, : V - max(1, V // 10)] = -np.inf
    elif mask == "offset":
        z += 500.0
    z = z.to(DT[dtype])
    tok = rng.integers(0, V, (T, K))
    if K > 1:
        tok[:, -1] = tok[:, 0]
    if K:
        tok[rng.random((T, K)) < 0.1] = IGNORE
    return z, torch.from_numpy(tok), torch.from_numpy(rng.uniform(0.4, 2.0, T).astype(np.float32))


def strided(x, pad, off=0):
    """x on the GPU as a view with `pad` elements after (and `off` before) each row."""
    T, V = x.shape
    buf = torch.full((T, off + V + pad), 7.0, dtype=x.dtype, device=dev())
    buf[:, off:off + V] = x.to(dev())
    return buf[:, off:off + V]


def check(z, tok, temp, top_n, out):
    T, V = z.shape
    r = ref.token_logprobs(z.double().numpy(), tok.numpy(), None if temp is None else temp.double().numpy(), top_n,
                           IGNORE)
    t64 = np.ones(T) if temp is None else temp.double().numpy()
    base = U * (sums(V) + 16)

    def near(a, b, tol, what):
        a, b = a.double().cpu().numpy(), np.asarray(b)
        assert a.shape == b.shape
        b = np.where(np.abs(b) > np.finfo(np.float32).max, np.copysign(np.inf, b), b)   # fp32's range
        fin = np.isfinite(b)
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b)), what
        assert np.all(a[np.isinf(b)] < 0), what
        tol = np.broadcast_to(tol, b.shape)
        bad = np.abs(a[fin] - b[fin]) > tol[fin]
        assert not bad.any(), (what, float(np.abs(a[fin] - b[fin]).max()), float(tol[fin][bad].min()))

    lse = np.nan_to_num(np.abs(r["lse"]), nan=0.0, posinf=0.0, neginf=0.0)
    near(out["lse"], r["lse"], base + 4 * U * lse, "lse")
    near(out["entropy"], r["entropy"], base * (2 + 2 * np.log(V)), "entropy")
    near(out["logprob"], r["logprob"], base + 4 * U * np.nan_to_num(np.abs(r["logprob"]), posinf=0.0), "logprob")
    if top_n:
        assert np.array_equal(out["top_id"].cpu().numpy(), r["top_id"]), "alternatives differ"
        near(out["top_logprob"], r["top_logprob"], base + 4 * U * np.nan_to_num(np.abs(r["top_logprob"]), posinf=0.0),
             "top_logprob")
    st = out["stats"].cpu()
    zmax = z.double().max(1).values.numpy()
    good = ~r["bad"]
    assert np.array_equal(st[:, 0].numpy()[good], zmax[good].astype(np.float32))
    assert torch.isnan(st[torch.from_numpy(r["bad"])]).all()
    assert torch.equal(st[:, 2].isnan(), out["entropy"].cpu().isnan())
    del t64
    return r


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V,K,top_n,pad", [
    (1, 1, 1, 1, 0), (3, 2, 1, 5, 1), (5, 7, 3, 7, 0), (2, 63, 2, 64, 1), (4, 255, 1, 20, 0), (4, 256, 0, 20, 3),
    (3, 257, 5, 1, 0), (2, 1000, 64, 128, 8), (3, 2047, 1, 0, 1), (3, 4097, 5, 20, 7), (2, 8193, 2, 128, 0),
    (2, 32001, 5, 20, 2), (1, 151936, 1, 20, 0), (1, 151936, 1, 128, 1),
])
def test_sizes(rng, dtype, T, V, K, top_n, pad):
    say(f"token_logprobs {dtype} T={T} V={V} K={K} top_n={top_n} pad={pad}")
    z, tok, temp = make(rng, T, V, K, dtype, None)
    for tt in (None, temp):
        out = binding.token_logprobs(strided(z, pad, pad), tok.to(dev()), None if tt is None else tt.to(dev()),
                                     top_n=top_n, ignore_index=IGNORE)
        check(z, tok, tt, top_n, out)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("mask", ["ties", "equal", "sorted", "lowest", "masked", "late", "offset"])
@pytest.mark.parametrize("T,V", [(3, 50), (5, 3001), (3, 40000)])
def test_masks(rng, dtype, mask, T, V):
    say(f"token_logprobs mask={mask} {dtype} T={T} V={V}")
    z, tok, temp = make(rng, T, V, 4, dtype, mask)
    for top_n in (1, 20, 100):
        out = binding.token_logprobs(z.to(dev()), tok.to(dev()), temp.to(dev()), top_n=top_n, ignore_index=IGNORE)
        check(z, tok, temp, top_n, out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,V", [(2, 32768), (2, 32769), (39, 40960), (40, 40960), (41, 40961), (255, 8193)])
def test_sizes_about_the_cut_of_rows(rng, dtype, T, V):
    """Rows of up to four tiles of 8,192, or of eight rows a tile, are one
    workgroup's; others are cut into segments."""
    say(f"token_logprobs {dtype} T={T} V={V}")
    z, tok, temp = make(rng, T, V, 2, dtype, "masked")
    for pad, top_n in ((0, 20), (1, 0)):
        z_dev = strided(z, pad)
        out = binding.token_logprobs(z_dev, tok.to(dev()), temp.to(dev()), top_n=top_n,
                                     ignore_index=IGNORE)
        check(z, tok, temp, top_n, out)


@pytest.mark.parametrize("T", [300, 384])
def test_many_long_rows_are_cut_or_not(T):
    """300 rows of 49 tiles of 8,192 are cut into segments, 384 are not: the same
    values either way, from rows repeated in a batch and scored alone."""
    V = 400000
    gen = torch.Generator(device=dev()).manual_seed(5)
    base = torch.randn(3, V, generator=gen, device=dev()).bfloat16()
    tok = torch.randint(0, V, (3, 2), generator=gen, device=dev())
    z, tk = base.repeat(T // 3, 1), tok.repeat(T // 3, 1)
    out = binding.token_logprobs(z, tk, top_n=20)
    check(base.cpu(), tok.cpu(), None, 20, {k: v[:3] for k, v in out.items()})
    for v in out.values():
        v = v.view(T // 3, -1)
        assert torch.equal(v, v[:1].expand_as(v))


@pytest.mark.parametrize("T", [700, 5000])
def test_many_rows(rng, T):
    V = 1203
    say(f"token_logprobs T={T} V={V}")
    z, tok, temp = make(rng, T, V, 2, "bf16", "masked")
    out = binding.token_logprobs(z.to(dev()), tok.to(dev()), temp.to(dev()), top_n=8, ignore_index=IGNORE)
    check(z, tok, temp, 8, out)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("mask", ["ties", "equal", "lowest", "zeros", "columns"])
def test_tied_rows_of_several_tiles(rng, dtype, mask):
    """Whole rows in one workgroup, more equal logits than its lists hold."""
    T, V = 260, 20000
    say(f"token_logprobs tied rows {mask} {dtype}")
    z, tok, temp = make(rng, T, V, 2, dtype, {"zeros": "lowest", "columns": None}.get(mask, mask))
    if mask == "columns":                        # the large logits all in a few threads' places, thousands of them
        e = 16 // z.element_size()
        z = torch.where((torch.arange(V) // e) % 256 < 14, z + 20, torch.full_like(z, 1.0))
    if mask == "zeros":                          # both zeros are one value; a few above them
        z[:] = 0.0
        z[:, ::2] = -0.0
        z[1::2, 7000:7004] = torch.finfo(DT[dtype]).smallest_normal
        z[2::3, 300:15000:7] = 2.0
    if mask == "lowest":                         # four tokens left by a mask of the lowest value
        z[3:] = torch.finfo(DT[dtype]).min
        z[3:, 9000:9004] = torch.randn(T - 3, 4, generator=torch.Generator().manual_seed(5)).to(z.dtype)
    for top_n in (20, 128):
        out = binding.token_logprobs(z.to(dev()), tok.to(dev()), temp.to(dev()), top_n=top_n, ignore_index=IGNORE)
        check(z, tok, temp, top_n, out)


@pytest.mark.parametrize("V", [40, 5000, 70000])
def test_invalid_rows(rng, V):
    """NaN, +inf, invalid temperatures and tokens: NaN outputs, no alternatives, and the report."""
    z, tok, temp = make(rng, 8, V, 3, "fp32", None)
    tok = tok.clamp(min=0)
    z[1, V // 2] = np.nan
    z[2, V - 1] = np.inf
    z[3] = np.nan
    z[3, 0] = -np.inf
    temp[4], temp[5] = 0.0, float("nan")
    tok[6, 1], tok[6, 2] = V, -1
    out = binding.token_logprobs(z.to(dev()), tok.to(dev()), temp.to(dev()), top_n=3, check=False)
    r = check(z, tok, temp, 3, out)
    assert r["bad"].sum() == 5 and torch.isnan(out["logprob"][6]).cpu().tolist() == [False, True, True]
    assert torch.all(out["top_id"][1:6].cpu() == -1) and torch.all(torch.isnan(out["top_logprob"][1:6]).cpu())
    with pytest.raises(ValueError, match=r"invalid temperature\[4\]"):
        binding.token_logprobs(z.to(dev()), tok.to(dev()), temp.to(dev()))
    with pytest.raises(ValueError, match=r"invalid target\[6\]"):
        binding.token_logprobs(z.to(dev()), tok.to(dev()))


def test_smallest_temperature_and_no_rows(rng):
    z, tok, _ = make(rng, 2, 300, 1, "fp32", None)
    temp = torch.tensor([1e-45, 3e38])
    out = binding.token_logprobs(z.to(dev()), tok.to(dev()), temp.to(dev()), top_n=2, ignore_index=IGNORE)
    assert out["entropy"][0].item() == 0.0                      # the largest logit alone
    assert abs(out["entropy"][1].item() - np.log(300)) < 1e-5   # uniform
    assert out["top_id"][0, 0].item() == z[0].argmax().item()
    e = binding.token_logprobs(torch.empty(0, 5, device=dev()), torch.empty(0, 2, dtype=torch.int64, device=dev()),
                               top_n=2)
    assert e["logprob"].shape == (0, 2) and e["top_id"].shape == (0, 2) and e["stats"].shape == (0, 4)
    g = binding.token_logprobs_backward(torch.empty(0, 5, device=dev()), None, e["stats"], grad_lse=e["lse"])
    assert g.shape == (0, 5)


def grad_reference(z, tok, temp, stats, g, ge, gl):
    """(gradient, tolerance) with the kernel's own log sum and entropy as inputs"""
    z64 = z.double().numpy()
    T, V = z64.shape
    t64 = np.ones(T) if temp is None else temp.double().numpy()
    st = stats.double().cpu().numpy()
    d = np.zeros((T, V))
    tol = np.zeros((T, V))
    for t in range(T):
        if not (np.isfinite(st[t, 0]) and np.isfinite(st[t, 1])):
            continue
        with np.errstate(over="ignore"):
            lp = (z64[t] - st[t, 0]) / t64[t] - st[t, 1]
        p = np.exp(lp)
        lpz = np.where(p > 0, lp, 0.0)
        G = A = 0.0
        own, ownmag = np.zeros(V), np.zeros(V)
        for y, w in zip(tok[t].tolist(), g[t].double().tolist()):
            if 0 <= y < V and z64[t, y] > -np.inf:
                G += w
                A += abs(w)
                own[y] += w
                ownmag[y] += abs(w)
        e, l, H = float(ge[t]), float(gl[t]), st[t, 2]
        d[t] = (p * (l - G - e * (lpz + H)) + own) / t64[t]
        size = abs(l) + A + abs(e) * (np.abs(lpz) + abs(H))
        K = tok.shape[1]
        tol[t] = U * (p * size * (24 + 4 * (np.abs(lpz) + abs(st[t, 1])) + K) + (K + 8) * ownmag) / t64[t] + 2e-38
    return d, tol


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,V,K,pad,mask", [
    (1, 1, 1, 0, None), (3, 2, 2, 1, None), (4, 257, 3, 0, "masked"), (3, 1000, 64, 5, "ties"), (2, 4096, 1, 0, None),
    (3, 4099, 5, 1, "lowest"), (2, 9001, 1024, 3, "masked"), (2, 33000, 7, 2, "offset"), (600, 515, 2, 0, "masked"),
])
def test_gradient(rng, dtype, T, V, K, pad, mask):
    say(f"token_logprobs_backward {dtype} T={T} V={V} K={K} pad={pad} mask={mask}")
    z, tok, temp = make(rng, T, V, K, dtype, mask)
    tok[0, 0] = V                                               # an invalid token passes nothing
    g = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32))
    ge, gl = (torch.from_numpy(rng.standard_normal(T).astype(np.float32)) for _ in range(2))
    zg = strided(z, pad, pad)
    for tt in (None, temp):
        tg = None if tt is None else tt.to(dev())
        out = binding.token_logprobs(zg, tok.to(dev()), tg, ignore_index=IGNORE, check=False)
        buf = torch.full((T, V + 2 * pad + 1), 3.0, dtype=z.dtype, device=dev())
        got = binding.token_logprobs_backward(zg, tok.to(dev()), out["stats"], g.to(dev()), ge.to(dev()), gl.to(dev()),
                                              temperature=tg, ignore_index=IGNORE, grad_logits=buf[:, pad:pad + V])
        assert got.data_ptr() == buf[:, pad:].data_ptr()
        assert torch.all(buf[:, :pad] == 3) and torch.all(buf[:, pad + V:] == 3)      # the rest left as it was
        want, tol = grad_reference(z, tok, tt, out["stats"], g, ge, gl)
        tol = tol + np.abs(want) * torch.finfo(z.dtype).eps / 2
        if dtype == "fp16":
            tol = tol + 2.0 ** -25                              # half a subnormal step
        a = got.double().cpu().numpy()
        # (a gradient past the type's range rounds to infinity as any conversion does)
        over = np.abs(want) >= torch.finfo(z.dtype).max
        assert np.all((np.abs(a - want) <= tol) | over), float((np.abs(a - want) - tol)[~over].max())
        # and whole, against the oracle's own forward
        whole = ref.token_logprobs_backward(z.double().numpy(), tok.numpy(), g.numpy(), ge.numpy(), gl.numpy(),
                                            None if tt is None else tt.numpy(), IGNORE)
        n = np.linalg.norm(whole[~over])
        assert np.linalg.norm((a - whole)[~over]) <= (torch.finfo(z.dtype).eps + U * (sums(V) + 64) * 8) * n + 1e-30


def test_gradient_parts_and_invalid_rows(rng):
    z, tok, temp = make(rng, 6, 700, 2, "fp32", None)
    z[1, 5] = np.nan
    z[2, 6] = np.inf
    z[3] = -np.inf
    temp[4] = -1.0
    zg, tg, pg = z.to(dev()), tok.to(dev()), temp.to(dev())
    out = binding.token_logprobs(zg, tg, pg, ignore_index=IGNORE, check=False)
    g = torch.ones(6, 2, device=dev())
    ones = torch.ones(6, device=dev())
    kw = dict(temperature=pg, ignore_index=IGNORE)
    parts = [binding.token_logprobs_backward(zg, tg, out["stats"], a, b, c, **kw)
             for a, b, c in ((g, None, None), (None, ones, None), (None, None, ones), (g, ones, ones))]
    for d in parts:
        assert torch.all(d[1:5] == 0) and torch.isfinite(d).all()
    # the parts' sum and the whole differ by roundings of p times their sizes (at most 30 here)
    assert torch.allclose(parts[0] + parts[1] + parts[2], parts[3], rtol=0, atol=1e-5)
    assert torch.allclose(parts[2][0].sum(), 1 / pg[0], rtol=1e-5)     # d lse sums to 1 / T


def test_deterministic(rng):
    z, tok, temp = make(rng, 3, 60000, 8, "bf16", "ties")
    a = [binding.token_logprobs(z.to(dev()), tok.to(dev()), temp.to(dev()), top_n=50, ignore_index=IGNORE)
         for _ in range(3)]
    for o in a[1:]:
        for k in o:
            assert torch.equal(o[k], a[0][k]), k


def test_autograd(rng):
    z, tok, temp = make(rng, 4, 900, 3, "fp32", "masked")
    tok = tok.clamp(min=0)
    x = z.to(dev()).requires_grad_()
    lp, lse, ent, tl, ti = binding.TokenLogprobFunction.apply(x, tok.to(dev()), temp.to(dev()), None, 5)
    w = torch.from_numpy(rng.standard_normal((4, 3)).astype(np.float32)).to(dev())
    live = torch.tensor([0, 1, 3], device=dev())
    finite = torch.isfinite(lp[live])
    loss = (torch.where(finite, lp[live], 0.0) * w[live]).sum() + (ent[live] * 0.3).sum() + (lse[live] ** 2).sum()
    loss.backward()
    r = ref.token_logprobs(z.double().numpy(), tok.numpy(), temp.numpy())
    gl = np.where(np.isfinite(r["lse"]), 2 * r["lse"], 0.0)
    ge = np.array([0.3, 0.3, 0.0, 0.3])
    want = ref.token_logprobs_backward(z.double().numpy(), tok.numpy(), w.cpu().double().numpy(), ge, gl, temp.numpy())
    assert np.allclose(x.grad.double().cpu().numpy(), want, atol=2e-5)
    assert not tl.requires_grad and not ti.requires_grad
    x.grad = None
    binding.TokenLogprobFunction.apply(x, tok.to(dev()))[2][live].sum().backward()      # entropy alone
    want = ref.token_logprobs_backward(z.double().numpy(), tok.numpy(), None, np.array([1.0, 1, 0, 1]))
    assert np.allclose(x.grad.double().cpu().numpy(), want, atol=2e-5)


def test_captured_calls_replay_bitwise(rng):
    """Forward and backward of two shapes (one split over workgroups, one not)
    captured in two graphs that run one after the other."""
    made = []
    for T, V in ((2, 50000), (300, 700)):
        z, tok, temp = make(rng, T, V, 2, "bf16", "masked")
        zg, tg, pg = z.to(dev()), tok.to(dev()), temp.to(dev())
        g = torch.from_numpy(rng.standard_normal((T, 2)).astype(np.float32)).to(dev())

        def step(zg=zg, tg=tg, pg=pg, g=g):
            o = binding.token_logprobs(zg, tg, pg, top_n=7, ignore_index=IGNORE, check=False)
            d = binding.token_logprobs_backward(zg, tg, o["stats"], g, temperature=pg, ignore_index=IGNORE)
            return [o["logprob"], o["lse"], o["entropy"], o["top_logprob"], o["top_id"], d]
        eager = step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        made.append((graph, held, eager, step))             # (step holds the inputs)
    for _ in range(3):
        for graph, held, eager, _ in made:
            for t in held:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for graph, held, eager, _ in made:
            for a, b in zip(held, eager):
                assert torch.equal(a, b)


def test_another_stream(rng):
    z, tok, temp = make(rng, 3, 20000, 2, "bf16", None)
    zg, tg, pg = z.to(dev()), tok.to(dev()), temp.to(dev())
    want = binding.token_logprobs(zg, tg, pg, top_n=9, ignore_index=IGNORE)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = binding.token_logprobs(zg, tg, pg, top_n=9, ignore_index=IGNORE, check=False)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k])


def test_refusals(rng):
    z, tok, temp = make(rng, 3, 50, 2, "fp32", None)
    zg, tg = z.to(dev()), tok.to(dev())
    with pytest.raises(ValueError, match="temperature must have shape"):
        binding.token_logprobs(zg, tg, torch.ones(4, device=dev()))
    with pytest.raises(TypeError, match="int64"):
        binding.token_logprobs(zg, tg.int())
    with pytest.raises(ValueError, match="tokens must have shape"):
        binding.token_logprobs(zg, tg[:2])
    with pytest.raises(ValueError, match="tokens is on"):
        binding.token_logprobs(zg, tok)
    with pytest.raises(binding.StceError, match="top_n=129"):
        binding.token_logprobs(zg, tg, top_n=129)
    with pytest.raises(binding.StceError, match="V=0"):
        binding.token_logprobs(zg[:, :0])
    out = binding.token_logprobs(zg, tg, ignore_index=IGNORE, check=False)
    with pytest.raises(ValueError, match="grad_logprob must have"):
        binding.token_logprobs_backward(zg, tg, out["stats"], torch.ones(3, device=dev()))
    with pytest.raises(ValueError, match="stats must be"):
        binding.token_logprobs_backward(zg, tg, out["stats"][:2])
    with pytest.raises(binding.StceError, match="overlaps"):
        binding.token_logprobs_backward(zg, tg, out["stats"], grad_logits=zg)
