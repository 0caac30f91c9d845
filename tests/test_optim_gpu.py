"""The AdamW step over many tensors and the global gradient norm, against the fp64 oracle on the
same rounded inputs.

Tolerances, in units of u = 2^-24 (fp32 rounding).  m = b1 m + c1 g: b1, c1 and the scaled gradient
are rounded once each, then two products and a sum: 5 u (|b1 m| + |c1 g|).  v: 7 u v (all terms are
positive; g enters twice).  The update m / (da sqrt(v) + db): the step size lr / (1 - b1^t) takes lr's rounding, expm1f
(2 u, and 1 of its argument) and a division, 5 u; da = 1 / (size sqrt(1 - b2^t)) adds 3 u / 2 and a
root, a product and a reciprocal, 9.5 u; db = eps / size has 7 u; the root of v has half of v's 7 and
2 of its own, so the denominator has at most 5.5 + 9.5 + 1 = 16 u; the reciprocal adds 2, the
product 1, and the first moment's terms 5: 24 u of size (|b1 m| + |c1 g|) / (sqrt(v / (1 - b2^t)) +
eps).  The weight: 3 u |w| for its decay and the difference, and half a step of its type for the
store.
8-bit states: the scale is a maximum's 5 (7/2) units and a division, under 8 u.  A code is the
nearest to a quotient known to within the value's error over the scale and 10 u of itself: it has
to be one of the codes between the ends of that interval.
"""
import numpy as np
import pytest

from oracle import train as ot

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GROUP = dict(lr=0.01, betas=(0.8, 0.96), eps=1e-10, weight_decay=0.1)


def _np(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _quantized(x):
    """(codes, scales) tensors of a 1-D float array, by the oracle."""
    import torch
    s = ot.block_scales(x).astype(np.float32)
    per = np.repeat(s.astype(np.float64), 256)[:len(x)]
    q = ot.encode_e4m3(np.divide(x, per, out=np.zeros_like(x), where=per > 0))
    return (torch.from_numpy(q).float().cuda().to(torch.float8_e4m3fn), torch.from_numpy(s).cuda())


def _make(n, param="f32", grad="f32", bits=32, master=False, seed=0, offset=0, shape=None):
    """(parameter, gradient, state): a run in progress, sizes spread over decades, some zeros.
    ``offset``: elements in front of every array in its allocation (alignment)."""
    import torch
    rng = np.random.default_rng(seed + n)

    def place(a, dt):
        t = torch.zeros(offset + n, dtype=dt, device="cuda")[offset:]
        t.copy_(torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a)
        return t

    scale = 10.0 ** rng.uniform(-5, -1, n)
    g = rng.standard_normal(n) * scale * (rng.random(n) > 0.1)
    m = rng.standard_normal(n) * scale * (rng.random(n) > 0.1)
    v = (scale * (0.1 + rng.random(n))) ** 2 * (rng.random(n) > 0.1)
    w = rng.standard_normal(n) * 0.1
    p = place(w, _dtype(param))
    gt = place(g, _dtype(grad))
    if bits == 8:
        s = {}
        for name, x in (("m", m), ("r", np.sqrt(v))):
            q, sc = _quantized(x)
            s[name] = place(q.view(torch.uint8), torch.uint8).view(torch.float8_e4m3fn)
            s[name + "_scale"] = sc
    else:
        s = {"m": place(m, torch.float32), "v": place(v, torch.float32)}
    if master:
        s["master"] = place(w, torch.float32)
        p.copy_(s["master"])
    if shape is not None:
        p, gt = p.view(shape), gt.view(shape)
    return p, gt, s


def _before(p, g, s):
    """What the step reads, in float64."""
    out = dict(w=_np(s["master"] if "master" in s else p), g=_np(g))
    if "r" in s:
        out["m"] = ot.dequantize_blocks(_np(s["m"]), _np(s["m_scale"]))
        out["v"] = ot.dequantize_blocks(_np(s["r"]), _np(s["r_scale"])) ** 2
    else:
        out["m"], out["v"] = _np(s["m"]), _np(s["v"])
    return out


def _check_codes(got, scales, x, err, floor):
    """Codes and scales of values x known to within err; floor: nonzero values get a code."""
    want = ot.block_scales(x)
    blocks = len(want)
    tops = np.array([err[i * 256:(i + 1) * 256].max() for i in range(blocks)])
    assert np.all(np.abs(scales - want) <= tops / 448 + 8 * U * want)
    per = np.repeat(scales, 256)[:len(x)]
    on = per > 0
    assert not got[~on].any()
    lo, hi = ((x[on] + s * (err[on] + 10 * U * np.abs(x[on]))) / per[on] for s in (-1, 1))
    if floor:
        small = 2.0 ** -9
        lo, hi = (np.where(x[on] > 0, np.maximum(e, small), e) for e in (lo, hi))
        assert np.all(got[on][x[on] > 0] > 0)
    assert np.all(got[on] >= ot.encode_e4m3(lo)) and np.all(got[on] <= ot.encode_e4m3(hi))


def _check(before, p, s, t, lr, betas, eps, weight_decay, scale=1.0):
    b1, b2 = betas
    w, m, v = ot.adamw(before["w"], before["g"], before["m"], before["v"], t, lr, b1, b2, eps,
                       weight_decay, scale)
    m_size = np.abs(b1 * before["m"]) + np.abs((1 - b1) * scale * before["g"])
    denom = np.sqrt(v / (1 - b2 ** t)) + eps
    update = lr / (1 - b1 ** t) * np.divide(m_size, denom, out=np.zeros_like(denom),
                                            where=denom > 0)
    exact = 3 * U * np.abs(before["w"]) + 24 * U * update + 2.0 ** -140
    half = {2: 2.0 ** -8, 4: U}[p.element_size()]
    if "master" in s:
        assert np.all(np.abs(_np(s["master"]) - w) <= exact + U * np.abs(w))
        assert bool((s["master"].to(p.dtype).view(-1) == p.view(-1)).all())
    else:
        assert np.all(np.abs(_np(p) - w) <= exact + half * (np.abs(w) + exact))
    if "r" in s:
        _check_codes(_np(s["m"]), _np(s["m_scale"]), m, 5 * U * m_size, False)
        _check_codes(_np(s["r"]), _np(s["r_scale"]), np.sqrt(v), 5 * U * np.sqrt(v), True)
    else:
        assert np.all(np.abs(_np(s["m"]) - m) <= 5 * U * m_size + 2.0 ** -140)
        assert np.all(np.abs(_np(s["v"]) - v) <= 7 * U * v + 2.0 ** -140)


SIZES = [1, 7, 8, 255, 256, 257, 2048, 4095, 4096, 4097, 12345]
KINDS = [("f32", "f32", 32, False), ("bf16", "bf16", 32, False), ("bf16", "f32", 32, True),
         ("f32", "bf16", 8, False), ("bf16", "f32", 8, False), ("bf16", "bf16", 8, True)]


@pytest.mark.parametrize("param,grad,bits,master", KINDS)
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_step_every_type_size_and_alignment(cuda_device, param, grad, bits, master, offset):
    import torch
    import lm_head_linear_gemm_b200 as flce
    made = [_make(n, param, grad, bits, master, seed=3, offset=offset) for n in SIZES]
    before = [_before(*x) for x in made]
    step = torch.full((1,), 6, dtype=torch.int64, device="cuda")
    opt = flce.AdamW([dict(params=[x[0] for x in made], states=[x[2] for x in made], **GROUP)],
                     step=step)
    opt.step([x[1] for x in made], grad_scale=0.75)
    assert int(step) == 7 and not opt._scratch.any()
    for b, (p, _, s) in zip(before, made):
        _check(b, p, s, 7, scale=0.75, **GROUP)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("param,master", [("f32", False), ("bf16", False), ("bf16", True)])
def test_long_launches_equal_short_ones(cuda_device, param, master, grad, bits, offset):
    """A launch of many elements works in larger tiles than one of few: a tensor, and the same cut at
    multiples of 256 elements into tensors of launches of their own, move bit for bit alike."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    n, piece = 6_000_011, 1_000_192
    gen = torch.Generator(device="cuda").manual_seed(n)
    rand = lambda dt: torch.randn(offset + n, device="cuda", generator=gen).to(dt)[offset:]
    p, grads = rand(_dtype(param)), [rand(_dtype(grad)) for _ in range(2)]
    q = torch.empty(offset + n, dtype=p.dtype, device="cuda")[offset:].copy_(p)
    make = dict(state_bits=bits, min_8bit_size=0, master_weights=master, **GROUP)
    whole = flce.AdamW([p], **make)
    parts = [flce.AdamW([part], **make) for part in q.split(piece)]
    for g in grads:
        whole.step([g], grad_scale=0.5)
        for opt, part in zip(parts, g.split(piece)):
            opt.step([part], grad_scale=0.5)
    assert torch.equal(p, q)
    for name, t in whole.state[0].items():
        joined = torch.cat([opt.state[0][name].view(torch.uint8) for opt in parts])
        assert torch.equal(t.view(torch.uint8), joined), name


def test_neighbours_in_one_buffer_stay(cuda_device):
    """Tensors that end inside a vector, a warp's block and a chunk: what lies behind them stays."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    for bits in (32, 8):
        for n in (1, 9, 250, 4100):
            store = torch.full((n + 600,), 5.0, dtype=torch.bfloat16, device="cuda")
            code = torch.float8_e4m3fn if bits == 8 else torch.float32
            keep = [torch.full((n + 600,), 3, dtype=torch.uint8 if bits == 8 else torch.float32,
                               device="cuda") for _ in range(2)]
            s = dict(zip(("m", "r" if bits == 8 else "v"), (k[:n].view(code) for k in keep)))
            if bits == 8:
                for name in ("m_scale", "r_scale"):
                    s[name] = torch.ones(n // 256 + 3, device="cuda")[:-(-n // 256)]
            opt = flce.AdamW([dict(params=[store[:n]], states=[s])])
            opt.step([torch.ones(n, device="cuda")])
            # the step moves every state; a weight of 5 rounds back to itself (lr = 1e-3 is below
            # half a bf16 step there, 2^-6)
            assert bool((store == 5).all())
            assert not any(bool((k[:n] == 3).any()) for k in keep)
            assert all(bool((k[n:] == 3).all()) for k in keep)


def test_many_tensors_groups_and_missing_gradients(cuda_device):
    """800 tensors in three launches of two groups, mixed types, some without a gradient."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    kinds = [KINDS[i % len(KINDS)] for i in range(800)]
    made = [_make(1 + (37 * i) % 700, *k, seed=i) for i, k in enumerate(kinds)]
    other = dict(lr=0.003, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0)
    groups = [dict(params=[x[0] for x in made[a::2]], states=[x[2] for x in made[a::2]], **h)
              for a, h in ((0, GROUP), (1, other))]
    made = made[0::2] + made[1::2]
    before = [_before(*x) for x in made]
    raw = [[t.clone() for t in (x[0], *x[2].values())] for x in made]
    opt = flce.AdamW(groups)
    opt.step([None if i % 5 == 4 else x[1] for i, x in enumerate(made)])
    assert int(opt.step_count) == 1 and not opt._scratch.any()
    for i, (b, (p, _, s)) in enumerate(zip(before, made)):
        if i % 5 == 4:
            assert all(torch.equal(a.view(torch.uint8), t.view(torch.uint8))
                       for a, t in zip(raw[i], (p, *s.values())))
        else:
            _check(b, p, s, 1, **(GROUP if i < 400 else other))
    # no gradient at all: a step that moves nothing is still a step
    opt.step([None] * 800)
    assert int(opt.step_count) == 2


@pytest.mark.parametrize("count", [40, 450])
def test_long_launches_of_every_type_at_once(cuda_device, count):
    """More elements than the short tiling takes, in tensors of every type, width and alignment with
    whole tiles and tails: a launch's ring has stages for the widest of them.  450 tensors, all with
    a gradient, take two launches."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    rng = np.random.default_rng(count)
    sizes = rng.integers(1, 2 * 6_000_000 // count, count)
    assert sizes.sum() > 5_000_000
    made = [_make(int(n), *KINDS[i % len(KINDS)], seed=i, offset=(0, 0, 0, 1)[i % 4])
            for i, n in enumerate(sizes)]
    before = [_before(*x) for x in made]
    other = dict(lr=0.003, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0)
    cut = count // 3
    opt = flce.AdamW([dict(params=[x[0] for x in part], states=[x[2] for x in part], **h)
                      for part, h in ((made[:cut], GROUP), (made[cut:], other))],
                     step=torch.full((1,), 9, dtype=torch.int64, device="cuda"))
    opt.step([x[1] for x in made], grad_scale=0.5)
    assert int(opt.step_count) == 10 and not opt._scratch.any()
    for i, (b, (p, _, s)) in enumerate(zip(before, made)):
        _check(b, p, s, 10, scale=0.5, **(GROUP if i < cut else other))


@pytest.mark.parametrize("bits", [32, 8])
def test_run_from_zero_states_against_the_oracle(cuda_device, bits):
    """Six steps from fresh states; each is checked from what the one before it left."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    W = torch.randn(40, 333, device="cuda").to(torch.bfloat16)
    gamma = torch.ones(333, device="cuda")
    opt = flce.AdamW([W, gamma], state_bits=bits, master_weights=True, **GROUP)
    assert ("r" in opt.state[0]) == (bits == 8) and "v" in opt.state[1]   # 333 < min_8bit_size
    assert "master" in opt.state[0] and "master" not in opt.state[1]
    for t in range(1, 7):
        W.main_grad = torch.randn(40, 333, device="cuda") * 0.1 ** t
        gamma.grad = torch.randn(333, device="cuda")
        before = [_before(p, g, s) for p, g, s in zip(opt.params, opt.grads(), opt.state)]
        opt.step()
        for b, p, s in zip(before, opt.params, opt.state):
            _check(b, p, s, t, **GROUP)


def test_zero_infinite_and_nan_gradients(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce
    for bits in (32, 8):
        p = torch.ones(1024, device="cuda")
        opt = flce.AdamW([p], state_bits=bits, min_8bit_size=0, lr=0.1, weight_decay=0.0)
        opt.step([torch.zeros(1024, device="cuda")])
        assert bool((p == 1).all())                       # 0 / (0 + eps)
        s = opt.state[0]
        assert not any(t.view(torch.uint8).any() for t in s.values())
        g = torch.ones(1024, device="cuda")
        g[300], g[700] = float("nan"), float("inf")
        opt.step([g])
        bad = torch.isnan(p)
        assert bool(bad[300]) and bool(bad[700]) and int(bad.sum()) == 2
        assert bool(torch.isnan(s["m"].float()[300]))
        if bits == 8:                                     # the scale tells the block is lost
            assert bool(torch.isnan(s["m_scale"][1])) and bool(torch.isfinite(s["m_scale"][[0, 3]]
                                                                              ).all())
    # tiny states: a block below 448 x 2^-126 holds zeros, and nothing becomes NaN
    p = torch.ones(256, device="cuda")
    opt = flce.AdamW([p], state_bits=8, min_8bit_size=0)
    opt.step([torch.full((256,), 1e-37, device="cuda")])
    opt.step([torch.full((256,), 1e-30, device="cuda")])
    assert bool(torch.isfinite(p).all())
    assert bool((opt.state[0]["r"].float() >= 0).all())


def test_small_second_moments_keep_a_code(cuda_device):
    """One element far above the rest of its block: the others' denominators do not vanish."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    p = torch.zeros(256, device="cuda")
    g = torch.full((256,), 1e-7, device="cuda")
    g[0] = 1.0
    opt = flce.AdamW([p], state_bits=8, min_8bit_size=0, lr=0.1, weight_decay=0.0, eps=1e-12)
    for _ in range(3):
        opt.step([g])
    r = opt.state[0]["r"].float()
    assert float(r[0]) == 448 and bool((r[1:] == 2.0 ** -9).all())
    assert bool((p.abs() <= 3 * 0.1 * 1.2).all())         # steps stay near lr


def test_second_moments_below_the_normal_range_keep_a_code(cuda_device):
    """v below 2^-126, which the approximate root takes for 0, keeps its code: the largest of a block
    448, a small one next to a large one the smallest.  g = 1e-19 and c2 = 0.04 give v = 2^-130.9,
    known to half of 2^-149: its root is off by under 2^-19, the scale by 8 u more."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    g = torch.full((512,), 1e-19, device="cuda")
    g[256], g[300], g[3] = 1.0, 0.0, 0.0
    p = torch.zeros(512, device="cuda")
    opt = flce.AdamW([p], state_bits=8, min_8bit_size=0, **GROUP)
    opt.step([g])
    r, scale = opt.state[0]["r"].float(), opt.state[0]["r_scale"]
    want = torch.full((512,), 448.0, device="cuda")
    want[257:] = 2.0 ** -9
    want[300] = want[3] = 0
    assert torch.equal(r, want)
    root = float(torch.tensor(1e-19)) * 0.04 ** 0.5
    assert abs(float(scale[0]) * 448 / root - 1) <= 2.0 ** -19 + 8 * U
    assert bool((opt.state[0]["m"].float()[g > 0] != 0)[:255].all())


def test_skip_on_a_factor_that_is_not_finite(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce
    p, g, s = _make(5000, "bf16", "f32", 8, seed=1)
    g[77] = float("inf")
    raw = [t.clone() for t in (p, *s.values())]
    opt = flce.AdamW([dict(params=[p], states=[s])])
    norm, factor = flce.grad_norm([g], max_norm=1.0)
    assert torch.isinf(norm) and torch.isnan(factor)
    opt.step([g], grad_scale=factor)
    assert int(opt.step_count) == 0 and not opt._scratch.any()
    assert all(torch.equal(a.view(torch.uint8), t.view(torch.uint8))
               for a, t in zip(raw, (p, *s.values())))
    opt.skip_nonfinite = False
    opt.step([g], grad_scale=factor)
    assert int(opt.step_count) == 1 and bool(torch.isnan(p).all())


def test_captured_steps_count_and_read_the_rate(cuda_device):
    """A captured step replayed with other gradients and another rate equals eager steps."""
    import torch
    import lm_head_linear_gemm_b200 as flce

    def fresh():
        made = [_make(n, "bf16", "f32", 8, seed=2) for n in (5000, 300)]
        lr = torch.full((1,), 0.01, device="cuda")
        opt = flce.AdamW([dict(params=[x[0] for x in made], states=[x[2] for x in made], lr=lr)])
        return made, opt, lr

    a, eager, lr_a = fresh()
    b, captured, lr_b = fresh()
    grads = [torch.empty_like(x[1]) for x in b]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, factor = flce.grad_norm(grads, max_norm=0.5)
        captured.step(grads, grad_scale=factor)
    assert int(captured.step_count) == 0
    for t in range(3):
        for i, (x, y) in enumerate(zip(a, grads)):
            y.copy_(x[1] * (t + 1))
        lr_a.fill_(0.01 / (t + 1))
        lr_b.copy_(lr_a)
        n, f = flce.grad_norm(grads, max_norm=0.5)
        eager.step(grads, grad_scale=f)
        graph.replay()
        assert torch.equal(n, norm) and torch.equal(f, factor)
    assert int(eager.step_count) == int(captured.step_count) == 3
    for (p, _, s), (q, _, r) in zip(a, b):
        assert torch.equal(p, q)
        assert all(torch.equal(s[k].view(torch.uint8), r[k].view(torch.uint8)) for k in s)


@pytest.mark.parametrize("scale", [0.5, 0.1, 2])
def test_a_number_as_the_factor_waits_for_nothing(cuda_device, scale):
    """A factor given as a number is filled in on the device: a step with it may be captured, and an
    eager one does not wait for what the stream still has to do."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    g = torch.randn(300, device="cuda")
    made = [torch.ones(300, device="cuda") for _ in range(3)]
    opts = [flce.AdamW([p]) for p in made]
    opts[0].step([g], grad_scale=torch.tensor(float(scale), device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opts[1].step([g], grad_scale=scale)
    graph.replay()
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)                      # about 0.5 s
    opts[2].step([g], grad_scale=scale)
    assert not torch.cuda.current_stream().query()
    assert torch.equal(made[0], made[1]) and torch.equal(made[0], made[2])


def test_numbers_beyond_fp32_as_the_factor(cuda_device):
    """They are infinite on the device, and the step is skipped."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    p = torch.ones(300, device="cuda")
    opt = flce.AdamW([p])
    for scale in (1e39, float("inf"), float("nan")):
        opt.step([p.clone()], grad_scale=scale)
    assert bool((p == 1).all()) and int(opt.step_count) == 0
    with pytest.raises(TypeError):
        opt.step([p.clone()], grad_scale="half")


def test_eight_bit_states_take_the_definitions_roundings(cuda_device):
    """m, v, scales and codes equal, bit for bit, the definition computed by torch in fp32 one
    operation at a time; two steps, so that the second starts from the first's codes."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    n = 300 * 256 + 100
    p, g, s = _make(n, "bf16", "f32", 8, seed=11)
    pad = lambda t: torch.nn.functional.pad(t.float(), (0, -n % 256)).view(-1, 256)
    b1, c1, b2, c2 = (torch.tensor(x, dtype=torch.float64, device="cuda").float()
                      for x in (0.8, 1 - 0.8, 0.96, 1 - 0.96))
    gs = torch.tensor(0.83, device="cuda")
    m8, r8 = pad(s["m"]), pad(s["r"])
    ms, rs = s["m_scale"].clone()[:, None], s["r_scale"].clone()[:, None]
    opt = flce.AdamW([dict(params=[p], states=[s])], **GROUP)
    for _ in range(2):
        opt.step([g], grad_scale=gs)
        gg = pad(g) * gs
        m = b1 * (m8 * ms) + c1 * gg
        v = b2 * (r8 * rs).square() + c2 * gg.square()
        r = v.sqrt()
        scale = lambda x: x.abs().amax(1, keepdim=True) * torch.tensor(1 / 448, device="cuda")
        code = lambda x, sc: torch.where(sc == 0, 0.0, (x / sc).clamp(-448, 448)).to(
            torch.float8_e4m3fn).float()
        ms, rs = scale(m), scale(r)
        m8 = code(m, ms)
        r8 = code(torch.where(r > 0, torch.maximum(r, 2.0 ** -9 * rs), r), rs)
        assert torch.equal(s["m_scale"], ms[:, 0]) and torch.equal(s["r_scale"], rs[:, 0])
        assert torch.equal(s["m"].float(), m8.view(-1)[:n])
        assert torch.equal(s["r"].float(), r8.view(-1)[:n])


def test_a_graph_that_saved_a_parameter_notices_the_step(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce
    p = torch.ones(300, device="cuda", requires_grad=True)
    opt = flce.AdamW([p], lr=0.1)
    y = (p * p).sum()
    opt.step([torch.ones(300, device="cuda")])
    with pytest.raises(RuntimeError):
        y.backward()
    assert opt.status() == 0


def test_a_parameter_left_alone_stays_usable_in_its_graph(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce
    p, q = (torch.full((300,), 2.0, device="cuda", requires_grad=True) for _ in range(2))
    opt = flce.AdamW([p, q], lr=0.1)
    y = (p * p).sum()
    opt.step([None, torch.ones(300, device="cuda")])
    y.backward()
    assert bool((p.grad == 4).all()) and not bool((q == 2).any())


@pytest.mark.parametrize("why", ["eps", "factor", "gradient", "moved"])
def test_a_refused_step_leaves_the_parameters_graphs_usable(cuda_device, why):
    import torch
    import lm_head_linear_gemm_b200 as flce
    p, q = (torch.full((300,), 2.0, device="cuda", requires_grad=True) for _ in range(2))
    opt = flce.AdamW([p, q], lr=0.1)
    y, g = (p * p).sum(), [torch.ones(300, device="cuda") for _ in range(2)]
    scale = None
    if why == "eps":
        opt.param_groups[0]["eps"] = 0.0
    elif why == "factor":
        scale = torch.ones(1, dtype=torch.float64, device="cuda")
    elif why == "gradient":
        g[1] = g[1].half()
    else:
        q.data = q.data[:100]
        g[1] = g[1][:100]
    with pytest.raises((flce.FlceError, TypeError, ValueError)):
        opt.step(g, grad_scale=scale)
    y.backward()
    assert bool((p.grad == 4).all()) and int(opt.step_count) == 0


def test_a_lone_tensor_is_one_parameter(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce
    p = torch.ones(3, 5, device="cuda")
    opt = flce.AdamW([dict(params=p)])
    assert len(opt.params) == 1
    opt.step([torch.ones(3, 5, device="cuda")])
    assert not bool((p == 1).any())
    with pytest.raises(TypeError):
        flce.AdamW(p)


def test_states_are_not_replaced_and_a_device_rate_is_copied(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce
    rate = lambda x: torch.full((1,), x, device="cuda")
    p, q = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    mine = rate(0.5)
    opt, other = flce.AdamW([p], lr=mine), flce.AdamW([q], lr=rate(0.25))
    with pytest.raises(TypeError):
        opt.state[0]["m"] = torch.zeros(300, device="cuda")
    opt.load_state_dict(other.state_dict())
    assert opt.param_groups[0]["lr"] is mine and float(mine) == 0.25
    third = flce.AdamW([torch.ones(300, device="cuda")], lr=0.125)
    third.load_state_dict(other.state_dict())
    other.param_groups[0]["lr"].fill_(1.0)
    assert float(third.param_groups[0]["lr"]) == 0.25
    opt.load_state_dict(flce.AdamW([q], lr=0.125).state_dict())
    assert opt.param_groups[0]["lr"] == 0.125


@pytest.mark.parametrize("saved_on", ["host", "device"])
def test_a_captured_step_follows_a_loaded_rate(cuda_device, saved_on):
    """A step captured with its rate on the device reads the rate that load_state_dict brings,
    whether that was saved as a number or as a tensor."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    g = torch.randn(300, device="cuda")
    rate = torch.full((1,), 0.5, device="cuda")
    p, q = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    opt = flce.AdamW([p], lr=rate)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step([g])
    lr = 0.125 if saved_on == "host" else torch.full((1,), 0.125, device="cuda")
    other = flce.AdamW([q], lr=lr)
    opt.load_state_dict(other.state_dict())
    assert opt.param_groups[0]["lr"] is rate and float(rate) == 0.125
    other.step([g])
    graph.replay()
    assert torch.equal(p, q)


def test_optimizers_at_once_on_two_streams(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce

    def make(seed):
        made = [_make(n, "bf16", "bf16", 8, seed=seed) for n in (70000, 300, 4096)]
        return made, flce.AdamW([dict(params=[x[0] for x in made], states=[x[2] for x in made])])

    pairs = [(make(s), make(s)) for s in (21, 22)]
    streams = [torch.cuda.Stream() for _ in pairs]
    torch.cuda.synchronize()
    for _ in range(6):
        for (a, _), st in zip(pairs, streams):
            a[1].step([x[1] for x in a[0]], stream=st)
    torch.cuda.synchronize()
    for (a, b) in pairs:
        for _ in range(6):
            b[1].step([x[1] for x in b[0]])
        for (p, _, s), (q, _, r) in zip(a[0], b[0]):
            assert torch.equal(p, q) and all(
                torch.equal(s[k].view(torch.uint8), r[k].view(torch.uint8)) for k in s)


def test_other_stream_moved_parameter_and_checkpoint(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce
    p, g, s = _make(3000, "bf16", "bf16", 32, seed=4)
    opt = flce.AdamW([dict(params=[p], states=[s])], **GROUP)
    b = _before(p, g, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    opt.step([g], grad_scale=0.5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(b, p, s, 1, scale=0.5, **GROUP)
    old = p.data
    p.data = p.data.clone()                               # moved: the step follows the parameter
    b = _before(p, g, s)
    frozen = old.clone()
    opt.step([g])
    assert torch.equal(old, frozen)
    _check(b, p, s, 2, **GROUP)
    saved = {k: v for k, v in opt.state_dict().items()}
    saved["state"] = [{k: t.clone() for k, t in st.items()} for st in saved["state"]]
    saved["step"] = saved["step"].clone()
    q = p.clone()
    twin = flce.AdamW([q])
    twin.load_state_dict(saved)
    assert twin.param_groups[0]["lr"] == GROUP["lr"] and int(twin.step_count) == 2
    opt.step([g])
    twin.step([g])
    assert torch.equal(p, q)
    with pytest.raises(ValueError):
        flce.AdamW([q], state_bits=8, min_8bit_size=0).load_state_dict(saved)


def test_a_parameter_replaced_at_the_same_address(cuda_device):
    """p.data cut short or made another type in place is noticed, although its address stays."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    p = torch.ones(600, device="cuda")
    opt = flce.AdamW([p])
    whole = p.data
    p.data = whole[:100]
    with pytest.raises(ValueError):                       # its states have 600 elements
        opt.step([torch.ones(100, device="cuda")])
    assert bool((whole == 1).all()) and int(opt.step_count) == 0
    p.data = whole
    opt.step([torch.ones(600, device="cuda")])
    assert not bool((whole == 1).any())


def test_offsets_past_32_bits(cuda_device):
    """2^31 + 4133 elements in 8-bit states: the last block's values equal a small tensor's."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    tail, n = 4133, 2 ** 31 + 4133
    p, g, s = _make(tail, "bf16", "bf16", 8, seed=5)
    big_p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    big_g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    big_p[-tail:], big_g[-tail:] = p, g
    st = {k: torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
          for k in ("m", "r")}
    blocks = -(-n // 256)
    for k in ("m_scale", "r_scale"):
        st[k] = torch.zeros(blocks, device="cuda")
        st[k][-(-(-tail // 256)):] = s[k]
    for k in ("m", "r"):
        st[k].view(torch.uint8)[-tail:] = s[k].view(torch.uint8)
    norm_big, _ = flce.grad_norm([big_g], 1.0)
    norm_small, _ = flce.grad_norm([g], 1.0)
    assert abs(float(norm_big) - float(norm_small)) <= 70 * U * float(norm_small)
    flce.AdamW([dict(params=[big_p], states=[st])]).step([big_g])
    flce.AdamW([dict(params=[p], states=[s])]).step([g])
    assert torch.equal(big_p[-tail:], p) and not big_p[:2 ** 31].any()
    for k in ("m", "r"):
        assert torch.equal(st[k].view(torch.uint8)[-tail:], s[k].view(torch.uint8))


def test_binding_refuses(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce
    p = torch.ones(600, device="cuda")
    opt = flce.AdamW([p])
    for g, err in ((torch.ones(600, 1, device="cuda"), ValueError), (torch.ones(601, device="cuda"), ValueError), (torch.ones(600), ValueError),
                   (torch.ones(600, device="cuda").half(), TypeError),
                   (torch.ones(1200, device="cuda")[::2], ValueError)):
        with pytest.raises(err):
            opt.step([g])
    with pytest.raises(ValueError):
        opt.step([])
    with pytest.raises(TypeError):
        opt.step([p.clone()], grad_scale=torch.ones(1, dtype=torch.float64, device="cuda"))
    for bad in ([p, p], [p[:300], p[200:]]):              # overlapping memory
        with pytest.raises(ValueError):
            flce.AdamW(bad)
    ok = dict(m=torch.zeros(600, device="cuda"), v=torch.zeros(600, device="cuda"))
    for change, err in ((dict(v=torch.zeros(599, device="cuda")), ValueError),
                        (dict(v=torch.zeros(600, device="cuda").bfloat16()), TypeError),
                        (dict(r=torch.zeros(600, device="cuda")), ValueError),
                        (dict(master=torch.zeros(600, device="cuda")), ValueError),
                        (dict(m=ok["v"]), ValueError)):
        with pytest.raises(err):
            flce.AdamW([dict(params=[p], states=[{**ok, **change}])])
    with pytest.raises(TypeError):
        flce.AdamW([p], step=torch.zeros(1, device="cuda"))


# ------------------------------------------------------------------------------- gradient norm
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1])
def test_grad_norm(cuda_device, dtype, offset):
    """A thread sums 64 squares in fp32 before it goes on in 64 bits: 64 units of the sum, half of
    them in its root, and the root's rounding."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    rng = np.random.default_rng(8)
    grads = []
    for n in SIZES + [0, 16384, 16385, 3000000]:
        t = torch.zeros(n + offset, dtype=_dtype(dtype), device="cuda")[offset:]
        t.copy_(torch.from_numpy(rng.standard_normal(n) * 10.0 ** rng.uniform(-4, 0)))
        grads.append(t)
    for max_norm in (0.5, 1e9):
        want, wf = ot.grad_norm([_np(g) for g in grads], max_norm)
        norm, factor = flce.grad_norm(grads + [None], max_norm)
        assert norm.dtype == torch.float32 and norm.dim() == 0
        assert abs(float(norm) - want) <= 34 * U * want
        assert abs(float(factor) - wf) <= 40 * U * wf
        again, _ = flce.grad_norm(grads, max_norm)
        assert torch.equal(norm, again)
    assert flce.grad_norm(grads)[1] is None
    for bad, err in (([grads[5], grads[5].cpu()], ValueError), ([grads[5].cpu()], ValueError),
                     ([grads[5], grads[5].double()], TypeError), ([grads[6][::2]], ValueError)):
        with pytest.raises(err):
            flce.grad_norm(bad)


def test_grad_norm_of_many_large_tensors(cuda_device):
    """More tensors than the small launch takes, with whole chunks, tails, both types, any alignment."""
    import torch
    import lm_head_linear_gemm_b200 as flce
    rng = np.random.default_rng(12)
    grads = []
    for i in range(1100):                                 # two launches
        n, offset = int(rng.integers(1, 60000 if i % 10 == 0 else 2000)), i % 3
        t = torch.zeros(n + offset, dtype=_dtype(("bf16", "f32")[i % 2]), device="cuda")[offset:]
        t.copy_(torch.from_numpy(rng.standard_normal(n) * 10.0 ** rng.uniform(-4, 0)))
        grads.append(t)
    assert sum(g.numel() >= 16384 for g in grads) > 50
    want, wf = ot.grad_norm([_np(g) for g in grads], 0.5)
    norm, factor = flce.grad_norm(grads, 0.5)
    assert abs(float(norm) - want) <= 34 * U * want and abs(float(factor) - wf) <= 40 * U * wf
    assert torch.equal(norm, flce.grad_norm(grads)[0])


def test_grad_norm_of_many_none_zero_and_nan(cuda_device):
    import torch
    import lm_head_linear_gemm_b200 as flce
    grads = [torch.full((1 + i % 3,), 0.5, device="cuda") for i in range(2500)]   # three launches
    want = 0.5 * np.sqrt(sum(g.numel() for g in grads))
    norm, factor = flce.grad_norm(grads, 1.0)
    assert abs(float(norm) - want) <= 34 * U * want
    zero, factor = flce.grad_norm([torch.zeros(10, device="cuda")], 1.0)
    assert float(zero) == 0 and float(factor) == 1
    empty, _ = flce.grad_norm([torch.zeros(0, device="cuda")], 1.0)
    assert float(empty) == 0
    nan, factor = flce.grad_norm([torch.full((3,), float("nan"), device="cuda")], 1.0)
    assert torch.isnan(nan) and torch.isnan(factor)
