"""AdamW over many tensors (-m gpu): every result equals, bit for bit, the same
fp32 operations done one by one on the host (numpy rounds each), and lies within
their summed roundings of the formula in fp64."""
import ctypes

import numpy as np
import pytest

gpu = pytest.mark.gpu
BLOCK = 256
F = np.float32


def constants(t, lr, b1, b2, eps, wd):
    return dict(b1=F(b1), b2=F(b2), c1m=F(1.0 - b1), c2m=F(1.0 - b2), decay=F(1.0 - lr * wd),
                c1=F(lr / (1.0 - b1 ** t)), c2=F(1.0 / np.sqrt(1.0 - b2 ** t)), eps=F(eps))


def ref_update(p, g, m, v, c, scale=None):
    """fp32 operations, each rounded by itself."""
    if scale is not None:
        g = g * F(scale)
    m = m * c["b1"] + g * c["c1m"]
    v = v * c["b2"] + (g * g) * c["c2m"]
    root = np.sqrt(v)
    p = p * c["decay"] - (m * c["c1"]) / (root * c["c2"] + c["eps"])
    assert p.dtype == m.dtype == root.dtype == np.float32
    return p, m, v, root


def e4m3(x):
    import torch
    return torch.from_numpy(np.clip(x, F(-448), F(448))).to(torch.float8_e4m3fn)


def ref_encode(x, root):
    """(codes, scales) of one tensor, block by block."""
    import torch
    n = x.size
    codes, scales = torch.zeros(n, dtype=torch.uint8), np.zeros(-(-n // BLOCK), F)
    for b in range(scales.size):
        y = x[b * BLOCK:(b + 1) * BLOCK]
        top = np.max(np.abs(y))
        if top > F(2.0 ** -100):
            z = y * (F(448) * (F(1) / top))
            if root:
                z = np.where((y > 0) & (z < F(2.0 ** -9)), F(2.0 ** -9), z)
            codes[b * BLOCK:(b + 1) * BLOCK] = e4m3(z.astype(F)).view(torch.uint8)
            scales[b] = top * (F(1) / F(448))
    return codes, scales


def ref_decode(codes, scales):
    import torch
    return codes.view(torch.float8_e4m3fn).float().numpy() * np.repeat(scales, BLOCK)[:codes.numel()]


def bf16(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


SIZES = [1, 2, 7, 8, 255, 256, 257, 1000, 4096, 70_001]


class Case:
    """Tensors at any alignment inside larger ones, whose other elements must stay as they are."""

    def __init__(self, sizes, bits, grad="float32", copy=False, off=0, seed=0, spread=3.0):
        import torch
        self.sizes, self.bits, self.off = sizes, bits, off
        self.rng = np.random.default_rng(seed)
        self.big = {}
        self.p = self._tensors("p", torch.float32, 0.5)
        self.g = self._tensors("g", getattr(torch, grad), 0.0)
        self.spread = spread
        self.new_grads()
        eight = bits == 8
        self.m = self._tensors("m", torch.uint8 if eight else torch.float32, 0)
        self.v = self._tensors("v", torch.uint8 if eight else torch.float32, 0)
        self.copies = self._tensors("c", torch.bfloat16, 0.0) if copy else None
        rng = self.rng
        for p in self.p:
            p.copy_(torch.from_numpy(rng.standard_normal(p.numel()).astype(F)))
        self.state = None
        if eight:
            self.ms = self._tensors("ms", torch.float32, 0.0, [-(-n // BLOCK) for n in sizes], 0)
            self.vs = self._tensors("vs", torch.float32, 0.0, [-(-n // BLOCK) for n in sizes], 0)
        self.step = torch.zeros(1, dtype=torch.int32, device="cuda")

    def _tensors(self, name, dtype, fill, sizes=None, off=None):
        import torch
        off = self.off if off is None else off
        out = []
        for i, n in enumerate(sizes or self.sizes):
            big = torch.full((n + off + 16,), fill, dtype=dtype, device="cuda")
            self.big[name, i] = (big, off, n, big.clone())
            out.append(big[off:off + n])
        return out

    def new_grads(self):
        import torch
        for g in self.g:
            x = self.rng.standard_normal(g.numel()) * np.exp(self.spread * self.rng.standard_normal(g.numel()))
            g.copy_(torch.from_numpy(x.astype(F)))

    def make(self, **kw):
        import torch
        from token_dispatch_histogram_b200.optim import EpAdamW
        eight = self.bits == 8
        as8 = (lambda ts: [t.view(torch.float8_e4m3fn) for t in ts]) if eight else (lambda ts: ts)
        return EpAdamW(self.p, self.g, state_bits=self.bits, copies=self.copies,
                       state=dict(step=self.step, m=as8(self.m), v=as8(self.v), m_scale=self.ms if eight else None,
                                  v_scale=self.vs if eight else None), **kw)

    def numpy(self):
        get = lambda ts: [t.float().cpu().numpy() if t.dtype.is_floating_point else t.cpu() for t in ts]  # noqa: E731
        return dict(p=get(self.p), g=get(self.g), m=get(self.m), v=get(self.v),
                    ms=get(self.ms) if self.bits == 8 else None, vs=get(self.vs) if self.bits == 8 else None)

    def outside_is_untouched(self):
        import torch
        for (name, i), (big, off, n, was) in self.big.items():
            assert torch.equal(big[:off], was[:off]) and torch.equal(big[off + n:], was[off + n:]), (name, i)


def ref_step(s, bits, c, scale=None):
    out = dict(p=[], m=[], v=[], ms=[], vs=[])
    for i in range(len(s["p"])):
        m = ref_decode(s["m"][i], s["ms"][i]) if bits == 8 else s["m"][i]
        v = ref_decode(s["v"][i], s["vs"][i]) if bits == 8 else s["v"][i]
        v = v * v if bits == 8 else v
        p, m, v, root = ref_update(s["p"][i], s["g"][i], m, v, c, scale)
        out["p"].append(p)
        if bits == 8:
            for x, k, r in ((m, "m", False), (root, "v", True)):
                codes, scales = ref_encode(x, r)
                out[k].append(codes)
                out[k + "s"].append(scales)
        else:
            out["m"].append(m)
            out["v"].append(v)
    return out


def same(case, want):
    import torch
    got = case.numpy()
    for k in ("p", "m", "v") + (("ms", "vs") if case.bits == 8 else ()):
        for i in range(len(case.sizes)):
            a, b = np.asarray(got[k][i]), np.asarray(want[k][i])
            assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f"), (k, i, int((a != b).sum()))
    if case.copies is not None:
        for c, p in zip(case.copies, got["p"]):
            assert torch.equal(c.cpu(), bf16(p))
    case.outside_is_untouched()


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["float32", "bfloat16"])
@pytest.mark.parametrize("off,copy", [(0, True), (1, True), (4, False), (3, False)])
def test_steps_equal_the_operations_one_by_one(bits, grad, off, copy):
    kw = dict(lr=2e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    case = Case(SIZES, bits, grad, copy, off)
    opt = case.make(**kw)
    for t in range(1, 5):
        case.new_grads()
        want = ref_step(case.numpy(), bits, constants(t, 2e-2, 0.9, 0.95, 1e-8, 0.1))
        opt.step()
        assert int(case.step) == t
        same(case, want)


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_steps_stay_near_the_formula_in_64_bits(bits):
    """One step from an earlier state: m and v take three roundings, p about ten of numbers no larger than |p| and the
    update's size; a code adds half a unit of its last place, or the smallest code where a root is held above zero."""
    import torch
    case = Case([1000, 4096], bits, spread=1.0)
    opt = case.make(lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.05)
    for _ in range(3):
        case.new_grads()
        opt.step()
    case.new_grads()
    s = case.numpy()
    opt.step()
    got = case.numpy()
    eps = 2.0 ** -24
    for i in range(2):
        g, p = s["g"][i].astype(np.float64), s["p"][i].astype(np.float64)
        m0 = ref_decode(s["m"][i], s["ms"][i]) if bits == 8 else s["m"][i]
        v0 = ref_decode(s["v"][i], s["vs"][i]).astype(np.float64) ** 2 if bits == 8 else s["v"][i].astype(np.float64)
        m = 0.9 * m0.astype(np.float64) + 0.1 * g
        v = 0.99 * v0 + 0.01 * g * g
        u = 1e-2 / (1 - 0.9 ** 4) * m / (np.sqrt(v / (1 - 0.99 ** 4)) + 1e-6)
        mag = 0.9 * np.abs(m0) + 0.1 * np.abs(g)
        um = np.abs(u) * mag / np.maximum(np.abs(m), 1e-300)
        assert np.all(np.abs(got["p"][i] - (p * (1 - 5e-4) - u)) <= eps * (3 * np.abs(p) + 12 * um + 2 * np.abs(u)))
        if bits == 32:
            assert np.all(np.abs(got["m"][i] - m) <= 4 * eps * mag)
            assert np.all(np.abs(got["v"][i] - v) <= 6 * eps * v)
        else:
            gm, gv = ref_decode(got["m"][i], got["ms"][i]), ref_decode(got["v"][i], got["vs"][i])
            sm, sv = (np.repeat(x, BLOCK)[:gm.size] for x in (got["ms"][i], got["vs"][i]))
            assert np.all(np.abs(gm - m) <= np.maximum(2.0 ** -4 * np.abs(m), sm * 2.0 ** -10) + 8 * eps * mag)
            r = np.sqrt(v)
            assert np.all(np.abs(gv - r) <= np.maximum(2.0 ** -4 * r, sv * 2.0 ** -9) + 8 * eps * r)
            assert np.all(gv[r > 0] > 0)
    assert torch.all(torch.isfinite(case.p[0]))


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_blocks_of_zeros_and_of_very_small_and_large_values(bits):
    import torch
    case = Case([256 * 6 + 30], bits, spread=0.0)
    opt = case.make(lr=1e-3, betas=(0.9, 0.999), eps=0.0 if bits == 8 else 1e-8, weight_decay=0.0)
    g = case.g[0]
    g[:256] = 1e-20
    g[256:512] *= 1e-38        # squares vanish; the first moment is subnormal or below 2^-100
    g[512:768] *= 1e18
    g[768:1024] *= 1e-18
    g[1024] = 1e9              # one element far above the others of its block
    g[1536:] = 0.0
    c = constants(1, 1e-3, 0.9, 0.999, 0.0 if bits == 8 else 1e-8, 0.0)
    with np.errstate(all="ignore"):
        want = ref_step(case.numpy(), bits, c)
    opt.step()
    same(case, want)
    assert torch.all(torch.isfinite(case.p[0][512:1536]))


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_bad_gradient_stays_where_it_is(bits):
    """A NaN keeps to its element, an infinity to its block of 256; the other blocks step as if it were not there."""
    case, clean = Case([256 * 4], bits), Case([256 * 4], bits)
    case.g[0][300], case.g[0][700] = float("nan"), float("inf")
    kw = dict(lr=1e-3)
    for c in (case, clean):
        o = c.make(**kw)
        o.step()
        c.g[0].fill_(0.5)
        o.step()
    a, b = case.numpy(), clean.numpy()
    ok = np.ones(1024, bool)
    ok[300] = False
    ok[512:768] = False
    for k in ("p", "m", "v"):
        x, y = np.asarray(a[k][0]), np.asarray(b[k][0])
        sel = ok if bits == 32 or k == "p" else ok & ~((np.arange(1024) >= 256) & (np.arange(1024) < 512))
        np.testing.assert_array_equal(x[sel & ~((np.arange(1024) >= 256) & (np.arange(1024) < 512))],
                                      y[sel & ~((np.arange(1024) >= 256) & (np.arange(1024) < 512))])
    assert np.isnan(a["p"][0][300]) and np.all(np.isfinite(a["p"][0][ok]))


@gpu
def test_more_tensors_than_a_launch_takes_and_empty_ones():
    import token_dispatch_histogram_b200 as tdh
    sizes = [int(n) for n in np.random.default_rng(3).integers(0, 600, 700)]
    sizes[5:9] = [0, 0, 0, 0]
    sizes[-1] = 0
    case = Case(sizes, 8, copy=True)
    opt = case.make(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    s = case.numpy()
    want = ref_step({k: [x for x, n in zip(v, sizes) if n] if v is not None else None for k, v in s.items()}, 8,
                    constants(1, 1e-2, 0.9, 0.95, 1e-8, 0.1))
    before = tdh.ep_launch_count()
    opt.step()
    assert tdh.ep_launch_count() - before == -(-sum(n > 0 for n in sizes) // 256)
    got = case.numpy()
    at = 0
    for i, n in enumerate(sizes):
        if n:
            for k in ("p", "m", "v", "ms", "vs"):
                np.testing.assert_array_equal(np.asarray(got[k][i]), np.asarray(want[k][at]))
            at += 1
    case.outside_is_untouched()


@gpu
def test_a_tensor_of_many_blocks_is_covered_once():
    import torch
    n = 148 * 8 * 8 * 256 * 2 + 77  # more than two rounds of the grid
    g = torch.Generator(device="cuda").manual_seed(0)
    p, grad = (torch.randn(n, generator=g, device="cuda") for _ in range(2))
    was = p.clone()
    from token_dispatch_histogram_b200.optim import EpAdamW
    opt = EpAdamW([p], [grad], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    opt.step()
    c = constants(1, 1e-2, 0.9, 0.95, 1e-8, 0.1)
    w, m, v, _ = ref_update(was.cpu().numpy(), grad.cpu().numpy(), np.zeros(n, F), np.zeros(n, F), c)
    np.testing.assert_array_equal(p.cpu().numpy(), w)
    np.testing.assert_array_equal(opt.m[0].cpu().numpy(), m)
    np.testing.assert_array_equal(opt.v[0].cpu().numpy(), v)


@gpu
def test_offsets_past_32_bits():
    import torch
    from token_dispatch_histogram_b200.optim import EpAdamW
    n, tail = (1 << 31) + 256 * 3 + 50, 5000
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-tail:], g[-tail:] = torch.randn(tail, device="cuda"), torch.randn(tail, device="cuda").bfloat16()
    was, grad = p[-tail:].cpu().numpy(), g[-tail:].float().cpu().numpy()
    opt = EpAdamW([p], [g], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, state_bits=8)
    opt.step()
    c = constants(1, 1e-2, 0.9, 0.95, 1e-8, 0.1)
    w, m, v, root = ref_update(was, grad, np.zeros(tail, F), np.zeros(tail, F), c)
    np.testing.assert_array_equal(p[-tail:].cpu().numpy(), w)
    assert torch.all(p[:-tail] == 0) and torch.all(opt.m[0].view(torch.uint8)[:-tail] == 0)
    # whole blocks of the tail, which starts inside one
    skip = (-(n - tail)) % BLOCK
    codes, scales = ref_encode(m[skip:], False)
    assert torch.equal(opt.m[0][-tail + skip:].view(torch.uint8).cpu(), codes)
    np.testing.assert_array_equal(opt.m_scale[0][-scales.size:].cpu().numpy(), scales)


@gpu
def test_learning_rate_and_scale_on_the_device_and_a_replayed_graph():
    import torch
    case, other = Case([1000, 300], 8, copy=True), Case([1000, 300], 8, copy=True)
    lr = torch.full((1,), 1e-2, device="cuda")
    scale = torch.full((1,), 0.5, device="cuda")
    a = case.make(lr=lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    want = ref_step(case.numpy(), 8, constants(1, float(lr), 0.9, 0.95, 1e-8, 0.1), 0.5)
    a.step(grad_scale=scale)
    same(case, want)
    # the same steps, eager and replayed, while rate, scale and gradients change between them
    b = other.make(lr=lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    b.step(grad_scale=scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(grad_scale=scale)
    for k in range(3):
        lr.fill_(1e-2 / (k + 2))
        scale.fill_(1.0 / (k + 1))
        case.new_grads()
        for x, y in zip(case.g, other.g):
            y.copy_(x)
        a.step(grad_scale=scale)
        graph.replay()
    assert int(other.step) == 4
    for x, y in ((case.p, other.p), (case.m, other.m), (case.v, other.v), (case.copies, other.copies),
                 (case.ms, other.ms), (case.vs, other.vs)):
        assert all(torch.equal(i, j) for i, j in zip(x, y))


@gpu
def test_another_stream_and_going_on_from_a_state():
    import torch
    from token_dispatch_histogram_b200.optim import EpAdamW
    case = Case([5000], 32)
    a = EpAdamW(case.p, case.g, lr=1e-2)
    q = case.p[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(stream=side)
    a.step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b = EpAdamW([q], case.g, lr=1e-2)
    b.step()
    c = EpAdamW([q], case.g, lr=1e-2, state=b.state_dict())
    c.step()
    assert torch.equal(q, case.p[0]) and int(c.steps) == 2 and torch.equal(c.m[0], a.m[0])


@gpu
@pytest.mark.parametrize("noisy", [False, True])
@pytest.mark.parametrize("change", [5.0, 0.2])
@pytest.mark.parametrize("beta2,steps", [(0.99, 600), (0.999, 3000)])
def test_moments_in_8_bits_follow_those_in_32(beta2, steps, change, noisy):
    """Half of the gradients change their size for good, and the 8-bit roots follow as the fp32 ones do.

    With c = 1 - beta2, a step moves a root r by c/2 (k - 1) r, k = g^2 / v (E|k - 1| < 1), so its code by chance: a
    variance of at most c/2 r * r/8 a step (a code is at most r/8), which decays at 2 c a step: 0.18 r in all, twice that
    while k is not 1.  Rounding by chance has no bias; that of a root of noisy v is half the variance, 2 %."""
    import torch
    from token_dispatch_histogram_b200.optim import EpAdamW
    n = 256 * 64
    g = torch.Generator(device="cuda").manual_seed(1)
    size = torch.exp(torch.randn(n, generator=g, device="cuda"))
    moved = torch.rand(n, generator=g, device="cuda") < 0.5
    grad = torch.empty(n, device="cuda")
    a, b = (EpAdamW([torch.zeros(n, device="cuda")], [grad], lr=1e-6, betas=(0.9, beta2), weight_decay=0.0,
                    state_bits=bits) for bits in (8, 32))
    for t in range(2 * steps):
        grad.copy_(size * torch.randn(n, generator=g, device="cuda") if noisy else size)
        if t >= steps:
            grad[moved] *= change
        a.step()
        b.step()
    ratio = a.v[0].float() * a.v_scale[0].repeat_interleave(BLOCK) / b.v[0].sqrt()
    for part in (ratio[moved], ratio[~moved]):
        assert 0.9 <= float(part.mean()) <= 1.1 and float(part.std()) <= 0.36


@gpu
@pytest.mark.parametrize("off,n", [(0, 256 * 400), (3, 70_001)])
def test_roots_are_rounded_by_chance_where_steps_are_small(off, n):
    """Far into a run each root goes to one of the two codes around it, in proportion; all else is as before."""
    import torch
    b2 = 0.999
    cases = [Case([300, n], 8, off=off, spread=1.0) for _ in range(2)]
    opts = [c.make(lr=1e-2, betas=(0.9, b2), eps=1e-8, weight_decay=0.1) for c in cases]
    for c, o in zip(cases, opts):
        for _ in range(3):  # still to nearest: 0.001 / (1 - 0.999^t) is near 1 / t
            o.step()
        c.step.fill_(1000)
        c.new_grads()
        c.g[1][7::1000] = 0.0
    s = cases[0].numpy()
    con = constants(1001, 1e-2, 0.9, b2, 1e-8, 0.1)
    want = ref_step(s, 8, con)
    for o in opts:
        o.step()
    got, other = (c.numpy() for c in cases)
    for k in ("p", "m", "v", "ms", "vs"):
        for i in range(2):
            np.testing.assert_array_equal(np.asarray(got[k][i]), np.asarray(other[k][i]))  # the same chance
            if k != "v":
                np.testing.assert_array_equal(np.asarray(got[k][i]), np.asarray(want[k][i]))
    cases[0].outside_is_untouched()
    v = ref_decode(s["v"][1], s["vs"][1])
    root = ref_update(s["p"][1], s["g"][1], np.zeros_like(v), v * v, con)[3].astype(np.float64)
    vs = np.repeat(got["vs"][1], BLOCK)[:n].astype(np.float64)
    z = root / vs  # in units of the codes' values; 3 roundings of fp32 off what the kernel rounds
    held = got["v"][1].view(torch.float8_e4m3fn).double().numpy()
    unit = 2.0 ** np.maximum(np.floor(np.log2(z)) - 3, -9)
    assert np.all(np.abs(held - z) <= unit * (1 + 2.0 ** -15)) and np.all(held > 0)
    # those above the smallest code and below the largest: no bias, within five deviations of a mean of n (1/2 each at most)
    sel = (z > 2.0 ** -9) & (z < 447)
    assert abs(np.mean(((held - z) / unit)[sel])) <= 5 * 0.5 / np.sqrt(sel.sum())
    # and by chance indeed: farther than half a code as often as that says, 1/4 if places in between are evenly taken
    assert 0.2 <= np.mean((np.abs(held - z) > unit / 2)[sel]) <= 0.3
    # another step, another chance
    for c, t in zip(cases, (1000, 1001)):
        c.step.fill_(t)
    for o in opts:
        o.step()
    assert not torch.equal(cases[0].v[1], cases[1].v[1])


@gpu
def test_a_refused_step_does_not_count():
    import torch
    import token_dispatch_histogram_b200 as tdh
    case = Case([100], 32)
    opt = case.make(lr=1e-2)
    opt.step()
    for bad, err in ((dict(grad_scale=torch.ones(1, dtype=torch.float64, device="cuda")), TypeError),
                     (dict(grad_scale=torch.ones(2, device="cuda")), ValueError),
                     (dict(grad_scale=torch.ones(1)), ValueError)):
        with pytest.raises(err):
            opt.step(**bad)
        assert int(case.step) == 1
    opt.lr = float("nan")
    with pytest.raises(tdh.EpError):
        opt.step()
    assert int(case.step) == 1
    opt.lr = 1e-2
    opt.step()
    assert int(case.step) == 2


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_nan_changes_no_other_element_of_its_block(bits):
    """Every other element, code and scale as if the element with the NaN had gradients of 0."""
    case, clean = Case([256 * 4], bits), Case([256 * 4], bits)
    case.g[0][300], clean.g[0][300] = float("nan"), 0.0
    for c in (case, clean):
        o = c.make(lr=1e-3)
        o.step()
        c.new_grads()
        c.g[0][300] = 0.0
        o.step()
    a, b = case.numpy(), clean.numpy()
    rest = np.arange(1024) != 300
    for k in ("p", "m", "v"):
        x, y = np.asarray(a[k][0]), np.asarray(b[k][0])
        np.testing.assert_array_equal(x[rest], y[rest])
        assert np.isnan(x[300]) if x.dtype == np.float32 else (x[300] & 0x7F) == 0x7F
    if bits == 8:
        np.testing.assert_array_equal(a["ms"][0], b["ms"][0])
        np.testing.assert_array_equal(a["vs"][0], b["vs"][0])


# ------------------------------------------------------------------ refusals (no GPU needed)

def test_adamw_argument_errors():
    import token_dispatch_histogram_b200 as tdh
    L = tdh.lib()
    p = ctypes.c_void_p(0x1000)

    def call(n_tensors=1, bits=32, gdt=0, step=p, lr=1e-3, lr_dev=None, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, gs=None,
             table=True, **fields):
        t = (tdh.EpAdamWTensor * 1)()
        for k, v in dict(p=0x1000, g=0x1000, m=0x1000, v=0x1000, m_scale=0x1000, v_scale=0x1000, n=10).items():
            setattr(t[0], k, v)
        for k, v in fields.items():
            setattr(t[0], k, v)
        return L.ep_adamw(t if table else None, n_tensors, bits, gdt, step, lr, lr_dev, b1, b2, eps, wd, gs, None)

    nan = float("nan")
    for kw in [dict(n_tensors=-1), dict(bits=16), dict(gdt=2), dict(step=None), dict(step=ctypes.c_void_p(0x1001)),
               dict(lr=nan), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=nan), dict(eps=-1.0), dict(eps=nan),
               dict(wd=float("inf")), dict(table=False), dict(p=None), dict(g=None), dict(m=None), dict(v=None),
               dict(bits=8, m_scale=None), dict(bits=8, v_scale=None), dict(p=0x1002), dict(g=0x1002), dict(m=0x1001),
               dict(copy=0x1001), dict(n=-1), dict(n=1 << 40), dict(gdt=1, g=0x1001), dict(gs=ctypes.c_void_p(0x1002)),
               dict(lr_dev=ctypes.c_void_p(0x1002)), dict(bits=8, m_scale=0x1002)]:
        assert call(**kw) == tdh.EP_ERR_ARG, kw
    assert call(n_tensors=0, table=False) == tdh.EP_OK
    assert call(n=0, p=None, g=None, m=None, v=None) == tdh.EP_OK


def test_adamw_refuses_wrong_tensors():
    import torch
    from token_dispatch_histogram_b200.optim import EpAdamW
    x = torch.zeros(8)
    with pytest.raises(ValueError):
        EpAdamW([x], [x])  # CPU tensors
    with pytest.raises(ValueError):
        EpAdamW([], [])
    with pytest.raises(ValueError):
        EpAdamW([x], [x], state_bits=16)
    with pytest.raises(ValueError):
        EpAdamW([x], [x, x])
    with pytest.raises(ValueError):
        EpAdamW([x, x], [x, x])
    with pytest.raises(TypeError):
        EpAdamW([x], [x.half()])
    with pytest.raises(ValueError):
        EpAdamW([x], [x[:7]])
    with pytest.raises(TypeError):
        EpAdamW([x.double()], [x])
