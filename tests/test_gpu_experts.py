"""The experts' products over the slots of a buffer, and their gradients (-m gpu),
against the same sums in fp64.

A result is a sum of K products of bf16 values (exact in fp32), taken 16 at a
time into an fp32 accumulator: each of the K / 16 additions, and a few more
around it, is off by at most 2^-23 of the magnitudes' sum (cut off rather than
rounded); then one rounding to the output's type."""
import ctypes

import numpy as np
import pytest

gpu = pytest.mark.gpu

LENS = {
    "one row": [1],
    "empty slots": [0, 3, 0, 0, 40, 0],
    "around a tile": [127, 128, 129, 1, 255, 257],
    "many short": [2, 0, 1, 5, 3, 1, 0, 8, 1, 1, 2, 7, 4, 0, 0, 6, 33, 1, 2, 3],
    "long": [1500, 0, 900],
}


class Buffer:
    """Slots in a buffer: rows before the first and behind the last belong to none; the last two slots are replicas,
    and one entry of slot_order is no slot at all."""

    def __init__(self, lens, before=5, behind=9, replicas=True):
        import torch
        self.lens = list(lens)
        n = len(self.lens)
        self.E = n - 2 if replicas and n > 3 else n
        self.reps = n - self.E
        cu = np.cumsum([before] + self.lens + [0])  # the entry of no slot has no rows
        self.P = int(cu[-1]) + behind
        self.begin = [int(v) for v in cu[:n]]
        self.expert = list(range(self.E)) + [(3 * m + 1) % self.E for m in range(self.reps)]
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.order = torch.tensor(list(range(n)) + [-1], dtype=torch.int32, device="cuda")
        self.rep = torch.tensor(self.expert[self.E:] or [0], dtype=torch.int32, device="cuda")
        self.outside = np.ones(self.P, bool)
        self.outside[before:cu[-1]] = False
        self.kw = dict(slot_order=self.order, rep_expert=self.rep)

    def slots(self):
        for s, (b, n) in enumerate(zip(self.begin, self.lens)):
            yield s, self.expert[s], slice(b, b + n)


def values(shape, seed, ints=False, scale=1.0):
    """bf16 values; ints: whole numbers so small that every fp32 sum is exact."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    if ints:
        return torch.randint(-2, 3, shape, generator=g, device="cuda").to(torch.bfloat16)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def product(buf, x, w, transposed):
    """(sum, sum of magnitudes) in fp64, zeros outside the slots."""
    import torch
    N = w.shape[2 if transposed else 1]
    y, mag = (torch.zeros((buf.P, N), dtype=torch.float64, device="cuda") for _ in range(2))
    for _, e, r in buf.slots():
        we = w[e].double() if transposed else w[e].double().T
        y[r] = x[r].double() @ we
        mag[r] = x[r].double().abs() @ we.abs()
    return y, mag


def sum_bound(K, mag):
    return (K / 16 + 8) * 2.0 ** -23 * mag


def rounded(bound, want, dtype):
    """The bound of a value that is `bound` off `want`, after one rounding."""
    import torch
    return bound + (want.abs() + bound) * (torch.finfo(dtype).eps / 2) + torch.finfo(dtype).smallest_normal


def check(got, want, bound, buf=None, fill=None):
    import torch
    d = (got.double() - want).abs()
    ok = d <= bound
    if buf is not None:
        out = torch.from_numpy(buf.outside).cuda()
        assert torch.all(got[out] == fill)
        ok = ok | out[:, None]
    assert torch.all(ok), f"{int((~ok).sum())} of {ok.numel()} off, worst {float((d / bound)[~ok].max()):.3g} bounds"


def out(shape, fill=7.0, dtype=None):
    import torch
    return torch.full(shape, fill, dtype=dtype or torch.bfloat16, device="cuda")


def status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def poison_outside(buf, *ts):
    """Values that must take no part, in rows of no slot."""
    import torch
    o = torch.from_numpy(buf.outside).cuda()
    for t in ts:
        t[o] = float("nan")
        t[-1] = float("inf")


SHAPES = [(8, 8), (64, 256), (72, 264), (200, 136), (1024, 8), (520, 520)]


@gpu
@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_gemm(lens, K, N, transposed, ints):
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer(LENS[lens])
    x, w = values((buf.P, K), 1, ints), values((buf.E, K, N) if transposed else (buf.E, N, K), 2, ints)
    poison_outside(buf, x)
    y, st = out((buf.P, N)), status()
    tdh.ep_expert_gemm(x, w, buf.cu, y, transpose_w=transposed, dev_status=st, **buf.kw)
    assert tdh.ep_status_read(st) == 0
    want, mag = product(buf, x, w, transposed)
    if ints:
        check(y, want.to(torch.bfloat16).double(), torch.zeros_like(want), buf, 7.0)
    check(y, want, rounded(sum_bound(K, mag), want, y.dtype), buf, 7.0)


@gpu
@pytest.mark.parametrize("lens", [[1] * 8, [0, 3, 0, 8, 1, 33, 0, 0, 2, 1, 0, 5], [64] + [0] * 9 + [65] + [0] * 9],
                         ids=str)
@pytest.mark.parametrize("K,N", [(8, 8), (72, 264), (200, 136), (1024, 128), (64, 392), (2048, 520)])
def test_gemm_of_few_rows_a_slot(lens, K, N):
    """The form for decoding: the average is what decides, and a slot may have more than it takes at a time."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer(lens, before=1, behind=2)
    assert buf.P <= 8 * buf.E
    for ints in (True, False):
        x, w = values((buf.P, K), 1, ints), values((buf.E, N, K), 2, ints)
        poison_outside(buf, x)
        y, st = out((buf.P, N)), status()
        tdh.ep_expert_gemm(x, w, buf.cu, y, dev_status=st, **buf.kw)
        want, mag = product(buf, x, w, False)
        if ints:
            check(y, want.to(torch.bfloat16).double(), torch.zeros_like(want), buf, 7.0)
        check(y, want, rounded(sum_bound(K, mag), want, y.dtype), buf, 7.0)
        if N % 16 == 0 and not ints:
            I = N // 2
            h, gu = out((buf.P, I)), out((buf.P, N))
            tdh.ep_expert_up(x, w, buf.cu, h, gu, dev_status=st, **buf.kw)
            check(gu, want, rounded(sum_bound(K, mag), want, gu.dtype), buf, 7.0)
            g, u = want[:, :I], want[:, I:]
            e = sum_bound(K, mag)
            act = silu(g) * u
            bound = (1.1 * e[:, :I] * (u.abs() + e[:, I:]) + (silu(g).abs() + 1.1 * e[:, :I]) * e[:, I:]
                     + act.abs() * (g.abs() + 16) * 2.0 ** -22)
            check(h, act, rounded(bound, act, h.dtype), buf, 7.0)
        assert tdh.ep_status_read(st) == 0


def silu(g):
    import torch
    return g * torch.sigmoid(g)


@gpu
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("H,I", [(8, 8), (64, 128), (72, 136), (200, 264), (1024, 8)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_up(lens, H, I, keep):
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer(LENS[lens])
    x, w = values((buf.P, H), 3), values((buf.E, 2 * I, H), 4, scale=2.0 / H ** 0.5)
    poison_outside(buf, x)
    h, st = out((buf.P, I)), status()
    gu = out((buf.P, 2 * I)) if keep else None
    tdh.ep_expert_up(x, w, buf.cu, h, gu, dev_status=st, **buf.kw)
    assert tdh.ep_status_read(st) == 0
    p, mag = product(buf, x, w, False)
    e = sum_bound(H, mag)
    if keep:
        check(gu, p, rounded(e, p, gu.dtype), buf, 7.0)
    g, u, eg, eu = p[:, :I], p[:, I:], e[:, :I], e[:, I:]
    # |silu'| < 1.1; the fast exponential's argument is off by |g| 2^-23, it and the quotient by a few units of 2^-22
    want = silu(g) * u
    bound = 1.1 * eg * (u.abs() + eu) + (silu(g).abs() + 1.1 * eg) * eu + want.abs() * (g.abs() + 16) * 2.0 ** -22
    check(h, want, rounded(bound, want, h.dtype), buf, 7.0)


@gpu
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("H,I", [(8, 8), (64, 256), (72, 264), (200, 136), (1024, 8)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_up_backward(lens, H, I, keep):
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer(LENS[lens])
    dy, w2, gu = values((buf.P, H), 5), values((buf.E, H, I), 6, scale=H ** -0.5), values((buf.P, 2 * I), 7, scale=3.0)
    poison_outside(buf, dy, gu)
    dgu, st = out((buf.P, 2 * I)), status()
    h = out((buf.P, I)) if keep else None
    tdh.ep_expert_up_backward(dy, w2, gu, buf.cu, dgu, h, dev_status=st, **buf.kw)
    assert tdh.ep_status_read(st) == 0
    dh, mag = product(buf, dy, w2, True)
    e = sum_bound(H, mag)
    gate = torch.nan_to_num(gu[:, :I].double(), posinf=0.0).requires_grad_(True)
    up = torch.nan_to_num(gu[:, I:].double(), posinf=0.0).requires_grad_(True)
    act = silu(gate) * up
    dg, du = torch.autograd.grad(act, (gate, up), dh)
    gate, up, act = gate.detach(), up.detach(), act.detach()
    sg = torch.sigmoid(gate)
    fast = (gate.abs() + 16) * 2.0 ** -22
    # dg = dh u (sg + g sg (1 - sg)): each part of the bracket is off by `fast` of its magnitude, 1 - sg by `fast` of 1
    part = sg + (gate * sg).abs() * (1 - sg + fast)
    bg = e * up.abs() * 1.1 + (dh.abs() + e) * up.abs() * (part * 3 * fast + (gate * sg).abs() * fast)
    bu = e * silu(gate).abs() + (dh.abs() + e) * silu(gate).abs() * 2 * fast
    want, bound = torch.cat([dg, du], 1), torch.cat([bg, bu], 1)
    check(dgu, want, rounded(bound, want, dgu.dtype), buf, 7.0)
    if keep:
        check(h, act, rounded(act.abs() * 2 * fast, act, h.dtype), buf, 7.0)


@gpu
@pytest.mark.parametrize("H,I", [(64, 256), (72, 264), (200, 136), (64, 8)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_up_backward_over_the_kept_products(lens, H, I):
    """dgu in the place of gu: bit for bit what it is in a place of its own."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer(LENS[lens])
    dy, w2, gu = values((buf.P, H), 5), values((buf.E, H, I), 6, scale=H ** -0.5), values((buf.P, 2 * I), 7, scale=3.0)
    dgu, h, own, kept = out((buf.P, 2 * I)), out((buf.P, I)), out((buf.P, I)), gu.clone()
    tdh.ep_expert_up_backward(dy, w2, gu, buf.cu, dgu, h, **buf.kw)
    tdh.ep_expert_up_backward(dy, w2, gu, buf.cu, gu, own, **buf.kw)
    inside = torch.from_numpy(~buf.outside).cuda()[:, None]
    assert torch.equal(gu, torch.where(inside, dgu, kept)) and torch.equal(own, h)


def wgrad_want(buf, a, b):
    import torch
    n = len(buf.lens)
    want, mag = (torch.zeros((n, a.shape[1], b.shape[1]), dtype=torch.float64, device="cuda") for _ in range(2))
    for s, _, r in buf.slots():
        want[s] = a[r].double().T @ b[r].double()
        mag[s] = a[r].double().abs().T @ b[r].double().abs()
    return want, mag


@gpu
@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rep_dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,N", [(8, 8), (128, 256), (136, 264), (72, 520), (520, 72)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_wgrad(lens, M, N, rep_dtype, accumulate, ints):
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer(LENS[lens])
    a, b = values((buf.P, M), 8, ints), values((buf.P, N), 9, ints)
    poison_outside(buf, a, b)
    # the gradient is a part of a longer row; one row more than there are slots stays as it is
    wide = out((buf.E + 1, M * N + 24), 3.0, torch.float32)
    rep = out((buf.reps + 2, M * N + 8), 3.0, getattr(torch, rep_dtype))
    home_v, rep_v = wide[:, 16:16 + M * N].view(-1, M, N), rep[:, 8:].view(-1, M, N)
    st = status()
    tdh.ep_expert_wgrad(a, b, buf.cu, home_v[:buf.E], rep_v, accumulate=accumulate, dev_status=st, **buf.kw)
    assert tdh.ep_status_read(st) == 0
    want, mag = wgrad_want(buf, a, b)
    if accumulate:
        want = want + 3.0
        mag = mag + 3.0
    longest = max(buf.lens)
    for got, w, m in ((home_v[:buf.E], want[:buf.E], mag[:buf.E]), (rep_v[:buf.reps], want[buf.E:], mag[buf.E:])):
        if ints:
            check(got, w.to(got.dtype).double(), torch.zeros_like(w))
        check(got, w, rounded(sum_bound(longest, m), w, got.dtype))
    assert torch.all(wide[buf.E] == 3.0) and torch.all(wide[:, :16] == 3.0) and torch.all(wide[:, 16 + M * N:] == 3.0)
    assert torch.all(rep[buf.reps:] == 3.0) and torch.all(rep[:, :8] == 3.0)


@gpu
@pytest.mark.parametrize("rep_dtype", ["float32", "bfloat16"])
def test_wgrad_added_to_the_home_rows_only(rep_dtype):
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer([40, 0, 129, 3, 70, 0])  # the last two are replicas
    a, b = values((buf.P, 136), 1, True), values((buf.P, 72), 2, True)
    home, rep = out((buf.E, 136, 72), 3.0, torch.float32), out((buf.reps, 136, 72), 3.0, getattr(torch, rep_dtype))
    tdh.ep_expert_wgrad(a, b, buf.cu, home, rep, accumulate="home", **buf.kw)
    want, _ = wgrad_want(buf, a, b)
    assert torch.equal(home.double(), want[:buf.E] + 3.0)
    assert torch.equal(rep, want[buf.E:].to(rep.dtype))


@gpu
def test_rows_of_other_slots_take_no_part():
    """An infinity or NaN in one slot's rows stays in that slot: in the products' rows and in the weight gradients,
    whose last block of rows reaches into the next slot's."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer([70, 3, 64, 10, 1], replicas=False)
    a, b, w = values((buf.P, 72), 1), values((buf.P, 136), 2), values((buf.E, 136, 72), 3)
    bad = [slice(buf.begin[s], buf.begin[s] + buf.lens[s]) for s in (1, 3)]
    a[bad[0]], b[bad[0]], a[bad[1]], b[bad[1]] = float("inf"), float("nan"), float("nan"), -float("inf")
    y, g = out((buf.P, 136)), out((buf.E, 72, 136), dtype=torch.float32)
    tdh.ep_expert_gemm(a, w, buf.cu, y, **buf.kw)
    tdh.ep_expert_wgrad(a, b, buf.cu, g, **buf.kw)
    want, mag = product(buf, torch.nan_to_num(a, 0.0, 0.0, 0.0), w, False)
    gwant, gmag = wgrad_want(buf, a, b)
    for s, e, r in buf.slots():
        if s in (1, 3):
            assert not torch.any(torch.isfinite(y[r])) and not torch.any(torch.isfinite(g[e]))
        else:
            check(y[r], want[r], rounded(sum_bound(72, mag[r]), want[r], y.dtype))
            check(g[e], gwant[s], rounded(sum_bound(70, gmag[s]), gwant[s], g.dtype))


@gpu
def test_the_weight_gradient_keeps_32_bits_over_long_slots():
    """One sign throughout, so that cut-off bits would add up: 60,000 rows into one slot."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    P = 60_000
    a = values((P, 64), 1).abs() + 0.5
    b = values((P, 64), 2).abs() + 0.5
    g = torch.empty((1, 64, 64), device="cuda")
    tdh.ep_expert_wgrad(a, b, torch.tensor([0, P], dtype=torch.int32, device="cuda"), g)
    want = a.double().T @ b.double()
    # partial sums of at most 1024 rows (64 additions of a cut-off each), then at most 60 rounded additions
    assert torch.all((g[0].double() - want).abs() <= (64 * 2.0 ** -23 + 60 * 2.0 ** -24) * want)


@gpu
def test_the_weight_gradient_sums_512_rows_at_a_time():
    """One sign throughout: the accumulator cuts off up to 4.5e-9 of a partial sum for each of its 512 rows; the eight
    partial sums are added with seven roundings, the j-th of a sum of j + 1 parts in 8 (half a unit, 2^-24, each)."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    P = 4096
    a, b = values((P, 64), 1).abs() + 0.5, values((P, 64), 2).abs() + 0.5
    g = torch.empty((1, 64, 64), device="cuda")
    tdh.ep_expert_wgrad(a, b, torch.tensor([0, P], dtype=torch.int32, device="cuda"), g)
    want = a.double().T @ b.double()
    assert torch.all((g[0].double() - want).abs() <= (512 * 4.5e-9 + 35 / 8 * 2.0 ** -24) * want)


@gpu
def test_slots_that_do_not_fit_are_left_out_and_flagged():
    import torch
    import token_dispatch_histogram_b200 as tdh
    P, K, N, E = 300, 64, 64, 4
    x, w = values((P, K), 1), values((E, N, K), 2)
    ok = torch.tensor([0, 50, 50, 200, 300], dtype=torch.int32, device="cuda")

    def run(cu, order=None, rep=None):
        y, st = out((P, N)), status()
        tdh.ep_expert_gemm(x, w, torch.as_tensor(cu, dtype=torch.int32, device="cuda"), y, dev_status=st,
                           slot_order=None if order is None else torch.tensor(order, dtype=torch.int32, device="cuda"),
                           rep_expert=None if rep is None else torch.tensor(rep, dtype=torch.int32, device="cuda"))
        g, gst = out((E, K, N), dtype=torch.float32), status()
        tdh.ep_expert_wgrad(x, y, torch.as_tensor(cu, dtype=torch.int32, device="cuda"), g, dev_status=gst,
                            slot_order=None if order is None else torch.tensor(order, dtype=torch.int32,
                                                                               device="cuda"))
        return y, tdh.ep_status_read(st), tdh.ep_status_read(gst)

    full, st, gst = run(ok)
    assert st == 0 and gst == 0 and not torch.any(torch.all(full == 7.0, 1))
    for cu, untouched, bits in (
            ([0, 50, 40, 200, 301], [(200, 300)], tdh.EP_DEV_BAD_ROW),     # descending, and past the buffer
            ([-1, 50, 50, 200, 300], [(0, 50)], tdh.EP_DEV_BAD_ROW),
            ([0, 50, 50, 1 << 30, 300], [(50, 300)], tdh.EP_DEV_BAD_ROW)):
        y, st, gst = run(cu)
        assert st == bits and gst == bits
        for b, e in untouched:
            assert torch.all(y[b:e] == 7.0)
    y, st, gst = run(ok, [0, 1, 4, -1])           # a replica, but no table of replicas
    assert st == tdh.EP_DEV_BAD_EXPERT_ID and gst == tdh.EP_DEV_BAD_EXPERT_ID
    assert torch.all(y[50:] == 7.0) and torch.equal(y[:50], full[:50])
    y, st, _ = run(ok, [0, 1, 4, 3], [4])         # a replica of no expert
    assert st == tdh.EP_DEV_BAD_EXPERT_ID and torch.all(y[50:200] == 7.0) and torch.equal(y[200:], full[200:])
    y, st, _ = run(ok, [0, 1, 5, 3], [2])         # past the table
    assert st == tdh.EP_DEV_BAD_EXPERT_ID and torch.all(y[50:200] == 7.0)
    y, st, _ = run(ok, [0, 1, 4, 3], [2])         # and a replica as it should be
    assert st == 0 and torch.equal(y, full)


@gpu
@pytest.mark.parametrize("n", [20, 600])
@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("hidden", [False, True])
def test_slots_that_overlap_are_left_out_and_flagged(hidden, few, n):
    """Behind an entry of cu_seqlens below the one before it (hidden: at an entry that is no slot) a slot may begin inside
    an earlier one: of rows that two slots claim, the first has them."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    K, N, E = 64, 136, n
    # slot 0 [0, 30), 1 goes back, 2 [10, 40) overlaps, 3 [40, 47) and the rest, one row each, do not
    cu = np.concatenate([[0, 30, 10, 40, 47], 47 + np.arange(1, n - 3)]).astype(np.int32)
    order = np.arange(n, dtype=np.int32)
    if hidden:
        order[1] = -1
    P = int(cu[-1]) + (0 if few else 8 * n)
    x, w, wt = values((P, K), 1, True), values((E, N, K), 2, True), values((E, K, N), 3, True)
    assert few == (P <= 8 * n)  # the form for few rows is chosen by the rows of the buffer
    to = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    owner = np.full(P, -1)
    for s in range(n):
        if s != 1 and s != 2:
            owner[cu[s]:cu[s + 1]] = s
    mine = to(owner)
    for t, weights in ((False, w), (True, wt)):
        y, st = out((P, N)), status()
        tdh.ep_expert_gemm(x, weights, to(cu), y, transpose_w=t, slot_order=to(order), dev_status=st)
        assert tdh.ep_status_read(st) == tdh.EP_DEV_BAD_ROW
        full = torch.einsum("pk,pnk->pn", x.double(), (weights.transpose(1, 2) if t else weights)[mine.clamp(min=0)]
                            .double())
        assert torch.equal(y, torch.where(mine[:, None] >= 0, full, 7.0).to(torch.bfloat16))
    b, g, st = values((P, 40), 4, True), out((E, K, 40), dtype=torch.float32), status()
    tdh.ep_expert_wgrad(x, b, to(cu), g, slot_order=to(order), dev_status=st)
    assert tdh.ep_status_read(st) == tdh.EP_DEV_BAD_ROW
    for s in [0, 2, 3, 4, n - 1]:
        r = slice(int(cu[s]), int(cu[s + 1]))
        assert torch.equal(g[s].double(), x[r].double().T @ b[r].double() if s != 2 else torch.full_like(g[s], 7.0).double())


@gpu
@pytest.mark.parametrize("n", [6, 700])
def test_an_id_at_two_slots_has_no_gradient_row(n):
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer([20, 0, 70, 3, 64, 1] + [1] * (n - 6), replicas=False)
    a, b = values((buf.P, 72), 1, True), values((buf.P, 40), 2, True)
    order = np.arange(n, dtype=np.int32)
    order[4] = 2
    g, st = out((n, 72, 40), dtype=torch.float32), status()
    tdh.ep_expert_wgrad(a, b, buf.cu[:n + 1], g, slot_order=torch.from_numpy(order).cuda(), dev_status=st)
    assert tdh.ep_status_read(st) == tdh.EP_DEV_BAD_EXPERT_ID
    want, _ = wgrad_want(buf, a, b)
    assert torch.all(g[[2, 4]] == 7.0)
    rest = [e for e in range(n) if e not in (2, 4)]
    check(g[rest], want[rest], torch.zeros_like(want[rest]))


@gpu
@pytest.mark.parametrize("n_slots", [40, 700])
def test_weight_gradients_of_the_largest_ids(n_slots):
    """1024 experts and as many replica rows as a call takes: ids up to 4094, some of them at two slots."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    E, cap, M, N = 1024, 3071, 8, 8
    lens = [int(v) for v in np.random.default_rng(n_slots).integers(0, 5, n_slots)]
    buf = Buffer(lens, replicas=False)
    a, b = values((buf.P, M), 1, True), values((buf.P, N), 2, True)
    # the highest ids, and as many below them as the slots of a call, in whole words of 32
    high = E + cap - 1 - np.arange(n_slots - n_slots // 2)
    order = np.concatenate([high[:n_slots // 2] - (cap + 31) // 32 * 32, high]).astype(np.int32)
    for twice in (False, True):
        if twice:
            order[3] = order[n_slots - 1]
        home, rep, st = out((E, M, N), dtype=torch.float32), out((cap, M, N), dtype=torch.float32), status()
        tdh.ep_expert_wgrad(a, b, buf.cu[:n_slots + 1], home, rep, slot_order=torch.from_numpy(order).cuda(),
                            dev_status=st)
        assert tdh.ep_status_read(st) == (tdh.EP_DEV_BAD_EXPERT_ID if twice else 0)
        want = torch.full((E + cap, M, N), 7.0, dtype=torch.float64, device="cuda")
        left_out = (3, n_slots - 1) if twice else ()
        grads, _ = wgrad_want(buf, a, b)
        for s in range(n_slots):
            if s not in left_out:
                want[order[s]] = grads[s]
        assert torch.equal(torch.cat([home, rep]).double(), want)


@gpu
def test_no_rows_and_no_slots():
    import torch
    import token_dispatch_histogram_b200 as tdh
    E, K, N = 3, 64, 72
    cu = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    none = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    tdh.ep_expert_gemm(none, values((E, N, K), 1), cu, torch.empty((0, N), dtype=torch.bfloat16, device="cuda"))
    g = out((E, K, N), dtype=torch.float32)
    tdh.ep_expert_wgrad(none, torch.empty((0, N), dtype=torch.bfloat16, device="cuda"), cu, g, accumulate=True)
    assert torch.all(g == 7.0)
    tdh.ep_expert_wgrad(none, torch.empty((0, N), dtype=torch.bfloat16, device="cuda"), cu, g)
    assert torch.all(g == 0.0)
    x, y = values((5, K), 2), out((5, N))
    tdh.ep_expert_gemm(x, values((E, N, K), 1), cu[:1], y)
    tdh.ep_expert_gemm(x, values((E, N, K), 1), cu, y)
    assert torch.all(y == 7.0)


@gpu
def test_many_slots_more_than_a_block_of_threads():
    """The largest table of slots: 1024 experts and 1023 replicas, most of them with a row or none."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    E, K, N = 1024, 64, 40
    rng = np.random.default_rng(0)
    lens = rng.choice([0, 0, 1, 2, 5], size=2 * E - 1)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    order = rng.permutation(2 * E - 1).astype(np.int32)
    rep = rng.integers(0, E, E - 1).astype(np.int32)
    P = int(cu[-1])
    x, w, y, st = values((P, K), 1), values((E, N, K), 2), out((P, N)), status()
    to = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    tdh.ep_expert_gemm(x, w, to(cu), y, slot_order=to(order), rep_expert=to(rep), dev_status=st)
    assert tdh.ep_status_read(st) == 0
    e = np.where(order < E, order, rep[np.maximum(order - E, 0)])
    of = to(np.repeat(e, lens))
    want = torch.einsum("pk,pnk->pn", x.double(), w[of].double())
    mag = torch.einsum("pk,pnk->pn", x.double().abs(), w[of].double().abs())
    check(y, want, rounded(sum_bound(K, mag), want, y.dtype))


@gpu
@pytest.mark.parametrize("n,M,N", [(40, 520, 520), (600, 72, 136), (513, 8, 264), (512, 264, 8)])
def test_weight_gradients_of_many_slots_of_unlike_length(n, M, N):
    """More tiles than are at work at once, from slots of 0 to 900 rows, below and above the table that is sorted."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    rng = np.random.default_rng(n)
    lens = np.minimum(900, rng.geometric(1 / 60, n)) * rng.integers(0, 2, n)
    lens[n // 2] = 900
    buf = Buffer([int(v) for v in lens], replicas=False)
    order = rng.permutation(n).astype(np.int32)
    a, b = values((buf.P, M), 1, True), values((buf.P, N), 2, True)
    poison_outside(buf, a, b)
    g, st = out((n, M, N), dtype=torch.float32), status()
    tdh.ep_expert_wgrad(a, b, buf.cu[:n + 1], g, slot_order=torch.from_numpy(order).cuda(), dev_status=st)
    assert tdh.ep_status_read(st) == 0
    want, _ = wgrad_want(buf, a, b)
    check(g[torch.from_numpy(order.astype(np.int64)).cuda()], want, torch.zeros_like(want))
    tdh.ep_expert_wgrad(a, b, buf.cu[:n + 1], g, slot_order=torch.from_numpy(order).cuda(), accumulate=True)
    check(g[torch.from_numpy(order.astype(np.int64)).cuda()], 2 * want, torch.zeros_like(want))


@gpu
def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31: the last slot's results, in every form."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    N, K, E = 8192, 64, 3
    P = (1 << 31) // N + 700
    cu = torch.tensor([0, P - 500, P - 130, P], dtype=torch.int32, device="cuda")
    x = torch.zeros((P, K), dtype=torch.bfloat16, device="cuda")
    x[P - 600:] = values((600, K), 1, True)
    w = values((E, N, K), 2, True)
    last = [slice(P - 500, P - 130), slice(P - 130, P)]

    def exact(got, a, b, e):
        want = a.double() @ b.double()
        assert torch.equal(got, want.to(torch.bfloat16)), e

    y = torch.empty((P, N), dtype=torch.bfloat16, device="cuda")
    tdh.ep_expert_gemm(x, w, cu, y)
    for e, r in enumerate(last, 1):
        exact(y[r], x[r], w[e].T, e)
    assert torch.all(y[:1000] == 0)
    back = torch.empty((P, K), dtype=torch.bfloat16, device="cuda")
    tdh.ep_expert_gemm(y, values((E, N, K), 3, True), cu, back, transpose_w=True)
    w3 = values((E, N, K), 3, True)
    for e, r in enumerate(last, 1):
        want, mag = y[r].double() @ w3[e].double(), y[r].double().abs() @ w3[e].double().abs()
        check(back[r], want, rounded(sum_bound(N, mag), want, back.dtype))
    h = torch.empty((P, N // 2), dtype=torch.bfloat16, device="cuda")
    gu = torch.empty((P, N), dtype=torch.bfloat16, device="cuda")
    tdh.ep_expert_up(x, w, cu, h, gu)
    assert torch.equal(gu[P - 500:], y[P - 500:])
    dgu = y.zero_()
    w2 = values((E, K, N // 2), 4, True)
    tdh.ep_expert_up_backward(x, w2, gu, cu, dgu, h)
    for e, r in enumerate(last, 1):
        dh = x[r].double() @ w2[e].double()
        g, u = gu[r].double().chunk(2, 1)
        act = silu(g) * u
        check(h[r], act, rounded(act.abs() * (g.abs() + 16) * 2.0 ** -21, act, h.dtype))
        du = dh * silu(g)
        check(dgu[r][:, N // 2:], du, rounded(du.abs() * (g.abs() + 16) * 2.0 ** -21, du, dgu.dtype))
    g = torch.empty((E, N, K), device="cuda")
    tdh.ep_expert_wgrad(gu, x, cu, g)
    for e, r in enumerate(last, 1):
        want, mag = gu[r].double().T @ x[r].double(), gu[r].double().abs().T @ x[r].double().abs()
        check(g[e], want, rounded(sum_bound(512, mag), want, g.dtype))


@gpu
def test_two_streams_and_a_replayed_graph_give_the_same_bits():
    import torch
    import token_dispatch_histogram_b200 as tdh
    buf = Buffer([300, 17, 0, 513, 128, 40])
    H, I = 256, 136
    x, w13 = values((buf.P, H), 1), values((buf.E, 2 * I, H), 2, scale=H ** -0.5)
    w2, dy = values((buf.E, H, I), 3, scale=I ** -0.5), values((buf.P, H), 4)
    names = dict(h=(buf.P, I), gu=(buf.P, 2 * I), y=(buf.P, H), dgu=(buf.P, 2 * I), h2=(buf.P, I), dx=(buf.P, H))

    def passes(o, stream=None):
        kw = dict(stream=stream, **buf.kw)
        tdh.ep_expert_up(x, w13, buf.cu, o["h"], o["gu"], **kw)
        tdh.ep_expert_gemm(o["h"], w2, buf.cu, o["y"], **kw)
        tdh.ep_expert_up_backward(dy, w2, o["gu"], buf.cu, o["dgu"], o["h2"], **kw)
        tdh.ep_expert_gemm(o["dgu"], w13, buf.cu, o["dx"], transpose_w=True, **kw)
        tdh.ep_expert_wgrad(dy, o["h2"], buf.cu, o["g2"], o["r2"], **kw)

    def outs():
        o = {k: out(s) for k, s in names.items()}
        o["g2"] = out((buf.E, H, I), dtype=torch.float32)
        o["r2"] = out((buf.reps, H, I), dtype=torch.float32)
        return o

    first = outs()
    passes(first)
    torch.cuda.synchronize()
    sides = [(torch.cuda.Stream(), outs()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o in sides:
            passes(o, s)
    torch.cuda.synchronize()
    graph, o = torch.cuda.CUDAGraph(), outs()
    with torch.cuda.graph(graph):
        passes(o)
    graph.replay()
    graph.replay()
    for other in (sides[0][1], sides[1][1], o):
        for k in first:
            assert torch.equal(first[k], other[k]), k


# ------------------------------------------------------------------ refusals (no GPU needed)

def test_expert_argument_errors():
    import token_dispatch_histogram_b200 as tdh
    L = tdh.lib()
    p, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)

    def gemm(x=p, rows=10, K=64, w=p, n_w=4, N=64, t=0, cu=p, n=4, order=None, rep=None, n_rep=0, y=p):
        return L.ep_expert_gemm(x, rows, K, w, n_w, N, t, cu, n, order, rep, n_rep, y, None, None)

    shapes = [dict(rows=-1), dict(rows=1 << 31), dict(n_w=0), dict(n_w=1025), dict(n=-1), dict(n=4000), dict(n_rep=-1),
              dict(cu=None)]
    for kw in shapes + [dict(K=0), dict(K=12), dict(N=4), dict(N=100), dict(x=None), dict(w=None), dict(y=None),
                        dict(x=odd), dict(w=odd), dict(y=odd), dict(K=1 << 29), dict(K=1 << 20, N=1 << 20)]:
        assert gemm(**kw) == tdh.EP_ERR_ARG, kw
        assert gemm(t=1, **kw) == tdh.EP_ERR_ARG, kw
    assert gemm(rows=0, x=None, y=None) == tdh.EP_OK
    assert gemm(n=0, cu=None) == tdh.EP_OK

    def up(x=p, rows=10, H=64, w=p, n_w=4, I=64, cu=p, n=4, n_rep=0, h=p, gu=p):
        return L.ep_expert_up(x, rows, H, w, n_w, I, cu, n, None, None, n_rep, h, gu, None, None)

    for kw in shapes + [dict(H=12), dict(I=12), dict(x=None), dict(w=None), dict(h=None), dict(gu=odd), dict(h=odd)]:
        assert up(**kw) == tdh.EP_ERR_ARG, kw
    assert up(rows=0, x=None, h=None, gu=None) == tdh.EP_OK

    def back(dy=p, rows=10, H=64, w=p, n_w=4, I=64, gu=p, cu=p, n=4, n_rep=0, dgu=p, h=p):
        return L.ep_expert_up_backward(dy, rows, H, w, n_w, I, gu, cu, n, None, None, n_rep, dgu, h, None, None)

    for kw in shapes + [dict(H=12), dict(I=12), dict(dy=None), dict(w=None), dict(gu=None), dict(dgu=None),
                        dict(h=odd), dict(dgu=odd), dict(gu=odd)]:
        assert back(**kw) == tdh.EP_ERR_ARG, kw

    def wg(a=p, b=p, rows=10, M=64, N=64, cu=p, n=4, g=p, n_w=4, ld=4096, rep=None, dt=0, n_rep=0, ldr=4096):
        return L.ep_expert_wgrad(a, b, rows, M, N, cu, n, None, g, n_w, ld, rep, dt, n_rep, ldr, 0, None, None)

    for kw in shapes + [dict(M=12), dict(N=12), dict(a=None), dict(b=odd), dict(g=None), dict(g=odd), dict(ld=4095),
                        dict(ld=4098), dict(rep=odd), dict(rep=p, ldr=4095), dict(rep=p, ldr=4100, dt=1), dict(dt=2)]:
        assert wg(**kw) == tdh.EP_ERR_ARG, kw
    assert wg(n=0, cu=None) == tdh.EP_OK


def test_expert_binding_refuses_wrong_tensors():
    import torch
    import token_dispatch_histogram_b200 as tdh
    bf = dict(dtype=torch.bfloat16)
    x, w, y = torch.zeros(4, 64, **bf), torch.zeros(2, 72, 64, **bf), torch.zeros(4, 72, **bf)
    cu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        tdh.ep_expert_gemm(x, w, cu, y)  # CPU tensors
    with pytest.raises(TypeError):
        tdh.ep_expert_gemm(x.float(), w, cu, y)
    with pytest.raises(ValueError):
        tdh.ep_expert_gemm(x, w, cu, y[:, :64])
    with pytest.raises(ValueError):
        tdh.ep_expert_gemm(x, w, cu, y, transpose_w=True)
    with pytest.raises(ValueError):
        tdh.ep_expert_up(x, w, cu, y)
    with pytest.raises(ValueError):
        tdh.ep_expert_up_backward(x, torch.zeros(2, 64, 72, **bf), torch.zeros(4, 72, **bf), cu,
                                  torch.zeros(4, 144, **bf))
    with pytest.raises(TypeError):
        tdh.ep_expert_wgrad(x, y, cu, torch.zeros(2, 64, 72, **bf))
    with pytest.raises(ValueError):
        tdh.ep_expert_wgrad(x, y, cu, torch.zeros(2, 72, 64))


def test_wgrad_refuses_another_word_for_accumulate():
    import torch
    import token_dispatch_histogram_b200 as tdh
    x, y = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 72, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="accumulate"):
        tdh.ep_expert_wgrad(x, y, torch.zeros(3, dtype=torch.int32), torch.zeros(2, 64, 72), accumulate="replicas")
