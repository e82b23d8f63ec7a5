"""The router and its gradient (-m gpu) against the definition in 64 bits: which
experts, in which order, and the weights within the bounds of their fp32 steps."""
import ctypes

import numpy as np
import pytest

gpu = pytest.mark.gpu


def ref_router(x, K, score, bias=None, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    """(ids, w) from the definition, token by token, in fp64.  x: fp64 logits."""
    T, E = x.shape
    ids, w = np.zeros((T, K), np.int32), np.zeros((T, K))
    length = E // n_group
    for t in range(T):
        s = ref_scores(x[t], score)
        key = x[t].copy() if bias is None else np.where(np.isinf(x[t]), -np.inf, s + bias)
        by = s if bias is None and n_group > 1 and group_top == 2 else key
        by = np.where(np.isinf(x[t]), -np.inf, by)
        groups = []
        for g in range(n_group):
            best = sorted((v for v in by[g * length:(g + 1) * length] if v != -np.inf), reverse=True)[:group_top]
            groups.append(sum(best) if best else -np.inf)
        kept = sorted(range(n_group), key=lambda g: (-groups[g], g))[:topk_group]
        order = sorted((e for e in range(E) if e // length in kept), key=lambda e: (-key[e], e))
        ids[t] = order[:K]
        c = s[ids[t]]
        if renorm:
            c = ref_ratio(x[t][ids[t]], score)
        w[t] = scale * c
    return ids, w


def ref_scores(x, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-x))
    m = x.max()
    if m == -np.inf:
        return np.zeros_like(x)
    e = np.exp(x - m)
    return e / e.sum()


def ref_ratio(x, score):
    if np.all(x == -np.inf):
        return np.zeros_like(x)
    # logs of the scores, so that scores far below the smallest double still have their ratio
    log = x if score == "softmax" else -np.logaddexp(0.0, -x)
    e = np.exp(log - log.max())
    return e / e.sum()


def w_bound(x, want, ids, scale):
    """|w - want| of the fp32 steps: exp(x - m) is off by |x - m| half-units (the rounded difference) and two units of
    its own; sum, quotient and scale add a few more; the smallest results are subnormal."""
    chosen = np.take_along_axis(x, ids.astype(np.int64), 1)
    top = np.max(x, 1, keepdims=True)
    far = np.where(np.isfinite(chosen) & np.isfinite(top), np.abs(chosen - top), 0.0)
    return (far + 16) * 2.0 ** -23 * np.abs(want) + abs(scale) * 2.0 ** -140


def logits_of(T, E, dtype, seed, spread=1.0, masked=0.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = spread * (torch.randn((T, E), generator=g) + torch.randn(E, generator=g))
    if masked:
        x[torch.rand((T, E), generator=g) < masked] = -float("inf")
        if T > 3:
            x[3] = -float("inf")      # a row whose mask leaves nothing
            x[2, :-1] = -float("inf")  # and one that it leaves one expert
    return x.to(dtype)


def call(x, K, dtype_w=None, **kw):
    import torch
    import token_dispatch_histogram_b200 as tdh
    T = x.shape[0]
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), 77.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    b = kw.pop("bias", None)
    tdh.ep_router(x, ids, w, bias=None if b is None else torch.from_numpy(b.astype(np.float32)).cuda(), dev_status=st,
                  **kw)
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64), tdh.ep_status_read(st)


CASES = [  # T, E, K, score, bias scale, n_group, topk_group, group_top, renorm, scale
    (1, 1, 1, "softmax", None, 1, 1, 1, True, 1.0),
    (1, 256, 8, "sigmoid", 0.1, 8, 4, 2, True, 2.5),
    (65, 64, 6, "softmax", None, 1, 1, 1, False, 1.0),
    (65, 64, 6, "softmax", None, 1, 1, 1, True, 1.0),
    (40, 384, 8, "sigmoid", 0.1, 1, 1, 1, True, 1.0),
    (33, 17, 17, "sigmoid", None, 1, 1, 1, False, 0.5),
    (33, 33, 32, "softmax", 0.01, 1, 1, 1, False, 1.0),
    (20, 1024, 8, "softmax", 0.01, 32, 5, 2, True, 1.0),
    (20, 1000, 7, "sigmoid", None, 8, 3, 2, True, 1.0),
    (20, 1000, 7, "softmax", None, 8, 3, 1, False, 1.0),
    (20, 160, 6, "softmax", None, 8, 3, 1, False, 16.0),
    (31, 16, 2, "softmax", None, 16, 2, 2, True, 1.0),
    (9, 72, 32, "sigmoid", 0.1, 2, 2, 1, True, 1.0),
    (9, 100, 3, "sigmoid", 1.0, 5, 1, 2, True, 1.0),
    (700, 128, 4, "softmax", None, 1, 1, 1, True, 1.0),
    (50, 40, 1, "sigmoid", 0.1, 1, 1, 1, True, 1.0),
]


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(str(v) for v in c))
def test_router_matches_the_definition(case, masked, dtype):
    import torch
    T, E, K, score, b, ng, tg, gt, renorm, scale = case
    x = logits_of(T, E, getattr(torch, dtype), T + E + K, masked=masked)
    bias = None if b is None else (b * np.random.default_rng(E).standard_normal(E)).astype(np.float32)
    kw = dict(score=score, n_group=ng, topk_group=tg, group_top=gt, renorm=renorm, scale=scale)
    ids, w, st = call(x.cuda(), K, bias=bias, **kw)
    x64 = x.double().numpy()
    want_ids, want = ref_router(x64, K, bias=None if bias is None else bias.astype(np.float64), **kw)
    assert st == 0
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= w_bound(x64, want, ids, scale))


MANY = [  # more tokens than there are warps at work: several to a warp
    (5003, 64, 6, "softmax", None, 1, 1, 1, False, 1.0),
    (5003, 40, 8, "sigmoid", 0.1, 1, 1, 1, True, 2.5),
    (4801, 96, 12, "sigmoid", 0.1, 4, 2, 2, True, 1.0),
    (4801, 33, 20, "softmax", 0.05, 1, 1, 1, True, 1.0),
    (4801, 32, 32, "sigmoid", None, 1, 1, 1, True, 1.0),
    (4801, 16, 16, "softmax", 0.1, 1, 1, 1, True, 1.0),
    (4802, 128, 8, "sigmoid", 0.1, 1, 1, 1, True, 1.0),
    (4803, 128, 5, "softmax", None, 1, 1, 1, False, 1.0),
    (4801, 100, 8, "softmax", 0.02, 1, 1, 1, True, 1.0),
    (4801, 65, 1, "sigmoid", None, 1, 1, 1, False, 1.0),
    (4801, 8, 8, "softmax", 0.1, 1, 1, 1, False, 1.0),
    (4801, 3, 2, "sigmoid", 0.1, 1, 1, 1, True, 1.0),
]


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "_".join(str(v) for v in c))
def test_many_tokens(case, masked, dtype):
    test_router_matches_the_definition(case, masked, dtype)


@gpu
def test_close_keys_among_many_tokens():
    """Tokens that fp32 cannot decide, next to others of the same warp that it can."""
    import torch
    T, E, K = 5001, 32, 4
    x = logits_of(T, E, torch.float32, 12)
    x[::3, 5] = x[::3, 9]
    close = np.nextafter(x[1::7, 3].numpy(), np.float32(np.inf))
    x[1::7, 4] = torch.from_numpy(close)
    x[::5, :6] += 3.0
    bias = np.zeros(E, np.float32)
    ids, w, st = call(x.cuda(), K, score="sigmoid", bias=bias)
    want_ids, want = ref_router(x.double().numpy(), K, "sigmoid", bias=bias.astype(np.float64))
    assert st == 0
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= w_bound(x.double().numpy(), want, ids, 1.0))


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
def test_experts_closer_than_32_bit_scores_tell_apart(score, groups, bias):
    """Neighbouring fp32 logits: the scores differ by less than an fp32 score's last place, and equal logits tie."""
    import torch
    T, E, K = 64, 64, 8
    rng = np.random.default_rng(5)
    base = rng.choice([0.5, 2.0, -3.0], size=(T, 1)).astype(np.float32)
    step = rng.choice([0, 1, 3, 9, 27], size=(T, E))  # no two different pairs have the same sum
    x = base.copy().repeat(E, 1)
    for i in range(27):
        x = np.where(step > i, np.nextafter(x, np.float32(np.inf)), x)
    b = None if bias is None else np.full(E, bias, np.float32)
    kw = dict(score=score, n_group=groups[0], topk_group=groups[1], group_top=groups[2])
    ids, w, st = call(torch.from_numpy(x).cuda(), K, bias=b, **kw)
    want_ids, want = ref_router(x.astype(np.float64), K, bias=None if b is None else b.astype(np.float64), **kw)
    assert st == 0
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= w_bound(x.astype(np.float64), want, ids, 1.0))


@gpu
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("E,K", [(64, 8), (100, 8), (128, 3), (200, 8)])
def test_ties_and_unusual_logits_of_many_tokens(E, K, score, bias):
    """Few different values, so that most choices are ties; masks, NaN and infinities among them."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    T = 4777
    rng = np.random.default_rng(E + K)
    x = rng.integers(-2, 3, (T, E)).astype(np.float32)
    x[rng.random((T, E)) < 0.2] = -np.inf
    x[5] = -np.inf
    b = np.zeros(E, np.float32) if bias else None
    kw = dict(score=score)
    ids, w, st = call(torch.from_numpy(x).cuda(), K, bias=b, **kw)
    b64 = None if b is None else b.astype(np.float64)
    want_ids, want = ref_router(x.astype(np.float64), K, bias=b64, **kw)
    assert st == 0
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= w_bound(x.astype(np.float64), want, ids, 1.0))
    x[7, 3], x[9, 1] = np.nan, np.inf
    ids, w, st = call(torch.from_numpy(x).cuda(), K, bias=b, **kw)
    assert st == tdh.EP_DEV_BAD_LOGIT
    y = np.nan_to_num(x, nan=-np.inf, posinf=np.finfo(np.float32).max, neginf=-np.inf)
    np.testing.assert_array_equal(ids, ref_router(y.astype(np.float64), K, bias=b64, **kw)[0])


@gpu
@pytest.mark.parametrize("T", [200, 4801])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_whose_large_biases_cancel(score, T):
    """Keys near 1000 and -999 whose sum is decided far below their own last place in 32 bits."""
    import torch
    E, K = 16, 2
    rng = np.random.default_rng(3)
    x = (rng.uniform(-1, 1, (T, 1)) + 2e-6 * rng.standard_normal((T, E))).astype(np.float32)
    bias = np.array([1000, -999] + [-2000] * 6 + [0.5, 0.5] + [-5] * 6, np.float32)
    kw = dict(score=score, n_group=2, topk_group=1, group_top=2)
    ids, w, st = call(torch.from_numpy(x).cuda(), K, bias=bias, **kw)
    want_ids, want = ref_router(x.astype(np.float64), K, bias=bias.astype(np.float64), **kw)
    assert st == 0
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= w_bound(x.astype(np.float64), want, ids, 1.0))


@gpu
@pytest.mark.parametrize("E,K", [(64, 8), (96, 32), (1024, 5)])
@pytest.mark.parametrize("what", ["equal", "lowest", "two values", "signed zeros"])
def test_ties_go_to_the_lower_index(E, K, what):
    import torch
    x = torch.zeros((5, E))
    if what == "lowest":
        x += torch.finfo(torch.float32).min
    if what == "two values":
        x[:, 1::2] = 1.0
    if what == "signed zeros":
        x[:, ::3] = -0.0
    ids, w, st = call(x.cuda(), K, score="softmax")
    want = np.arange(K) if what != "two values" else np.concatenate([np.arange(1, E, 2), np.arange(0, E, 2)])[:K]
    assert st == 0
    np.testing.assert_array_equal(ids, np.tile(want, (5, 1)))
    ones = np.array([1.0 if what != "two values" or e % 2 else np.exp(-1.0) for e in want])
    np.testing.assert_allclose(w, np.tile(ones / ones.sum(), (5, 1)), rtol=20 * 2.0 ** -23)


@gpu
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_far_logits_keep_their_ratios(score, renorm):
    import torch
    x = torch.tensor([[-300.0, -301.0, -302.5, -299.0], [300.0, 299.0, 250.0, -300.0], [-95.0, -96.0, -97.0, -120.0],
                      [torch.finfo(torch.float32).min] * 3 + [0.0], [88.0, 30.0, 17.0, 16.0]])
    ids, w, st = call(x.cuda(), 3, score=score, renorm=renorm)
    want_ids, want = ref_router(x.double().numpy(), 3, score, renorm=renorm)
    assert st == 0
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= w_bound(x.double().numpy(), want, ids, 1.0))


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("E", [64, 100, 256])
def test_many_rows_of_a_wider_matrix(E, dtype):
    """The forms for many tokens at any row stride and start, and the rows next to theirs left alone."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    T, K = 4801, 6
    wide = logits_of(T, E + 67, getattr(torch, dtype), 9).cuda()
    for off in (0, 1, 4):
        x = wide[:, off:off + E]
        ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T, K), 77.0, device="cuda")
        tdh.ep_router(x, ids, w, score="softmax", renorm=False)
        want_ids, want = ref_router(x.double().cpu().numpy(), K, "softmax", renorm=False)
        np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
        assert np.all(np.abs(w.cpu().numpy() - want) <= w_bound(x.double().cpu().numpy(), want, want_ids, 1.0))
        out = torch.full((T, E + 67), 5.0, dtype=wide.dtype, device="cuda")
        dw = torch.randn((T, K), device="cuda")
        tdh.ep_router_backward(dw, x, ids, out[:, off:off + E], score="softmax", renorm=False)
        want, mag = ref_backward(dw.double().cpu().numpy(), x.double().cpu().numpy(), want_ids, "softmax", False, 1.0)
        check_backward(out[:, off:off + E], want, mag, x)
        assert torch.all(out[:, :off] == 5.0) and torch.all(out[:, off + E:] == 5.0)


@gpu
@pytest.mark.parametrize("E", [96, 384])
def test_offsets_past_32_bits(E):
    import torch
    import token_dispatch_histogram_b200 as tdh
    T, K = (1 << 31) // E + 5000, 4
    x = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 1 << 22):
        x[i:i + (1 << 22)] = torch.randn((min(1 << 22, T - i), E), device="cuda", dtype=torch.bfloat16)
    ids, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")
    tdh.ep_router(x, ids, w)
    out = torch.empty_like(x)
    tdh.ep_router_backward(w, x, ids, out)
    for rows in (slice(0, 100), slice(T - 300, T)):
        x64 = x[rows].double().cpu().numpy()
        want_ids, want = ref_router(x64, K, "softmax")
        np.testing.assert_array_equal(ids[rows].cpu().numpy(), want_ids)
        assert np.all(np.abs(w[rows].cpu().numpy() - want) <= w_bound(x64, want, want_ids, 1.0))
        want, mag = ref_backward(w[rows].double().cpu().numpy(), x64, want_ids, "softmax", True, 1.0)
        check_backward(out[rows], want, mag, x[rows])


@gpu
def test_nan_and_infinite_logits_are_flagged_and_defined():
    import torch
    import token_dispatch_histogram_b200 as tdh
    x = logits_of(6, 20, torch.float32, 3)
    x[1, 4] = float("nan")
    x[2, 7] = float("inf")
    x[4] = float("nan")
    ids, w, st = call(x.cuda(), 4, score="softmax", renorm=False)
    assert st == tdh.EP_DEV_BAD_LOGIT
    y = torch.nan_to_num(x, nan=-float("inf"), posinf=torch.finfo(torch.float32).max, neginf=-float("inf"))
    want_ids, want = ref_router(y.double().numpy(), 4, "softmax", renorm=False)
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= w_bound(y.double().numpy(), want, ids, 1.0))
    assert ids[2, 0] == 7 and w[2, 0] == 1.0 and list(ids[4]) == [0, 1, 2, 3] and np.all(w[4] == 0)


@gpu
@pytest.mark.parametrize("E", [20, 64, 1000])
@pytest.mark.parametrize("groups", [(1, 1, 1), (4, 2, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_are_not_finite_exclude_or_prefer(score, groups, E):
    """-inf and NaN exclude their experts (taken last, by index), +inf puts its expert first."""
    import torch
    T, K = 40, 8
    x = logits_of(T, E, torch.float32, 6)
    bias = (0.1 * np.random.default_rng(1).standard_normal(E)).astype(np.float32)
    bias[[1, 7]], bias[[2, 11]], bias[5] = -np.inf, np.nan, np.inf
    kw = dict(score=score, n_group=groups[0], topk_group=groups[1], group_top=groups[2])
    ids, w, st = call(x.cuda(), K, bias=bias, **kw)
    want_ids, want = ref_router(x.double().numpy(), K, bias=np.where(np.isnan(bias), -np.inf, bias).astype(np.float64), **kw)
    assert st == 0 and np.all(ids[:, 0] == 5)
    if E > 20 or groups[0] == 1:  # two groups of five experts are too few without those excluded
        assert not np.any(np.isin(ids, [1, 2, 7, 11]))
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= w_bound(x.double().numpy(), want, ids, 1.0))
    if groups[0] == 1:
        bias[:] = np.nan  # nothing left to prefer: by index
        ids, w, st = call(x.cuda(), K, bias=bias, **kw)
        np.testing.assert_array_equal(ids, np.tile(np.arange(K), (T, 1)))
        assert np.all(np.isfinite(w))


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_rows_of_a_wider_matrix(dtype):
    """Any row stride and any start: the logits as columns of a wider projection, outputs into slices."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    T, E, K = 50, 64, 6
    wide = logits_of(T, 131, getattr(torch, dtype), 9).cuda()
    for off in (0, 1, 3, 64):
        x = wide[:, off:off + E]
        ids = torch.full((T + 2, K), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T + 2, K), 77.0, device="cuda")
        tdh.ep_router(x, ids[1:T + 1], w[1:T + 1], score="sigmoid")
        want_ids, want = ref_router(x.double().cpu().numpy(), K, "sigmoid")
        np.testing.assert_array_equal(ids[1:T + 1].cpu().numpy(), want_ids)
        assert np.all(np.abs(w[1:T + 1].cpu().numpy() - want) <= w_bound(x.double().cpu().numpy(), want, want_ids, 1.0))
        assert torch.all(ids[[0, T + 1]] == -7) and torch.all(w[[0, T + 1]] == 77.0)
        out = torch.full((T, 131), 5.0, dtype=wide.dtype, device="cuda")
        dw = torch.randn((T, K), device="cuda")
        tdh.ep_router_backward(dw, x, ids[1:T + 1], out[:, off:off + E], score="softmax", renorm=False)
        want, mag = ref_backward(dw.double().cpu().numpy(), x.double().cpu().numpy(), want_ids, "softmax", False, 1.0)
        check_backward(out[:, off:off + E], want, mag, x)
        assert torch.all(out[:, :off] == 5.0) and torch.all(out[:, off + E:] == 5.0)


# ------------------------------------------------------------------ backward

def ref_backward(dw, x, ids, score, renorm, scale):
    """(dlogits, sum of the magnitudes of its terms) from the Jacobian of the definition, in fp64."""
    T, E = x.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ok = (ids[t] >= 0) & (ids[t] < E)
        j, d = ids[t][ok], scale * dw[t][ok]
        s = ref_scores(x[t], score)
        if renorm:
            r = ref_ratio(x[t][j], score)
            slope = 1 - s[j] if score == "sigmoid" else 1.0
            inner, absinner = (d * r).sum(), np.abs(d * r).sum()
            np.add.at(out[t], j, r * slope * (d - inner))
            np.add.at(mag[t], j, r * slope * (np.abs(d) + absinner))
        elif score == "sigmoid":
            np.add.at(out[t], j, d * s[j] * (1 - s[j]))
            np.add.at(mag[t], j, np.abs(d) * s[j] * (1 - s[j]))
        else:
            out[t] -= s * (d * s[j]).sum()
            mag[t] += s * np.abs(d * s[j]).sum()
            np.add.at(out[t], j, d * s[j])
            np.add.at(mag[t], j, np.abs(d) * s[j])
    return out, mag


def check_backward(got, want, mag, x):
    """fp32 steps: each term within (range + 32) units of 2^-23 of its magnitude (exp of rounded differences, sums over
    at most 1024 scores by 32 lanes); then one rounding to the output's type."""
    import torch
    xs = x.double().cpu().numpy()
    fin = np.where(np.isfinite(xs), xs, 0.0)
    far = min(120.0, float(fin.max() - fin.min())) if fin.size else 0.0
    half, tiny = torch.finfo(got.dtype).eps / 2, torch.finfo(got.dtype).smallest_normal
    if got.dtype == torch.float16:
        tiny *= 2.0 ** -10  # its subnormals
    bound = (far + 32) * 2.0 ** -23 * mag
    bound = bound + (np.abs(want) + bound) * half + tiny
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound)


@gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (65, 64, 6), (33, 17, 17), (9, 1024, 32), (200, 384, 8),
                                   (21, 100, 5), (5003, 64, 6), (4801, 45, 12), (4801, 300, 20), (4802, 128, 8), (4803, 99, 3),
                                   (4801, 5, 5), (4803, 300, 4)])
def test_backward_matches_the_jacobian(T, E, K, score, renorm, masked, dtype):
    import torch
    import token_dispatch_histogram_b200 as tdh
    x = logits_of(T, E, getattr(torch, dtype), T + E, spread=2.0, masked=masked)
    ids, _, _ = call(x.cuda(), K, score=score)
    dw = torch.randn((T, K), generator=torch.Generator().manual_seed(K))
    out = torch.full((T, E), float("nan"), dtype=x.dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tdh.ep_router_backward(dw.cuda(), x.cuda(), torch.from_numpy(ids).cuda(), out, score=score, renorm=renorm, scale=1.5,
                           dev_status=st)
    assert tdh.ep_status_read(st) == 0
    want, mag = ref_backward(dw.double().numpy(), x.double().numpy(), ids, score, renorm, 1.5)
    check_backward(out, want, mag, x)


@gpu
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_backward_matches_differences_of_the_forward(score, renorm):
    """Central differences of the definition (fp64 on the host) at the experts that were chosen."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    T, E, K = 6, 24, 4
    x = logits_of(T, E, torch.float32, 4)
    ids, _, _ = call(x.cuda(), K, score=score)
    dw = np.random.default_rng(2).standard_normal((T, K)).astype(np.float32)
    out = torch.empty((T, E), device="cuda")
    tdh.ep_router_backward(torch.from_numpy(dw).cuda(), x.cuda(), torch.from_numpy(ids).cuda(), out, score=score,
                           renorm=renorm)

    def loss(v):
        w = np.array([ref_ratio(v[t][ids[t]], score) if renorm else ref_scores(v[t], score)[ids[t]] for t in range(T)])
        return (w * dw).sum(1)

    x64, eps = x.double().numpy(), 1e-5
    for e in range(E):
        hi, lo = x64.copy(), x64.copy()
        hi[:, e] += eps
        lo[:, e] -= eps
        # the difference quotient is off by eps^2 times a third derivative below 1
        np.testing.assert_allclose(out[:, e].cpu().numpy(), (loss(hi) - loss(lo)) / (2 * eps), atol=2e-6)


@gpu
@pytest.mark.parametrize("T,E", [(4, 12), (4904, 12), (4904, 120), (4904, 130)])
def test_backward_of_repeated_and_bad_ids(T, E):
    import torch
    import token_dispatch_histogram_b200 as tdh
    K = 5
    x = logits_of(T, E, torch.float32, 8)
    ids = np.array([[3, 3, 3, 1, 0], [2, 5, 2, 5, 2], [0, E, -1, 4, 7], [-1, -1, 999, -5, 1 << 30]], np.int32)
    ids = np.tile(ids, (T // 4, 1))
    dw = torch.randn((T, K), generator=torch.Generator().manual_seed(1))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            out = torch.full((T, E), float("nan"), device="cuda")
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            tdh.ep_router_backward(dw.cuda(), x.cuda(), torch.from_numpy(ids).cuda(), out, score=score, renorm=renorm,
                                   dev_status=st)
            assert tdh.ep_status_read(st) == tdh.EP_DEV_BAD_EXPERT_ID
            want, mag = ref_backward(dw.double().numpy(), x.double().numpy(), ids, score, renorm, 1.0)
            check_backward(out, want, mag, x)


@gpu
def test_zero_tokens_and_another_stream_and_a_graph():
    import torch
    import token_dispatch_histogram_b200 as tdh
    e = torch.empty((0, 64), device="cuda")
    tdh.ep_router(e, torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda"))
    tdh.ep_router_backward(torch.empty((0, 4), device="cuda"), e, torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                           torch.empty((0, 64), device="cuda"))
    T, E, K = 300, 64, 6
    x = logits_of(T, E, torch.float32, 1).cuda()
    ids = torch.zeros((T, K), dtype=torch.int32, device="cuda")
    w = torch.zeros((T, K), device="cuda")
    dx = torch.zeros((T, E), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tdh.ep_router(x, ids, w, score="sigmoid", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    first = (ids.clone(), w.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tdh.ep_router(x, ids, w, score="sigmoid")
        tdh.ep_router_backward(w, x, ids, dx, score="sigmoid")
    x.copy_(logits_of(T, E, torch.float32, 2))
    graph.replay()
    want_ids, want = ref_router(x.double().cpu().numpy(), K, "sigmoid")
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    assert not torch.equal(ids, first[0])
    d, mag = ref_backward(w.double().cpu().numpy(), x.double().cpu().numpy(), want_ids, "sigmoid", True, 1.0)
    check_backward(dx, d, mag, x)


@gpu
@pytest.mark.parametrize("T,dtype", [(40, "float32"), (40, "float16"), (4801, "bfloat16")])
@pytest.mark.parametrize("E,K,n_group,topk_group,group_top", [
    (64, 6, 1, 1, 1), (128, 8, 1, 1, 1), (200, 12, 1, 1, 1), (256, 8, 1, 1, 1), (384, 1, 1, 1, 1), (1000, 8, 1, 1, 1),
    (64, 2, 8, 3, 1), (256, 8, 8, 4, 2), (320, 8, 8, 4, 1)])
def test_zeros_of_either_sign_are_equal(E, K, n_group, topk_group, group_top, T, dtype):
    """Rows led by a few zeros of mixed signs above distinct negative logits: equal keys, so in the order of their ids,
    whether they lead or stand at the K-th place."""
    import torch
    rng = np.random.default_rng(E + K)
    lower = -1.0 - np.arange(E) / 128  # distinct, 16-bit types too, down to -8.8
    if dtype != "float32":
        lower = -2.0 ** (np.arange(E) // 64 % 10) * (1 + np.arange(E) % 64 / 64)
    x = np.stack([rng.permutation(lower) for _ in range(T)])
    for t in range(T):
        at = rng.choice(E, min(E, 1 + t % (K + 2)), replace=False)
        x[t, at] = np.where(rng.random(len(at)) < 0.5, 0.0, -0.0)
    kw = dict(score="softmax", n_group=n_group, topk_group=topk_group, group_top=group_top)
    xd = torch.from_numpy(x).to(getattr(torch, dtype))
    ids, w, st = call(xd.cuda(), K, **kw)
    want_ids, want = ref_router(xd.double().numpy(), K, **kw)
    assert st == 0
    np.testing.assert_array_equal(ids, want_ids)
    assert np.all(np.abs(w - want) <= w_bound(xd.double().numpy(), want, ids, 1.0))


@gpu
@pytest.mark.parametrize("kind", ["logits", "bias", "infinite"])
def test_a_group_that_is_left_out_costs_nothing(kind):
    """One group without an expert to take (its logits masked, or its biases -inf), or with a key of +inf, does not send
    every token through fp64, which takes many times as long: the time stays near that of the batch without it."""
    import torch
    import token_dispatch_histogram_b200 as tdh
    T, E, K = 65536, 256, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((T, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    x2, bias2 = x.clone(), bias.clone()
    if kind == "logits":
        x2[:, 32:64] = -float("inf")
    elif kind == "bias":
        bias2[32:64] = -float("inf")
    else:
        bias2[40] = float("inf")
    ids, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")

    def best(x, b):
        times = []
        for _ in range(8):
            a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                tdh.ep_router(x, ids, w, score="sigmoid", bias=b, n_group=8, topk_group=4, group_top=2)
            z.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(z))
        return min(times)

    plain, other = best(x, bias), best(x2, bias2)
    assert other <= 2 * plain


@gpu
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_of_infinite_keys(score, group_top):
    """Groups masked by logits or by biases, with infinite biases, and with finite biases whose sum is too large for fp32:
    the order is that of the definition."""
    import torch
    T, E, K, n_group = 60, 128, 6, 8
    x = logits_of(T, E, torch.float32, 5)
    rng = np.random.default_rng(6)
    top = float(np.finfo(np.float32).max)
    for kind in range(6):
        bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
        y = x.clone()
        if kind in (0, 5):
            y[:, 16:32] = -float("inf")
        if kind in (1, 5):
            bias[32:48] = -np.inf
        if kind in (2, 5):
            bias[[50, 70]] = np.inf
        if kind in (3, 5):
            bias[[80, 81, 96, 97]] = top * np.array([0.8, 0.8, 0.9, 0.9])
        if kind in (4, 5):
            bias[112:128] = -top
            bias[2:4] = -top
        for topk_group in (2, 5, 7):
            kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
            ids, w, st = call(y.cuda(), K, bias=bias, **kw)
            with np.errstate(over="ignore"):
                want_ids, want = ref_router(y.double().numpy(), K, bias=bias.astype(np.float64), **kw)
            np.testing.assert_array_equal(ids, want_ids)


@gpu
@pytest.mark.parametrize("T,E", [(64, 384), (4864, 384), (64, 1024), (4864, 96)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_expert_of_low_bias_and_high_score_at_the_border(score, T, E):
    """The last chosen expert and the next ones are held up by their biases, and behind them stands one of a score near
    1 and a low bias, whose key passes theirs, or does not, by less than its score's error in fp32."""
    import torch
    K = 8
    rng = np.random.default_rng(E)
    x = 0.1 * rng.standard_normal(E)
    x[7] = 9.0 if score == "softmax" else 4.0
    x = x.astype(np.float32)
    s = ref_scores(x.astype(np.float64), score)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    key = np.sort(np.delete(s + bias, 7))[::-1]
    # keys within a few 1e-8 around the border
    at = np.argsort(-np.where(np.arange(E) == 7, -9.0, s + bias))[K - 1:K + 2]
    bias[at] = (key[K - 1] - s[at] + np.array([0.0, -3e-8, -6e-8])).astype(np.float32)
    bias[7] = np.float32(key[K - 1] - s[7])
    rows = np.repeat(x[None], T, 0)
    rows[:, 7] += (np.arange(T) % 16 - 8) * np.float32(2.0 ** -19)  # a few units of the last place
    kw = dict(score=score)
    ids, w, st = call(torch.from_numpy(rows).cuda(), K, bias=bias, **kw)
    want_ids, want = ref_router(rows[:16].astype(np.float64), K, bias=bias.astype(np.float64), **kw)
    assert len({tuple(r) for r in want_ids}) > 1  # 7 among them or not
    np.testing.assert_array_equal(ids, np.tile(want_ids, (T // 16, 1)))


# ------------------------------------------------------------------ refusals (no GPU needed)

def test_router_argument_errors():
    import token_dispatch_histogram_b200 as tdh
    L = tdh.lib()
    fake, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001)

    def fwd(logits=fake, dtype=0, T=4, E=16, ld=16, K=2, score=0, bias=None, ng=1, tg=1, gt=1, scale=1.0, ids=fake,
            w=fake):
        return L.ep_router(logits, dtype, T, E, ld, K, score, bias, ng, tg, gt, 1, scale, ids, w, None, None)

    bad = [dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(E=0), dict(E=1025, ld=1025), dict(ld=15), dict(K=0),
           dict(K=17), dict(E=64, ld=64, K=33), dict(score=2), dict(ng=0), dict(ng=3), dict(E=33, ld=33, ng=33, tg=33),
           dict(ng=4, tg=0), dict(ng=4, tg=5), dict(ng=16, tg=1), dict(gt=0), dict(gt=3), dict(scale=float("nan")),
           dict(scale=float("inf")), dict(logits=None), dict(ids=None), dict(w=None), dict(logits=odd), dict(ids=odd),
           dict(w=odd), dict(bias=odd), dict(T=1 << 31, K=2)]
    for kw in bad:
        assert fwd(**kw) == tdh.EP_ERR_ARG, kw
    assert fwd(T=0, logits=None, ids=None, w=None) == tdh.EP_OK

    def bwd(dw=fake, logits=fake, dtype=0, T=4, E=16, ld=16, ids=fake, K=2, score=0, scale=1.0, out=fake, ldo=16):
        return L.ep_router_backward(dw, logits, dtype, T, E, ld, ids, K, score, 1, scale, out, ldo, None, None)

    for kw in [dict(dtype=3), dict(T=-1), dict(ld=15), dict(ldo=15), dict(K=17), dict(score=5), dict(dw=None),
               dict(ids=None), dict(out=None), dict(logits=None), dict(out=odd), dict(dw=odd), dict(scale=float("nan"))]:
        assert bwd(**kw) == tdh.EP_ERR_ARG, kw
    assert bwd(T=0, dw=None, logits=None, ids=None, out=None) == tdh.EP_OK


def test_router_binding_refuses_wrong_tensors():
    import torch
    import token_dispatch_histogram_b200 as tdh
    x, ids, w = torch.zeros(4, 16), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        tdh.ep_router(x, ids, w)  # CPU tensors
    with pytest.raises(TypeError):
        tdh.ep_router(x.double(), ids, w)
    with pytest.raises(TypeError):
        tdh.ep_router(x, ids.long(), w)
    with pytest.raises(TypeError):
        tdh.ep_router(x, ids, w.half())
    with pytest.raises(ValueError):
        tdh.ep_router(x, ids, w, score="tanh")
    with pytest.raises(ValueError):
        tdh.ep_router(x.T, ids, w)


@gpu
def test_router_binding_refuses_wrong_shapes():
    import torch
    import token_dispatch_histogram_b200 as tdh
    x = torch.zeros((4, 16), device="cuda")
    ids, w = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    with pytest.raises(ValueError):
        tdh.ep_router(x, ids[:3], w)
    with pytest.raises(ValueError):
        tdh.ep_router(x, ids, w[:, :1])
    with pytest.raises(ValueError):
        tdh.ep_router(x, ids, w, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(tdh.EpError):
        tdh.ep_router(x[:1].expand(4, 16), ids, w)  # rows on top of each other
    with pytest.raises(tdh.EpError):
        tdh.ep_router(x, ids, w, n_group=3, topk_group=1)
    with pytest.raises(TypeError):
        tdh.ep_router_backward(w, x, ids, torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda"))
