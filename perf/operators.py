"""Cases, plain forms and 64-bit definitions of the operators around the dispatch path: the router in front of it, the
experts' products between dispatch and combine, and the optimizer step behind the gradient reduction.

Each case is one call:

  router           logits [T, E] -> the K experts of each token and their gate weights
  router_backward  dw [T, K] -> dlogits [T, E]
  up               rows [P, H] grouped by expert -> silu(x Wg^T) * (x Wu^T), and with `save` the products before it
  down             rows [P, I] grouped by expert -> x W^T
  dgrad            rows [P, 2I] grouped by expert -> x W, W as the forward holds it
  up_backward      dy [P, H], and up's saved products -> their gradients, and the activation again
  wgrad            a [P, M], b [P, N] grouped by expert -> a_s^T b_s for each slot s
  adamw            one step over many tensors at once, moments in 32 or in 8 bits

The sizes are those of this repository's workloads: the moderate eight-rank layer (32,768 tokens, 64 experts, K = 6,
H = 2048, I = 1024), one rank of the DeepSeek-V3-shaped layer (8 home experts and the replicas it received, 32,768 rows,
H = 7168, I = 2048) and the fine-grained layer (524,288 tokens, 384 experts, K = 8).
"""
import math

import torch

own = False

BLOCK = 256     # elements that share a scale where the moments are held in 8 bits
FP8_MAX = 448.0
FP8_MIN = 2.0 ** -9
TINY = 2.0 ** -100  # a block with nothing above it is held as zeros

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # serving: one decoded token through a router with a balance bias and expert groups (launch latency)
        dict(name="router 1 token", op="router", T=1, E=256, K=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renorm=True, scale=2.5, dtype="f32"),
        # training: the fine-grained layer's whole batch, sigmoid scores with a balance bias
        dict(name="router 524288 tokens", op="router", T=524288, E=384, K=8, score="sigmoid", bias=True, n_group=1,
             topk_group=1, group_top=1, renorm=True, scale=1.0, dtype="f32"),
        # training: the moderate layer, softmax over all experts (a dense gradient), logits in 16 bits
        dict(name="router backward 32768", op="router_backward", T=32768, E=64, K=6, score="softmax", renorm=False,
             scale=1.0, dtype="bf16"),
        # training: the fine-grained layer's gradient (zero but at the chosen experts)
        dict(name="router backward 524288", op="router_backward", T=524288, E=384, K=8, score="sigmoid", renorm=True,
             scale=1.0, dtype="f32"),
        # serving: 32 decoded tokens over 64 experts, three rows an expert (bound by the weights' bytes)
        dict(name="up decode", op="up", P=192, H=2048, I=1024, G=64, reps=0, save=False, spread=0.5),
        # training: the moderate layer's first two projections
        dict(name="up 196608 rows", op="up", P=196608, H=2048, I=1024, G=64, reps=0, save=True, spread=0.5),
        # serving's prefill and training: one rank's second projection, with replicas of hot experts
        dict(name="down one rank", op="down", P=32768, H=7168, I=2048, G=8, reps=5, spread=0.5),
        # training: the gradient that goes back into dispatch, on an odd, ragged rank
        dict(name="dgrad odd rank", op="dgrad", P=20011, H=2048, I=1000, G=33, reps=7, spread=1.0),
        # training: one rank's gradient through the second projection and the activation
        dict(name="up backward one rank", op="up_backward", P=32768, H=7168, I=2048, G=8, reps=5, spread=0.5),
        # training: the weight gradients of the moderate layer's second projection, for the replica reduction
        dict(name="wgrad 196608 rows", op="wgrad", P=196608, M=2048, N=1024, G=64, reps=0, spread=0.5),
        # training: a model's smaller tensors (norms, routers, biases among them), of every size
        dict(name="adamw 300 tensors", op="adamw", tensors=300, total=100_000_000, bits=32, copy=False),
        # training: one rank's expert weights with moments in 8 bits and the bf16 weights that the products read
        dict(name="adamw 8 bits one rank", op="adamw", tensors=16, total=352_321_536, bits=8, copy=True),
    ]


def draw(rng):
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["router", "router_backward", "up", "down", "dgrad", "up_backward", "wgrad", "adamw"])
    if op in ("router", "router_backward"):
        n_group = rng.choice([1, 1, 4, 8])
        E = n_group * span(max(1, 16 // n_group), 384 // n_group)
        K = rng.randint(1, 8)
        topk_group = rng.randint(min(n_group, -(-K * n_group // E)), n_group)
        c = dict(op=op, T=span(1, 262144), E=E, K=K, score=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "f32", "bf16", "f16"]))
        if op == "router":
            c.update(bias=rng.random() < 0.5, n_group=n_group, topk_group=topk_group,
                     group_top=rng.choice([1, 2]) if E >= 2 * n_group else 1)
        return c
    if op == "adamw":
        return dict(op=op, tensors=span(1, 300), total=span(10_000, 200_000_000), bits=rng.choice([32, 8]),
                    copy=rng.random() < 0.5)
    P = span(1, 40_000)
    H, I = 8 * span(16, 512), 8 * span(16, 256)
    G = span(1, 64)
    reps = rng.choice([0, 0, 3, 6])
    c = dict(op=op, P=P, G=G, reps=reps, spread=rng.choice([0.2, 0.5, 1.0]))
    if op == "wgrad":
        return dict(c, M=H, N=I)
    return dict(c, H=H, I=I, **({"save": rng.random() < 0.5} if op == "up" else {}))


# ------------------------------------------------------------------ inputs

def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(int(seed))


def _normal(g, shape, dtype=torch.bfloat16, scale=1.0):
    """Normal values; large ones slice by slice, so that no fp32 copy of the whole is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(scale))
    return out


def _sizes(case, seed):
    """Rows of each slot: multinomial over lognormal weights, as a router with a bias per expert gives; they sum to P."""
    g = _gen(seed + 77, "cpu")
    n = case["G"] + case["reps"]
    p = torch.softmax(case["spread"] * torch.randn(n, generator=g, dtype=torch.float64), 0)
    u = torch.rand(case["P"], generator=g, dtype=torch.float64)
    return torch.bincount(torch.bucketize(u, torch.cumsum(p, 0)).clamp_(max=n - 1), minlength=n)


def _slots(case, seed):
    """The slots of a rank's buffer: its home experts, then the replicas it received, as a replica plan gives them."""
    n = _sizes(case, seed)
    cu = torch.zeros(len(n) + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(n, 0)
    rep = torch.randint(0, case["G"], (max(1, case["reps"]),), generator=_gen(seed + 78, "cpu"))
    weight = torch.cat([torch.arange(case["G"]), rep[:case["reps"]]])
    return dict(cu=cu.to(torch.int32).cuda(), slots=torch.arange(len(n), dtype=torch.int32, device="cuda"),
                rep=rep.to(torch.int32).cuda(), weight=weight.cuda(), longest=int(n.max()), sizes=n.tolist(),
                where=weight.tolist())


def _tensor_sizes(case, seed):
    """Element counts of the tensors: spread over their logarithm (a norm's weight to an expert's), they sum to total.
    Equal ones where there are few (a rank's expert weights)."""
    k, total = case["tensors"], case["total"]
    if k <= 16:
        n = [total // k] * k
    else:
        u = torch.exp(3.0 * torch.rand(k, generator=_gen(seed + 79, "cpu"), dtype=torch.float64) * math.log(10))
        n = [max(1, int(x)) for x in u / u.sum() * total]
    return n


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=dict(case))
    if op in ("router", "router_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        skew = torch.randn(E, generator=g, device="cuda")
        logits = torch.randn((T, E), generator=g, device="cuda").add_(skew).to(DTYPES[case["dtype"]])
        s.update(logits=logits)
        if op == "router":
            s.update(bias=torch.randn(E, generator=g, device="cuda").mul_(0.1) if case["bias"] else None,
                     ids=torch.empty((T, K), dtype=torch.int32, device="cuda"),
                     w=torch.empty((T, K), dtype=torch.float32, device="cuda"))
        else:
            ids = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :K].to(torch.int32)
            s.update(ids=ids.contiguous(), dw=torch.randn((T, K), generator=g, device="cuda"),
                     dlogits=torch.empty_like(logits))
        return s
    if op == "adamw":
        n = _tensor_sizes(case, seed)
        pad = [-(-x // BLOCK) * BLOCK for x in n]
        at = [0]
        for x in pad:
            at.append(at[-1] + x)
        mine = torch.zeros(at[-1], dtype=torch.bool, device="cuda")
        for a, x in zip(at, n):
            mine[a:a + x] = True

        def flat(scale):
            return _normal(g, at[-1], torch.float32, scale).mul_(mine)

        p, grad = flat(0.02), flat(1e-3)
        m, v = flat(3e-4), flat(1e-3).square_()
        s.update(p=p, grad=grad, n=n, at=at, step=torch.full((1,), 100, dtype=torch.int32, device="cuda"),
                 copy=p.to(torch.bfloat16) if case["copy"] else None)
        if case["bits"] == 8:
            m, s["m_scale"] = _encode(m, False)
            v, s["v_scale"] = _encode(v.sqrt_(), True)
        s.update(m=m, v=v)
        if own:
            s["optimizer"] = _optimizer(s)
        return s
    P, sl = case["P"], _slots(case, seed)
    s.update(sl)
    G, n_slots = case["G"], case["G"] + case["reps"]
    if op == "wgrad":
        M, N = case["M"], case["N"]
        s.update(a=_normal(g, (P, M)), b=_normal(g, (P, N)),
                 g_home=torch.empty((G, M, N), dtype=torch.float32, device="cuda"),
                 g_rep=torch.empty((max(1, case["reps"]), M, N), dtype=torch.float32, device="cuda"))
        return s
    H, I = case["H"], case["I"]

    def rows(width):
        return torch.empty((P, width), dtype=torch.bfloat16, device="cuda")

    if op == "up":
        s.update(x=_normal(g, (P, H)), w=_normal(g, (G, 2 * I, H), scale=H ** -0.5), h=rows(I),
                 gu=rows(2 * I) if case["save"] else None)
    elif op == "down":
        s.update(x=_normal(g, (P, I)), w=_normal(g, (G, H, I), scale=I ** -0.5), y=rows(H))
    elif op == "dgrad":
        s.update(x=_normal(g, (P, 2 * I)), w=_normal(g, (G, 2 * I, H), scale=H ** -0.5), y=rows(H))
    else:
        s.update(x=_normal(g, (P, H)), w=_normal(g, (G, H, I), scale=I ** -0.5), gu=_normal(g, (P, 2 * I)),
                 dgu=rows(2 * I), h=rows(I))
    return s


def _optimizer(s):
    """What a training program builds once: the optimizer over its tensors, here with the moments of a run under way."""
    from token_dispatch_histogram_b200.optim import EpAdamW

    def views(flat):
        return [flat[a:a + x] for a, x in zip(s["at"], s["n"])]

    def scales(flat):
        return [flat[a // BLOCK:a // BLOCK + -(-x // BLOCK)] for a, x in zip(s["at"], s["n"])]

    eight = s["case"]["bits"] == 8
    return EpAdamW(views(s["p"]), views(s["grad"]), lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1,
                   state_bits=s["case"]["bits"], copies=views(s["copy"]) if s["copy"] is not None else None,
                   state=dict(step=s["step"], m=views(s["m"]), v=views(s["v"]),
                              m_scale=scales(s["m_scale"]) if eight else None,
                              v_scale=scales(s["v_scale"]) if eight else None))


# ------------------------------------------------------------------ plain forms

def _plain_router(s):
    """Scores and keys in 64 bits: which of two experts comes first is decided next to a border."""
    c = s["case"]
    K, ng = c["K"], c["n_group"]
    x = s["logits"].double()
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else _softmax(x)
    key = p + s["bias"].double() if s["bias"] is not None else x
    if ng > 1:
        of = (p + s["bias"].double()) if s["bias"] is not None else p if c["group_top"] == 2 else x
        best = of.view(len(x), ng, -1).topk(c["group_top"], dim=2).values.sum(2)
        top = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, top, True)
        key = key.masked_fill(~keep.repeat_interleave(x.shape[1] // ng, dim=1), -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(ids=ids.to(torch.int32), w=(w * c["scale"]).float())


def _softmax(x):
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_router_backward(s):
    c = s["case"]
    x, ids, dw = s["logits"].float(), s["ids"].long(), s["dw"]
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else _softmax(x)
    chosen = p.gather(1, ids)
    dp = dw * c["scale"]
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        dp = (dp - (dp * chosen).sum(1, keepdim=True) / total) / total
    if c["score"] == "sigmoid":
        return dict(dlogits=torch.zeros_like(x).scatter_add_(1, ids, dp * chosen * (1 - chosen)).to(s["logits"].dtype))
    inner = (dp * chosen).sum(1, keepdim=True)
    return dict(dlogits=(torch.zeros_like(x).scatter_add_(1, ids, dp * chosen) - p * inner).to(s["logits"].dtype))


def _padded(s, rows):
    """Grouped rows as [slots, longest, width] in 32 bits, zeros behind each slot's rows."""
    at = s["cu"][:-1, None].long() + torch.arange(s["longest"], device="cuda")
    there = at < s["cu"][1:, None]
    return rows[at.clamp_(max=len(rows) - 1)].float().mul_(there[..., None]), there


def _plain_product(s, x, transposed):
    xp, there = _padded(s, x)
    w = s["w"][s["weight"]].float()
    return torch.bmm(xp, w if transposed else w.transpose(1, 2))[there]  # rows of a slot follow each other: in order


def _silu(g):
    return g / (1 + torch.exp(-g))


def _plain_up_backward(s):
    I = s["case"]["I"]
    dh = _plain_product(s, s["x"], True)
    g, u = s["gu"][:, :I].float(), s["gu"][:, I:].float()
    sg = 1 / (1 + torch.exp(-g))
    dg, du = dh * u * sg * (1 + g * (1 - sg)), dh * g * sg
    return dict(dgu=torch.cat([dg, du], 1).bfloat16(), h=(g * sg * u).bfloat16())


def _encode(x, root):
    """8-bit codes (e4m3) and one scale for each block of BLOCK elements: its largest magnitude stands at FP8_MAX.
    Second moments are held as roots, and a nonzero one never at zero: a later step divides by it."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1)
    inv = torch.where(top > TINY, FP8_MAX / top, 0.0)
    y = b * inv[:, None]
    if root:
        y = torch.where(b > 0, y.clamp(min=FP8_MIN), y)
    return y.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(-1), torch.where(top > TINY, top / FP8_MAX, 0.0)


def _decode(code, scale):
    return (code.to(scale.dtype).view(-1, BLOCK) * scale[:, None]).view(-1)


def _plain_adamw(s):
    """Each product and sum rounded by itself: the codes of 8-bit moments are defined by these 32-bit steps."""
    lr, b1, b2, eps, wd = 1e-3, 0.9, 0.95, 1e-8, 0.1
    eight = s["case"]["bits"] == 8
    s["step"] += 1
    t = s["step"].double()
    c1, c2 = (lr / (1 - b1 ** t)).float(), (1 / torch.sqrt(1 - b2 ** t)).float()
    g = s["grad"]
    m = _decode(s["m"], s["m_scale"]) if eight else s["m"]
    v = _decode(s["v"], s["v_scale"]).square_() if eight else s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    root = torch.sqrt(v)
    s["p"].copy_(s["p"] * (1 - lr * wd) - (m * c1) / (root * c2 + eps))
    if s["copy"] is not None:
        s["copy"].copy_(s["p"])
    if eight:
        code, scale = _encode(m, False)
        s["m"].copy_(code)
        s["m_scale"].copy_(scale)
        code, scale = _encode(root, True)
        s["v"].copy_(code)
        s["v_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_out(s)


def _adamw_out(s):
    names = ["p", "m", "v"] + (["m_scale", "v_scale"] if s["case"]["bits"] == 8 else [])
    return {k: s[k] for k in names + (["copy"] if s["copy"] is not None else [])}


def _plain(s):
    op = s["case"]["op"]
    if op == "router":
        return _plain_router(s)
    if op == "router_backward":
        return _plain_router_backward(s)
    if op == "up":
        I = s["case"]["I"]
        gu = _plain_product(s, s["x"], False)
        h = (_silu(gu[:, :I]) * gu[:, I:]).bfloat16()
        return dict(h=h, gu=gu.bfloat16()) if s["case"]["save"] else dict(h=h)
    if op == "down":
        return dict(y=_plain_product(s, s["x"], False).bfloat16())
    if op == "dgrad":
        return dict(y=_plain_product(s, s["x"], True).bfloat16())
    if op == "up_backward":
        return _plain_up_backward(s)
    if op == "wgrad":
        a, b = _padded(s, s["a"])[0], _padded(s, s["b"])[0]
        d = torch.bmm(a.transpose(1, 2), b)
        G = s["case"]["G"]
        return dict(home=d[:G], rep=d[G:]) if s["case"]["reps"] else dict(home=d)
    return _plain_adamw(s)


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import token_dispatch_histogram_b200 as tdh
    c = s["case"]
    op = c["op"]
    if op == "router":
        tdh.ep_router(s["logits"], s["ids"], s["w"], score=c["score"], bias=s["bias"], n_group=c["n_group"],
                      topk_group=c["topk_group"], group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"])
        return dict(ids=s["ids"], w=s["w"])
    if op == "router_backward":
        tdh.ep_router_backward(s["dw"], s["logits"], s["ids"], s["dlogits"], score=c["score"], renorm=c["renorm"],
                               scale=c["scale"])
        return dict(dlogits=s["dlogits"])
    if op == "adamw":
        s["optimizer"].step()
        return _adamw_out(s)
    slots = dict(slot_order=s["slots"], rep_expert=s["rep"])
    if op == "up":
        tdh.ep_expert_up(s["x"], s["w"], s["cu"], s["h"], s["gu"], **slots)
        return dict(h=s["h"], gu=s["gu"]) if c["save"] else dict(h=s["h"])
    if op == "down":
        tdh.ep_expert_gemm(s["x"], s["w"], s["cu"], s["y"], **slots)
        return dict(y=s["y"])
    if op == "dgrad":
        tdh.ep_expert_gemm(s["x"], s["w"], s["cu"], s["y"], transpose_w=True, **slots)
        return dict(y=s["y"])
    if op == "up_backward":
        tdh.ep_expert_up_backward(s["x"], s["w"], s["gu"], s["cu"], s["dgu"], s["h"], **slots)
        return dict(dgu=s["dgu"], h=s["h"])
    tdh.ep_expert_wgrad(s["a"], s["b"], s["cu"], s["g_home"], s["g_rep"], **slots)
    return dict(home=s["g_home"], rep=s["g_rep"]) if c["reps"] else dict(home=s["g_home"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ bytes and operations of one pass

def work(case):
    op = case["op"]
    if op in ("router", "router_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        size = 2 if case["dtype"] != "f32" else 4
        if op == "router":
            return {"bytes": T * E * size + T * K * 8 + (4 * E if case["bias"] else 0), "flops": 0}
        # only a softmax over all experts has a gradient that needs every logit
        read = E if case["score"] == "softmax" and not case["renorm"] else K
        return {"bytes": T * read * size + T * E * size + T * K * 8, "flops": 0}
    if op == "adamw":
        n, b = case["total"], 1 if case["bits"] == 8 else 4
        return {"bytes": n * (12 + 4 * b + (2 if case["copy"] else 0)) + (16 * (n // BLOCK) if b == 1 else 0), "flops": 0}
    P, used = case["P"], min(case["P"], case["G"])
    if op == "wgrad":
        M, N = case["M"], case["N"]
        return {"bytes": 2 * P * (M + N) + 4 * M * N * (case["G"] + case["reps"]), "flops": 2 * P * M * N}
    H, I = case["H"], case["I"]
    if op == "up":
        return {"bytes": 2 * (P * H + used * 2 * I * H + P * I * (3 if case["save"] else 1)), "flops": 4 * P * H * I}
    if op == "down":
        return {"bytes": 2 * (P * I + used * H * I + P * H), "flops": 2 * P * H * I}
    if op == "dgrad":
        return {"bytes": 2 * (P * 2 * I + used * 2 * I * H + P * H), "flops": 4 * P * H * I}
    return {"bytes": 2 * (P * H + used * H * I + P * 5 * I), "flops": 2 * P * H * I}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "router":
        return _exact_router(s)
    if op == "router_backward":
        return _exact_router_backward(s)
    if op == "adamw":
        return _exact_adamw(s)
    if op == "wgrad":
        out = torch.empty((case["G"] + case["reps"], case["M"], case["N"]), dtype=torch.float64, device="cuda")
        for i, (a, b) in enumerate(_bounds(s)):
            torch.mm(s["a"][a:b].double().T, s["b"][a:b].double(), out=out[i])
        G = case["G"]
        return dict(home=out[:G], rep=out[G:]) if case["reps"] else dict(home=out)
    width = s["w"].shape[1 if op in ("up", "down") else 2]
    y = torch.empty((case["P"], width), dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(_bounds(s)):
        w = s["w"][s["where"][i]].double()
        torch.mm(s["x"][a:b].double(), w.T if op in ("up", "down") else w, out=y[a:b])
    if op in ("down", "dgrad"):
        return dict(y=y)
    I = case["I"]
    if op == "up":
        h = y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]
        return dict(h=h, gu=y) if case["save"] else dict(h=h)
    gate, up = s["gu"].double().split(I, dim=1)
    sig = torch.sigmoid(gate)
    dgate = y * up * (sig + gate * sig * (1 - sig))  # d silu(g) / dg, by the product rule
    return dict(dgu=torch.cat([dgate, y * gate * sig], 1), h=gate * sig * up)


def _bounds(s):
    at = 0
    for n in s["sizes"]:
        yield at, at + n
        at += n


def _exact_router(s):
    c, bias = s["case"], s["bias"]
    T, E = s["logits"].shape
    ids = torch.empty((T, c["K"]), dtype=torch.int64, device="cuda")
    w = torch.empty((T, c["K"]), dtype=torch.float64, device="cuda")
    for a in range(0, T, 65536):
        x = s["logits"][a:a + 65536].to(torch.float64)
        if c["score"] == "sigmoid":
            score = torch.where(x >= 0, 1 / (1 + (-x).exp()), x.exp() / (1 + x.exp()))
        else:
            score = (x - torch.logsumexp(x, 1, keepdim=True)).exp()
        key = x.clone() if bias is None else score + bias.to(torch.float64)
        if c["n_group"] > 1:
            by = (key if bias is not None or c["group_top"] == 1 else score).view(len(x), c["n_group"], -1)
            first = by.amax(2)
            if c["group_top"] == 2:
                at = by.argmax(2, keepdim=True)
                first = first + by.scatter(2, at, -math.inf).amax(2)
            # a group's place: how many groups stand before it, equal ones by their index
            lower = torch.arange(c["n_group"], device="cuda")
            before = (first[:, None, :] > first[:, :, None]) | ((first[:, None, :] == first[:, :, None])
                                                                & (lower[None, :] < lower[:, None]))
            out = before.sum(2) >= c["topk_group"]
            key = torch.where(out[:, :, None], -math.inf, key.view(len(x), c["n_group"], -1)).view(len(x), E)
        for k in range(c["K"]):
            best = key.amax(1, keepdim=True)
            at = torch.where(key == best, torch.arange(E, device="cuda"), E).amin(1)
            ids[a:a + 65536, k] = at
            w[a:a + 65536, k] = score.gather(1, at[:, None])[:, 0]
            key.scatter_(1, at[:, None], -math.inf)
    if c["renorm"]:
        w /= w.sum(1, keepdim=True)
    return dict(ids=ids.to(torch.int32), w=w * c["scale"])


def _exact_router_backward(s):
    """The weights' Jacobian, from the definition: dw_j/dx_e for every chosen j, summed with dL/dw_j."""
    c, K = s["case"], s["case"]["K"]
    out = torch.empty(s["logits"].shape, dtype=torch.float64, device="cuda")
    for a in range(0, len(out), 65536):
        x, ids = s["logits"][a:a + 65536].double(), s["ids"][a:a + 65536].long()
        dw = c["scale"] * s["dw"][a:a + 65536].double()
        o = out[a:a + 65536].zero_()
        xs = x.gather(1, ids)
        if c["score"] == "sigmoid":
            z = torch.sigmoid(xs)
            dz = z * torch.sigmoid(-xs)
            if c["renorm"]:
                t = z.sum(1, keepdim=True)
                jac = (torch.eye(K, device="cuda", dtype=torch.float64) / t[..., None]
                       - z[:, :, None] / (t * t)[..., None])  # dw_j / dz_k
                o.scatter_(1, ids, torch.einsum("tj,tjk->tk", dw, jac) * dz)
            else:
                o.scatter_(1, ids, dw * dz)
        elif c["renorm"]:
            z = torch.softmax(xs, 1)
            jac = torch.diag_embed(z) - z[:, :, None] * z[:, None, :]
            o.scatter_(1, ids, torch.einsum("tj,tjk->tk", dw, jac))
        else:
            z = torch.softmax(x, 1)
            zs = z.gather(1, ids)
            o -= z * (dw * zs).sum(1, keepdim=True)
            o.scatter_add_(1, ids, dw * zs)
    return dict(dlogits=out)


def _exact_adamw(s):
    eight = s["case"]["bits"] == 8
    t = int(s["step"]) + 1
    p, g = s["p"].double(), s["grad"].double()
    m = s["m"].double() if not eight else s["m"].double() * s["m_scale"].double().repeat_interleave(BLOCK)
    v = s["v"].double() if not eight else (s["v"].double() * s["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    m = 0.9 * m + 0.1 * g
    v = 0.95 * v + 0.05 * g * g
    p = p - 1e-3 * 0.1 * p - 1e-3 * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.95 ** t)).sqrt() + 1e-8)
    out = dict(p=p)
    if eight:
        out["m"], out["m_scale"] = _encode(m, False)
        out["v"], out["v_scale"] = _encode(v.sqrt(), True)
        out["m"], out["v"] = out["m"].double(), out["v"].double()
    else:
        out.update(m=m, v=v)
    if s["copy"] is not None:
        out["copy"] = p
    return out
