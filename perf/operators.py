"""The home rank's operators of a mixture-of-experts layer, as cases that can be timed and compared.

Four operators, each with the directions that a user has of it:

  route   top-k choice of experts and router weights from logits, and the logits' gradient
  sort    rows of tokens sorted by expert, from fp32, bf16 or 8-bit rows
  merge   the experts' rows back in token order with the router weights applied, and its gradient; with unit
          weights it is the gradient of sort
  norm    root-mean-square norm of x + residual, written in fp32, bf16 or 8 bits with scales, and its gradient

Where `own` is false, run() computes them from elementary torch operations in 32 bits, rounded once at the end; where
it is true, run() calls the framework's entry points on the same inputs and the same caller-owned buffers.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1}
MOST = 1 << 28   # T * K * H of the largest listed case
EPS = 1e-5


def listed():
    return [
        # a decode step's tokens on one home rank: 128 experts, top-4, weights renormalised over the chosen
        dict(name="route-decode", op="route", T=64, E=128, K=4, dtype="bf16", score="softmax", renorm=True, bias=False,
             train=False, pad=0),
        # a long prompt through 256 experts, sigmoid scores with the balancing bias
        dict(name="route-prefill", op="route", T=16384, E=256, K=8, dtype="f32", score="sigmoid", renorm=True,
             bias=True, train=False, pad=0),
        # a training step's router: probabilities over all experts, forward and the logits' gradient
        dict(name="route-train", op="route", T=8191, E=128, K=4, dtype="f32", score="softmax", renorm=False, bias=False,
             train=True, pad=0),
        # decode: 256 pairs to the expert FFN
        dict(name="sort-decode", op="sort", T=64, E=128, K=4, H=2880, dtype="bf16", group=0, masked=0.0, pad=0),
        # prefill or training: each row to eight experts
        dict(name="sort-prefill", op="sort", T=8192, E=256, K=8, H=4096, dtype="bf16", group=0, masked=0.0, pad=0),
        # rows that came in 8 bits with a scale per 128 columns, a ragged count with padding tokens
        dict(name="sort-8bit", op="sort", T=4099, E=128, K=4, H=2880, dtype="fp8", group=128, masked=0.05, pad=0),
        # decode: 256 result rows back to 64 tokens
        dict(name="merge-decode", op="merge", T=64, E=128, K=4, H=2880, dtype="bf16", weighted=True, train=False,
             masked=0.0, pad=0),
        # prefill: eight result rows per token
        dict(name="merge-prefill", op="merge", T=8192, E=256, K=8, H=4096, dtype="bf16", weighted=True, train=False,
             masked=0.0, pad=0),
        # training: gradients of the experts' rows and of the router weights, padding tokens among them
        dict(name="merge-backward", op="merge", T=6554, E=128, K=4, H=2880, dtype="bf16", weighted=True, train=True,
             masked=0.05, pad=0),
        # decode: the next layer's input in 8 bits, one scale per row
        dict(name="norm-decode", op="norm", T=64, H=2880, dtype="bf16", residual="bf16", out="fp8", group=0, share=1.0,
             train=False, pad=0),
        # prefill: 8 bits with a scale per 128 columns
        dict(name="norm-prefill", op="norm", T=16384, H=4096, dtype="bf16", residual="bf16", out="fp8", group=128,
             share=1.0, train=False, pad=0),
        # training: gradients of the input and of the weight
        dict(name="norm-backward", op="norm", T=8191, H=2880, dtype="bf16", residual="bf16", out="bf16", group=0,
             share=1.0, train=True, pad=0),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "sort", "merge", "norm"])
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 256, rng.randint(2, 512)])
        K = rng.randint(1, min(8, E))
        return dict(op=op, T=_spread(rng, 1, min(16384, (16384 * 256) // E)), E=E, K=K, dtype=rng.choice(["f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6, bias=rng.random() < 0.4,
                    train=rng.random() < 0.4, pad=rng.choice([0, 0, 1, 5]))
    H = 8 * _spread(rng, 8, 1024)
    dtype = rng.choice(["f32", "bf16", "bf16"])
    pad = rng.choice([0, 0, 8, 64])
    if op == "norm":
        T = _spread(rng, 1, min(16384, (1 << 26) // H))
        train = rng.random() < 0.35
        out = dtype if train else rng.choice(["bf16", "fp8", "fp8", dtype])
        return dict(op=op, T=T, H=H, dtype=dtype, residual=rng.choice([dtype, dtype, "f32"]), out=out,
                    group=rng.choice([0, 32, 64, 128]) if out == "fp8" else 0,
                    share=1.0 if train else rng.choice([1.0, 1.0, 0.5]), train=train, pad=pad)
    E = rng.choice([8, 16, 60, 64, 128, 256])
    K = rng.choice([1, 2, 4, 6, 8])
    T = _spread(rng, 1, min(16384, MOST // (K * H) // (2 if dtype == "f32" else 1)))
    masked = rng.choice([0.0, 0.05, 0.3])
    if op == "sort":
        dtype = rng.choice([dtype, "fp8"])
        return dict(op=op, T=T, E=E, K=K, H=H, dtype=dtype, group=rng.choice([0, 32, 64, 128]) if dtype == "fp8" else 0,
                    masked=masked, pad=pad)
    train = rng.random() < 0.5
    return dict(op=op, T=T, E=E, K=K, H=H, dtype=dtype, weighted=train or rng.random() < 0.6, train=train,
                masked=masked, pad=pad)


# ------------------------------------------------------------------------------------------------ inputs
class _Make:
    """Inputs on the GPU from the seed alone."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda")

    def rows(self, T, H, pad, dtype):
        """[T][H] rows of a buffer whose rows are H + pad apart."""
        return self.normal(T, H + pad).to(TYPES[dtype])[:, :H]

    def order(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")


def _buffer(T, H, pad, dtype):
    return torch.zeros(T, H + pad, dtype=torch.uint8 if dtype == "fp8" else TYPES[dtype], device="cuda").view(TYPES[dtype])[:, :H]


def _groups(H, group):
    return -(-H // group) if group else 1


def _experts(m, T, E, K, masked):
    """K distinct experts a token, some of them chosen far more often than others; padding tokens have none (-1)."""
    taste = m.normal(E)
    expert = torch.topk(m.normal(T, E) + taste, K, dim=1).indices.to(torch.int32)
    if masked:
        expert[m.uniform(T) < masked] = -1
    return expert


def _positions(expert, E):
    """The row of each (token, position) in the order sorted by expert, -1 for none."""
    flat = expert.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    perm = torch.argsort(key, stable=True)
    pos = torch.empty_like(perm)
    pos[perm] = torch.arange(flat.numel(), device="cuda")
    return torch.where(flat < 0, torch.full_like(pos, -1), pos).to(torch.int32).view(expert.shape)


def prepare(case, seed):
    m, s = _Make(seed), dict(case=case)
    T, op, pad = case["T"], case["op"], case["pad"]
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "route":
        E, K = case["E"], case["K"]
        s["logits"] = (1.5 * m.normal(T, E + pad)).to(TYPES[case["dtype"]])[:, :E]
        s["bias"] = 0.2 * m.normal(E) if case["bias"] else None
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        s["expert"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, K, device="cuda")
        if case["train"]:
            s["dw"] = m.normal(T, K)
            s["dlogits"] = _buffer(T, E, pad, case["dtype"])
        return s
    H = case["H"]
    if op == "norm":
        s["x"] = m.rows(T, H, pad, case["dtype"])
        s["gamma"] = (1 + 0.1 * m.normal(H)).to(TYPES[case["dtype"]])
        if case["train"]:
            s["dout"] = m.rows(T, H, pad, case["dtype"])
            s["h"] = m.rows(T, H, pad, case["residual"])
            s["dres"] = m.rows(T, H, pad, case["residual"])
            s["rstd"] = (s["h"].float().square().mean(1) + EPS).rsqrt()
            s["dx"] = _buffer(T, H, pad, case["dtype"])
            s["dgamma"] = torch.empty(H, device="cuda")
            s["workspace"] = torch.empty(2048 * H, dtype=torch.uint8, device="cuda")
            return s
        s["residual"] = (3 * m.normal(T, H + pad)).to(TYPES[case["residual"]])[:, :H]
        s["residual_out"] = _buffer(T, H, pad, case["residual"])
        s["out"] = _buffer(T, H, 2 * pad, case["out"])
        s["out_scale"] = torch.zeros(T, _groups(H, case["group"]), device="cuda") if case["out"] == "fp8" else None
        s["rstd"] = torch.zeros(T, device="cuda")
        s["rows"] = s["count"] = None
        if case["share"] < 1:  # the rows that a step released, and their number on the device
            listed_rows = torch.full((T,), -1, dtype=torch.int32, device="cuda")
            n = max(1, int(case["share"] * T))
            listed_rows[:n] = m.order(T)[:n].sort().values.to(torch.int32)
            s["rows"], s["count"], s["chosen"] = listed_rows, torch.tensor([n], dtype=torch.int32, device="cuda"), n
        return s
    E, K = case["E"], case["K"]
    n = T * K
    expert = _experts(m, T, E, K, case["masked"])
    if op == "sort":
        s["expert"] = expert
        s["x"] = m.rows(T, H, pad, case["dtype"])
        s["x_scale"] = 0.01 + 0.01 * m.uniform(T, _groups(H, case["group"])) if case["dtype"] == "fp8" else None
        for k, count in (("perm", n), ("pos", n), ("counts", E), ("offsets", E + 1)):
            s[k] = torch.empty(count, dtype=torch.int32, device="cuda")
        s["xs"] = torch.zeros(n, H, dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16, device="cuda")
        s["workspace"] = torch.empty(1 << 18, dtype=torch.uint8, device="cuda")
        return s
    s["pos"] = _positions(expert, E)
    s["rows"] = m.rows(n, H, pad, case["dtype"])
    s["w"] = torch.softmax(m.normal(T, K), 1) if case["weighted"] else None
    if case["train"]:
        s["dout"] = m.rows(T, H, pad, case["dtype"])
        s["drows"] = _buffer(n, H, pad, case["dtype"])
        s["dw"] = torch.empty(T, K, device="cuda")
    else:
        s["out"] = _buffer(T, H, pad, case["dtype"])
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _route_own(s):
    import asynchronous_moe_expert_amd as M

    c = s["case"]
    how = dict(score=M.MOE_SIGMOID if c["score"] == "sigmoid" else M.MOE_SOFTMAX, renorm=c["renorm"], scale=s["scale"])
    M.moe_route(s["logits"], s["expert"], s["w"], bias=s["bias"], **how)
    if not c["train"]:
        return s["expert"], s["w"]
    M.moe_route_backward(s["logits"], s["expert"], s["dw"], s["dlogits"], s["err"], **how)
    return s["expert"], s["w"], s["dlogits"]


def _sort_own(s):
    import asynchronous_moe_expert_amd as M

    M.moe_sort_rows(s["expert"], s["case"]["E"], s["x"], s["xs"], s["perm"], s["pos"], s["counts"], s["offsets"],
                    s["err"], s["workspace"], x_scale=s["x_scale"], group=s["case"]["group"])
    return s["perm"], s["pos"], s["counts"], s["offsets"], s["xs"]


def _merge_own(s):
    import asynchronous_moe_expert_amd as M

    if not s["case"]["train"]:
        M.moe_merge_rows(s["rows"], s["pos"], s["w"], s["out"], s["err"])
        return s["out"]
    M.moe_merge_rows_backward(s["dout"], s["rows"], s["pos"], s["w"], s["drows"], s["dw"], s["err"])
    return s["drows"], s["dw"]


def _norm_own(s):
    import asynchronous_moe_expert_amd as M

    c = s["case"]
    if c["train"]:
        M.moe_residual_norm_backward(s["dout"], s["h"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], s["workspace"],
                                     dres=s["dres"])
        return s["dx"], s["dgamma"]
    M.moe_residual_norm(s["x"], s["residual"], s["gamma"], EPS, s["out"], residual_out=s["residual_out"],
                        rstd=s["rstd"], out_scale=s["out_scale"], group=c["group"], row_list=s["rows"],
                        row_count=s["count"], err=s["err"])
    return [t for t in (s["out"], s["residual_out"], s["rstd"], s["out_scale"]) if t is not None]


def _route_plain(s):
    c = s["case"]
    l = s["logits"].float()
    score = l if s["bias"] is None else l + s["bias"]
    chosen = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["K"]]
    lc = l.gather(1, chosen)
    if c["score"] == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.exp(lc - m)
        p = e / (e if c["renorm"] else torch.exp(l - m)).sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-lc))
        if c["renorm"]:
            p = p / p.sum(1, keepdim=True)
    expert, w = chosen.to(torch.int32), p * s["scale"]
    if not c["train"]:
        return expert, w
    dp = s["dw"] * s["scale"]
    if c["score"] == "softmax" and not c["renorm"]:
        every = torch.exp(l - m)
        every = every / every.sum(1, keepdim=True)
        dl = -every * (dp * p).sum(1, keepdim=True)
        dl = dl.scatter_add(1, chosen, p * dp)
    else:
        dc = p * (dp - (dp * p).sum(1, keepdim=True)) if c["renorm"] else p * dp
        if c["score"] == "sigmoid":
            dc = dc / (1 + torch.exp(lc))
        dl = torch.zeros_like(l).scatter_add(1, chosen, dc)
    return expert, w, dl.to(s["logits"].dtype)


def _spread_scale(scale, H, group):
    return scale if not group else scale.repeat_interleave(group, dim=1)[:, :H]


def _sort_plain(s):
    E, K, H = s["case"]["E"], s["case"]["K"], s["case"]["H"]
    flat = s["expert"].reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    perm = torch.argsort(key, stable=True)
    places = torch.arange(flat.numel(), device=flat.device)
    pos = torch.empty_like(perm)
    pos[perm] = places
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device).scatter_add(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    there = places < offsets[E]
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * _spread_scale(s["x_scale"], H, s["case"]["group"])
    xs = (x[perm // K] * there[:, None]).to(s["xs"].dtype)
    none = torch.full_like(perm, -1)
    return (torch.where(there, perm, none).int(), torch.where(flat < 0, none, pos).int(), counts.int(), offsets.int(), xs)


def _merge_plain(s):
    c, (T, K) = s["case"], s["pos"].shape
    there = s["pos"] >= 0
    at = s["pos"].clamp(min=0).long()
    w = there.float() if s["w"] is None else s["w"] * there
    rows = s["rows"].float()[at.reshape(-1)].view(T, K, c["H"])
    if not c["train"]:
        return (rows * w[:, :, None]).sum(1).to(s["out"].dtype)
    dout = s["dout"].float()
    dw = (rows * dout[:, None, :]).sum(2) * there
    drows = torch.zeros(T * K + 1, c["H"], dtype=s["drows"].dtype, device=dout.device)
    drows[torch.where(there, at, T * K).reshape(-1)] = (w[:, :, None] * dout[:, None, :]).to(drows.dtype).view(T * K, -1)
    return drows[:T * K], dw


def _norm_plain(s):
    c = s["case"]
    gamma = s["gamma"].float()
    if c["train"]:
        dout, h, r = s["dout"].float(), s["h"].float(), s["rstd"][:, None]
        g = dout * gamma
        dx = r * (g - h * (r * r * (g * h).mean(1, keepdim=True))) + s["dres"].float()
        return dx.to(s["dx"].dtype), (dout * h * r).sum(0)
    at = slice(None) if s["rows"] is None else s["rows"][:s["chosen"]].long()
    h = s["x"][at].float() + s["residual"][at].float()
    r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    y, scale = h * r * gamma, None
    if c["out"] == "fp8":
        T, H = y.shape
        group = c["group"] or H
        amax = torch.nn.functional.pad(y.abs(), (0, -H % group)).view(T, -1, group).amax(2)
        scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        y = (y / _spread_scale(scale, H, c["group"])).clamp(-448, 448)
    got = [y.to(s["out"].dtype), h.to(s["residual_out"].dtype), r[:, 0]] + ([] if scale is None else [scale])
    if s["rows"] is None:
        return got
    return [_placed(part, at, s["x"].shape[0]) for part in got]


def _placed(part, at, T):
    """`part` at the rows `at` of T; rows that the list leaves out stay as they were."""
    plain = torch.uint8 if part.dtype == TYPES["fp8"] else part.dtype
    full = torch.zeros(T, *part.shape[1:], dtype=plain, device=part.device)
    full[at] = part.view(plain)
    return full.view(part.dtype)


_plain = dict(route=_route_plain, sort=_sort_plain, merge=_merge_plain, norm=_norm_plain)
_own = dict(route=_route_own, sort=_sort_own, merge=_merge_own, norm=_norm_own)


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    T, s = case["T"], BYTES[case["dtype"]]
    if case["op"] == "route":
        E, n = case["E"], T * case["K"]
        return dict(bytes=T * E * s * (2 if case["train"] else 1) + 8 * n + (4 * n if case["train"] else 0),
                    flops=T * E * (6 if case["train"] else 3))
    H = case["H"]
    if case["op"] == "norm":
        r = BYTES[case["residual"]]
        if case["train"]:
            return dict(bytes=T * H * (2 * s + 2 * r) + 4 * T + H * (s + 4), flops=10 * T * H)
        rows = T if case["share"] == 1 else max(1, int(case["share"] * T))
        return dict(bytes=rows * (H * (s + 2 * r + BYTES[case["out"]]) + 4 + 4 * _groups(H, case["group"])) + H * s,
                    flops=7 * rows * H)
    n = T * case["K"]
    kept = int(n * (1 - case["masked"]))
    if case["op"] == "sort":
        o = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=T * H * s + kept * H * o + 12 * n + (4 * T * _groups(H, case["group"]) if s == 1 else 0),
                    flops=T * H if s == 1 else n)
    if case["train"]:
        return dict(bytes=T * H * s + 2 * kept * H * s + 12 * n, flops=3 * kept * H)
    return dict(bytes=kept * H * s + T * H * s + (8 if case["weighted"] else 4) * n, flops=2 * kept * H)


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_route_exact, sort=_sort_exact, merge=_merge_exact, norm=_norm_exact)[case["op"]](s)


def _route_exact(s):
    c = s["case"]
    l = s["logits"].double()
    T, E = l.shape
    score = (s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]).clone()
    chosen = torch.zeros(T, c["K"], dtype=torch.long, device="cuda")
    places = torch.arange(E, device="cuda").expand(T, E)
    for j in range(c["K"]):  # the largest of what is left, the lowest index among equals
        best = score.amax(1, keepdim=True)
        chosen[:, j] = torch.where(score == best, places, torch.full_like(places, E)).amin(1)
        score.scatter_(1, chosen[:, j:j + 1], -math.inf)
    l = l.requires_grad_()
    lc = l.gather(1, chosen)
    if c["score"] == "softmax":
        w = torch.softmax(lc, 1) if c["renorm"] else torch.softmax(l, 1).gather(1, chosen)
    else:
        w = torch.sigmoid(lc)
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    w = w * s["scale"]
    if not c["train"]:
        return None, w.detach()
    (w * s["dw"].double()).sum().backward()
    return None, w.detach(), l.grad


def _sort_exact(s):
    E, K, H = s["case"]["E"], s["case"]["K"], s["case"]["H"]
    x = s["x"].double()
    if s["x_scale"] is not None:
        group = s["case"]["group"] or H
        x = x * s["x_scale"].double()[:, torch.arange(H, device="cuda") // group]
    xs = torch.zeros(s["xs"].shape, dtype=torch.float64, device="cuda")
    flat, at = s["expert"].reshape(-1), 0
    for e in range(E):
        pairs = torch.nonzero(flat == e)[:, 0]
        xs[at:at + pairs.numel()] = x[pairs // K]
        at += pairs.numel()
    return None, None, None, None, xs


def _merge_exact(s):
    c, (T, K) = s["case"], s["pos"].shape
    out = torch.zeros(T, c["H"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    drows = torch.zeros(T * K, c["H"], dtype=torch.float64, device="cuda") if c["train"] else None
    for j in range(K):
        t = torch.nonzero(s["pos"][:, j] >= 0)[:, 0]
        p = s["pos"][t, j].long()
        w = torch.ones(t.numel(), 1, dtype=torch.float64, device="cuda") if s["w"] is None else s["w"][t, j:j + 1].double()
        if c["train"]:
            dout = s["dout"][t].double()
            dw[t, j] = torch.linalg.vecdot(dout, s["rows"][p].double())
            drows[p] = dout * w
        else:
            out[t] += s["rows"][p].double() * w
    return (drows, dw) if c["train"] else out


def _norm_exact(s):
    c = s["case"]
    gamma, H = s["gamma"].double(), c["H"]
    if c["train"]:
        dout, h, r = s["dout"].double(), s["h"].double(), s["rstd"].double()
        xhat = h * r[:, None]
        g = dout * gamma
        dx = (g - xhat * (torch.linalg.vecdot(g, xhat) / H)[:, None]) * r[:, None] + s["dres"].double()
        return dx, torch.linalg.vecdot(dout, xhat, dim=0)
    T = c["T"]
    keep = torch.ones(T, 1, dtype=torch.float64, device="cuda")
    if s["rows"] is not None:
        keep.zero_()
        keep[s["rows"][:s["chosen"]].long()] = 1
    h = s["x"].double() + s["residual"].double()
    r = torch.rsqrt(torch.linalg.vecdot(h, h) / H + EPS)[:, None]
    y = h * gamma * r
    got = [y * keep, h * keep, (r * keep)[:, 0]]
    if c["out"] == "fp8":
        group = c["group"] or H
        codes, scales = torch.zeros_like(y), []
        for a in range(0, H, group):
            part = y[:, a:a + group]
            amax = part.abs().amax(1, keepdim=True)
            sc = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
            v = part / sc
            # four significant bits down to 2^-6, steps of 2^-9 below
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            codes[:, a:a + group] = torch.round(v / step) * step
            scales.append(sc * keep)
        got[0] = codes * keep
        got.append(torch.cat(scales, 1))
    return got
