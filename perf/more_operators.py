"""The experts' products of a mixture-of-experts layer and what stands between them, as cases that can be timed
and compared.  Rows are sorted by expert; how many each expert has is known on the device alone (offsets).

  matmul    each expert's rows times its weights, row-major weights in either orientation (the forward product, or
            the gradient of the rows), the rows in place or gathered from the tokens
  matmul8   the same with rows in 8 bits and a scale per 128 columns, weights in 8 bits and a scale per 128 x 128
  wgrad     the weights' gradient: each expert's rows of the outputs' gradient times its rows of the inputs
  swiglu    silu(gate) * up of the rows, written in fp32, bf16 or 8 bits with scales, and its gradient

Where `own` is false, run() computes them from elementary torch operations in 32 bits, rounded once at the end; where
it is true, run() calls the framework's entry points on the same inputs and the same caller-owned buffers.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1}
MOST = 16384 * 4096 * 4096       # n * N * D of the largest listed case
MOST_WEIGHTS = 32 * 4096 * 4096  # E * N * D of it


def listed():
    return [
        # a tiny fp32 layer: 64 pairs, 8 experts, 64 -> 2 * 128
        dict(name="matmul-tiny", op="matmul", n=64, E=8, N=256, D=64, dtype="f32", out="f32", transposed=False, topk=0,
             skew=0.0, masked=0.0, pad=0),
        # a decode step: 256 pairs over the 8 experts of a rank, gate and up of a 2880 x 2880 layer
        dict(name="matmul-decode", op="matmul", n=256, E=8, N=5760, D=2880, dtype="bf16", out="bf16", transposed=False,
             topk=4, skew=0.0, masked=0.0, pad=0),
        # a prefill wave: 6554 pairs over 32 skewed experts, gate and up, rows gathered from the tokens
        dict(name="matmul-prefill", op="matmul", n=6554, E=32, N=4096, D=4096, dtype="bf16", out="bf16",
             transposed=False, topk=8, skew=1.0, masked=0.0, pad=0),
        # a training step's gradient of the rows, with the same weights read in the other direction
        dict(name="matmul-rows-grad", op="matmul", n=16384, E=32, N=4096, D=4096, dtype="bf16", out="bf16",
             transposed=True, topk=0, skew=0.5, masked=0.0, pad=0),
        # the decode step in 8 bits
        dict(name="matmul8-decode", op="matmul8", n=256, E=8, N=5760, D=2880, out="bf16", topk=4, skew=0.0, masked=0.0,
             pad=0),
        # the prefill step in 8 bits: 16384 pairs gathered from 2048 tokens
        dict(name="matmul8-prefill", op="matmul8", n=16384, E=32, N=4096, D=4096, out="bf16", topk=8, skew=1.0,
             masked=0.0, pad=0),
        # a training step's weight gradient, kept in fp32
        dict(name="wgrad-train", op="wgrad", n=16384, E=32, N=4096, D=4096, dtype="bf16", out="f32", skew=0.5,
             masked=0.0, pad=0),
        # a ragged one: few rows, some experts with none, padding among the pairs
        dict(name="wgrad-ragged", op="wgrad", n=4099, E=8, N=2880, D=2880, dtype="bf16", out="bf16", skew=2.0,
             masked=0.05, pad=0),
        # decode: 256 rows to the down product, in 8 bits
        dict(name="swiglu-decode", op="swiglu", n=256, I=2880, dtype="bf16", out="fp8", group=128, train=False,
             masked=0.0, pad=0),
        # prefill in 8 bits
        dict(name="swiglu-prefill", op="swiglu", n=16384, I=2048, dtype="bf16", out="fp8", group=128, train=False,
             masked=0.0, pad=0),
        # training: gradients of gate and up, and the product's rows again for the weight gradient
        dict(name="swiglu-backward", op="swiglu", n=16384, I=2048, dtype="bf16", out="bf16", group=0, train=True,
             masked=0.05, pad=0),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul8", "wgrad", "swiglu"])
    pad = rng.choice([0, 0, 16, 64])
    masked = rng.choice([0.0, 0.0, 0.05, 0.3])
    if op == "swiglu":
        I = 8 * _spread(rng, 8, 1024)
        dtype = rng.choice(["f32", "bf16", "bf16"])
        train = rng.random() < 0.4
        out = dtype if train else rng.choice(["bf16", "fp8", "fp8", dtype])
        return dict(op=op, n=_spread(rng, 1, min(16384, 16384 * 2048 // I)), I=I, dtype=dtype, out=out,
                    group=rng.choice([0, 32, 64, 128]) if out == "fp8" else 0, train=train, masked=masked, pad=pad)
    E = rng.choice([1, 4, 8, 16, 32, rng.randint(2, 64)])
    step = 16 if op == "matmul8" else 8
    N, D = step * _spread(rng, 64 // step, 5760 // step), step * _spread(rng, 64 // step, 5760 // step)
    while E * N * D > MOST_WEIGHTS:
        E //= 2
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "matmul8":
        dtype = "fp8"
    most = MOST // (N * D) // (16 if dtype == "f32" else 1)
    case = dict(op=op, n=_spread(rng, 1, max(1, min(16384, most))), E=E, N=N, D=D, dtype=dtype,
                out="f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "f32"]), skew=rng.choice([0.0, 0.5, 1.0, 2.0]),
                masked=masked, pad=pad)
    if op != "wgrad":
        case["topk"] = rng.choice([0, 1, 4, 8])
    if op == "matmul":
        case["transposed"] = rng.random() < 0.4
    if op == "matmul8":
        del case["dtype"]
    return case


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

    def rows(self, n, H, pad, dtype):
        """[n][H] rows of a buffer whose rows are H + pad apart."""
        return self.normal(n, H + pad).to(TYPES[dtype])[:, :H]

    def sizes(self, n, E, skew):
        """How many of n pairs each of E experts has, some chosen more often than others."""
        share = (1.0 / torch.arange(1, E + 1, device="cuda") ** skew)[torch.randperm(E, generator=self.g, device="cuda")]
        share = torch.cumsum(share / share.sum(), 0)
        to = torch.searchsorted(share, self.uniform(n)).clamp(max=E - 1)
        return torch.bincount(to, minlength=E).tolist()


def _buffer(n, H, pad, dtype):
    return torch.zeros(n, H + pad, dtype=torch.uint8 if dtype == "fp8" else TYPES[dtype], device="cuda").view(TYPES[dtype])[:, :H]


def _groups(H, group):
    return -(-H // group) if group else 1


def _quantized(t, rows):
    """t [..][R][C] in 8 bits with a scale per `rows` rows and 128 columns: the codes and the scales."""
    R, C = t.shape[-2:]
    blocks = torch.nn.functional.pad(t, (0, -C % 128, 0, -R % rows))
    blocks = blocks.view(*t.shape[:-2], -(-R // rows), rows, -(-C // 128), 128)
    scale = (blocks.abs().amax((-3, -1)) / 448).clamp(min=1e-30)
    codes = (blocks / scale[..., :, None, :, None]).reshape(*t.shape[:-2], -(-R // rows) * rows, -1)
    return codes[..., :R, :C].to(TYPES["fp8"]), scale


def prepare(case, seed):
    m, s = _Make(seed), dict(case=case)
    n, op, pad = case["n"], case["op"], case["pad"]
    there = n - int(n * case["masked"])  # pairs that have an expert
    if op == "swiglu":
        I = case["I"]
        s["gu"] = (1.5 * m.normal(n, 2 * I + pad)).to(TYPES[case["dtype"]])[:, :2 * I]
        s["count"], s["there"] = torch.tensor([there], dtype=torch.int32, device="cuda"), there
        s["h"] = _buffer(n, I, pad, case["out"])
        s["scale"] = torch.zeros(n, _groups(I, case["group"]), device="cuda") if case["out"] == "fp8" else None
        if case["train"]:
            s["dh"] = m.rows(n, I, pad, case["dtype"])
            s["dgu"] = _buffer(n, 2 * I, pad, case["dtype"])
        return s
    E, N, D = case["E"], case["N"], case["D"]
    s["sizes"] = m.sizes(there, E, case["skew"])
    s["offsets"] = torch.tensor([0] + s["sizes"], device="cuda").cumsum(0).to(torch.int32)
    s["there"] = there
    if op == "wgrad":
        s["dout"], s["x"] = m.rows(n, N, pad, case["dtype"]), m.rows(n, D, pad, case["dtype"])
        s["dw"] = torch.empty(E, N, D, dtype=TYPES[case["out"]], device="cuda")
        return s
    tokens = -(-n // case["topk"]) if case["topk"] else n
    s["slot"] = s["x_scale"] = s["w_scale"] = None
    if case["topk"]:  # the token of each row, -1 behind the last
        s["slot"] = (torch.randperm(n, generator=m.g, device="cuda") // case["topk"]).to(torch.int32)
        s["slot"][there:] = -1
    if op == "matmul":
        s["x"] = m.rows(tokens, D, pad, case["dtype"])
        s["w"] = torch.empty(E, *((D, N) if case["transposed"] else (N, D)), dtype=TYPES[case["dtype"]], device="cuda")
        s["w"].normal_(0, 0.02, generator=m.g)
    else:
        codes, s["x_scale"] = _quantized(m.normal(tokens, D + pad), 1)
        s["x"] = codes[:, :D]
        s["x_scale"] = s["x_scale"][:, :-(-D // 128)].contiguous()
        s["w"] = torch.empty(E, N, D, dtype=torch.uint8, device="cuda").view(TYPES["fp8"])
        s["w_scale"] = torch.empty(E, -(-N // 128), -(-D // 128), device="cuda")
        for e in range(E):
            codes, s["w_scale"][e] = _quantized(0.02 * m.normal(N, D), 128)
            s["w"][e].view(torch.uint8).copy_(codes.view(torch.uint8))
    s["out"] = _buffer(n, N, pad, case["out"])
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _matmul_own(s):
    import asynchronous_moe_expert_amd as M

    M.moe_expert_matmul(s["x"], s["w"], s["offsets"], s["out"], s["err"], row_slot=s["slot"], x_scale=s["x_scale"],
                        w_scale=s["w_scale"], transposed=s["case"].get("transposed", False))
    return s["out"]


def _wgrad_own(s):
    import asynchronous_moe_expert_amd as M

    M.moe_expert_matmul_backward(s["dout"], s["x"], s["offsets"], s["dw"])
    return s["dw"]


def _swiglu_own(s):
    import asynchronous_moe_expert_amd as M

    if s["case"]["train"]:
        M.moe_swiglu_backward(s["gu"], s["dh"], s["dgu"], h=s["h"], count=s["count"])
        return s["dgu"], s["h"]
    M.moe_swiglu(s["gu"], s["h"], h_scale=s["scale"], group=s["case"]["group"], count=s["count"])
    return s["h"] if s["scale"] is None else (s["h"], s["scale"])


def _spread_scale(scale, H, group):
    return scale if not group else scale.repeat_interleave(group, dim=1)[:, :H]


def _rows_plain(s):
    """The rows in the order of the experts, one tensor for each expert, as the values that they stand for."""
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * _spread_scale(s["x_scale"], x.shape[1], 128)
    x = x[:s["there"]] if s["slot"] is None else x[s["slot"][:s["there"]].long()]
    return x.split(s["sizes"])


def _weight_plain(s, e):
    """Expert e's weights, [contraction][outputs]."""
    w = s["w"][e].float()
    if s["w_scale"] is not None:
        w = w * s["w_scale"][e].repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]
    return w if s["case"].get("transposed") else w.t()


def _matmul_plain(s):
    out = torch.zeros(s["out"].shape, dtype=s["out"].dtype, device=s["out"].device)
    parts = [(rows @ _weight_plain(s, e)).to(out.dtype) for e, rows in enumerate(_rows_plain(s))]
    out[:s["there"]] = torch.cat(parts)
    return out


def _wgrad_plain(s):
    pairs = zip(s["dout"][:s["there"]].split(s["sizes"]), s["x"][:s["there"]].split(s["sizes"]))
    return torch.stack([(dout.float().t() @ x.float()).to(s["dw"].dtype) for dout, x in pairs])


def _swiglu_plain(s):
    c, I, n = s["case"], s["case"]["I"], s["there"]
    g, u = s["gu"][:n, :I].float(), s["gu"][:n, I:].float()
    gate = 1 / (1 + torch.exp(-g))
    h = g * gate * u
    if c["train"]:
        dh = s["dh"][:n].float()
        dg, du = dh * u * gate * (1 + g * (1 - gate)), dh * g * gate
        return _padded(torch.cat([dg, du], 1).to(s["dgu"].dtype), c["n"]), _padded(h.to(s["h"].dtype), c["n"])
    if s["scale"] is None:
        return _padded(h.to(s["h"].dtype), c["n"])
    group = c["group"] or I
    amax = torch.nn.functional.pad(h.abs(), (0, -I % group)).view(n, -1, group).amax(2)
    scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    codes = (h / _spread_scale(scale, I, c["group"])).clamp(-448, 448).to(TYPES["fp8"])
    return _padded(codes, c["n"]), _padded(scale, c["n"])


def _padded(rows, n):
    """`rows` with zeros behind them, as the buffers hold them."""
    plain = torch.uint8 if rows.dtype == TYPES["fp8"] else rows.dtype
    full = torch.zeros(n, rows.shape[1], dtype=plain, device=rows.device)
    full[:rows.shape[0]] = rows.view(plain)
    return full.view(rows.dtype)


_plain = dict(matmul=_matmul_plain, matmul8=_matmul_plain, wgrad=_wgrad_plain, swiglu=_swiglu_plain)
_own = dict(matmul=_matmul_own, matmul8=_matmul_own, wgrad=_wgrad_own, swiglu=_swiglu_own)


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    n = case["n"] - int(case["n"] * case["masked"])
    if case["op"] == "swiglu":
        I, b, o = case["I"], BYTES[case["dtype"]], BYTES[case["out"]]
        if case["train"]:
            return dict(bytes=n * I * (5 * b + o), flops=16 * n * I)
        return dict(bytes=n * I * (2 * b + o) + (4 * n * _groups(I, case["group"]) if o == 1 else 0), flops=6 * n * I)
    E, N, D, o = case["E"], case["N"], case["D"], BYTES[case["out"]]
    b = BYTES[case.get("dtype", "fp8")]
    if case["op"] == "wgrad":
        return dict(bytes=n * (N + D) * b + E * N * D * o, flops=2 * n * N * D)
    tokens = -(-n // case["topk"]) if case["topk"] else n
    scales = 4 * (-(-D // 128)) * (tokens + E * (-(-N // 128))) if b == 1 else 0
    return dict(bytes=tokens * D * b + min(E, n) * N * D * b + n * N * o + scales + (4 * n if case["topk"] else 0),
                flops=2 * n * N * D)


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return dict(matmul=_matmul_exact, matmul8=_matmul_exact, wgrad=_wgrad_exact, swiglu=_swiglu_exact)[case["op"]](s)


def _values(codes, scale, rows):
    """What 8-bit codes stand for, with a scale per `rows` rows and 128 columns."""
    r = torch.arange(codes.shape[0], device="cuda") // rows
    c = torch.arange(codes.shape[1], device="cuda") // 128
    return codes.double() * scale.double()[r][:, c]


def _matmul_exact(s):
    c = s["case"]
    out = torch.zeros(c["n"], c["N"], dtype=torch.float64, device="cuda")
    x = s["x"].double() if s["x_scale"] is None else _values(s["x"], s["x_scale"], 1)
    a = 0
    for e in range(c["E"]):
        b = int(s["offsets"][e + 1])
        rows = torch.arange(a, b, device="cuda") if s["slot"] is None else s["slot"][a:b].long()
        w = s["w"][e].double() if s["w_scale"] is None else _values(s["w"][e], s["w_scale"][e], 128)
        out[a:b] = torch.mm(x.index_select(0, rows), w if c.get("transposed") else w.transpose(0, 1))
        a = b
    return out


def _wgrad_exact(s):
    c = s["case"]
    dw = torch.zeros(c["E"], c["N"], c["D"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        rows = slice(int(s["offsets"][e]), int(s["offsets"][e + 1]))
        dw[e] = torch.mm(s["dout"][rows].double().transpose(0, 1), s["x"][rows].double())
    return dw


def _swiglu_exact(s):
    c, I = s["case"], s["case"]["I"]
    keep = (torch.arange(c["n"], device="cuda") < s["count"]).double()[:, None]
    gu = s["gu"].double().requires_grad_()
    h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    if c["train"]:
        (h * s["dh"].double()).sum().backward()
        return gu.grad * keep, h.detach() * keep
    h = h.detach()
    if c["out"] != "fp8":
        return h * keep
    group, codes, scales = c["group"] or I, torch.zeros_like(h), []
    for a in range(0, I, group):
        part = h[:, a:a + group]
        amax = part.abs().amax(1, keepdim=True)
        scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        v = part / scale
        # four significant bits down to 2^-6, steps of 2^-9 below
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        codes[:, a:a + group] = torch.round(v / step) * step
        scales.append(scale * keep)
    return codes * keep, torch.cat(scales, 1)
