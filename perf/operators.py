"""The operators around a LoRA-wrapped attention input projection, as cases to
measure: the block-scaled 8-bit product that is the projection's base
y = x W^T, the quantiser that feeds it, and the rotation of the query and key
heads it produces, with and without the norm of each head.

Every case is one call of one entry point:

  quantize   x [T, K] -> e4m3 values and one fp32 scale per (token, 128 columns)
  matmul     e4m3 x e4m3 with those scales and one per 128 x 128 weight block
  linear     quantize + matmul: 16-bit x in, 16-bit y out, one call
  rope       rotary positions of the q and k heads of a fused projection
  norm_rope  root-mean-square norm of each q and k head, then the rotation

`own` false computes the plain form in elementary torch operations, `own` true
calls the library.
"""
import math

import torch

own = False

BLOCK = 128            # columns that share a scale
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -100  # a group whose largest magnitude is below this is scaled as if it were this

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one token's hidden state on its way into a projection
        dict(name="quantize one token", op="quantize", dtype="f16", T=1, K=4096),
        # the inputs of the down projection of a prefill batch of 8 x 1024 tokens
        dict(name="quantize prefill", op="quantize", dtype="bf16", T=8192, K=14336),
        # one token through the down projection: the weights are read once and that is all
        dict(name="matmul one token", op="matmul", dtype="bf16", T=1, N=4096, K=14336),
        # an odd batch through an odd layer, no side a multiple of any tile
        dict(name="matmul ragged", op="matmul", dtype="f16", T=77, N=1501, K=1000),
        # the fused q/k/v projection of a decode batch
        dict(name="matmul decode qkv", op="matmul", dtype="bf16", T=512, N=6144, K=4096),
        # the fused gate/up projection of a prefill batch
        dict(name="matmul prefill gate_up", op="matmul", dtype="bf16", T=8192, N=28672, K=4096),
        # the q projection of a decode batch, from 16-bit inputs
        dict(name="linear decode q", op="linear", dtype="f16", T=256, N=4096, K=4096),
        # a large mixed batch, from 16-bit inputs
        dict(name="linear large mixed", op="linear", dtype="bf16", T=4096, N=8192, K=8192),
        # adjacent pairs, half of each head rotated, a small decode batch
        dict(name="rope decode partial", op="rope", dtype="f16", T=32, q_heads=32, k_heads=8, dim=128, rot=64,
             interleaved=True, scaling="none", base=10000.0, longest=4096),
        # split halves, frequencies scaled for a long context, a prefill batch at far positions
        dict(name="rope prefill long", op="rope", dtype="bf16", T=8192, q_heads=32, k_heads=8, dim=128, rot=128,
             interleaved=False, scaling="yarn", base=500000.0, longest=131072),
        # the same heads with their norms, one token
        dict(name="norm_rope one token", op="norm_rope", dtype="bf16", T=1, q_heads=32, k_heads=8, dim=128, rot=128,
             interleaved=False, scaling="none", base=1000000.0, longest=40960),
        dict(name="norm_rope prefill", op="norm_rope", dtype="bf16", T=8192, q_heads=32, k_heads=8, dim=128, rot=128,
             interleaved=False, scaling="linear", base=1000000.0, longest=131072),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantize", "matmul", "matmul", "linear", "rope", "norm_rope"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "quantize":
        return dict(op=op, dtype=dtype, T=spread(1, 8192), K=spread(64, 14336))
    if op in ("matmul", "linear"):
        N, K = spread(64, 28672), spread(64, 14336) if rng.random() < 0.5 else 128 * spread(1, 112)
        return dict(op=op, dtype=dtype, T=min(spread(1, 8192), 8192 * 28672 * 4096 // (N * K)), N=N, K=K)
    dim = rng.choice([64, 80, 96, 128, 192, 256])
    rot = rng.choice([dim, dim, dim // 2, dim // 4])
    return dict(op=op, dtype=dtype, T=spread(1, 8192), q_heads=spread(1, 64), k_heads=spread(1, 8), dim=dim, rot=rot,
                interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]),
                base=float(rng.choice([10000, 500000, 1000000])), longest=spread(1024, 1 << 20))


# ---------------------------------------------------------------- the inputs

def frequencies(rot, base, scaling):
    """Radians per position of each pair, in 64 bits, and the factor on cos and sin.

    linear: positions stretched by 4.  yarn: pairs that turn more than 32 times
    over 32768 positions keep their frequency, those that turn less than once
    are stretched by 4, a ramp over the pair's index between."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f / 4.0 * ramp + f * (1 - ramp), 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def up(n, m):
    return -(-n // m) * m


def rows(T, K, multiple, dtype):
    """A [T, K] tensor whose rows start at multiples of `multiple` elements."""
    return torch.empty(T, up(K, multiple), dtype=dtype, device="cuda")[:, :K]


def hidden(g, T, K, dtype):
    """Hidden states: normal, each channel with its own size, a few channels far larger."""
    size = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
    size = torch.where(torch.rand(K, generator=g, device="cuda") < 0.002, size * 30, size)
    x = rows(T, K, 8, dtype)
    return x.copy_(torch.randn(T, K, generator=g, device="cuda") * size)


def blocks_of(x, block_rows):
    """The largest magnitude of each block of block_rows x 128 values."""
    T, K = x.shape
    p = torch.zeros(up(T, block_rows), up(K, BLOCK), device=x.device).index_put_(
        (torch.arange(T, device=x.device)[:, None], torch.arange(K, device=x.device)[None]), x.abs().float())
    return p.view(-1, block_rows, p.shape[1] // BLOCK, BLOCK).amax((1, 3)).clamp_min(SMALLEST)


def spread_out(s, T, K, block_rows):
    """A block's value at every place of the block."""
    return s.repeat_interleave(block_rows, 0)[:T].repeat_interleave(BLOCK, 1)[:, :K]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype, T = case["op"], TYPES[case["dtype"]], case["T"]
    s = dict(op=op)
    if op in ("quantize", "matmul", "linear"):
        K, KB = case["K"], up(case["K"], BLOCK) // BLOCK
        s["x"] = hidden(g, T, K, dtype)
    if op in ("quantize", "matmul"):
        s["q"] = rows(T, K, 16, torch.float8_e4m3fn)
        s["scale"] = torch.empty(T, KB, device="cuda")
    if op in ("matmul", "linear"):
        N = case["N"]
        w = 0.02 * torch.randn(N, K, generator=g, device="cuda")
        ws = blocks_of(w, BLOCK) / E4M3_MAX
        s["W"] = rows(N, K, 16, torch.float8_e4m3fn)
        s["W"].copy_(w / spread_out(ws, N, K, BLOCK))
        s["w_scale"] = ws.contiguous()
        s["y"] = rows(T, N, 8, dtype)
        del w
    if op == "matmul":
        x = s.pop("x").float()
        scale = blocks_of(x, 1) / E4M3_MAX
        s["scale"].copy_(scale)
        s["q"].copy_(x / spread_out(scale, T, K, 1))
    if op == "linear":
        s["work"] = torch.empty(up(T * up(K, 16), 256) + 4 * T * KB + 4096, dtype=torch.uint8, device="cuda")
    if op in ("rope", "norm_rope"):
        hq, hk, dim = case["q_heads"], case["k_heads"], case["dim"]
        # the fused projection: q heads, k heads, v heads
        s["x"] = torch.randn(T, (hq + 2 * hk) * dim, generator=g, device="cuda").to(dtype)
        s["y"] = torch.empty(T, (hq + hk) * dim, dtype=dtype, device="cuda")
        s["heads"], s["dim"], s["interleaved"], s["rot"] = [hq, hk], dim, case["interleaved"], case["rot"]
        start = torch.randint(0, max(1, case["longest"] - T), (1,), generator=g, device="cuda")
        # prompts of 1024 tokens (or fewer) from their own starts; single tokens each at its own place
        s["positions"] = (start + torch.arange(T, device="cuda") % 1024 if T > 256
                          else torch.randint(0, case["longest"], (T,), generator=g, device="cuda")).to(torch.int64)
        f, s["attn_scale"] = frequencies(case["rot"], case["base"], case["scaling"])
        s["inv_freq"] = f.cuda()
    if op == "norm_rope":
        s["weights"] = [(1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(dtype) for _ in range(2)]
        s["eps"] = 1e-6
    return s


# ---------------------------------------------------------------- one pass

def plain_quantize(x):
    a = blocks_of(x, 1)
    T, K = x.shape
    # the quotient in 64 bits: values next to a border of two 8-bit values
    q = (x.double() * E4M3_MAX / spread_out(a.double(), T, K, 1)).float().to(torch.float8_e4m3fn)
    return q, (a.double() / E4M3_MAX).float()


def plain_matmul(q, scale, W, w_scale, dtype):
    x = q.float() * spread_out(scale, q.shape[0], q.shape[1], 1)
    w = W.float() * spread_out(w_scale, W.shape[0], W.shape[1], BLOCK)
    return torch.matmul(x, w.t()).to(dtype)


def plain_rope(s):
    T, H, dim, rot = s["x"].shape[0], sum(s["heads"]), s["dim"], s["rot"]
    x = s["x"][:, :H * dim].reshape(T, H, dim).float()
    if "weights" in s:
        w = torch.cat([s["weights"][0].float().expand(s["heads"][0], dim), s["weights"][1].float().expand(s["heads"][1], dim)])
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    c = (torch.cos(angle) * s["attn_scale"]).float()[:, None]
    d = (torch.sin(angle) * s["attn_scale"]).float()[:, None]
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * d, b * c + a * d], -1).reshape(T, H, rot)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * d, b * c + a * d], -1)
    return torch.cat([turned, x[..., rot:]], -1).reshape(T, H * dim).to(s["x"].dtype)


def run(s):
    op = s["op"]
    if own:
        from gather_matmul_b200 import ops
        if op == "quantize":
            ops.quantize_fp8(s["x"], s["q"], s["scale"])
            return s["q"], s["scale"]
        if op == "matmul":
            return ops.matmul_fp8(s["q"], s["scale"], s["W"], s["w_scale"], s["y"])
        if op == "linear":
            return ops.linear_fp8(s["x"], s["W"], s["w_scale"], s["y"], s["work"])
        if op == "rope":
            return ops.rope(s["x"], s["y"], s["heads"], s["dim"], s["positions"], s["inv_freq"],
                            interleaved=s["interleaved"], attn_scale=s["attn_scale"])
        return ops.norm_rope(s["x"], s["weights"], s["y"], s["heads"], s["dim"], s["positions"], s["inv_freq"],
                             eps=s["eps"], interleaved=s["interleaved"], attn_scale=s["attn_scale"])
    if op == "quantize":
        return plain_quantize(s["x"])
    if op == "matmul":
        return plain_matmul(s["q"], s["scale"], s["W"], s["w_scale"], s["y"].dtype)
    if op == "linear":
        return plain_matmul(*plain_quantize(s["x"]), s["W"], s["w_scale"], s["y"].dtype)
    return plain_rope(s)


def work(case):
    op, T = case["op"], case["T"]
    if op in ("rope", "norm_rope"):
        n = T * (case["q_heads"] + case["k_heads"]) * case["dim"]
        turned = T * (case["q_heads"] + case["k_heads"]) * case["rot"]
        return {"bytes": 4 * n + 8 * T + 4 * case["rot"] + (4 * case["dim"] if op == "norm_rope" else 0),
                "flops": 3 * turned + (4 * n if op == "norm_rope" else 0)}
    K = case["K"]
    KB = up(K, BLOCK) // BLOCK
    if op == "quantize":
        return {"bytes": 3 * T * K + 4 * T * KB, "flops": 2 * T * K}
    N = case["N"]
    weights = N * K + 4 * KB * (up(N, BLOCK) // BLOCK)
    inputs = T * K + 4 * T * KB if op == "matmul" else 2 * T * K
    return {"bytes": weights + inputs + 2 * T * N, "flops": 2 * T * N * K}


# ---------------------------------------------------------------- in 64 bits

def exact_e4m3(v):
    """v (64 bits, at most 448 in magnitude) to the nearest e4m3 value, ties to the even code."""
    grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=v.device)
    middle = (grid[1:] + grid[:-1]) / 2
    below, above = torch.bucketize(v.abs(), middle), torch.bucketize(v.abs(), middle, right=True)
    code = torch.where(below != above, below + below % 2, below)
    return torch.copysign(grid[code], v)


def exact_scales(x):
    T, K = x.shape
    out = torch.empty(T, up(K, BLOCK) // BLOCK, dtype=torch.float64, device=x.device)
    for b in range(out.shape[1]):
        out[:, b] = x[:, b * BLOCK:(b + 1) * BLOCK].double().abs().max(1).values.clamp_min(SMALLEST)
    return out


def exact_quantize(x):
    a, q = exact_scales(x), torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for b in range(a.shape[1]):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        q[:, at] = exact_e4m3(x[:, at].double() * 448 / a[:, b:b + 1])
    return q, a / 448


def exact_product(q, scale, W, w_scale):
    y = torch.zeros(q.shape[0], W.shape[0], dtype=torch.float64, device=q.device)
    for b in range(scale.shape[1]):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        left = q[:, at].double() * scale[:, b:b + 1].double()
        right = W[:, at].double() * w_scale[:, b].double().repeat_interleave(BLOCK)[:W.shape[0], None]
        y.addmm_(left, right.t())
    return y


def exact_heads(s):
    T, dim, rot, half = s["x"].shape[0], s["dim"], s["rot"], s["rot"] // 2
    first, second = ((slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else (slice(0, half), slice(half, rot)))
    # the rotation as a product of complex numbers
    turn = torch.polar(torch.full((T, half), s["attn_scale"], dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] * s["inv_freq"][None])
    out = torch.empty(T, sum(s["heads"]) * dim, dtype=torch.float64, device="cuda")
    for h in range(sum(s["heads"])):
        x = s["x"][:, h * dim:(h + 1) * dim].double()
        if "weights" in s:
            x = x * s["weights"][0 if h < s["heads"][0] else 1].double() * torch.rsqrt(x.square().sum(1, keepdim=True) / dim + s["eps"])
        z = torch.complex(x[:, first], x[:, second]) * turn
        x[:, first], x[:, second] = z.real, z.imag
        out[:, h * dim:(h + 1) * dim] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        return exact_quantize(s["x"])
    if s["op"] == "matmul":
        return exact_product(s["q"], s["scale"], s["W"], s["w_scale"])
    if s["op"] == "linear":
        return exact_product(*exact_quantize(s["x"]), s["W"], s["w_scale"])
    return exact_heads(s)
