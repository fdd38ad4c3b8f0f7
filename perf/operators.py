"""Operators of the ZeRO-3 shard step over many tensors, their plain forms and their cases.

Five operators:

adamw32   AdamW over many tensors at once, moments in 32 bits
adamw8    the same with moments in 8 bits, one scale per 256 elements, each code rounded to
          nearest or stochastically (the random numbers are a hash of a seed and the element)
norm      the L2 norm over many gradient tensors and the factor that clips it
mxq       a bf16 or fp32 shard to microscaled 4-bit floating point, and the values that it then
          stands for
mxgather  a unit's full parameters from D shards in microscaled 4-bit floating point

A parameter list is laid out as the framework's flat unit: tensors end to end with no alignment,
so a ragged list's tensors start at odd offsets. States held in 8 or 4 bits are returned as the
values they stand for, in bf16, which holds them exactly.

The formulas, in the notation of the library's header. AdamW, every operation rounded to 32 bits:
    g = grad * grad_scale        m' = B1 m + B1c g        v' = B2 v + B2c (g g)
    p' = p DEC - SS (m' / (sqrt(v') / BC2S + EPS))         w = bf16(p')
8-bit moments: with u the bits of a block's largest magnitude, the scale byte is
s = min(254, (u + 0xfffff) >> 23) (at least 11 for v; 255, a block that holds no number, if the
magnitude is not finite), and a code c stands for float_of_bits(c << 20) * 2^(s - K), K = 15 for m
(sign in bit 7) and 31 for v (no sign): a float with 3 bits of mantissa. A positive v' never gets
code 0. Microscaled 4 bits: blocks of 32, scale byte max(0, exponent byte of the largest
magnitude - 2), elements +-{0, .5, 1, 1.5, 2, 3, 4, 6} rounded to nearest even, two a byte.
"""
import math

import torch

own = False

HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=100)
BLOCK = 256      # elements to a scale of the 8-bit moments
PAD = 1024       # a tensor's 8-bit moments start at a multiple of this
MX = 32          # elements to a scale of the 4-bit format
OPS = ("adamw32", "adamw8", "norm", "mxq", "mxgather")

# The tensors of one unit: (sizes of the 3.3M-parameter GPT, of one 7B decoder block, or a ragged
# list whose sizes are spread over their logarithm).
GPT = dict(unit="gpt", d=256, ff=1024, vocab=512, blocks=4)
DECODER = dict(unit="block", d=4096, ff=11008, blocks=1)


def listed():
    return [
        # a handful of small tensors (norms, biases, adapters): what a launch costs
        dict(name="adamw32 few small fp32", op="adamw32", grads="f32", w=False, clip=False,
             unit="ragged", count=5, lo=64, hi=4096, sizes=3),
        # the whole small GPT in one step, gradients clipped
        dict(name="adamw32 gpt bf16 clip", op="adamw32", grads="bf16", w=True, clip=True, **GPT),
        # one decoder block's parameters, bf16 gradients: the streaming rate
        dict(name="adamw32 block bf16", op="adamw32", grads="bf16", w=True, clip=True, **DECODER),
        # the small GPT with 8-bit moments, rounded to nearest
        dict(name="adamw8 gpt bf16 nearest", op="adamw8", grads="bf16", w=True, clip=True,
             stochastic=False, **GPT),
        # one decoder block with 8-bit moments, stochastic rounding
        dict(name="adamw8 block bf16 stochastic", op="adamw8", grads="bf16", w=True, clip=True,
             stochastic=True, **DECODER),
        # a thousand ragged tensors, fp32 gradients, most of them at odd offsets
        dict(name="adamw8 ragged fp32", op="adamw8", grads="f32", w=True, clip=False,
             stochastic=True, unit="ragged", count=1000, lo=64, hi=1 << 19, sizes=5),
        # the norm of the small GPT's gradients
        dict(name="norm gpt bf16", op="norm", grads="bf16", max_norm=1.0, **GPT),
        # the norm of two thousand ragged fp32 gradients
        dict(name="norm ragged fp32", op="norm", grads="f32", max_norm=1.0, unit="ragged",
             count=2000, lo=64, hi=1 << 20, sizes=7),
        # a small odd fp32 shard to 4 bits
        dict(name="mxq odd fp32", op="mxq", src="f32", S=100003),
        # a rank's bf16 working shard of one decoder block at D = 8
        dict(name="mxq block shard bf16", op="mxq", src="bf16", S=25298944),
        # the small GPT's unit from 4 shards
        dict(name="mxgather gpt D4 bf16", op="mxgather", D=4, S=820352, out="bf16"),
        # the decoder block's unit from 8 shards
        dict(name="mxgather block D8 bf16", op="mxgather", D=8, S=25298944, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))


def draw(rng):
    op = rng.choice(OPS)
    if op == "mxq":
        return dict(op=op, src=rng.choice(("bf16", "f32")), S=_log_int(rng, 1, 25_000_000))
    if op == "mxgather":
        D = rng.choice((1, 2, 3, 4, 8, 16, 32, 64))
        return dict(op=op, D=D, S=_log_int(rng, 1, 100_000_000 // D), out=rng.choice(("bf16", "f32")))
    lo = _log_int(rng, 1, 4096)
    hi = _log_int(rng, lo + 1, 1 << 19)
    most = 1_000 if op != "norm" else 2_000
    case = dict(op=op, grads=rng.choice(("bf16", "f32")), unit="ragged", lo=lo, hi=hi,
                count=_log_int(rng, 1, most), sizes=rng.randrange(1 << 20))
    if op == "norm":
        return dict(case, max_norm=rng.choice((0.1, 1.0, 1000.0)))
    case.update(w=rng.random() < 0.8, clip=rng.random() < 0.5)
    if op == "adamw8":
        case["stochastic"] = rng.random() < 0.5
    return case


def sizes_of(case):
    """Elements of each tensor of a case's unit."""
    if case["unit"] == "ragged":
        import random
        rng = random.Random(case["sizes"])
        return [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["count"])]
    d, ff = case["d"], case["ff"]
    if case["unit"] == "gpt":
        return [case["vocab"] * d] + case["blocks"] * [d, d, d * d, d * d, d * d, d * d, d, d,
                                                       ff * d, ff * d] + [d, d]
    return case["blocks"] * [d * d, d * d, d * d, d * d, ff * d, ff * d, ff * d, d, d]


def work(case):
    """Bytes: each input read once, each output written once (8-bit moments at 1 byte and 2/256 of
    scales, their values in bf16 as returned). flops: the formulas' operations."""
    if case["op"] == "mxq":
        S = case["S"]
        return dict(bytes=S * (2 if case["src"] == "bf16" else 4) + S * (0.5 + 1 / MX + 2), flops=4 * S)
    if case["op"] == "mxgather":
        n = case["D"] * case["S"]
        return dict(bytes=n * (0.5 + 1 / MX + (2 if case["out"] == "bf16" else 4)), flops=n)
    n = sum(sizes_of(case))
    g = n * (2 if case["grads"] == "bf16" else 4)
    if case["op"] == "norm":
        return dict(bytes=g, flops=2 * n)
    w = 2 * n if case["w"] else 0
    if case["op"] == "adamw32":
        return dict(bytes=g + w + 24 * n, flops=14 * n)
    return dict(bytes=g + w + 8 * n + 4 * n + 4 * n / BLOCK + 4 * n, flops=30 * n)


# ---------------------------------------------------------------- inputs


def _normal(n, std, gen):
    return torch.randn(n, generator=gen, device="cuda").mul_(std)


def _arena(sizes):
    """Where each tensor's 8-bit moments start, and the arena's length (as zs_state8_layout)."""
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // PAD) * PAD
    return starts, at


def _random_codes(n, lo, hi, gen):
    return torch.randint(lo, hi, (n,), generator=gen, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "mxq":
        S = case["S"]
        x = _normal(S, 0.02, gen)
        st["x"] = x.bfloat16() if case["src"] == "bf16" else x
        st["codes"] = torch.zeros(-(-S // 2), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.zeros(-(-S // MX), dtype=torch.uint8, device="cuda")
        st["out"] = torch.zeros(S, dtype=torch.bfloat16, device="cuda")
        return st
    if case["op"] == "mxgather":
        D, S = case["D"], case["S"]
        st["codes"] = [_random_codes(-(-S // 2), 0, 256, gen) for _ in range(D)]
        st["scales"] = [_random_codes(-(-S // MX), 116, 122, gen) for _ in range(D)]
        st["out"] = torch.zeros(D * S, device="cuda",
                                dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        return st
    sizes = sizes_of(case)
    n = sum(sizes)
    g = _normal(n, 1e-3, gen)
    st["g"] = g.bfloat16() if case["grads"] == "bf16" else g
    if case["op"] == "norm":
        st["sumsq"] = torch.zeros(1, dtype=torch.float64, device="cuda")
        st["norm_coef"] = torch.zeros(2, device="cuda")
        if own:
            import fsdp_sharded_optimizer_zs_amd as zs
            st["table"] = zs.MultiTable(grads=st["g"].split(sizes))
            st["workspace"] = torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device="cuda")
        return st
    st["p"] = _normal(n, 0.02, gen)
    st["w"] = torch.zeros(n, dtype=torch.bfloat16, device="cuda") if case["w"] else None
    st["grad_scale"] = (torch.rand(1, generator=gen, device="cuda") * 0.5 + 0.4) if case["clip"] else None
    lists = dict(p=st["p"].split(sizes), grads=st["g"].split(sizes),
                 w=st["w"].split(sizes) if case["w"] else None)
    if case["op"] == "adamw32":
        st["m"] = _normal(n, 3e-4, gen)
        st["v"] = _normal(n, 1e-3, gen).square_()
        if own:
            import fsdp_sharded_optimizer_zs_amd as zs
            st["table"] = zs.MultiTable(m=st["m"].split(sizes), v=st["v"].split(sizes), **lists)
        return st
    starts, total = _arena(sizes)
    st["seed"] = (seed * 2654435761 + 12345) % (1 << 63) if case["stochastic"] else None
    # moments as an earlier step left them: codes of a signed normal and of a spread-out square
    st["m8"] = _random_codes(total, 0, 256, gen)
    st["v8"] = _random_codes(total, 100, 256, gen)
    st["ms"] = _random_codes(total // BLOCK, 114, 119, gen)
    st["vs"] = _random_codes(total // BLOCK, 104, 110, gen)
    st["m_out"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
    st["v_out"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
    # the plan: each element's tensor, its place in the tensor and its place in the arena
    lens = torch.tensor(sizes, device="cuda")
    st["tensor"] = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), lens)
    first = torch.tensor([0] + sizes, device="cuda").cumsum(0)[:-1]
    st["index"] = torch.arange(n, device="cuda") - first[st["tensor"]]
    st["place"] = st["index"] + torch.tensor(starts, device="cuda")[st["tensor"]]
    st["count"] = len(sizes)
    # what lies between the tensors of an arena is never stepped
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    live[st["place"]] = True
    st["m8"].mul_(live)
    st["v8"].mul_(live)
    if own:
        import fsdp_sharded_optimizer_zs_amd as zs
        cut = [(a, a + k) for a, k in zip(starts, sizes)]
        blocks = [(a // BLOCK, a // BLOCK - (-k // BLOCK)) for a, k in zip(starts, sizes)]
        st["table"] = zs.MultiTable(
            m=[st["m8"][a:b] for a, b in cut], v=[st["v8"][a:b] for a, b in cut],
            m_scale=[st["ms"][a:b] for a, b in blocks], v_scale=[st["vs"][a:b] for a, b in blocks],
            **lists)
    return st


# ---------------------------------------------------------------- one pass


def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st, op)
    return dict(adamw32=_adamw32, adamw8=_adamw8, norm=_norm, mxq=_mxq, mxgather=_mxgather)[op](st)


def _own(st, op):
    import fsdp_sharded_optimizer_zs_amd as zs
    if op == "mxq":
        zs.zs_quantize_mx4(st["x"], st["codes"], st["scales"])
        zs.zs_gather_unit_mx4([st["codes"]], [st["scales"]], st["out"])
        return st["out"]
    if op == "mxgather":
        zs.zs_gather_unit_mx4(st["codes"], st["scales"], st["out"])
        return st["out"]
    if op == "norm":
        zs.zs_grad_norm(st["table"], st["case"]["max_norm"], st["sumsq"], st["norm_coef"],
                        st["workspace"])
        return dict(sumsq=st["sumsq"], norm_coef=st["norm_coef"])
    if op == "adamw32":
        zs.zs_adamw_multi(st["table"], HP, grad_scale=st["grad_scale"])
        return dict(p=st["p"], m=st["m"], v=st["v"], w=st["w"])
    zs.zs_adamw_multi(st["table"], HP, grad_scale=st["grad_scale"], seed=st["seed"])
    zs.zs_state8_decode(st["m8"], st["ms"], zs.ZS_STATE8_M, st["m_out"])
    zs.zs_state8_decode(st["v8"], st["vs"], zs.ZS_STATE8_V, st["v_out"])
    return dict(p=st["p"], m=st["m_out"], v=st["v_out"], w=st["w"])


def _consts():
    b1t, b2t = HP["beta1"] ** HP["step"], HP["beta2"] ** HP["step"]
    return dict(dec=1.0 - HP["lr"] * HP["weight_decay"], b1=HP["beta1"], b1c=1.0 - HP["beta1"],
                b2=HP["beta2"], b2c=1.0 - HP["beta2"], ss=HP["lr"] / (1.0 - b1t),
                bc2s=math.sqrt(1.0 - b2t), eps=HP["eps"])


def _moments(st, m, v):
    k, g = _consts(), st["g"].float()
    if st["grad_scale"] is not None:
        g = g * st["grad_scale"]
    return m * k["b1"] + g * k["b1c"], v * k["b2"] + (g * g) * k["b2c"]


def _parameters(st, m1, v1):
    k = _consts()
    # the divisor as a tensor: division by a number may be taken as a product with its inverse
    bc2s = torch.full((1,), k["bc2s"], device=v1.device)
    den = v1.sqrt() / bc2s + k["eps"]
    st["p"].copy_(st["p"] * k["dec"] - (m1 / den) * k["ss"])
    if st["w"] is not None:
        st["w"].copy_(st["p"])


def _adamw32(st):
    m1, v1 = _moments(st, st["m"], st["v"])
    st["m"].copy_(m1)
    st["v"].copy_(v1)
    _parameters(st, m1, v1)
    return dict(p=st["p"], m=st["m"], v=st["v"], w=st["w"])


def _pow2(e):
    """2^e for whole numbers e, in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _decode8(codes, scales, places, K, signed):
    c = codes[places].int()
    s = scales[places >> 8].int()
    mag = ((c & (0x7F if signed else 0xFF)) << 20).view(torch.float32)
    x = (mag.double() * _pow2(s - K)).float()
    if signed:
        x = torch.where(c >= 128, -x, x)
    return torch.where(s == 255, float("nan"), x)


def _mix(x):
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_words(st):
    """The 32 random bits of each element, from the seed, its tensor and its place in it."""
    lo, hi = st["seed"] & 0xFFFFFFFF, st["seed"] >> 32
    t = torch.arange(1, st["count"] + 1, device="cuda")
    key = _mix((_mix((lo + 0x9E3779B9 * t) & 0xFFFFFFFF) + hi) & 0xFFFFFFFF)
    return _mix((st["index"] & 0xFFFFFFFF) ^ key[st["tensor"]])


def _encode8(x, codes, scales, places, K, signed, add):
    """Codes and scale bytes of the values x at `places` of an arena, from their magnitudes' bits."""
    mag = torch.zeros(codes.numel(), device=x.device)
    mag[places] = x.abs()
    live = torch.zeros(scales.numel(), dtype=torch.bool, device=x.device)
    live[places >> 8] = True
    u = mag.view(-1, BLOCK).amax(1).view(torch.int32)
    s = ((u.long() + 0xFFFFF) >> 23).clamp(0 if signed else 11, 254)
    s = torch.where((u & 0x7FFFFFFF) >= 0x7F800000, 255, s).int()
    scales.copy_(torch.where(live, s.to(torch.uint8), scales))
    se = s[places >> 8]
    bits = (x.abs().double() * _pow2(K - se)).float().view(torch.int32)
    if add is None:
        add = 0x7FFFF + ((bits >> 20) & 1)
    c = (bits.long() + add) >> 20
    if signed:
        c = c.clamp(max=127) | (torch.signbit(x).long() << 7)
    else:
        c = torch.where(x > 0, c.clamp(1, 255), 0)
    codes[places] = torch.where(se == 255, 0, c).to(torch.uint8)


def _adamw8(st):
    at = st["place"]
    m1, v1 = _moments(st, _decode8(st["m8"], st["ms"], at, 15, True),
                      _decode8(st["v8"], st["vs"], at, 31, False))
    _parameters(st, m1, v1)
    am = av = None
    if st["seed"] is not None:
        r = _random_words(st)
        am, av = ((r & 0xFFFF) << 4) | 8, ((r >> 16) << 4) | 8
    _encode8(m1, st["m8"], st["ms"], at, 15, True, am)
    _encode8(v1, st["v8"], st["vs"], at, 31, False, av)
    every = torch.arange(st["m8"].numel(), device="cuda")
    st["m_out"].copy_(_decode8(st["m8"], st["ms"], every, 15, True))
    st["v_out"].copy_(_decode8(st["v8"], st["vs"], every, 31, False))
    return dict(p=st["p"], m=st["m_out"], v=st["v_out"], w=st["w"])


def _norm(st):
    s = st["g"].double().square().sum()
    norm = s.sqrt()
    c = st["case"]["max_norm"] / (norm + 1e-6)
    st["sumsq"].copy_(s)
    st["norm_coef"].copy_(torch.stack([norm, torch.where(c >= 1, 1.0, c)]))
    return dict(sumsq=st["sumsq"], norm_coef=st["norm_coef"])


def _mxq(st):
    x, S = st["x"].float(), st["case"]["S"]
    blocks = torch.zeros(st["scales"].numel() * MX, device=x.device)
    blocks[:S] = x
    u = blocks.view(-1, MX).abs().amax(1).view(torch.int32)
    s = torch.where(u >= 0x7F800000, 255, ((u >> 23) - 2).clamp(min=0))
    st["scales"].copy_(s)
    y = blocks.view(-1, MX) * _pow2(127 - s.clamp(max=254))[:, None].float()
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6)
    q = torch.where((s == 255)[:, None], torch.zeros_like(q), q)
    code = ((q * 2).int() - (q > 2).int() * (q - 2).int() - (q > 4).int() * ((q - 4) / 2).int())
    code = code | (torch.signbit(y).int() << 3)
    code = code.reshape(-1)[: 2 * st["codes"].numel()]
    st["codes"].copy_(code[0::2] | (code[1::2] << 4))
    st["out"].copy_(_mx_values(st["codes"][None], st["scales"][None], S)[0])
    return st["out"]


def _mx_values(codes, scales, S):
    """Values of D shards' codes [D, ceil(S / 2)] and scale bytes [D, ceil(S / 32)], in fp32."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=2).view(codes.shape[0], -1)[:, :S].int()
    s = scales.repeat_interleave(MX, dim=1)[:, :S].int()
    x = (grid[c & 7].double() * _pow2(s - 127)).float()
    x = torch.where(c >= 8, -x, x)
    return torch.where(s == 255, float("nan"), x)


def _mxgather(st):
    x = _mx_values(torch.stack(st["codes"]), torch.stack(st["scales"]), st["case"]["S"])
    st["out"].copy_(x.view(-1))
    return st["out"]


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total = sum(float(x.double().dot(x.double())) for x in st["g"].split(1 << 22))
        norm = math.sqrt(total)
        return dict(sumsq=torch.tensor([total], dtype=torch.float64),
                    norm_coef=torch.tensor([norm, min(1.0, case["max_norm"] / (norm + 1e-6))],
                                           dtype=torch.float64))
    if op == "mxq":
        x = torch.nn.functional.pad(st["x"].double(), (0, -case["S"] % MX)).view(-1, MX)
        top = x.abs().amax(1, keepdim=True)
        two = _two((torch.frexp(top)[1] - 3).clamp(min=-127))
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
        edge = (grid[1:] + grid[:-1]) / 2
        a = (x / two).abs().contiguous()
        # a tie goes to the even code: the lower one at edges 0, 2, 4, 6, the upper one at 1, 3, 5
        k = torch.bucketize(a, edge) + ((a == edge[1]) | (a == edge[3]) | (a == edge[5])).long()
        return (torch.where(x < 0, -1.0, 1.0) * grid[k] * two).view(-1)[: case["S"]]
    if op == "mxgather":
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
        grid, S = torch.cat([grid, -grid]), case["S"]
        at = torch.arange(S, device="cuda")
        return torch.cat([
            grid[((c.long()[at // 2] >> (4 * (at % 2))) & 15)] * _two(s.long()[at // MX] - 127)
            for c, s in zip(st["codes"], st["scales"])])
    return _exact_adamw(st, op)


def _two(e):
    """2^e from a table of powers."""
    table = torch.tensor([math.ldexp(1.0, k) for k in range(-400, 401)], device="cuda",
                         dtype=torch.float64)
    return table[(e + 400).long()]


def _exact_adamw(st, op):
    b1, b2, t = HP["beta1"], HP["beta2"], HP["step"]
    g = st["g"].double()
    if st["grad_scale"] is not None:
        g = g * st["grad_scale"].double()
    if op == "adamw32":
        m, v = st["m"].double(), st["v"].double()
    else:
        m = _value8(st["m8"], st["ms"], 127, 15)[st["place"]]
        v = _value8(st["v8"], st["vs"], 255, 31)[st["place"]]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    hat = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + HP["eps"])
    p = st["p"].double() * (1 - HP["lr"] * HP["weight_decay"]) - HP["lr"] * hat
    if op == "adamw8":
        rm = rv = None
        if st["seed"] is not None:
            r = _random_words(st)
            rm, rv = ((r % 65536) * 16 + 8) / 2**20, ((r // 65536) * 16 + 8) / 2**20
        m = _nearby8(m, st["m8"].numel(), st["place"], 15, rm, 0)
        v = _nearby8(v, st["v8"].numel(), st["place"], 31, rv, 11)
    return dict(p=p, m=m, v=v, w=p if st["w"] is not None else None)


def _value8(codes, scales, most, K):
    """Codes as a number with 3 bits behind the point and an exponent, from 64-bit arithmetic."""
    c = codes.double()
    sign = torch.where(c > most, -1.0, 1.0)
    c = torch.where(c > most, c - 128, c)
    field, part = torch.div(c, 8, rounding_mode="floor"), c % 8
    mag = torch.where(field > 0, (1 + part / 8) * _two(field), part / 8 * 2)
    return sign * mag * _two(scales.long().repeat_interleave(BLOCK) - K - 127)


def _nearby8(x, total, place, K, r, least):
    """Values of the 8-bit format near x, by its block's scale: x's neighbours in steps of an eighth
    of its binade, the nearest one or, with r in (0, 1), the lower one of x + r steps."""
    a = torch.zeros(total, dtype=torch.float64, device=x.device)
    a[place] = x.abs()
    top = a.view(-1, BLOCK).amax(1).clamp(min=2.0 ** -140)
    part, s = torch.frexp(top / 1.875)  # the smallest s with top <= 1.875 * 2^(s - 127)
    s = (s.long() + 127 - (part == 0.5).long()).clamp(least, 254).repeat_interleave(BLOCK)[place]
    unit = _two(s - K - 126)  # the smallest normal number of the block
    binade = _two(torch.frexp((x.abs() / unit).clamp(min=1.0))[1] - 1) * unit
    steps = x.abs() / (binade / 8)
    q = torch.round(steps) if r is None else torch.floor(steps + r)
    y = q * binade / 8
    if K == 31:
        y = torch.where(x > 0, torch.maximum(y, unit / 8), torch.zeros_like(y))
    out = torch.zeros(total, dtype=torch.float64, device=x.device)
    out[place] = torch.where(x < 0, -y, y)
    return out
