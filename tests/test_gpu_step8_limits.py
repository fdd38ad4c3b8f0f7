"""The parameters beside 8-bit moments where their bound is tight or numbers leave fp32's
normal range: tiny updates, large lr and eps, infinities and NaN, and tensors past 2^32
elements off HBM's sectors.

The bound, for the fp32 m' and v' that the step computes: with r = 2^-24 half an ulp, the
root is off by 2r (one ulp), 1 / BC2S and the fused divisor by r each, the reciprocal by 2r
and the product m' / den by r: 7 r < 2^-21 of the update in all; that product may round
into the subnormals, off by 2^-150, which SS multiplies; p * DEC and the result are off by
r of themselves or by 2^-150. In all 2^-21 |upd| + 2^-24 (|p DEC| + |p'|) + (1 + SS / 2) 2^-149."""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
import workloads as W
from gpu_util import check_bf16, check_bits, check_f32, device, to_np
from oracle import zs_formats as F
from oracle import zs_oracle as O

pytestmark = pytest.mark.gpu

HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)


def exact_form(k):
    """Whether the header promises the fp32 step's bits."""
    return bool(k["EPS"] * k["BC2S"] < np.float32(2.0**-38) or k["EPS"] > np.float32(2.0**125))


def formula(p, m, v, g, hp):
    """(p', room): the formula in float64 for the fp32 m' and v', and the bound."""
    k = O.adamw_constants(hp)
    f = np.float32
    with np.errstate(all="ignore"):
        m1 = (f(k["B1"]) * m + f(k["B1c"]) * g).astype(np.float64)
        v1 = (f(k["B2"]) * v + f(k["B2c"]) * (g * g)).astype(np.float64)
        k = {n: np.float64(x) for n, x in k.items()}
        upd = k["SS"] * (m1 / (np.sqrt(v1) / k["BC2S"] + k["EPS"]))
        pd = p.astype(np.float64) * k["DEC"]
        want = pd - upd
        return want, (2.0**-21 * np.abs(upd) + 2.0**-24 * (np.abs(pd) + np.abs(want))
                      + (1 + k["SS"] / 2) * 2.0**-149)


def step(p, mc, ms, vc, vs, g, hp, w=True):
    """One step of one tensor given as numpy arrays; the arrays after it, and w."""
    dev = device()
    t = [torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in (p, mc, ms, vc, vs, g)]
    wt = torch.zeros(p.size, dtype=torch.int16, device=dev)
    table = zs.MultiTable([t[0]], [t[1]], [t[3]], [t[5]], [wt] if w else None, [t[2]], [t[4]])
    zs.zs_adamw_multi(table, hp)
    torch.cuda.synchronize()
    return [to_np(x) for x in (*t[:5], wt)]


def check_near(got, want, room, what):
    """Finite values within the bound; infinities of the same sign and NaN in the same
    places."""
    fine = np.isfinite(want)
    got64 = got.astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN elsewhere"
    assert np.array_equal(got64[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    off = np.abs(got64[fine] - want[fine]) - room[fine]
    assert off.size == 0 or off.max() <= 0, f"{what}: off by {off.max()} more than the bound"


def moments(rng, n, lo, hi):
    """Codes and scales whose blocks' largest values are spread from 2^lo to 2^hi."""
    s = np.repeat(2.0 ** rng.uniform(lo, hi, -(-n // 256)), 256)[:n]
    m = (rng.standard_normal(n) * s).astype(np.float32)
    return m, F.state8_encode(m, F.M)


@pytest.mark.parametrize("eps", (1e-8, 1.0, 2.0**60, 2.0**124, 2.0**125, 2.0**126, 2.0**126.5, 2.0**127,
                                 3e38, 1e39))
@pytest.mark.parametrize("lr", (3e-4, 0.1, 1.0, 100.0, 1e6, 1e12))
def test_tiny_updates_and_large_lr_and_eps(lr, eps):
    """Moments down to 2^-149, from stored codes and from the gradient, beside v of 0 to
    2^20, parameters of 0, subnormal and ordinary ones; SS up to 1e13."""
    rng = np.random.default_rng(12)
    n = 256 * 60 + 19
    _, (mc, ms) = moments(rng, n, -150, 10)
    v = np.square(rng.standard_normal(n) * np.repeat(2.0 ** rng.uniform(-70, 10, -(-n // 256)), 256)[:n])
    vc, vs = F.state8_encode(v.astype(np.float32), F.V)
    g = (rng.standard_normal(n) * 2.0 ** rng.uniform(-149, 8, n)).astype(np.float32)
    g[rng.random(n) < 0.5] = 0
    p = (rng.standard_normal(n) * 2.0 ** rng.uniform(-149, 2, n)).astype(np.float32)
    p[rng.random(n) < 0.5] = 0
    hp = O.AdamWHP(**dict(HP, lr=lr, eps=eps, weight_decay=0.01))
    with np.errstate(all="ignore"):
        want = F.adamw_step8(p, mc, ms, vc, vs, g, hp)
    got = step(p, mc, ms, vc, vs, g, hp)
    for j, what in enumerate(("m codes", "m scales", "v codes", "v scales"), 1):
        check_bits(got[j], want[j], what)
    check_bf16(got[5], O.bf16_round(got[0]), "w", exact=True)
    if exact_form(O.adamw_constants(hp)):
        check_f32(got[0], want[0], "p", exact=True)
    else:
        near, room = formula(p, F.state8_values(mc, ms, F.M), F.state8_values(vc, vs, F.V), g, hp)
        check_near(got[0], near, room, f"lr {lr}, eps {eps}")


def test_infinities_and_nan_reach_the_same_parameters():
    """Infinite and NaN gradients, gradients whose square overflows, NaN blocks, infinite and
    NaN parameters, and quotients m' / den that overflow: NaN, signs of infinity and finite
    values where the fp32 step has them."""
    rng = np.random.default_rng(13)
    n = 256 * 40 + 5
    m, (mc, ms) = moments(rng, n, -20, 126)
    vc, vs = F.state8_encode(np.zeros(n, np.float32), F.V)
    g = np.zeros(n, np.float32)
    g[::7] = rng.choice(np.array([np.inf, -np.inf, np.nan, 1e20, -1e25, 3e38, 1e-30, 5.0], np.float32),
                        g[::7].size)
    p = (rng.standard_normal(n) * 0.02).astype(np.float32)
    p[::5] = rng.choice(np.array([np.inf, -np.inf, np.nan, 3e38, -3e38, -0.0], np.float32), p[::5].size)
    ms[3] = 255
    vs[9] = 255
    hp = O.AdamWHP(**HP)
    assert not exact_form(O.adamw_constants(hp))
    with np.errstate(all="ignore"):
        want = F.adamw_step8(p, mc, ms, vc, vs, g, hp)
    assert np.isnan(want[0]).any() and (want[0] == np.inf).any() and (want[0] == -np.inf).any()
    got = step(p, mc, ms, vc, vs, g, hp)
    for j, what in enumerate(("m codes", "m scales", "v codes", "v scales"), 1):
        check_bits(got[j], want[j], what)
    nan, inf = np.isnan(want[0]), np.isinf(want[0])
    assert np.array_equal(np.isnan(got[0]), nan)
    assert np.array_equal(np.isinf(got[0]), inf) and np.array_equal(got[0][inf], want[0][inf])
    near, room = formula(p, F.state8_values(mc, ms, F.M), F.state8_values(vc, vs, F.V), g, hp)
    keep = ~nan & ~inf
    check_near(got[0][keep], near[keep], room[keep], "the rest")
    check_bf16(got[5], O.bf16_round(got[0]), "w", exact=True)


def test_past_32_bits_off_the_sectors():
    """A tensor of 2^32 + 5,000 elements with ordinary hyperparameters, p and w one element
    off a 64-byte sector: windows at its start, around elements 2^31 and 2^32 and at its end.
    Codes, scales and w bit for bit, p within its bound."""
    dev = device()
    n = (1 << 32) + 5000
    whole = n >> 20
    block = W.as_bf16_bits(W.normal_f32(1 << 20, 1e-3, 77, dev))
    g = torch.empty(n, dtype=torch.int16, device=dev)
    g[:whole << 20].view(whole, 1 << 20).copy_(block)
    g[whole << 20:].copy_(block[:n - (whole << 20)])
    p = torch.full((n + 1,), 0.01, device=dev)[1:]
    w = torch.zeros(n + 1, dtype=torch.int16, device=dev)[1:]
    assert p.data_ptr() % 64 and w.data_ptr() % 64
    m, v = (torch.empty(n, dtype=torch.uint8, device=dev) for _ in range(2))
    for x in (m, v):
        codes = torch.randint(0, 256, (1 << 20,), dtype=torch.uint8, device=dev)
        x[:whole << 20].view(whole, 1 << 20).copy_(codes)
        x[whole << 20:].copy_(codes[:n - (whole << 20)])
    nb = -(-n // 256)
    ms, vs = (torch.full((nb,), x, dtype=torch.uint8, device=dev) for x in (117, 107))
    where = [(0, 8192), ((1 << 31) - 4096, 8192), ((1 << 32) - 4096, 8192),
             (n - n % 4096 - 4096, 4096 + n % 4096)]

    def window(a, k):
        b = slice(a // 256, -(-(a + k) // 256))
        return [to_np(x).copy() for x in (p[a:a + k], m[a:a + k], ms[b], v[a:a + k], vs[b], g[a:a + k],
                                          w[a:a + k])]

    before = [window(a, k) for a, k in where]
    table = zs.MultiTable([p], [m], [v], [g], [w], [ms], [vs])
    hp = O.AdamWHP(**dict(HP, step=4))
    assert not exact_form(O.adamw_constants(hp))
    zs.zs_adamw_multi(table, hp, seed=99)
    torch.cuda.synchronize()
    for (a, k), (p0, mc, m_s, vc, v_s, gg, _) in zip(where, before):
        g32 = O.bf16_widen(gg)
        want = F.adamw_step8(p0, mc, m_s, vc, v_s, g32, hp, 99, 0, a)
        got = window(a, k)
        for j, what in enumerate(("m codes", "m scales", "v codes", "v scales"), 1):
            check_bits(got[j], want[j], f"{what} at {a}")
        near, room = formula(p0, F.state8_values(mc, m_s, F.M), F.state8_values(vc, v_s, F.V), g32, hp)
        check_near(got[0], near, room, f"p at {a}")
        check_bf16(got[6], O.bf16_round(got[0]), f"w at {a}", exact=True)
