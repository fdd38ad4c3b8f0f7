"""AdamW over many tensors, 8-bit moments and the gradient norm against the oracle.

The step with fp32 moments is elementwise with a fixed operation order, and the codes of
8-bit moments follow from m' and v' by an exact rule, so these are compared bit for bit.
The parameters beside 8-bit moments have a bound (Case.near). The norm's sum is in
fp64 in an order of its own: n terms, all of one sign, each product exact, so that any
order is within n * 2^-53 of the correctly rounded sum; its float results are then off
by half a step (2^-24) more."""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
import workloads as W
from gpu_util import check_bf16, check_bits, check_f32, device, to_np
from oracle import zs_formats as F
from oracle import zs_oracle as O

pytestmark = pytest.mark.gpu

SIZES = [0, 1, 2, 3, 4, 5, 63, 64, 255, 256, 257, 1000, 1023, 1024, 1025, 3333, 4095, 4096, 4097,
         0, 8192, 12289]
GUARD = 37                     # elements between the tensors of an arena, never written
HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


class Arena:
    """Tensors with GUARD sentinel elements before, between and after them, in one
    allocation: odd starts, and a write beside a tensor shows."""

    def __init__(self, values, dtype, dev, guard=GUARD):
        self.guard, self.sizes = guard, [len(v) for v in values]
        n = sum(self.sizes) + guard * (len(values) + 1)
        self.all = torch.full((n,), 77, dtype=dtype, device=dev)
        self.views, at = [], guard
        for v in values:
            t = self.all[at:at + len(v)]
            t.copy_(torch.from_numpy(np.ascontiguousarray(v)).to(dev))
            self.views.append(t)
            at += len(v) + guard

    def check_guards(self, what):
        keep = torch.ones_like(self.all, dtype=torch.bool)
        at = self.guard
        for n in self.sizes:
            keep[at:at + n] = False
            at += n + self.guard
        assert bool((self.all[keep] == 77).all()), f"{what}: written beside a tensor"


def grads_of(sizes, dtype, seed, scale=1e-3):
    rng = np.random.default_rng(seed)
    g = [(rng.standard_normal(n) * scale).astype(np.float32) for n in sizes]
    return [O.bf16_round(x) for x in g] if dtype == "bf16" else g


def widen(g):
    return O.bf16_widen(g) if g.dtype == np.uint16 else g


def bits16(a):
    return a.view(np.int16) if a.dtype == np.uint16 else a


class Case:
    """A list of tensors on the device in guarded arenas, and the oracle's copy."""

    def __init__(self, sizes, grads, state, w=True, seed=0, p_scale=0.02):
        rng = np.random.default_rng(seed + 1000)
        dev = device()
        self.sizes, self.state = sizes, state
        self.p = [(rng.standard_normal(n) * p_scale).astype(np.float32) for n in sizes]
        self.g = grads
        m = [(rng.standard_normal(n) * 3e-4).astype(np.float32) for n in sizes]
        v = [np.square(rng.standard_normal(n) * 1e-3).astype(np.float32) for n in sizes]
        gt = torch.int16 if grads and grads[0].dtype == np.uint16 else torch.float32
        self.dp = Arena(self.p, torch.float32, dev)
        self.dg = Arena([bits16(g) for g in grads], gt, dev, GUARD + 2)
        self.dw = Arena([np.zeros(n, np.int16) for n in sizes], torch.int16, dev, GUARD + 4) if w else None
        args = dict(p=self.dp.views, grads=self.dg.views, w=self.dw.views if w else None)
        if state == zs.ZS_STATE_F32:
            self.m, self.v = m, v
            self.dm = Arena(m, torch.float32, dev, GUARD + 1)
            self.dv = Arena(v, torch.float32, dev, GUARD + 6)
            self.arenas = [self.dp, self.dg, self.dm, self.dv]
        else:
            self.m = [F.state8_encode(x, F.M) for x in m]
            self.v = [F.state8_encode(x, F.V) for x in v]
            self.dm = Arena([c for c, _ in self.m], torch.uint8, dev, GUARD + 1)
            self.dv = Arena([c for c, _ in self.v], torch.uint8, dev, GUARD + 6)
            self.dms = Arena([s for _, s in self.m], torch.uint8, dev, 5)
            self.dvs = Arena([s for _, s in self.v], torch.uint8, dev, 3)
            self.arenas = [self.dp, self.dg, self.dm, self.dv, self.dms, self.dvs]
            args.update(m_scale=self.dms.views, v_scale=self.dvs.views)
        if w:
            self.arenas.append(self.dw)
        self.table = zs.MultiTable(m=self.dm.views, v=self.dv.views, **args)

    def step_oracle(self, hp, scale=None, seed=None):
        torch.cuda.synchronize()
        self.w = []
        for t in range(len(self.sizes)):
            g = widen(self.g[t])
            if scale is not None:
                g = (g * np.float32(scale)).astype(np.float32)
            with np.errstate(all="ignore"):
                if self.state == zs.ZS_STATE_F32:
                    self.p[t], self.m[t], self.v[t], w = O.adamw_step(self.p[t], self.m[t], self.v[t],
                                                                      g, hp)
                else:
                    (mc, ms), (vc, vs) = self.m[t], self.v[t]
                    p0 = self.p[t]
                    self.p[t], mc, ms, vc, vs, w = F.adamw_step8(p0, mc, ms, vc, vs, g, hp, seed, t)
                    k = O.adamw_constants(hp)
                    if k["EPS"] * k["BC2S"] >= np.float32(2.0**-38):
                        self.p[t], w = self.near(t, p0, g, hp)
                    self.m[t], self.v[t] = (mc, ms), (vc, vs)
            self.w.append(w)

    def near(self, t, p0, g, hp):
        """The device's p, held to its bound: within 2^-21 of the update (root and
        reciprocal one ulp or 2^-23 each, 1 / BC2S, the divisor and the product half of
        that each: 2^-22 + 2^-23 + 2^-24 in all) and half an ulp each of p * DEC and of
        the result. It is then the start of the next step."""
        k = {n: np.float64(x) for n, x in O.adamw_constants(hp).items()}
        f = np.float32
        m = F.state8_values(*self.m[t], F.M)
        v = F.state8_values(*self.v[t], F.V)
        m1 = (f(k["B1"]) * m + f(k["B1c"]) * g).astype(np.float64)
        v1 = (f(k["B2"]) * v + f(k["B2c"]) * (g * g)).astype(np.float64)
        upd = k["SS"] * (m1 / (np.sqrt(v1) / k["BC2S"] + k["EPS"]))
        want = p0 * k["DEC"] - upd
        got = to_np(self.dp.views[t])
        ok = np.isfinite(want)
        assert np.array_equal(ok, np.isfinite(got)), f"tensor {t}: p is finite elsewhere"
        room = 2.0**-21 * np.abs(upd) + 2.0**-24 * (np.abs(p0 * k["DEC"]) + np.abs(want)) + 2.0**-149
        off = np.abs(got[ok] - want[ok]) - room[ok]
        assert off.size == 0 or off.max() <= 0, f"tensor {t}: p off by {off.max()} more than its bound"
        return got, O.bf16_round(got)

    def check(self, what):
        torch.cuda.synchronize()
        for t, n in enumerate(self.sizes):
            tag = f"{what}: tensor {t} ({n})"
            check_f32(to_np(self.dp.views[t]), self.p[t], tag + " p", exact=True)
            if self.dw:
                check_bf16(to_np(self.dw.views[t]), self.w[t], tag + " w", exact=True)
            if self.state == zs.ZS_STATE_F32:
                check_f32(to_np(self.dm.views[t]), self.m[t], tag + " m", exact=True)
                check_f32(to_np(self.dv.views[t]), self.v[t], tag + " v", exact=True)
            else:
                for name, codes, scales, want in (("m", self.dm, self.dms, self.m[t]),
                                                  ("v", self.dv, self.dvs, self.v[t])):
                    check_bits(to_np(scales.views[t]), want[1], f"{tag} {name} scales")
                    check_bits(to_np(codes.views[t]), want[0], f"{tag} {name} codes")
        for a in self.arenas:
            a.check_guards(what)


# ------------------------------------------------------------------ the step
@pytest.mark.parametrize("w", (True, False))
@pytest.mark.parametrize("scale", (None, 0.37))
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_adamw_multi_fp32_moments(dtype, scale, w):
    c = Case(SIZES, grads_of(SIZES, dtype, 1), zs.ZS_STATE_F32, w)
    gs = None if scale is None else torch.tensor([scale], device=device())
    for t in (1, 2, 3):
        zs.zs_adamw_multi(c.table, dict(step=t, **HP), grad_scale=gs)
        c.step_oracle(O.AdamWHP(step=t, **HP), scale)
        c.check(f"step {t}")


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_adamw_multi_gives_the_bits_of_adamw_step(dtype):
    dev = device()
    sizes = [5000, 70_003, 1024]
    c = Case(sizes, grads_of(sizes, dtype, 2), zs.ZS_STATE_F32)
    one = [[x.clone() for x in (c.dp.views[t], c.dm.views[t], c.dv.views[t], c.dw.views[t])]
           for t in range(3)]
    for step in (1, 2):
        zs.zs_adamw_multi(c.table, dict(step=step, **HP))
        for t in range(3):
            zs.zs_adamw_step(*one[t], [c.dg.views[t].clone()], dict(step=step, **HP))
    torch.cuda.synchronize()
    for t in range(3):
        for a, b in zip(one[t], (c.dp.views[t], c.dm.views[t], c.dv.views[t], c.dw.views[t])):
            assert torch.equal(a.view(torch.int16), b.clone().view(torch.int16))


@pytest.mark.parametrize("eps", (1e-8, 1e-13, 0.0))
@pytest.mark.parametrize("seed", (None, 5, (1 << 63) + 12345))
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_adamw_multi_8bit_moments(dtype, seed, eps):
    HP = dict(globals()["HP"], eps=eps)
    c = Case(SIZES, grads_of(SIZES, dtype, 3), zs.ZS_STATE_8BIT, w=dtype == "bf16")
    gs = torch.tensor([0.8], device=device())
    for t in (1, 2, 3):
        s = None if seed is None else seed + t
        zs.zs_adamw_multi(c.table, dict(step=t, **HP), grad_scale=gs if t > 1 else None, seed=s)
        c.step_oracle(O.AdamWHP(step=t, **HP), 0.8 if t > 1 else None, s)
        c.check(f"step {t}")


def test_adamw_multi_8bit_wide_ranges_and_specials():
    """Blocks whose elements span the type's whole range, blocks of zeros, and blocks
    with an infinity or NaN (from the gradient, then from the stored scale)."""
    rng = np.random.default_rng(9)
    n = 256 * 24 + 77
    g = (rng.standard_normal(n) * 10.0 ** rng.uniform(-44, 18, n)).astype(np.float32)
    g[256:512] = 0
    g[600] = np.inf
    g[900] = np.nan
    g[1300] = -np.inf
    g[256 * 24:] = 0
    for seed, eps in ((None, 1e-8), (3, 1e-8), (None, 0.0), (3, 0.0)):
        HP = dict(globals()["HP"], eps=eps)
        c = Case([n, 300], [g, np.zeros(300, np.float32)], zs.ZS_STATE_8BIT)
        for t in (1, 2, 3):
            zs.zs_adamw_multi(c.table, dict(step=t, **HP), seed=seed)
            c.step_oracle(O.AdamWHP(step=t, **HP), None, seed)
            c.check(f"step {t}, seed {seed}")


def test_adamw_multi_8bit_against_64_bits():
    """One step against the formula in float64. Nearest codes are off by at most half a
    step, 2^-4 of the value, or half a subnormal step 2^(s - K - 130); fp32 arithmetic
    adds at most 4 roundings (2^-22 relative for v, and of |B1 m| + |B1c g| for m)."""
    n = 100_003
    c = Case([n], grads_of([n], "f32", 4), zs.ZS_STATE_8BIT)
    m0 = F.state8_values(*c.m[0], F.M).astype(np.float64)
    v0 = F.state8_values(*c.v[0], F.V).astype(np.float64)
    p0, g = c.p[0].astype(np.float64), c.g[0].astype(np.float64)
    zs.zs_adamw_multi(c.table, dict(step=5, **HP))
    torch.cuda.synchronize()
    m1, v1 = 0.9 * m0 + 0.1 * g, 0.95 * v0 + 0.05 * g * g
    hat = (m1 / (1 - 0.9**5)) / (np.sqrt(v1 / (1 - 0.95**5)) + 1e-8)
    p1 = p0 * (1 - 3e-5) - 3e-4 * hat
    room = 2.0**-22 * (np.abs(p0) + 3e-4 * (np.abs(0.9 * m0) + np.abs(0.1 * g))
                       / (1 - 0.9**5) / (np.sqrt(v1 / (1 - 0.95**5)) + 1e-8) * 4)
    assert np.all(np.abs(to_np(c.dp.views[0]) - p1) <= room)
    for kind, codes, scales, want, size in (
            (F.M, c.dm, c.dms, m1, np.abs(0.9 * m0) + np.abs(0.1 * g)), (F.V, c.dv, c.dvs, v1, v1)):
        s = to_np(scales.views[0])
        got = F.state8_values(to_np(codes.views[0]), s, kind).astype(np.float64)
        sub = np.ldexp(1.0, np.repeat(s.astype(int), 256)[:n] - F.TOP[kind] - 130)
        sub = sub if kind == F.M else 2 * sub               # v: never 0, a whole step
        assert np.all(np.abs(got - want) <= 2.0**-4 * np.abs(want) + sub + 2.0**-22 * size)


def test_adamw_multi_large_and_many():
    """A tensor past 2^31 bytes of parameters beside small ones, and 5,000 tensors: the
    whole against zs_adamw_step, which the other tests hold to the oracle."""
    dev = device()
    sizes = [1 << 29, 7, 1_000_001]
    g = [W.normal_f32(n, 1e-3, 50 + i, dev) for i, n in enumerate(sizes)]
    p = [W.normal_f32(n, 0.02, 60 + i, dev) for i, n in enumerate(sizes)]
    m = [torch.zeros(n, device=dev) for n in sizes]
    v = [torch.zeros(n, device=dev) for n in sizes]
    w = [torch.zeros(n, dtype=torch.bfloat16, device=dev) for n in sizes]
    ref = [[x.clone() for x in y] for y in zip(p, m, v, w)]
    zs.zs_adamw_multi(zs.MultiTable(p, m, v, g, w), dict(step=1, **HP))
    for t in range(3):
        zs.zs_adamw_step(*ref[t], [g[t]], dict(step=1, **HP))
    torch.cuda.synchronize()
    for t in range(3):
        for a, b in zip(ref[t], (p[t], m[t], v[t], w[t])):
            assert torch.equal(a, b), t
    del p, m, v, w, g, ref
    rng = np.random.default_rng(6)
    sizes = [int(x) for x in np.exp(rng.uniform(0, 9, 5000))]
    n = sum(sizes)
    flat = [W.normal_f32(n, s, 70 + i, dev) for i, s in enumerate((0.02, 1e-4, 1e-3))]
    p, m, g = flat
    v, w = torch.zeros(n, device=dev), torch.zeros(n, dtype=torch.bfloat16, device=dev)
    ref = [x.clone() for x in (p, m, v, w)]
    table = zs.MultiTable(p.split(sizes), m.split(sizes), v.split(sizes), g.split(sizes),
                          w.split(sizes))
    zs.zs_adamw_multi(table, dict(step=7, **HP))
    zs.zs_adamw_step(*ref, [g], dict(step=7, **HP))
    torch.cuda.synchronize()
    for a, b in zip(ref, (p, m, v, w)):
        assert torch.equal(a, b)


def test_adamw_multi_8bit_past_32_bits():
    """A tensor of 2^32 + 5,000 elements (17 GB of p, 4 GB of each moment's codes):
    windows at its start, around element 2^31 and 2^32 and at its end against the oracle;
    p to the last bit (eps = 0 takes the exact operations), codes stochastic. The norm of
    its gradients, a repeated block of 2^20, against that block's."""
    dev = device()
    n = (1 << 32) + 5000
    block = W.as_bf16_bits(W.normal_f32(1 << 20, 1e-3, 77, dev))
    g = torch.empty(n, dtype=torch.int16, device=dev)
    whole = n >> 20
    g[:whole << 20].view(whole, 1 << 20).copy_(block)
    g[whole << 20:].copy_(block[:n - (whole << 20)])
    p = torch.full((n,), 0.01, device=dev)
    m = torch.randint(0, 256, (1 << 20,), dtype=torch.uint8, device=dev).repeat(whole + 1)[:n]
    v = torch.randint(0, 256, (1 << 20,), dtype=torch.uint8, device=dev).repeat(whole + 1)[:n]
    nb = -(-n // 256)
    ms, vs = (torch.full((nb,), x, dtype=torch.uint8, device=dev) for x in (117, 107))
    where = [(0, 4096), (1 << 31, 4096), ((1 << 32) - 2048, 4096), (n - n % 256 - 2048, 2048 + n % 256)]

    def window(a, k):
        b = slice(a // 256, -(-(a + k) // 256))
        return [to_np(x).copy() for x in (p[a:a + k], m[a:a + k], ms[b], v[a:a + k], vs[b], g[a:a + k])]

    before = [window(a, k) for a, k in where]
    table = zs.MultiTable([p], [m.contiguous()], [v], [g], None, [ms], [vs])
    m = table.tensors[1]
    hp = dict(HP, eps=0.0)
    zs.zs_adamw_multi(table, dict(step=4, **hp), seed=99)
    torch.cuda.synchronize()
    for (a, k), (p0, mc, m_s, vc, v_s, gg) in zip(where, before):
        with np.errstate(all="ignore"):
            want = F.adamw_step8(p0, mc, m_s, vc, v_s, O.bf16_widen(gg), O.AdamWHP(step=4, **hp), 99,
                                 0, a)
        got = window(a, k)
        check_f32(got[0], want[0], f"p at {a}", exact=True)
        for j, what in enumerate(("m codes", "m scales", "v codes", "v scales"), 1):
            check_bits(got[j], want[j], f"{what} at {a}")
    s, nc = norm_of(zs.MultiTable(grads=[g]))
    part = F.sumsq([O.bf16_widen(to_np(block))])
    tail = F.sumsq([O.bf16_widen(to_np(block[:n - (whole << 20)]))])
    assert abs(float(s) - (whole * part + tail)) <= n * 2.0**-53 * (whole * part + tail)


def test_adamw_multi_empty_and_side_stream():
    dev = device()
    zs.zs_adamw_multi(zs.MultiTable([], [], [], [], device=dev), dict(step=1, **HP))
    e = [torch.zeros(0, device=dev)]
    zs.zs_adamw_multi(zs.MultiTable(e, e, e, e), dict(step=1, **HP))
    sizes = [50_000, 33]
    c = Case(sizes, grads_of(sizes, "f32", 8), zs.ZS_STATE_8BIT)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        zs.zs_adamw_multi(c.table, dict(step=1, **HP))
    zs.zs_adamw_multi(c.table, dict(step=2, **HP), stream=side)
    side.synchronize()
    eager = Case(sizes, grads_of(sizes, "f32", 8), zs.ZS_STATE_8BIT)
    for t in (1, 2):
        zs.zs_adamw_multi(eager.table, dict(step=t, **HP))
        eager.step_oracle(O.AdamWHP(step=t, **HP))
    c.p, c.m, c.v, c.w = eager.p, eager.m, eager.v, eager.w
    c.check("side stream")


# ------------------------------------------------------------------ conversions
@pytest.mark.parametrize("kind", (F.M, F.V))
def test_decode_of_every_code_and_scale(kind):
    dev = device()
    codes = np.tile(np.arange(256, dtype=np.uint8), 256)
    scales = np.arange(256, dtype=np.uint8)
    want = F.state8_values(codes, scales, kind)
    dc, ds = torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev)
    out = torch.zeros(65536, device=dev)
    zs.zs_state8_decode(dc, ds, kind, out)
    check_f32(to_np(out), want, "fp32", exact=True)
    half = torch.zeros(65536, dtype=torch.bfloat16, device=dev)
    zs.zs_state8_decode(dc, ds, kind, half)
    check_bf16(to_np(half), O.bf16_round(want), "bf16", exact=True)
    ok = scales != 255                                  # and back: the same values
    c2, s2 = torch.zeros_like(dc), torch.zeros_like(ds)
    zs.zs_state8_encode(out, kind, c2, s2)
    back = F.state8_values(to_np(c2), to_np(s2), kind)
    keep = np.repeat(ok & (scales >= max(1, F.LEAST_SCALE[kind])), 256)
    check_f32(back[keep], want[keep], "again", exact=True)


@pytest.mark.parametrize("S", (1, 3, 255, 256, 257, 1021, 4096, 100_001))
@pytest.mark.parametrize("kind", (F.M, F.V))
def test_encode(kind, S):
    dev = device()
    rng = np.random.default_rng(S)
    x = (rng.standard_normal(S) * 10.0 ** rng.uniform(-45, 38, S)).astype(np.float32)
    if S > 1000:
        x[700] = np.nan
        x[:256] = (rng.standard_normal(256) * 1e-3).astype(np.float32)
        x[256:512] = 0
    if kind == F.V:
        x = np.abs(x)
        x[0] = -0.0
    codes, scales = F.state8_encode(x, kind)
    dx = Arena([x], torch.float32, dev)
    dc = Arena([np.zeros(S, np.uint8)], torch.uint8, dev)
    ds = Arena([np.zeros(scales.size, np.uint8)], torch.uint8, dev)
    zs.zs_state8_encode(dx.views[0], kind, dc.views[0], ds.views[0])
    check_bits(to_np(ds.views[0]), scales, "scales")
    check_bits(to_np(dc.views[0]), codes, "codes")
    for a in (dx, dc, ds):
        a.check_guards("encode")
    out = Arena([np.zeros(S, np.int16)], torch.int16, dev)
    zs.zs_state8_decode(dc.views[0], ds.views[0], kind, out.views[0])
    check_bf16(to_np(out.views[0]), O.bf16_round(F.state8_values(codes, scales, kind)), "back",
               exact=True)
    out.check_guards("decode")
    if kind == F.V and S > 1:
        x[1] = -1.0                                    # no second moment: the block is NaN
        zs.zs_state8_encode(torch.from_numpy(x).to(dev), kind, dc.views[0], ds.views[0])
        assert int(ds.views[0][0]) == 255


# ------------------------------------------------------------------ the norm
def norm_of(table, max_norm=1.0, ws=None):
    dev = device()
    s, nc = torch.full((1,), 5.0, dtype=torch.float64, device=dev), torch.full((2,), 5.0, device=dev)
    ws = torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device=dev) if ws is None else ws
    zs.zs_grad_norm(table, max_norm, s, nc, ws)
    return s, nc


def check_norm(s, nc, total, n, max_norm):
    s, nc = float(s), to_np(nc).astype(np.float64)
    rel = max(1, n) * 2.0**-53
    assert abs(s - total) <= rel * total
    norm, coef = F.clip_coef(total, max_norm)
    assert abs(nc[0] - float(norm)) <= (2.0**-23 + rel) * float(norm)
    assert abs(nc[1] - float(coef)) <= (2.0**-23 + rel) * float(coef)


@pytest.mark.parametrize("sizes", ([1], [5], [256], [4096], [4097], SIZES, [3_000_001], [17] * 3000))
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_grad_norm(dtype, sizes):
    g = grads_of(sizes, dtype, 11)
    a = Arena([bits16(x) for x in g], torch.int16 if dtype == "bf16" else torch.float32, device())
    table = zs.MultiTable(grads=a.views)
    total = F.sumsq([widen(x) for x in g])
    for max_norm in (1e-2, 1e6, math.inf):
        s, nc = norm_of(table, max_norm)
        check_norm(s, nc, total, sum(sizes), max_norm)
    ws = torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device=device())
    again = [norm_of(table, ws=ws)[0] for _ in range(20)]          # one workspace, call after call
    for s in again:
        assert torch.equal(s, norm_of(table)[0])                  # and the same order every time


@pytest.mark.parametrize("scale", (1e-30, 1e25))
def test_grad_norm_neither_over_nor_underflows(scale):
    g = grads_of([10_000], "f32", 12, scale)
    table = zs.MultiTable(grads=[torch.from_numpy(g[0]).to(device())])
    check_norm(*norm_of(table), F.sumsq(g), 10_000, 1.0)


def test_grad_norm_specials_and_empty():
    dev = device()
    g = torch.ones(5000, device=dev)
    table = zs.MultiTable(grads=[g])
    g[4999] = math.inf
    s, nc = norm_of(table)
    assert float(s) == math.inf and to_np(nc).tolist() == [math.inf, 0.0]
    assert float(norm_of(table, math.inf)[1][1]) == 1.0
    g[17] = math.nan
    s, nc = norm_of(table)
    assert math.isnan(float(s)) and np.isnan(to_np(nc)).all()
    for empty in (zs.MultiTable(grads=[], device=dev), zs.MultiTable(grads=[g[:0]])):
        s, nc = norm_of(empty)
        assert float(s) == 0 and to_np(nc).tolist() == [0.0, 1.0]


@pytest.mark.parametrize("D", (1, 3, 64))
def test_clip_coef_joins_ranks(D):
    dev = device()
    rng = np.random.default_rng(D)
    sums = rng.uniform(0.1, 5, D)
    dev_sums = [torch.tensor([x], dtype=torch.float64, device=dev) for x in sums]
    for max_norm in (0.5, 1e9):
        nc = torch.zeros(2, device=dev)
        zs.zs_clip_coef(dev_sums, max_norm, nc)
        total = 0.0
        for x in sums:
            total += x
        norm, coef = F.clip_coef(total, max_norm)
        # the kernel's root and quotient are correctly rounded in fp64 or one step off:
        # at most one step of the float apart
        assert abs(float(nc[0]) - norm) <= 2.0**-23 * norm
        assert abs(float(nc[1]) - coef) <= 2.0**-23 * coef


def test_refusals_on_the_device():
    dev = device()
    g = torch.zeros(100, device=dev)
    p, m, v = (torch.zeros(100, device=dev) for _ in range(3))
    for bad in (dict(p=[p], grads=[g]), dict(p=[p], m=[m], v=[v], grads=[g, g]),
                dict(p=[p], m=[m], v=[v], grads=[g], m_scale=[g]),
                dict(p=[p], m=[m[::2]], v=[v], grads=[g]), dict(p=[p], m=[m[:50]], v=[v], grads=[g]),
                dict(p=[p.double()], m=[m], v=[v], grads=[g])):
        with pytest.raises((ValueError, TypeError)):
            zs.MultiTable(**bad)
    with pytest.raises((ValueError, TypeError)):
        zs.MultiTable(grads=[g, g.bfloat16()])
    with pytest.raises(zs.ZsError) as e:
        zs.MultiTable([p], [p], [v], [g])
    assert e.value.status == zs.ZS_EALIAS
    table = zs.MultiTable([p], [m], [v], [g])
    for bad in (torch.zeros(2, device=dev), torch.zeros(1), torch.zeros(1, device=dev).double()):
        with pytest.raises(ValueError):
            zs.zs_adamw_multi(table, dict(step=1, **HP), grad_scale=bad)
    with pytest.raises(zs.ZsError):
        zs.zs_adamw_multi(table, dict(step=0, **HP))
    with pytest.raises(zs.ZsError):
        zs.zs_adamw_multi(zs.MultiTable(grads=[g]), dict(step=1, **HP))
    with pytest.raises(ValueError):
        norm_of(table, ws=torch.zeros(100, dtype=torch.uint8, device=dev))


# ------------------------------------------------------------------ together
def test_norm_clip_and_step_replayed_from_a_graph():
    """The run of a training step: two ranks' norms, the joined clip factor and the 8-bit
    step that reads it, captured once and replayed with new gradients, against the same
    calls made eagerly and against the oracle."""
    dev = device()
    sizes = [40_000, 1, 777, 5000]
    c = Case(sizes, grads_of(sizes, "bf16", 20, 0.05), zs.ZS_STATE_8BIT)
    e = Case(sizes, grads_of(sizes, "bf16", 20, 0.05), zs.ZS_STATE_8BIT)
    other = zs.MultiTable(grads=[torch.full((999,), 0.03, device=dev)])

    def buffers():
        return ([torch.zeros(1, dtype=torch.float64, device=dev) for _ in range(2)],
                torch.zeros(2, device=dev),
                [torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device=dev) for _ in range(2)])

    def pass_(case, b):
        sums, nc, ws = b
        zs.zs_grad_norm(case.table, 1.0, sums[0], nc, ws[0])
        zs.zs_grad_norm(other, 1.0, sums[1], nc, ws[1])
        zs.zs_clip_coef(sums, 1.0, nc)
        zs.zs_adamw_multi(case.table, dict(step=3, **HP), grad_scale=nc[1:], seed=42)

    gb, eb = buffers(), buffers()
    warm = Case(sizes, grads_of(sizes, "bf16", 20), zs.ZS_STATE_8BIT)
    pass_(warm, buffers())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        pass_(c, gb)
    c.w = [np.zeros(n, np.uint16) for n in sizes]
    c.check("capturing runs nothing")
    for rep in range(4):
        g = grads_of(sizes, "bf16", 30 + rep, 0.05)
        for case in (c, e):
            case.g = g
            for view, x in zip(case.dg.views, g):
                view.copy_(torch.from_numpy(bits16(x)).to(dev))
        graph.replay()
        pass_(e, eb)
        torch.cuda.synchronize()
        total = F.sumsq([widen(x) for x in g]) + F.sumsq([np.full(999, 0.03, np.float32)])
        check_norm(float(gb[0][0]) + float(gb[0][1]), gb[1], total,
                   sum(sizes) + 999, 1.0)
        assert torch.equal(gb[1], eb[1])
        c.step_oracle(O.AdamWHP(step=3, **HP), to_np(gb[1])[1], 42)
        e.p, e.m, e.v, e.w = c.p, c.m, c.v, c.w
        c.check(f"replay {rep}")
        e.check(f"eager {rep}")


def test_tables_on_streams_of_their_own_at_once():
    """Three tables' norm, clip factor and step enqueued together on three streams, each
    with its own workspace, several times over; then the same from three host threads."""
    import threading
    dev = device()
    sizes = [[60_000, 5], [4097] * 30, [123]]
    cases = [Case(s, grads_of(s, "bf16", 40 + i, 0.05), zs.ZS_STATE_F32) for i, s in enumerate(sizes)]
    outs = [(torch.zeros(1, dtype=torch.float64, device=dev), torch.zeros(2, device=dev),
             torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device=dev)) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()

    def enqueue(i, t):
        s, nc, ws = outs[i]
        zs.zs_grad_norm(cases[i].table, 0.5, s, nc, ws, stream=streams[i])
        zs.zs_adamw_multi(cases[i].table, dict(step=t, **HP), grad_scale=nc[1:], stream=streams[i])

    for t in (1, 2, 3):
        for i in range(3):
            enqueue(i, t)
    threads = [threading.Thread(target=lambda i=i: [enqueue(i, t) for t in (4, 5)]) for i in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        check_norm(outs[i][0], outs[i][1], F.sumsq([widen(x) for x in c.g]), sum(c.sizes), 0.5)
        for t in range(1, 6):
            c.step_oracle(O.AdamWHP(step=t, **HP), to_np(outs[i][1])[1])
        c.check(f"table {i}")


def test_two_graphs_of_one_table_and_workspace_in_turn():
    """Two captured norms that share a workspace, replayed one after the other with eager
    calls between: each leaves the workspace as the next one needs it."""
    dev = device()
    g = [torch.randn(n, device=dev) for n in (70_000, 3)]
    table = zs.MultiTable(grads=g)
    ws = torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device=dev)
    outs = [(torch.zeros(1, dtype=torch.float64, device=dev), torch.zeros(2, device=dev))
            for _ in range(2)]
    zs.zs_grad_norm(table, 1.0, *outs[0], ws)
    torch.cuda.synchronize()
    graphs = []
    for o in outs:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            zs.zs_grad_norm(table, 1.0, *o, ws)
        graphs.append(graph)
    for rep in range(3):
        for x in g:
            x.mul_(1.5)
        for graph in graphs:
            graph.replay()
        eager = norm_of(table, ws=ws)
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o[0], eager[0]) and torch.equal(o[1], eager[1])
        check_norm(*eager, F.sumsq([to_np(x) for x in g]), 70_003, 1.0)


def test_32bit_run_goes_on_in_8_bits_and_back():
    """A 32-bit run's moments encoded, stepped in 8 bits in one buffer laid out by
    zs_state8_layout, decoded and stepped in 32 bits again."""
    dev = device()
    sizes = [300, 5000, 1]
    c = Case(sizes, grads_of(sizes, "f32", 21), zs.ZS_STATE_F32)
    off = zs.zs_state8_layout(sizes)
    buf = {k: torch.zeros(off[-1], dtype=torch.uint8, device=dev) for k in "mv"}
    sc = {k: torch.zeros(off[-1] // 256, dtype=torch.uint8, device=dev) for k in "mv"}
    codes = {k: [buf[k][a:a + n] for a, n in zip(off, sizes)] for k in "mv"}
    scales = {k: [sc[k][a // 256:a // 256 - (-n // 256)] for a, n in zip(off, sizes)] for k in "mv"}
    for t in range(3):
        zs.zs_state8_encode(c.dm.views[t].clone(), zs.ZS_STATE8_M, codes["m"][t], scales["m"][t])
        zs.zs_state8_encode(c.dv.views[t].clone(), zs.ZS_STATE8_V, codes["v"][t], scales["v"][t])
    table = zs.MultiTable(c.dp.views, codes["m"], codes["v"], c.dg.views, c.dw.views, scales["m"],
                          scales["v"])
    zs.zs_adamw_multi(table, dict(step=2, **HP))
    torch.cuda.synchronize()
    after = [to_np(x).copy() for x in c.dp.views]
    flat = {k: torch.zeros(off[-1], device=dev) for k in "mv"}
    zs.zs_state8_decode(buf["m"], sc["m"], zs.ZS_STATE8_M, flat["m"])
    zs.zs_state8_decode(buf["v"], sc["v"], zs.ZS_STATE8_V, flat["v"])
    for t, (a, n) in enumerate(zip(off, sizes)):
        c.dm.views[t].copy_(flat["m"][a:a + n])
        c.dv.views[t].copy_(flat["v"][a:a + n])
    zs.zs_adamw_multi(c.table, dict(step=3, **HP))
    for t in range(3):
        p, mc, ms, vc, vs, _ = F.adamw_step8(c.p[t], *F.state8_encode(c.m[t], F.M),
                                             *F.state8_encode(c.v[t], F.V), c.g[t],
                                             O.AdamWHP(step=2, **HP))
        # p: the bound of Case.near is tested elsewhere; here a coarser one suffices
        assert np.abs(after[t] - p).max(initial=0) <= 2.0**-20 * np.abs(p).max(initial=0) + 1e-9
        c.p[t], c.m[t], c.v[t] = after[t], F.state8_values(mc, ms, F.M), F.state8_values(vc, vs, F.V)
    c.step_oracle(O.AdamWHP(step=3, **HP))
    c.check("32 -> 8 -> 32")
    gaps = torch.ones(off[-1], dtype=torch.bool, device=dev)
    for a, n in zip(off, sizes):
        gaps[a:a + n] = False
    for k in "mv":
        assert not flat[k][gaps].any() and not buf[k][gaps].any()
