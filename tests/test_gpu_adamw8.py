"""GPU: AdamW with 8-bit states against its oracle, bit for bit.

Every operation of the update is one IEEE float32 operation, in the kernel and in
the oracle alike, so parameters, codes, scales, EMA and bf16 copies have to be
equal in every bit; the oracle's update is held against the float64 AdamW in
test_train_host.py.
"""

import numpy as np
import pytest

import oracle.adamw as oa
import oracle.adamw8 as o8
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

KW = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.01)


def _bf16(x):
    import torch
    return torch.from_numpy(x).to(torch.bfloat16)


def _same(got, want, what):
    got, want = np.ascontiguousarray(got), np.ascontiguousarray(want)
    u = {1: np.uint8, 2: np.uint16, 4: np.uint32}[got.dtype.itemsize]
    a, b = got.view(u), want.astype(got.dtype, copy=False).view(u)
    if got.dtype == np.float32:
        a, b = np.where(np.isnan(got), 0x7FC00000, a), np.where(np.isnan(want), 0x7FC00000, b)
    bad = np.nonzero(a != b)[0]
    assert bad.size == 0, f"{what}: {bad.size} of {a.size} differ, first at {bad[0]}: {got[bad[0]]} {want[bad[0]]}"


class Case:
    """One tensor: host arrays, device tensors (offset into a larger buffer), and the oracle's step."""

    def __init__(self, rng, n, *, q8=True, grad_bf16=False, ema=False, copy=False, offset=0, zero_state=False):
        import torch
        import muon_optimizer_step_amd as ms
        self.n = n
        self.p = (0.02 * rng.standard_normal(n)).astype(np.float32)
        self.g = (1e-3 * rng.standard_normal(n)).astype(np.float32)
        self.grad_bf16 = grad_bf16
        m = (3e-4 * rng.standard_normal(n)).astype(np.float32) * (not zero_state)
        r = (1e-3 * np.exp(rng.standard_normal(n))).astype(np.float32) * (not zero_state)
        self.q8 = q8
        near = np.full(n, 0x7FFFF, dtype=np.int64)
        self.state = (o8.encode(m, near, False), o8.encode(r, near, True)) if q8 else (m, r * r)
        self.ema = (0.02 * rng.standard_normal(n)).astype(np.float32) if ema else None

        def put(t):
            flat = torch.zeros(t.numel() + offset + 8, dtype=t.dtype, device="cuda") if t.dtype != torch.float8_e4m3fn else \
                torch.zeros(t.numel() + offset + 8, dtype=torch.uint8, device="cuda").view(t.dtype)
            v = flat[offset:offset + t.numel()]
            v.view(torch.uint8).copy_(t.view(torch.uint8)) if t.numel() else None
            return v

        f8 = lambda c: torch.from_numpy(c).view(torch.float8_e4m3fn)  # noqa: E731
        self.P = put(torch.from_numpy(self.p))
        self.G = put(_bf16(self.g) if grad_bf16 else torch.from_numpy(self.g))
        if grad_bf16:
            self.g = _bf16(self.g).float().numpy()
        if q8:
            (mc, ms_), (rc, rs) = self.state
            self.S = ms.AdamW8State(put(f8(mc)), put(torch.from_numpy(ms_)), put(f8(rc)), put(torch.from_numpy(rs)))
        else:
            self.S = (put(torch.from_numpy(self.state[0])), put(torch.from_numpy(self.state[1])))
        self.E = put(torch.from_numpy(self.ema)) if ema else None
        self.C = put(torch.zeros(n, dtype=torch.bfloat16)) if copy else None

    def step(self, place, **kw):
        self.p, self.state, self.ema = o8.step(self.p, self.g, self.state, place=place, ema=self.ema, **kw)

    def check(self, label):
        import torch
        _same(gu.host(self.P), self.p, f"{label} param")
        if self.q8:
            for t, want, what in ((self.S.exp_avg.view(torch.uint8), self.state[0][0], "exp_avg"),
                                  (self.S.exp_avg_scale, self.state[0][1], "exp_avg_scale"),
                                  (self.S.rms.view(torch.uint8), self.state[1][0], "rms"),
                                  (self.S.rms_scale, self.state[1][1], "rms_scale")):
                _same(gu.host(t), want, f"{label} {what}")
        else:
            _same(gu.host(self.S[0]), self.state[0], f"{label} m")
            _same(gu.host(self.S[1]), self.state[1], f"{label} v")
        if self.E is not None:
            _same(gu.host(self.E), self.ema, f"{label} ema")
        if self.C is not None:
            _same(gu.host(self.C.float()), _bf16(self.p).float().numpy(), f"{label} copy")


def _run(cases, steps=2, seed=None, kw=KW, t0=5):
    import torch
    import muon_optimizer_step_amd as ms
    decay = 0.9965
    call = ms.PreparedAdamW8([c.P for c in cases], [c.G for c in cases], [c.S for c in cases], emas=[c.E for c in cases],
                             copies=[c.C for c in cases])
    for t in range(t0, t0 + steps):
        call(lr=kw["lr"], betas=(kw["beta1"], kw["beta2"]), eps=kw["eps"], weight_decay=kw["wd"], step=t, seed=seed,
             ema_decay=decay)
        torch.cuda.synchronize()
        for i, c in enumerate(cases):
            c.step(i, t=t, seed=seed, decay=decay, **kw)
            c.check(f"step {t} tensor {i} ({c.n})")


@pytest.mark.parametrize("seed", [None, 12345678901])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_sizes_around_a_block_in_every_alignment(seed, offset):
    rng = np.random.default_rng(offset)
    sizes = [1, 3, 255, 256, 257, 511, 2047, 2048, 2049, 5000, 70001]
    gu.say(f"[adamw8] offset {offset}, seed {seed}")
    _run([Case(rng, n, offset=offset) for n in sizes], seed=seed)


@pytest.mark.parametrize("grad_bf16", [False, True])
@pytest.mark.parametrize("ema", [False, True])
@pytest.mark.parametrize("copy", [False, True])
def test_mixed_states_and_options(grad_bf16, ema, copy):
    rng = np.random.default_rng(7)
    cases = [Case(rng, n, q8=q8, grad_bf16=grad_bf16, ema=ema, copy=copy, offset=o)
             for n, q8, o in ((4096, True, 0), (4096, False, 0), (301, True, 2), (301, False, 3), (1, False, 0))]
    _run(cases, seed=3)


def test_more_tensors_than_a_launch_holds_and_empty_ones():
    rng = np.random.default_rng(8)
    sizes = [0, 92, 512, 0] + [int(k) for k in rng.integers(1, 3000, size=120)] + [0]
    cases = [Case(rng, n, q8=i % 3 != 0, ema=i % 2 == 0) for i, n in enumerate(sizes)]
    gu.say(f"[adamw8] {len(cases)} tensors")
    _run(cases, steps=1, seed=99)


@pytest.mark.parametrize("step,kw", [
    (1, KW), (1, dict(KW, beta1=0.0, beta2=0.0)), (100000, dict(KW, wd=0.0, eps=1e-3)), (3, dict(KW, lr=0.0)),
])
def test_hyperparameters(step, kw):
    rng = np.random.default_rng(9)
    _run([Case(rng, 3000, zero_state=step == 1), Case(rng, 300, q8=False, zero_state=step == 1)], steps=1, kw=kw, t0=step)


def test_values_at_the_ends_of_the_range():
    """Zero gradients and states, one value far above the rest of its block, tiny and huge values, NaN and infinity."""
    import torch
    rng = np.random.default_rng(10)
    c = Case(rng, 8 * 256, ema=True, copy=True)
    g = c.g.reshape(8, 256)
    g[0] = 0
    g[1, 5] = 1e6
    g[2] *= 1e-30
    g[3] = 1e-42                                  # subnormal
    g[4] *= 1e18
    g[5, 7] = np.nan
    g[6, 9] = np.inf
    c.G.copy_(torch.from_numpy(c.g))
    z = c.state
    for codes, scale in z:
        codes.reshape(8, 256)[[0, 2, 3]] = 0
        scale[[0, 2, 3]] = 0
    c.S.exp_avg.view(torch.uint8).copy_(torch.from_numpy(z[0][0]))
    c.S.rms.view(torch.uint8).copy_(torch.from_numpy(z[1][0]))
    c.S.exp_avg_scale.copy_(torch.from_numpy(z[0][1]))
    c.S.rms_scale.copy_(torch.from_numpy(z[1][1]))
    _run([c], steps=1)
    scale = gu.host(c.S.exp_avg_scale)
    assert np.isnan(scale[5]) and np.isnan(scale[6]) and np.isfinite(scale[[0, 1, 2, 3, 4, 7]]).all()
    rms = gu.host(c.S.rms.view(torch.uint8)).reshape(8, 256)
    assert (rms[0] == 0).all() and (rms[1] > 0).all()       # a second moment above zero keeps a code above zero


def test_stochastic_rounding_keeps_small_decay_on_the_average():
    """A second moment that decays by 0.1 % a step under a block maximum that stays: far below a code's step.

    r = sqrt(v) falls by 0.05 % a step in codes 6-12 % apart.  Stochastic rounding moves a value with
    probability ~0.008 by one code, a variance of ~4e-5 of r^2 a step: 200 steps give a deviation of 0.09, the mean of
    65280 values 4e-4; 1 % is 28 of them.  Nearest rounding never leaves the first code.
    """
    import torch
    import muon_optimizer_step_amd as ms
    n = 256 * 256
    v0 = np.full(n, 0.25, dtype=np.float32)
    v0[::256] = 1.0
    g = np.zeros(n, dtype=np.float32)
    steps = 200
    g[::256] = 1.0                                            # keeps the block's largest at 1
    mean = {}
    for seed in (None, 5):
        P, G = torch.zeros(n, device="cuda"), gu.dev(g)
        s = ms.AdamW8State.from_moments(torch.zeros(n, device="cuda"), gu.dev(v0))
        call = ms.PreparedAdamW8([P], [G], [s])
        for t in range(1, steps + 1):
            call(lr=0.0, weight_decay=0.0, step=t, seed=seed)
        v = gu.host(s.moments()[1]).reshape(256, 256)
        mean[seed] = float(np.sqrt(v[:, 1:]).mean())
    want = 0.5 * 0.999 ** (steps / 2)
    gu.say(f"[adamw8] mean sqrt(v) after {steps} steps: stochastic {mean[5]:.4f}, nearest {mean[None]:.4f}, exact {want:.4f}")
    assert abs(mean[5] - want) <= 0.01 * want
    assert abs(mean[None] - 0.5) <= 0.02 * 0.5


def test_every_bit_of_the_seed_counts():
    import torch
    import muon_optimizer_step_amd as ms
    n = 4096
    rng = np.random.default_rng(16)
    p, g = rng.standard_normal(n).astype(np.float32), gu.dev(rng.standard_normal(n).astype(np.float32))
    seen = []
    for seed in [7] + [7 ^ (1 << b) for b in range(64)] + [-7]:
        s = ms.AdamW8State.zeros_like(g)
        ms.adamw8_step([gu.dev(p)], [g], [s], lr=1e-3, step=1, seed=seed)
        seen.append((s.exp_avg.view(torch.uint8), s.rms.view(torch.uint8)))
    for i, a in enumerate(seen):
        for b in seen[:i]:
            assert not torch.equal(a[0], b[0]) and not torch.equal(a[1], b[1])


@pytest.mark.parametrize("n", [1, 255, 256, 1000, 70000])
def test_conversion_from_and_to_float32_moments(n):
    import torch
    import muon_optimizer_step_amd as ms
    rng = np.random.default_rng(n)
    m = (rng.standard_normal(n) * np.exp(rng.standard_normal(n))).astype(np.float32)
    v = np.square(rng.standard_normal(n)).astype(np.float32)
    s = ms.AdamW8State.from_moments(gu.dev(m), gu.dev(v))
    near = np.full(n, 0x7FFFF, dtype=np.int64)
    (mc, msc), (rc, rsc) = o8.encode(m, near, False), o8.encode(np.sqrt(v), near, True)
    _same(gu.host(s.exp_avg.view(torch.uint8)), mc, "exp_avg codes")
    _same(gu.host(s.exp_avg_scale), msc, "exp_avg scale")
    _same(gu.host(s.rms.view(torch.uint8)), rc, "rms codes")
    _same(gu.host(s.rms_scale), rsc, "rms scale")
    m2, v2 = (gu.host(x) for x in s.moments())
    _same(m2, o8.decode(mc, msc), "moments m")
    # half a code's step is 1/16 of the value, or half of 2^-9 scales
    blocks = lambda x: np.repeat(x, 256)[:n]  # noqa: E731
    assert (np.abs(m2 - m) <= np.maximum(np.abs(m) / 16, blocks(msc) * 2.0 ** -10) * 1.001).all()
    r, r2 = np.sqrt(v), np.sqrt(v2)
    assert (np.abs(r2 - r) <= np.maximum(r / 16, blocks(rsc) * 2.0 ** -9) * 1.001).all()


def test_training_with_8_bit_states_follows_32_bit_states():
    """400 steps of least squares: the 8-bit run ends as low as the 32-bit one within a factor of two."""
    import torch
    import muon_optimizer_step_amd as ms
    rng = np.random.default_rng(2)
    a, x0 = gu.dev(rng.standard_normal((2048, 512)).astype(np.float32)), gu.dev(rng.standard_normal((512, 64)).astype(np.float32))
    y = a @ x0
    last = {}
    for q8 in (False, True):
        x = torch.zeros(512, 64, device="cuda")
        s = ms.AdamW8State.zeros_like(x) if q8 else (torch.zeros_like(x), torch.zeros_like(x))
        g = torch.empty_like(x)
        call = ms.PreparedAdamW8([x], [g], [s])
        for t in range(1, 401):
            g.copy_(a.T @ (a @ x - y) / 2048)
            call(lr=0.02, weight_decay=0.0, step=t, seed=1)
        last[q8] = float(((a @ x - y) ** 2).mean())
    start = float((y ** 2).mean())
    gu.say(f"[adamw8] mean square error {start:.3g} -> 32-bit {last[False]:.3g}, 8-bit {last[True]:.3g}")
    assert last[False] < 1e-2 * start and last[True] < 2 * last[False] + 1e-3 * start


def test_on_another_stream_and_in_a_graph():
    import torch
    import muon_optimizer_step_amd as ms
    rng = np.random.default_rng(4)
    a, b = Case(rng, 5000, ema=True, copy=True), None
    b = Case(np.random.default_rng(4), 5000, ema=True, copy=True)
    run = lambda c, stream=None: ms.adamw8_step([c.P], [c.G], [c.S], lr=1e-3, step=9, seed=2, emas=[c.E], copies=[c.C],  # noqa: E731
                                                ema_decay=0.99, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(a, side)
    torch.cuda.current_stream().wait_stream(side)
    run(b)
    torch.cuda.synchronize()
    eq = lambda: all(bool((x.view(torch.uint8) == y.view(torch.uint8)).all()) for x, y in (  # noqa: E731
        (a.P, b.P), (a.S.exp_avg, b.S.exp_avg), (a.S.rms, b.S.rms), (a.S.rms_scale, b.S.rms_scale), (a.E, b.E), (a.C, b.C)))
    assert eq()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(a)
    for _ in range(3):
        g.replay()
        run(b)
        float(torch.randn(1 << 16, device="cuda").sum())
        torch.cuda.synchronize()
        assert eq()


def test_binding_refusals():
    import torch
    import muon_optimizer_step_amd as ms
    x = torch.zeros(512, device="cuda")
    s = ms.AdamW8State.zeros_like(x)
    with pytest.raises(TypeError, match="pair"):
        ms.PreparedAdamW8([x], [x.clone()], [3])
    with pytest.raises(ValueError, match="elements"):
        ms.PreparedAdamW8([x], [x.clone()], [ms.AdamW8State.zeros_like(x[:256])])
    with pytest.raises(TypeError, match="grads"):
        ms.PreparedAdamW8([x], [x.half()], [s])
    with pytest.raises(ValueError, match="contiguous"):
        ms.PreparedAdamW8([x[::2]], [x[::2].clone()], [s])
    with pytest.raises(ValueError, match="elements"):
        ms.AdamW8State(s.exp_avg, s.exp_avg_scale[:1], s.rms, s.rms_scale)
    with pytest.raises(ms.MuonError) as e:
        ms.adamw8_step([x], [x], [s], lr=1e-3, step=1)
    assert e.value.code == ms._lib.MUON_ERR_UNSUPPORTED       # the gradient is the parameter itself
    with pytest.raises(ms.MuonError):
        ms.adamw8_step([x], [x.clone()], [s], lr=1e-3, step=0)


def test_one_step_against_the_float64_formula():
    rng = np.random.default_rng(6)
    c = Case(rng, 100000, grad_bf16=True)
    m, r = o8.decode(*c.state[0]), o8.decode(*c.state[1])
    p0 = c.p.copy()
    import torch
    import muon_optimizer_step_amd as ms
    ms.adamw8_step([c.P], [c.G], [c.S], lr=1e-3, weight_decay=0.01, step=50)
    torch.cuda.synchronize()
    f = gu.f32
    want, _, _ = oa.adamw_update(p0, c.g, m, r.astype(np.float64) ** 2, lr=f(1e-3), beta1=f(0.9), beta2=f(0.999), eps=f(1e-8),
                                 wd=f(0.01), step=50)
    assert gu.rel_max(gu.host(c.P), want) <= gu.ELEM_TOL
