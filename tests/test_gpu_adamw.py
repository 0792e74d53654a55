"""The AdamW step over many tensors: 32-bit moments within float32 roundings of the FP64
definition, 8-bit moments equal to the float32 sequence's codes bit for bit.

u = 2^-24.  m and v: each scalar is rounded once, and there are at most four further roundings:
5u of the terms' magnitudes.  p: the kernel's sqrt and quotient are within 2 ulp, the scalars
within u each; v's relative error halves under the root (all its terms are positive): 24 u of
lr/(1-b1^t) |m|/den covers them, with m's own error over den, and 3u of |p|."""
import numpy as np
import pytest
import torch

import weight_patches_gb300 as wpg
from oracle import adamw as oa
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def _rand(n, seed, std=1.0):
    return torch.randn(n, generator=torch.Generator().manual_seed(seed)) * std


def _f64(t):
    return t.detach().double().cpu().numpy()


class Set:
    """Tensors of given sizes, cut (with an optional odd offset) out of one buffer with canaries."""

    def __init__(self, sizes, param, bits, grad=torch.float32, seed=0, gap=256, off=0):
        self.sizes, self.bits = sizes, bits
        total = sum(-(-n // 256) * 256 + gap for n in sizes) + off + 256
        self.p = torch.full((total,), 3.0, dtype=torch.float32 if param == "fp32" else torch.bfloat16)
        self.master = torch.full((total,), 3.0) if param == "master" else None
        self.g = torch.full((total,), 3.0, dtype=grad)
        self.used = torch.zeros(total, dtype=torch.bool)
        self.spans = []
        at = gap + off
        m, v = torch.full((total,), 3.0), torch.full((total,), 3.0)
        for i, n in enumerate(sizes):
            s = slice(at, at + n)
            w = _rand(n, seed + 10 * i, 0.05)
            self.p[s] = w.to(self.p.dtype)
            if self.master is not None:
                self.master[s] = w
            size = torch.exp(_rand(n, seed + 10 * i + 1, 1.5) - 4)
            self.g[s] = (_rand(n, seed + 10 * i + 2) * size).to(grad)
            m[s] = _rand(n, seed + 10 * i + 3, 0.3) * size
            v[s] = (torch.rand(n, generator=torch.Generator().manual_seed(seed + 10 * i + 4)) + 0.1) * size * size
            self.used[s] = True
            self.spans.append(s)
            at += -(-n // 256) * 256 + gap
        for k in ("p", "master", "g"):
            t = getattr(self, k)
            setattr(self, k, None if t is None else t.to(gu.DEV))
        if bits == 32:
            self.m, self.v = m.to(gu.DEV), v.to(gu.DEV)
            self.ml, self.vl = [self.m[s] for s in self.spans], [self.v[s] for s in self.spans]
        else:
            self.ml, self.vl = [], []
            for s in self.spans:
                for t, signed, lst in ((m, True, self.ml), (v, False, self.vl)):
                    q, top = oa.encode(t[s].numpy(), signed)
                    lst.append(wpg.Block8(torch.from_numpy(q.copy()).to(gu.DEV), torch.from_numpy(top.copy()).to(gu.DEV)))
        self.cut = lambda t: None if t is None else [t[s] for s in self.spans]
        self.plan = wpg.lora_adamw_plan(self.cut(self.p), self.ml, self.vl, masters=self.cut(self.master))

    def snapshot(self):
        c = lambda t: None if t is None else t.clone()  # noqa: E731
        if self.bits == 32:
            st = [(self.ml[i].clone(), self.vl[i].clone()) for i in range(len(self.sizes))]
        else:
            st = [tuple(x.clone() for x in (a.codes, a.absmax, b.codes, b.absmax)) for a, b in zip(self.ml, self.vl)]
        return c(self.p), c(self.master), st


def _check(s, before, t, grad_scale=1.0, skip=()):
    p0, ma0, st0 = before
    assert torch.equal(s.p[~s.used], p0[~s.used])
    if s.master is not None:
        assert torch.equal(s.master[~s.used], ma0[~s.used])
    for i, sp in enumerate(s.spans):
        if s.sizes[i] == 0:
            continue
        if i in skip:
            assert torch.equal(s.p[sp], p0[sp])
            now = (s.ml[i], s.vl[i]) if s.bits == 32 else (s.ml[i].codes, s.ml[i].absmax, s.vl[i].codes, s.vl[i].absmax)
            assert all(torch.equal(a, b) for a, b in zip(now, st0[i]))
            continue
        g = _f64(s.g[sp])
        if s.bits == 32:
            m0, v0 = _f64(st0[i][0]), _f64(st0[i][1])
        else:
            c = [x.cpu().numpy() for x in st0[i]]
            m0, v0 = oa.decode(c[0], c[1], True), oa.decode(c[2], c[3], False)
            mf, vf = oa.moments_f32(g.astype(np.float32), m0, v0, HYPER["beta1"], HYPER["beta2"], grad_scale)
            for lst, val, signed in ((s.ml, mf, True), (s.vl, vf, False)):
                q, top = oa.encode(val, signed)
                assert np.array_equal(lst[i].absmax.cpu().numpy().view(np.uint32), top.view(np.uint32))
                assert np.array_equal(lst[i].codes.cpu().numpy(), q)
        src = (p0 if ma0 is None else ma0)[sp]
        P = _f64(src)
        want, wm, wv = oa.step(P, g, m0, v0, HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"],
                               HYPER["weight_decay"], t, grad_scale)
        gs = np.abs(g * grad_scale)
        em = 5 * U * (HYPER["beta1"] * np.abs(m0) + (1 - HYPER["beta1"]) * gs) + 2.0 ** -149
        if s.bits == 32:
            gu.assert_elementwise(_f64(s.ml[i]), wm, em, "m")
            gu.assert_elementwise(_f64(s.vl[i]), wv, 6 * U * wv + 2.0 ** -147, "v")
        den = np.sqrt(wv) / np.sqrt(1 - HYPER["beta2"] ** t) + HYPER["eps"]
        a = HYPER["lr"] / (1 - HYPER["beta1"] ** t)
        e = 3 * U * np.abs(P) + a * (em + 24 * U * np.abs(wm)) / den
        if s.master is not None:
            gu.assert_elementwise(_f64(s.master[sp]), want, e + gu.ulp_f32(want), "master")
            assert torch.equal(s.p[sp], s.master[sp].to(torch.bfloat16))
        else:
            ulp = gu.ulp_f32(np.abs(want) + e) if s.p.dtype == torch.float32 else gu.ulp_bf16(np.abs(want) + e)
            gu.assert_elementwise(_f64(s.p[sp]), want, e + ulp, "p")


SIZES = [[1], [7, 8, 9], [255, 256, 257, 2047, 2048, 2049], [5000, 1, 33000, 12288]]


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("param", ["fp32", "bf16", "master"])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("sizes", SIZES)
def test_step(sizes, bits, param, grad):
    s = Set(sizes, param, bits, grad)
    for t, gs in ((1, 1.0), (2, 0.37), (1000, 1.0)):
        before = s.snapshot()
        wpg.lora_adamw_step(s.plan, s.cut(s.g), step=t, grad_scale=gs, **HYPER)
        _check(s, before, t, gs)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("off", [1, 2, 5])
def test_unaligned_views(bits, off):
    s = Set([700, 2049, 31], "master", bits, torch.bfloat16, off=off)
    before = s.snapshot()
    wpg.lora_adamw_step(s.plan, s.cut(s.g), step=3, **HYPER)
    _check(s, before, 3)


def test_many_tensors_cross_the_launch_and_table_batches():
    s = Set([3 + i % 40 for i in range(4100)], "fp32", 32, gap=0)
    before = s.snapshot()
    wpg.lora_adamw_step(s.plan, s.cut(s.g), step=5, **HYPER)
    p0, _, st0 = before
    assert torch.equal(s.p[~s.used], p0[~s.used])
    for i in (0, 1, 399, 400, 401, 3898, 3899, 3900, 3901, 4099):
        want, _, _ = oa.step(_f64(p0[s.spans[i]]), _f64(s.g[s.spans[i]]), _f64(st0[i][0]), _f64(st0[i][1]),
                             HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], HYPER["weight_decay"], 5)
        assert np.abs(_f64(s.p[s.spans[i]]) - want).max() < 1e-6
    changed = (s.p[s.used] != p0[s.used]).float().mean()
    assert float(changed) > 0.99


def test_missing_gradients_empty_tensors_and_device_scale():
    s = Set([300, 0, 5000, 77], "master", 8)
    grads = s.cut(s.g)
    grads[0] = grads[3] = None
    before = s.snapshot()
    scale = torch.tensor([0.25], device=gu.DEV)
    wpg.lora_adamw_step(s.plan, grads, step=2, grad_scale=0.5, grad_scale_tensor=scale, **HYPER)
    _check(s, before, 2, 0.125, skip=(0, 3))
    before = s.snapshot()
    wpg.lora_adamw_step(s.plan, [None] * 4, step=3, **HYPER)
    _check(s, before, 3, skip=(0, 1, 2, 3))


def test_zero_state_zero_gradient():
    p = torch.ones(600, device=gu.DEV)
    m, v = wpg.Block8.zeros(600, True, gu.DEV), wpg.Block8.zeros(600, False, gu.DEV)
    plan = wpg.lora_adamw_plan([p], [m], [v])
    wpg.lora_adamw_step(plan, [torch.zeros(600, device=gu.DEV)], lr=0.1, weight_decay=0.5, step=1)
    assert torch.equal(p, torch.full_like(p, float(np.float32(1 - 0.05))))
    assert int(m.codes.abs().sum()) == 0 and int(v.codes.sum()) == 0 and float(v.absmax.sum()) == 0


def test_gradients_that_are_not_finite_show():
    for bad in (float("nan"), float("inf")):
        p = torch.ones(1024, device=gu.DEV)
        m, v = wpg.Block8.zeros(1024, True, gu.DEV), wpg.Block8.zeros(1024, False, gu.DEV)
        plan = wpg.lora_adamw_plan([p], [m], [v])
        g = torch.full((1024,), 0.5, device=gu.DEV)
        g[300] = bad
        wpg.lora_adamw_step(plan, [g], lr=0.1, step=1)
        assert bool(p[300].isnan()) and int(p.isnan().sum()) == 1
        vm, vv = wpg.lora_block8_decode(m.codes, m.absmax), wpg.lora_block8_decode(v.codes, v.absmax)
        for x in (vm, vv):
            assert not bool(x[256:512].isfinite().any()) and bool(x[:256].isfinite().all() and x[512:].isfinite().all())


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-8, 1.0, 1e8, 1e19])
def test_codes_over_the_whole_range(scale):
    """Blocks of every magnitude, with values on and next to the boundaries between codes."""
    rng = np.random.default_rng(5)
    q = rng.integers(0, 255, 4096) + 0.5
    edge = np.nextafter(np.float32(1), np.float32(2)) - 1
    v = np.float32(scale) * ((q / 255) ** 4 * (1 + edge * rng.integers(-3, 4, 4096))).astype(np.float32)
    m = np.float32(scale) * ((q / 255) ** 2 * (1 + edge * rng.integers(-3, 4, 4096))).astype(np.float32) \
        * rng.choice([-1, 1], 4096).astype(np.float32)
    m[::256] = v[::256] = np.float32(scale)
    # beta 0: the moments are the gradient and its square
    g = np.sqrt(v) if scale < 1e10 else m
    s32 = torch.from_numpy(g.astype(np.float32)).to(gu.DEV)
    p = torch.zeros(4096, device=gu.DEV)
    mq, vq = wpg.Block8.zeros(4096, True, gu.DEV), wpg.Block8.zeros(4096, False, gu.DEV)
    plan = wpg.lora_adamw_plan([p], [mq], [vq])
    for grad in (s32, torch.from_numpy(m.astype(np.float32)).to(gu.DEV)):
        wpg.lora_adamw_step(plan, [grad], lr=1e-3, beta1=0.0, beta2=0.0, step=1)
        gn = grad.cpu().numpy()
        with np.errstate(over="ignore"):
            mf, vf = oa.moments_f32(gn, np.zeros(4096, np.float32), np.zeros(4096, np.float32), 0.0, 0.0, 1.0)
        for got, val, signed in ((mq, mf, True), (vq, vf, False)):
            want, top = oa.encode(val, signed)
            assert np.array_equal(got.absmax.cpu().numpy(), top)
            assert np.array_equal(got.codes.cpu().numpy(), want)


def test_decode_every_code():
    for dt, signed in ((torch.int8, True), (torch.uint8, False)):
        q = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(dt).repeat(5)[:1100].contiguous().to(gu.DEV)
        if signed:
            q = q.clamp(min=-127)
        top = torch.tensor([1.0, 3e-20, 7.5, 0.0, 2e30], device=gu.DEV)
        got = wpg.lora_block8_decode(q, top).cpu().numpy()
        want = oa.decode(q.cpu().numpy(), top.cpu().numpy(), signed)
        assert np.array_equal(got.view(np.uint32) & 0x7fffffff, want.view(np.uint32) & 0x7fffffff)
        assert np.array_equal(got, want)
        assert np.array_equal(wpg.lora_block8_decode(q[3:1001].contiguous()[:513], top[:3]).cpu().numpy(),
                              oa.decode(q[3:516].cpu().numpy(), top[:3].cpu().numpy(), signed))


def test_captured_in_a_graph():
    a, b = Set([3000, 129], "master", 8, seed=7), Set([3000, 129], "master", 8, seed=7)
    scale = torch.ones(1, device=gu.DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            wpg.lora_adamw_step(a.plan, a.cut(a.g), step=4, grad_scale_tensor=scale, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    for f in (1.0, 0.5):
        scale.fill_(f)
        graph.replay()
        wpg.lora_adamw_step(b.plan, b.cut(b.g), step=4, grad_scale=f, **HYPER)
    torch.cuda.synchronize()
    assert torch.equal(a.p, b.p) and torch.equal(a.ml[0].codes, b.ml[0].codes) and torch.equal(a.vl[1].codes, b.vl[1].codes)
