"""One projection for the rows of many adapters, element by element against the FP64 definition.

The bound is the single-rounding design's (tests/gpu_util.py): with K the inner size and R the rank,
  |y - y*| <= ulp(|y*| + e) + e,   e = 2^-8 E + 4 (K + R + 16) 2^-24 S,
E the adapters' magnitude |s|(|X||A|^T)|B|^T (s X A^T is rounded once to bf16) and S the whole
magnitude sum of the element."""
import numpy as np
import pytest
import torch

import weight_patches_gb300 as wpg
from oracle import multi as om
from oracle import nf4 as onf4
from tests import gpu_util as gu
import workloads

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().double().cpu().numpy()


class Layer:
    def __init__(self, T, K, N, G, R, S, base="bf16", bias=False, seed=0, ldx=None, nan_pad=True):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        full = torch.full((T, ldx or K), float("nan") if nan_pad else 0.0, dtype=torch.bfloat16)
        full[:, :K] = n(T, K).bfloat16()
        self.X = full.to(gu.DEV)[:, :K]
        self.W = None
        if base == "bf16":
            self.W = (n(N, K) / K ** 0.5).bfloat16().to(gu.DEV)
            self.Wf = _f64(self.W)
        elif base == "nf4":
            w = workloads.draw_nf4(np.random.default_rng(seed), N, K)
            w.absmax[:] = w.absmax * np.float32(2.0 / K ** 0.5)
            self.W = gu.dev(w)
            self.Wf = onf4.dequant_f64(w.data, w.absmax, N, K)
        else:
            self.Wf = None
        self.bias = (n(N) * 0.2).to(torch.float32 if bias == "fp32" else torch.bfloat16).to(gu.DEV) if bias else None
        self.A = (n(S, G * R, K) / K ** 0.5).bfloat16().to(gu.DEV)
        self.B = (n(S, N, R) * 0.1).bfloat16().to(gu.DEV)
        self.scale = (torch.rand(S, generator=g) + 0.5).to(gu.DEV)
        self.row_scale = (torch.rand(T, generator=g) + 0.5).to(gu.DEV)
        self.T, self.K, self.N, self.G, self.R, self.S = T, K, N, G, R, S
        self.bank = wpg.AdapterBank(self.A, self.B, self.scale, G)

    def run(self, slot, rs=1.0, row_scale=True, **kw):
        slot_t = torch.tensor(slot, dtype=torch.int32, device=gu.DEV)
        y = wpg.lora_linear_fwd_multi(self.X, self.W, self.bias, self.bank, slot_t,
                                      row_scale=self.row_scale if row_scale else None, request_scale=rs, **kw)
        torch.cuda.synchronize()
        assert wpg.lora_device_status() == 0
        return y

    def check(self, slot, rs=1.0, row_scale=True, **kw):
        y = self.run(slot, rs, row_scale, **kw)
        s = om.row_scales(slot, _f64(self.scale), _f64(self.row_scale) if row_scale else None, rs)
        want, S, E = om.forward(_f64(self.X), self.Wf, None if self.bias is None else _f64(self.bias),
                                _f64(self.A), _f64(self.B), self.G, slot, s, self.N)
        e = 2.0 ** -8 * E + 4 * (self.K + self.R + 16) * 2.0 ** -24 * S
        ulp = gu.ulp_f32 if y.dtype == torch.float32 else gu.ulp_bf16
        gu.assert_elementwise(_f64(y), want, ulp(np.abs(want) + e) + e, "y")
        return y


def _slots(T, S, how, seed=0):
    rng = np.random.default_rng(seed)
    if how == "none":
        return [-1] * T
    if how == "one":
        return [S - 1] * T
    if how == "each":
        return [t % S for t in range(T)]
    if how == "runs":
        out = []
        while len(out) < T:
            out += [int(rng.integers(-1, S))] * int(rng.integers(1, 40))
        return out[:T]
    # any order, with rows without an adapter and values outside the bank
    return [int(v) for v in rng.choice([-1, -7, S, S + 1000, 2 ** 31 - 1, -2 ** 31] + list(range(S)) * 3, T)]


TOKENS = [1, 2, 3, 5, 8, 9, 16, 17, 33, 64, 65, 127, 128, 129, 200, 256, 257, 400, 513]


@pytest.mark.parametrize("how", ["none", "one", "each", "runs", "any"])
@pytest.mark.parametrize("T", TOKENS)
def test_rows_and_orders(T, how):
    Layer(T, 256, 272, 1, 16, 7, seed=T).check(_slots(T, 7, how, T), 0.7)


@pytest.mark.parametrize("base", ["bf16", "nf4", None])
@pytest.mark.parametrize("T", [1, 4, 6, 40, 64, 66, 140, 300])
@pytest.mark.parametrize("G,R", [(1, 8), (1, 24), (1, 64), (1, 72), (2, 16), (3, 32), (1, 256), (3, 128), (2, 40)])
def test_ranks_groups_and_weights(G, R, T, base):
    lay = Layer(T, 320, G * 136, G, R, 5, base=base, bias="bf16", seed=G * R + T)
    lay.check(_slots(T, 5, "any", T))


@pytest.mark.parametrize("base", ["bf16", "nf4"])
@pytest.mark.parametrize("T,K,N", [(1, 64, 8), (1, 2048, 1000), (3, 8192, 64), (5, 1536, 4608), (20, 5120, 640),
                                   (64, 4096, 328), (130, 1088, 2056), (700, 512, 520)])
def test_sizes(T, K, N, base):
    Layer(T, K, N, 1, 16, 9, base=base, bias="fp32", seed=K).check(_slots(T, 9, "any", K))


@pytest.mark.parametrize("K", [8, 72, 136, 200, 1544])
@pytest.mark.parametrize("T", [1, 30, 290])
def test_odd_inner_sizes_and_pitches(K, T):
    lay = Layer(T, K, 152, 1, 24, 4, seed=K, ldx=K + 24)
    out = torch.full((T + 2, 152 + 16), 7.0, dtype=torch.bfloat16, device=gu.DEV)
    y = lay.check(_slots(T, 4, "any", K), out=out[1:T + 1, 8:160])
    assert y.data_ptr() == out[1:, 8:].data_ptr()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:T + 1, 8:160] = False
    assert bool((out[keep] == 7.0).all())


@pytest.mark.parametrize("T", [1, 7, 100, 300])
@pytest.mark.parametrize("base", ["bf16", "nf4", None])
def test_fp32_output(T, base):
    Layer(T, 256, 264, 1, 16, 3, base=base, bias="fp32", seed=T).check(_slots(T, 3, "any"), out_dtype=torch.float32)


@pytest.mark.parametrize("T", [1, 4, 50, 290])
@pytest.mark.parametrize("base", ["bf16", "nf4"])
def test_rows_without_adapter_equal_the_plain_rows_of_any_batch(T, base):
    lay = Layer(T, 256, 256, 1, 16, 6, base=base, seed=3)
    plain = lay.run([-1] * T)
    slot = _slots(T, 6, "each")
    for i in range(0, T, 2):
        slot[i] = -1
    mixed = lay.run(slot)
    assert torch.equal(mixed[0::2], plain[0::2])
    # a scale of exactly zero is no adapter
    lay.row_scale.zero_()
    assert torch.equal(lay.run(_slots(T, 6, "each")), plain)


@pytest.mark.parametrize("T", [6, 60, 290])
def test_values_that_are_not_finite_stay_in_their_rows_and_slots(T):
    lay = Layer(T, 256, 256, 2, 16, 6, seed=4)
    slot = [t % 5 for t in range(T)]
    clean = lay.run(slot)
    lay.A[5] = float("nan")                         # a slot no row uses
    lay.B[5] = float("inf")
    lay.scale[5] = float("nan")
    assert torch.equal(lay.run(slot), clean)
    lay.A[2, 3, 7] = float("inf")                   # a slot some rows use
    lay.B[3, 100, 2] = float("nan")
    lay.X[4, 9] = float("nan")                      # a row (slot 4 or, when short, its own)
    got = lay.run(slot)
    hit = torch.tensor([t % 5 in (2, 3) or t == 4 for t in range(T)], device=gu.DEV)
    assert torch.equal(got[~hit], clean[~hit])
    assert bool(got[2].isnan().any() | got[2].isinf().any()) and bool(got[3, 100].isnan()) and bool(got[4].isnan().all())
    assert torch.equal(got[3, :100], clean[3, :100])


def test_one_slot_agrees_with_the_plain_adapter_call():
    lay = Layer(333, 512, 768, 3, 32, 2, seed=9)
    lay.row_scale.fill_(1.0)
    y = lay.run([1] * 333)
    ads = [wpg.Adapter(lay.A[1, g * 32:(g + 1) * 32].contiguous(), lay.B[1, g * 256:(g + 1) * 256].contiguous(),
                       32.0, float(lay.scale[1])) for g in range(3)]
    want = wpg.lora_linear_fwd_grouped(lay.X, lay.W, None, ads)
    assert (y.float() - want.float()).abs().max() <= 2 ** -6


def test_no_rows_other_stream_and_graph():
    lay = Layer(0, 64, 64, 1, 8, 2)
    assert lay.run([]).shape == (0, 64)
    for T in (3, 70, 300):
        lay = Layer(T, 512, 520, 1, 16, 6, seed=T)
        first, second = _slots(T, 6, "any", 1), _slots(T, 6, "runs", 2)
        want = [lay.run(first), lay.run(second)]
        slot = torch.tensor(first, dtype=torch.int32, device=gu.DEV)
        ws = torch.empty(wpg.lora_multi_workspace_size(lay.X, lay.W, lay.bank), dtype=torch.uint8, device=gu.DEV)
        out = torch.empty_like(want[0])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                wpg.lora_linear_fwd_multi(lay.X, lay.W, lay.bias, lay.bank, slot, row_scale=lay.row_scale, out=out,
                                          workspace=ws)
        torch.cuda.current_stream().wait_stream(s)
        for sl, w in zip((first, second), want):
            slot.copy_(torch.tensor(sl, dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w)
    assert wpg.lora_device_status() == 0


@pytest.mark.parametrize("T", [1, 8, 9, 17, 24, 25, 33, 41, 48, 49, 64, 65, 97, 128, 129, 200, 256])
@pytest.mark.parametrize("K,N,G,R", [(64, 72, 1, 8), (960, 216, 3, 24), (6464, 40, 1, 16), (512, 5136, 2, 32)])
def test_rows_over_a_4_bit_weight(K, N, G, R, T):
    lay = Layer(T, K, N, G, R, 6, base="nf4", bias="bf16", seed=K + T, ldx=K + 8)
    first = lay.check(_slots(T, 6, "any", K + T), 0.8)
    assert torch.equal(lay.run(_slots(T, 6, "any", K + T), 0.8), first)


@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("base", ["bf16", None])
@pytest.mark.parametrize("K,N,G,R", [(72, 128, 1, 64), (2048, 384, 3, 32), (1000, 216, 3, 8), (5120, 1152, 2, 64),
                                     (1536, 80, 5, 8), (328, 1000, 1, 24)])
def test_one_or_two_rows(K, N, G, R, base, T):
    lay = Layer(T, K, N, G, R, 4, base=base, bias="fp32", seed=K + R, ldx=K + 8)
    for slot in ([3, 0], [1, 1], [-1, 2], [2, 9], [-1, -1]):
        y = lay.check(slot[:T], 0.6)
        assert torch.equal(lay.run(slot[:T], 0.6), y)
    lay.check([0, 2][:T], 1.0, row_scale=False, out_dtype=torch.float32)


@pytest.mark.parametrize("T", [3, 4, 13, 16, 17, 31, 64, 90])
@pytest.mark.parametrize("base", ["bf16", "nf4", None])
@pytest.mark.parametrize("K,N,G,R", [(512, 1000, 1, 16), (1536, 120, 3, 8), (256, 48, 6, 16), (2048, 192, 8, 8)])
def test_rows_with_a_slot_each(K, N, G, R, base, T):
    lay = Layer(T, K, N, G, R, 100, base=base, bias="bf16", seed=N + T)
    slot = [int(v) for v in np.random.default_rng(T).permutation(100)[:T]]
    lay.check(slot, 0.9)
    for i in range(0, T, 3):
        slot[i] = -1
    lay.check(slot, 0.9)


@pytest.mark.parametrize("base", ["bf16", "nf4"])
def test_a_workspace_for_more_rows_serves_fewer(base):
    big = Layer(700, 512, 5136, 1, 16, 5, base=base, seed=1)
    size = wpg.lora_multi_workspace_size(big.X, big.W, big.bank)
    for T in (1, 64, 120, 300):
        lay = Layer(T, 512, 5136, 1, 16, 5, base=base, seed=T)
        lay.check(_slots(T, 5, "any", T), workspace=torch.empty(size, dtype=torch.uint8, device=gu.DEV))
