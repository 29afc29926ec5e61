"""The linear layer (product, bias, activation, gating, residual in one
launch) against its formula in 64 bits on the oracle's unpacked weights, on
every rung, both activation layouts and both output layouts."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import quantized_weight_prefill_amd as qg
from quantized_weight_prefill_amd import synth
from tests.ffn_ref import assert_within, bits, bits64, linear64
from tests.helpers import bytes_to_device, to_device

pytestmark = pytest.mark.gpu

NAMES = [qg.rung_name(r) for r in range(qg.num_rungs())]
ACTS = list(qg.ACTS)


class Problem:
    """Seeded inputs of one linear layer, weights scaled so that outputs are
    of the size of a few units."""

    def __init__(self, fmt, M, N, K, dtype, seed, gated=False, group=64, zp=True):
        self.fmt, self.M, self.N, self.K, self.dtype, self.gated = fmt, M, N, K, dtype, gated
        self.group, self.zp = (group, zp) if fmt == "w4a16" else (0, False)
        nt = 2 * N if gated else N
        rx, rw, rb = synth.streams(seed, 3)
        f = synth.weight_fields(fmt, rw, nt, K, group, not zp)
        scale = 1.0 / (np.sqrt(K) * {"q4k": 1.5, "q6k": 7.0, "w4a16": 0.04}[fmt])
        for key in ("d", "dmin", "scales"):
            if key in f:
                f[key] = synth.f16_bits(f[key].view(np.float16).astype(np.float64) * scale)
        enc = synth.encode(fmt, f)
        self.X = synth.activations(rx, M, K, dtype)
        self.bias_bits = synth.activations(rb, 1, nt, dtype)[0]
        self.res_bits = synth.activations(rb, M, N, dtype)
        self.x, self.wp = to_device(self.X, dtype), bytes_to_device(qg.pack(fmt, enc, nt, K))
        self.bias, self.res = to_device(self.bias_bits, dtype), to_device(self.res_bits, dtype)
        self.x64, self.w64 = bits64(self.X, dtype), bits64(oracle.dequant(fmt, enc, nt, K, dtype), dtype)

    def want(self, bias, res, act):
        return linear64(self.x64, self.w64, self.N, bits64(self.bias_bits, self.dtype) if bias else None,
                        bits64(self.res_bits, self.dtype) if res else None, act, self.gated)

    def run(self, layout, bias=False, res=False, act="none", **kw):
        kw = dict(bias=self.bias if bias else None, residual=self.res if res else None, act=act, gated=self.gated,
                  group=self.group, has_zp=self.zp, **kw)
        if layout == qg.X_FRAG:
            return qg.linear_xf(self.fmt, qg.x_to_xf(self.x), self.wp, self.M, self.N, self.K, **kw)
        return qg.linear(self.fmt, self.x, self.wp, self.N, **kw)


def frag(y):
    """Fragment-major copy of y by the library's own copy kernel."""
    return qg.x_to_xf(y.contiguous())


@pytest.mark.parametrize("layout", [qg.X_ROW, qg.X_FRAG], ids=["row", "xf"])
@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["q4k", "q6k", "w4a16"])
def test_every_rung(fmt, dtype, layout):
    """Plain and gated on each rung, the epilogue's parts in turn; Y without
    an epilogue has the product's bits, and the fragment-major Y those of the
    row-major one."""
    K = 1024
    for n, (M, N) in enumerate(((37, 256), (70, 130))):
        p = Problem(fmt, M, N, K, dtype, 300 + n)
        xf = qg.x_to_xf(p.x)
        for r, name in enumerate(NAMES):
            if layout == qg.X_FRAG:
                plain = qg.gemm_xf(fmt, xf, p.wp, M, N, K, group=p.group, has_zp=p.zp, rung=r)
            else:
                plain = qg.gemm_rung(fmt, r, p.x, p.wp, N, group=p.group, has_zp=p.zp)
            assert torch.equal(bits(p.run(layout, rung=r)), bits(plain)), name
            bias, res, act = bool((r + n) & 1), bool((r + n) & 2) or r % 3 == 0, ACTS[(r + n) % 5]
            y = p.run(layout, bias, res, act, rung=r)
            assert_within(y, *p.want(bias, res, act), dtype, f"{fmt} {name} {M}x{N} {act} bias={bias} res={res}")
            if N % 128 == 0:
                yf = p.run(layout, bias, res, act, rung=r, out_layout=qg.X_FRAG)
                assert torch.equal(bits(yf), bits(frag(y))), name
    for n, (M, N) in enumerate(((37, 128), (70, 80), (5, 16))):
        p = Problem(fmt, M, N, K, dtype, 310 + n, gated=True)
        for r, name in enumerate(NAMES):
            if name.endswith("-sk"):
                continue
            bias, res, act = bool((r + n) & 1), bool((r + n) & 2), ACTS[(r + 2 + n) % 5]
            y = p.run(layout, bias, res, act, rung=r)
            assert_within(y, *p.want(bias, res, act), dtype, f"gated {fmt} {name} {M}x{N} {act} bias={bias} res={res}")
            if N % 128 == 0:
                yf = p.run(layout, bias, res, act, rung=r, out_layout=qg.X_FRAG)
                assert torch.equal(bits(yf), bits(frag(y))), name


@pytest.mark.parametrize("fmt,M,N,K", [("q4k", 1, 1, 256), ("q6k", 1, 33, 512), ("w4a16", 3, 50, 128), ("q4k", 16, 4, 768),
                                       ("w4a16", 33, 97, 384), ("q6k", 129, 18, 256), ("q4k", 300, 515, 512)])
@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16], ids=["f16", "bf16"])
def test_odd_sizes(fmt, M, N, K, dtype):
    """The ladder's own choice at widths that fill no panel or quad, with
    guard values around Y."""
    p = Problem(fmt, M, N, K, dtype, 320)
    for layout in (qg.X_ROW, qg.X_FRAG):
        for act in ("gelu", "relu"):
            buf = torch.full((M * N + 64,), 7.0, dtype=p.x.dtype, device="cuda")
            out = buf[:M * N].view(M, N)
            y = p.run(layout, True, True, act, out=out)
            assert y is out
            assert_within(y, *p.want(True, True, act), dtype, f"{fmt} {M}x{N}x{K} {act}")
            assert bool((buf[M * N:] == 7.0).all())


@pytest.mark.parametrize("fmt,M,N,K", [("q4k", 98, 640, 1024), ("q6k", 173, 61, 768), ("q4k", 17, 4112, 512), ("q6k", 300, 256, 512),
                                       ("q4k", 48, 8192, 256), ("w4a16", 47, 1000, 384), ("w4a16", 200, 50, 640)])
def test_one_panel_waves_through_the_ladder(fmt, M, N, K):
    """Sizes whose ladder gives each wave one panel where the products share
    four (in bf16; of 48 x 8192 fp16 has four, too), one row group and several."""
    assert qg.linear_select_rung(fmt, M, N, K, False, qg.BF16)["name"] == "direct-small-m"
    assert qg.select_rung(fmt, M, N, K, qg.BF16)["name"] != "direct-small-m"
    for dtype in (qg.F16, qg.BF16):
        p = Problem(fmt, M, N, K, dtype, 460)
        y, d = p.want(True, True, "silu")
        got = p.run(qg.X_ROW, True, True, "silu")
        assert_within(got, y, d, dtype, f"{fmt} {M} {N} {K}")
        if N % 128 == 0:
            assert torch.equal(bits(p.run(qg.X_ROW, True, True, "silu", out_layout=qg.X_FRAG)), bits(frag(got)))


@pytest.mark.parametrize("M", [1, 5, 17, 33, 40, 49, 65, 100])
@pytest.mark.parametrize("gated", [False, True])
def test_fragment_major_output_zeroes_its_padding(M, gated):
    """Rows past M of the fragment-major Y are zeros whatever was there, and
    nothing past the layout's end is written."""
    p = Problem("q4k", M, 256, 512, qg.BF16, 330, gated=gated)
    n = qg.xf_bytes(M, 256) // 2
    for rung in (-1, 0, 1, 2):
        for layout in (qg.X_ROW, qg.X_FRAG):
            buf = torch.full((n + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
            y = p.run(layout, True, True, "silu", rung=rung)
            yf = p.run(layout, True, True, "silu", rung=rung, out_layout=qg.X_FRAG, out=buf[:n])
            assert torch.equal(bits(yf), bits(frag(y)))
            assert bool((buf[n:] == 3.0).all())


@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16], ids=["f16", "bf16"])
def test_split_rungs_with_epilogue(dtype):
    """K split across workgroups: the epilogue runs in the reduction, once."""
    for name, fmt, M, N, K in (("mfma32-64x64-sk", "q4k", 50, 260, 4096), ("mfma32-64x64-sk", "w4a16", 33, 131, 4096),
                               ("mfma32-768x64-sk", "q6k", 70, 384, 2048)):
        r = NAMES.index(name)
        p = Problem(fmt, M, N, K, dtype, 340)
        assert qg.rung_info(r, fmt, M, N, K)["k_split"] > (4 if "64x64" in name and "768" not in name else 1)
        for layout in (qg.X_ROW, qg.X_FRAG):
            y = p.run(layout, True, True, "gelu_tanh", rung=r)
            assert_within(y, *p.want(True, True, "gelu_tanh"), dtype, f"{name} {fmt}")
            if N % 128 == 0:
                yf = p.run(layout, True, True, "gelu_tanh", rung=r, out_layout=qg.X_FRAG)
                assert torch.equal(bits(yf), bits(frag(y)))


@pytest.mark.parametrize("M", [3, 40, 200])
def test_residual_in_place(M):
    p = Problem("q4k", M, 272, 512, qg.F16, 350)
    for rung in (-1, NAMES.index("mfma32-64x64-sk")):
        y = p.run(qg.X_ROW, True, True, "silu", rung=rung)
        out = p.res.clone()
        z = qg.linear("q4k", p.x, p.wp, p.N, bias=p.bias, residual=out, act="silu", rung=rung, out=out)
        assert z is out and torch.equal(bits(z), bits(y))
    pf = Problem("q4k", M, 256, 512, qg.F16, 351)
    with pytest.raises(ValueError):
        qg.linear("q4k", pf.x, pf.wp, 256, residual=pf.res, out=pf.res, out_layout=qg.X_FRAG)


def test_wide_accumulator_values():
    """The activations over their whole range: the bias sweeps +-40 and the
    extremes; infinities and NaN go where the formula sends them."""
    M, N, K = 2, 1024, 256
    p = Problem("q4k", M, N, K, qg.F16, 360)
    x0 = torch.zeros_like(p.x)
    sweep = torch.linspace(-40, 40, N, dtype=torch.float64).to(torch.float16)
    special = torch.tensor([65504.0, -65504.0, float("inf"), float("nan"), 0.0, -0.0, 6e-8, -6e-8], dtype=torch.float16)
    sweep[:special.numel()] = special
    for act in ACTS:
        y = qg.linear("q4k", x0, p.wp, N, bias=sweep.cuda(), act=act).cpu().double()
        w = torch.zeros((K, N), dtype=torch.float64)
        want, d = linear64(torch.zeros((M, K), dtype=torch.float64), w, N, sweep.double(), None, act)
        fin = torch.isfinite(want)
        assert torch.equal(torch.isnan(want), torch.isnan(y))
        assert torch.equal(torch.isinf(want), torch.isinf(y))
        assert_within(torch.where(fin, y, torch.zeros_like(y)), torch.where(fin, want, torch.zeros_like(want)),
                      torch.where(fin, d, torch.zeros_like(d)), qg.F16, act)


def test_other_stream_and_graph():
    """The call on a stream of its own, and captured and replayed on inputs
    that change between replays."""
    p = Problem("w4a16", 12, 256, 512, qg.BF16, 370, gated=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = p.run(qg.X_ROW, True, True, "silu")
    torch.cuda.current_stream().wait_stream(s)
    assert_within(y, *p.want(True, True, "silu"), qg.BF16, "stream")
    x, out = p.x.clone(), torch.empty((12, 256), dtype=torch.bfloat16, device="cuda")
    kw = dict(bias=p.bias, residual=p.res, act="silu", gated=True, group=p.group, has_zp=p.zp)
    qg.linear("w4a16", x, p.wp, 256, out=out, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.linear("w4a16", x, p.wp, 256, out=out, **kw)
    for i in range(4):
        x.copy_(p.x.roll(i, 0))
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        eager = qg.linear("w4a16", x, p.wp, 256, **kw)
        assert torch.equal(bits(out), bits(eager)), i


def test_empty_batch():
    p = Problem("q4k", 1, 128, 256, qg.F16, 380)
    x = torch.empty((0, 256), dtype=torch.float16, device="cuda")
    assert qg.linear("q4k", x, p.wp, 128).shape == (0, 128)
    assert qg.linear("q4k", x, p.wp, 128, out_layout=qg.X_FRAG).numel() == 0
