"""The feed-forward operators where one expert is popular, where a weight
overflows the operand type, and where buffers, streams and sizes are at the
edge of what a call takes."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
import quantized_weight_prefill_amd as qg
from quantized_weight_prefill_amd import synth
from tests.ffn_ref import HALF, SUB, act64
from tests.helpers import bytes_to_device, from_device, same_bits
from tests.test_gpu_exact import DTYPES, double_rounded, wide_gap_fields

pytestmark = pytest.mark.gpu

TORCH = {qg.F16: torch.float16, qg.BF16: torch.bfloat16}


def eye_fields(n):
    """Q4_K fields of the n x n unit matrix (d = 1, one scale for all)."""
    f = {k: np.zeros_like(v) for k, v in synth.q4k_fields(np.random.default_rng(0), n, n).items()}
    f["d"][:], f["sc"][:], f["q"][:] = 0x3C00, 1, np.eye(n, dtype=np.uint8)
    return f


def pack(f, N, K):
    return qg.pack("q4k", synth.encode("q4k", f), N, K)


def square_layer(x64, ids, E, dtype, down, **kw):
    """The layer of E equal experts with gate = up = I and no activation: h = x * x."""
    T, n = x64.shape
    eye = eye_fields(n)
    up = pack({k: np.concatenate([v, v]) for k, v in eye.items()}, 2 * n, n)
    ids = torch.as_tensor(ids, dtype=torch.int32).reshape(T, -1).cuda()
    offs, rows = qg.moe_group(ids, E)
    return qg.moe("q4k", "q4k", x64.to(TORCH[dtype]).cuda(), bytes_to_device(np.tile(up, E)),
                  bytes_to_device(np.tile(pack(down, n, n), E)), torch.ones(ids.shape, device="cuda"), offs, rows, n,
                  act="none", **kw).cpu().double()


def popular(T, E, share, rng):
    """One expert per token, `share` of them on expert E // 2."""
    ids = rng.integers(0, E, T)
    ids[rng.random(T) < share] = E // 2
    return ids


@pytest.mark.parametrize("dtype", DTYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T,E,share", [(9, 8, 1.0), (16, 8, 1.0), (17, 8, 1.0), (20, 8, 1.0), (24, 8, 1.0), (25, 8, 0.7),
                                       (64, 16, 0.5), (120, 40, 0.4), (1024, 300, 0.3), (1024, 256, 1.0)])
def test_moe_keeps_both_parts_of_h_whatever_an_experts_share(T, E, share, dtype):
    """What is left of h = x * x after its rounding, exactly, when an expert
    has more rows than others (at most four per expert on average): x are
    whole numbers up to 255, so x * x has 16 bits, its rounding 11 or 8 and
    the rest at most 8, and Y = h - RN(h) has them all."""
    n = 256
    rng = np.random.default_rng(1200 + T)
    x64 = torch.from_numpy(rng.integers(-255, 256, (T, n)).astype(np.float64))
    res = -(x64 * x64).to(TORCH[dtype])
    left = x64 * x64 + res.double()
    assert bool((left != 0).any()) and torch.equal(left.to(TORCH[dtype]).double(), left)
    y = square_layer(x64, popular(T, E, share, rng), E, dtype, eye_fields(n), residual=res.cuda())
    bad = (y != left).any(1).nonzero().flatten().tolist()
    assert not bad, f"{len(bad)} rows differ, first {bad[:8]}"


@pytest.mark.parametrize("T,E", [(3, 2), (20, 8), (40, 2), (1024, 300), (1024, 200)])
def test_moe_infinite_weights(T, E):
    """A weight beyond fp16's range is an infinity, and an output takes its
    sign whatever the rounding of h left: few pairs per expert and many, one
    panel of Y per workgroup and two."""
    n = 256
    rng = np.random.default_rng(1300 + T)
    x64 = torch.from_numpy(rng.integers(1, 256, (T, n)).astype(np.float64))
    down = eye_fields(n)
    w = torch.eye(n, dtype=torch.float64)           # [K][N]
    for col, k in ((5, 7), (130, 200)):             # 2 * 65504 * 1 in one row of the column
        down["d"][col, 0], down["sc"][col, 0, k // 32] = 0x7BFF, 2
        down["q"][col] = 0
        down["q"][col, k] = 1
        w[:, col] = 0
        w[k, col] = math.inf
    down["d"][77, 0], down["dmin"][77, 0] = 0, 0x7BFF  # 0 - 65504 * 2 in a whole sub-block
    down["m"][77, 0, 3] = 2
    w[:, 77] = 0
    w[96:128, 77] = -math.inf
    h = x64 * x64
    want = torch.where(torch.isinf(w).any(0), torch.where(w.sum(0) > 0, math.inf, -math.inf), h).to(torch.float16).double()
    low = h - h.half().double()
    assert all(bool((low[:, 7].sign() == s).any()) or T < 20 for s in (-1, 0, 1))
    y = square_layer(x64, popular(T, E, 0.2, rng), E, qg.F16, down)
    assert torch.equal(y, want), (y != want).nonzero()[:5]


def test_moe_products_beyond_binary32():
    """h * w above the largest float is an infinity in bf16, and what the
    rounding of h left does not turn it into a NaN."""
    n, T = 256, 12
    x64 = torch.full((T, n), 1.0e19, dtype=torch.float64) * (1 + torch.arange(n) / 512.0)
    x64 = x64.bfloat16().double()
    down = eye_fields(n)
    down["sc"][:] = 63
    for E in (2, 8):
        y = square_layer(x64, [i % E for i in range(T)], E, qg.BF16, down)
        assert bool((x64 * x64 < 3.3e38).all()) and bool((x64 * x64 * 63 > 3.5e38).all())
        assert bool((y == math.inf).all())


def test_buffers_that_share_memory_are_refused():
    """A result that overlaps an input would depend on which workgroup comes
    first; the residual in place, and the layer's x, are what is allowed."""
    rng = np.random.default_rng(1400)
    M, n = 40, 512
    wp = bytes_to_device(pack(synth.q4k_fields(rng, n, n), n, n))
    flat = torch.randn(3 * M * n, device="cuda").half()
    x, res = flat[:M * n].view(M, n), flat[M * n:2 * M * n].view(M, n)
    shifted = flat[M * n + n:2 * M * n + n].view(M, n)   # the residual from its second row on
    bias = torch.randn(n, device="cuda").half()
    with_bias = flat[2 * M * n:].view(M, n)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    split = [r for r in range(qg.num_rungs()) if qg.rung_name(r) == "mfma32-64x64-sk"][0]
    need = qg.workspace_bytes("q4k", split, M, n, n)
    xf = qg.x_to_xf(x)
    before = flat.clone()
    for kw in (dict(), dict(workspace=ws)):            # the common calls and the others
        for bad in (dict(out=x), dict(out=x, residual=x), dict(out=shifted, residual=res),
                    dict(out=with_bias, bias=with_bias[-1])):
            with pytest.raises(ValueError, match="shares memory"):
                qg.linear("q4k", x, wp, n, **bad, **kw)
        with pytest.raises(ValueError, match="shares memory"):
            qg.linear_xf("q4k", xf, wp, M, n, n, out=xf, out_layout=qg.X_FRAG, **kw)
        buf = torch.zeros(qg.xf_bytes(M, n) // 2, dtype=torch.float16, device="cuda")
        with pytest.raises(ValueError, match="shares memory"):
            qg.linear("q4k", x, wp, n, residual=buf[:M * n].view(M, n), out=buf, out_layout=qg.X_FRAG, **kw)
    for bad in (flat, wp):
        with pytest.raises(ValueError, match="workspace shares memory"):
            qg.linear("q4k", x, wp, n, rung=split, workspace=bad)
    with pytest.raises(ValueError, match="workspace shares memory"):
        inside = ws[need - 16:need - 16 + 2 * M * n].view(torch.float16).view(M, n)
        qg.linear("q4k", x, wp, n, rung=split, out=inside, workspace=ws[:need])
    assert torch.equal(flat, before)
    # side by side in one allocation is no overlap
    y = qg.linear("q4k", x, wp, n, bias=bias, residual=res)
    assert torch.equal(qg.linear("q4k", x, wp, n, bias=bias, residual=res, out=with_bias), y)
    assert torch.equal(qg.linear("q4k", x, wp, n, bias=bias, residual=res, out=res), y)

    T, k, E, H, I = 6, 2, 4, 512, 256
    up = bytes_to_device(np.tile(pack(synth.q4k_fields(rng, 2 * I, H), 2 * I, H), E))
    down = bytes_to_device(np.tile(pack(synth.q4k_fields(rng, H, I), H, I), E))
    ids, w, offs, rows = qg.moe_route(torch.randn((T, E), device="cuda"), k)
    both = (torch.randn((2 * T, H), device="cuda") * 0.01).half()
    tx, tr = both[:T], both[T:]
    ws = torch.empty(qg.moe_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    args = ("q4k", "q4k", tx, up, down, w, offs, rows, I)
    before = both.clone()
    for kw in (dict(), dict(workspace=ws)):
        for out in (both[1:T + 1], *(t[:2 * T * H].view(torch.float16).view(T, H) for t in (up, down))):
            with pytest.raises(ValueError, match="shares memory"):
                qg.moe(*args, out=out, **kw)
        with pytest.raises(ValueError, match="shares memory"):
            qg.moe(*args, residual=tr, out=both[T - 1:2 * T - 1], **kw)
    for bad in (up, down):
        with pytest.raises(ValueError, match="workspace shares memory"):
            qg.moe(*args, workspace=bad)
    assert torch.equal(both, before)
    y = qg.moe(*args, residual=tr)
    assert torch.equal(qg.moe(*args, residual=tr, out=tx.clone()), y)
    for kw in (dict(), dict(workspace=ws)):
        both.copy_(before)
        assert torch.equal(qg.moe(*args, residual=tr, out=tr, **kw), y)
        both.copy_(before)
        assert torch.equal(qg.moe(*args, residual=tr, out=tx, **kw), y)


def test_moe_weight_bytes_beyond_64_bits():
    """Experts whose packed bytes add up to a multiple of 2^64: refused by
    their size, not taken for weights of no bytes."""
    E, H, I = 1 << 24, 1 << 20, 1 << 26
    up, down = (qg.packed_bytes("w4a16", n, k, 128) for n, k in ((2 * I, H), (H, I)))
    assert up > 0 and E * up % 2 ** 64 == 0 and E * down % 2 ** 64 == 0
    x = torch.zeros((1, H), dtype=torch.float16, device="cuda")
    w = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="w_up holds 1024 bytes"):
        qg.moe("w4a16", "w4a16", x, w, w, torch.ones((1, 1), device="cuda"), offs, offs[:1].clone(), I, group=128)


def home_stream(ptr):
    """The stream whose memory the allocator's block at `ptr` belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= ptr < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no block of torch's allocator")


def test_results_and_workspaces_belong_to_the_calls_stream(monkeypatch):
    """A call on an explicit stream writes memory of that stream: a block of
    the current one may still be read by work that was queued there."""
    rng = np.random.default_rng(1500)
    T, k, E, n = 12, 2, 4, 512
    wp = bytes_to_device(pack(synth.q4k_fields(rng, n, n), n, n))
    up = bytes_to_device(np.tile(pack(synth.q4k_fields(rng, 2 * n, n), 2 * n, n), E))
    down = bytes_to_device(np.tile(pack(synth.q4k_fields(rng, n, n), n, n), E))
    x = (torch.randn((T, n), device="cuda") * 0.01).half()
    logits = torch.randn((T, E), device="cuda")
    split = [r for r in range(qg.num_rungs()) if qg.rung_name(r) == "mfma32-64x64-sk"][0]
    spaces = []
    call = qg._call

    def spy(fn, index, stream, *args):
        if fn in ("qgemm_linear", "qgemm_moe"):
            spaces.append(args[-2])
        return call(fn, index, stream, *args)

    def run(**kw):
        ids, w, offs, rows = qg.moe_route(logits, k, **kw)
        o2, r2 = qg.moe_group(ids, E, **kw)
        return [ids, w, offs, rows, o2, r2, qg.linear("q4k", x, wp, n, rung=split, **kw),
                qg.linear("q4k", x, wp, n, out_layout=qg.X_FRAG, **kw),
                qg.moe("q4k", "q4k", x, up, down, w, offs, rows, n, **kw)]

    want = run()
    monkeypatch.setattr(qg, "_call", spy)
    side, default = torch.cuda.Stream(), torch.cuda.default_stream()
    torch.cuda.synchronize()
    for current, other in ((default, side), (side, default), (default, default), (side, side)):
        spaces.clear()
        with torch.cuda.stream(current):
            got = run(stream=other.cuda_stream)
            current.wait_stream(other)
            same = [torch.equal(a, b) for a, b in zip(got, want)]
        torch.cuda.synchronize()
        assert all(same), same
        assert len(spaces) == 3 and spaces[0] and not spaces[1] and spaces[2]
        for p in [t.data_ptr() for t in got] + [spaces[0], spaces[2]]:
            assert home_stream(p) == other.cuda_stream


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", DTYPES, ids=["f16", "bf16"])
def test_activations_relative_accuracy(act, dtype):
    """act(v) to the bits that its rounding leaves, the negative tail
    included: with X = 0, v the bias and -RN(act(v)) the residual, Y is what
    was left, exact in binary32 (the two are within a factor of two).

    Error: exp2 and rcp 2^-23 each, two products 2^-24 each, in all 2^-21;
    erfc's fit 4e-7 < 2^-21 more.  The exponent x takes at most 5.5 roundings
    of 2^-24 (GELU: |v| / sqrt 2 and its constant twice, the product with
    log2 e, its constant, one more product), ln 2 * 5.5 < 4.  Then Y's own
    rounding."""
    tt, half, sub = TORCH[dtype], HALF[dtype], SUB[dtype]
    wide = 60.0 if act == "silu" else 13.5
    v = torch.cat([torch.linspace(-wide, wide, 4000, dtype=torch.float64), torch.logspace(-3, 0, 48, dtype=torch.float64),
                   -torch.logspace(-3, 0, 48, dtype=torch.float64)]).to(tt)
    N, K = v.numel(), 256
    wp = bytes_to_device(pack(synth.q4k_fields(np.random.default_rng(1600), N, K), N, K))
    x0 = torch.zeros((1, K), dtype=tt, device="cuda")
    v64 = v.double()
    y = act64(v64, act)
    r = y.to(tt)
    got = qg.linear("q4k", x0, wp, N, bias=v.cuda(), act=act, residual=-r.cuda()[None])[0].cpu().double()
    want = y - r.double()
    order = {"silu": 1.4427 * v64.abs(), "gelu": 0.72135 * v64 ** 2,
             "gelu_tanh": v64.abs() * (2.3023 + 0.10295 * v64 ** 2)}[act]
    err = (2.0 ** -21 * (2 if act == "gelu" else 1) + 4 * order * 2.0 ** -24) * y.abs()
    tail = order > 100                       # below |v| 2^-100; from |v| 2^-125 on it may be 0
    bad = ((got - want).abs() > err + half * (want.abs() + err) + sub) & ~tail
    assert not bool(bad.any()), (v64[bad][:4], got[bad][:4], want[bad][:4])
    plain = qg.linear("q4k", x0, wp, N, bias=v.cuda(), act=act)[0].cpu().double()
    low = tail & (v64 < 0)
    assert bool((plain[low].abs() <= y[low].abs() * (1 + 2 * half) + sub).all())


@pytest.mark.parametrize("E", [300, 200], ids=["few_per_expert", "many_per_expert"])
@pytest.mark.parametrize("dtype", DTYPES, ids=["f16", "bf16"])
def test_unpack_contract_with_two_panels_per_workgroup(dtype, E):
    """Identity extraction of the down projection on blocks whose d and dmin
    are far apart, with more row tiles than two per wave of the down product
    (1024 pairs over 300 and 200 experts, 256 columns)."""
    n, T = 256, 1024
    wide = wide_gap_fields(1700 + dtype, n, n)
    enc = synth.encode("q4k", wide)
    W = oracle.dequant("q4k", enc, n, n, dtype)
    assert int((double_rounded(wide, dtype) != W).sum()) > 0
    eye = eye_fields(n)
    ones = {k: v.copy() for k, v in eye.items()}
    ones["q"][:] = 1
    up = pack({k: np.concatenate([eye[k], ones[k]]) for k in eye}, 2 * n, n)
    x = torch.eye(n, dtype=TORCH[dtype], device="cuda").repeat(T // n, 1)
    ids = torch.from_numpy(np.random.default_rng(1701).integers(0, E, (T, 1)).astype(np.int32)).cuda()
    offs, rows = qg.moe_group(ids, E)
    y = qg.moe("q4k", "q4k", x, bytes_to_device(np.tile(up, E)), bytes_to_device(np.tile(qg.pack("q4k", enc, n, n), E)),
               torch.ones((T, 1), device="cuda"), offs, rows, n, act="none")
    assert same_bits(from_device(y), np.tile(W, (T // n, 1)))


def test_explicit_stream_inside_a_capture():
    """Calls on a stream that joins a capture, captured and replayed on inputs
    that change: the results of the eager calls, memory of their own."""
    rng = np.random.default_rng(1800)
    T, k, E, n = 12, 2, 4, 512
    wp = bytes_to_device(pack(synth.q4k_fields(rng, n, n), n, n))
    up = bytes_to_device(np.tile(pack(synth.q4k_fields(rng, 2 * n, n), 2 * n, n), E))
    down = bytes_to_device(np.tile(pack(synth.q4k_fields(rng, n, n), n, n), E))
    x0 = (torch.randn((T, n), device="cuda") * 0.01).half()
    l0 = torch.randn((T, E), device="cuda")
    x, logits = x0.clone(), l0.clone()
    split = [r for r in range(qg.num_rungs()) if qg.rung_name(r) == "mfma32-64x64-sk"][0]

    def run(**kw):
        _, w, offs, rows = qg.moe_route(logits, k, **kw)
        return (qg.linear("q4k", x, wp, n, rung=split, act="silu", **kw),
                qg.moe("q4k", "q4k", x, up, down, w, offs, rows, n, residual=x, **kw))

    run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = run(stream=side.cuda_stream)
        here.wait_stream(side)
    for i in range(4):
        x.copy_(x0.roll(i, 0))
        logits.copy_(l0.roll(i, 1))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, run())), i
