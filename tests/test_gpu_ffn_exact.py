"""The unpack contract through the linear and the mixture-of-experts kernels,
bit for bit: identity extraction on Q4_K blocks whose d and dmin are far apart,
where a binary32 intermediate would round some weights differently."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import quantized_weight_prefill_amd as qg
from quantized_weight_prefill_amd import synth
from tests.helpers import bytes_to_device, from_device, same_bits, to_device
from tests.test_gpu_exact import DTYPES, _assert_sensitive, _eye, _wide_case, wide_gap_fields

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("layout", ["row", "xf"])
def test_linear_identity_every_rung(dtype, layout):
    """X = I, so Y = W; then as the up half of a gated call whose gate is 1."""
    K, N = 512, 48
    c = _wide_case(K, N, K, dtype, seed=940 + dtype, X=_eye(K, dtype))
    _assert_sensitive(c)
    x, wp = to_device(c.X, dtype), c.device_weights()
    ones = {k: np.zeros_like(v) for k, v in c.fields.items()}
    ones["d"][:], ones["sc"][:], ones["q"][:] = 0x3C00, 1, 1
    both = {k: np.concatenate([ones[k], c.fields[k]]) for k in c.fields}
    wg = bytes_to_device(qg.pack("q4k", synth.encode("q4k", both), 2 * N, K))
    xf = qg.x_to_xf(x)
    for rung in range(qg.num_rungs()):
        name = qg.rung_name(rung)
        for gated in (False, True):
            if gated and name.endswith("-sk"):
                continue
            w = wg if gated else wp
            if layout == "row":
                y = qg.linear("q4k", x, w, N, gated=gated, rung=rung)
            else:
                y = qg.linear_xf("q4k", xf, w, K, N, K, gated=gated, rung=rung)
            assert same_bits(from_device(y), c.W), f"{name} gated={gated}"
    for M in (1, 3, 16, 20, 40, 64):  # the ladder's decode-sized kernels, the same rows
        if layout == "row":
            y = qg.linear("q4k", x[:M], wp, N)
        else:
            y = qg.linear_xf("q4k", qg.x_to_xf(x[:M].contiguous()), wp, M, N, K)
        assert same_bits(from_device(y), c.W[:M]), M


@pytest.mark.parametrize("dtype", DTYPES, ids=["f16", "bf16"])
def test_moe_identity(dtype):
    """One expert, top-1, weight 1, no activation: with up = 1 and down = I
    the layer returns the gate's weights, with gate = I and up = 1 the down
    projection's."""
    n = 256
    wide = wide_gap_fields(960 + dtype, n, n)
    W = oracle.dequant("q4k", synth.encode("q4k", wide), n, n, dtype)

    def const(q):
        f = {k: np.zeros_like(v) for k, v in wide.items()}
        f["d"][:], f["sc"][:], f["q"][:] = 0x3C00, 1, q
        return f

    eye, ones = const(np.eye(n, dtype=np.uint8)), const(1)
    cat = lambda a, b: {k: np.concatenate([a[k], b[k]]) for k in a}
    pack = lambda f, N: bytes_to_device(qg.pack("q4k", synth.encode("q4k", f), N, n))
    x = to_device(_eye(n, dtype), dtype)
    w1 = torch.ones((n, 1), device="cuda")
    offs, rows = qg.moe_group(torch.zeros((n, 1), dtype=torch.int32, device="cuda"), 1)
    for up, down in ((cat(wide, ones), eye), (cat(eye, ones), wide)):
        y = qg.moe("q4k", "q4k", x, pack(up, 2 * n), pack(down, n), w1, offs, rows, n, act="none")
        assert same_bits(from_device(y), W)
        for T in (1, 5):
            o, r = qg.moe_group(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), 1)
            y = qg.moe("q4k", "q4k", x[:T], pack(up, 2 * n), pack(down, n), w1[:T], o, r, n, act="none")
            assert same_bits(from_device(y), W[:T])


@pytest.mark.parametrize("dtype", DTYPES, ids=["f16", "bf16"])
def test_moe_hidden_keeps_what_its_rounding_left(dtype):
    """Gate = up = down = I, so h = x * x and Y = h + residual, with the residual
    -RN(h): what is left has few bits, and Y is exactly that (x are whole numbers
    up to 255: x * x has 16 bits, its rounding 11 or 8, the rest at most 8).  A
    few pairs per expert and many, with one panel per workgroup of the down
    product and (many experts) two; then all pairs on one expert of several,
    where the tile of more than eight rows may keep the rounding alone."""
    n = 256
    f = {k: np.zeros_like(v) for k, v in wide_gap_fields(980, n, n).items()}
    f["d"][:], f["sc"][:], f["q"][:] = 0x3C00, 1, np.eye(n, dtype=np.uint8)
    up = qg.pack("q4k", synth.encode("q4k", {k: np.concatenate([v, v]) for k, v in f.items()}), 2 * n, n)
    down = qg.pack("q4k", synth.encode("q4k", f), n, n)
    for T, E, one in ((1, 1, 0), (3, 1, 0), (8, 1, 0), (20, 1, 0), (150, 3, 0), (600, 300, 0), (1024, 200, 0), (20, 8, 1)):
        rng = np.random.default_rng(981 + T)
        x64 = torch.from_numpy(rng.integers(-255, 256, (T, n)).astype(np.float64))
        tt = torch.float16 if dtype == qg.F16 else torch.bfloat16
        h = x64 * x64
        res = -h.to(tt)
        left = h + res.double()
        assert bool((left != 0).any()) and torch.equal(left.to(tt).double(), left)
        ids = (torch.arange(T, dtype=torch.int32) % E if not one else torch.full((T,), 3, dtype=torch.int32))[:, None].cuda()
        offs, rows = qg.moe_group(ids, E)
        y = qg.moe("q4k", "q4k", x64.to(tt).cuda(), bytes_to_device(np.tile(up, E)), bytes_to_device(np.tile(down, E)),
                   torch.ones((T, 1), device="cuda"), offs, rows, n, act="none", residual=res.cuda())
        first = 16 if one else 0
        assert torch.equal(y[first:].cpu().double(), left[first:]), (T, E)


def test_calls_with_and_without_the_common_path():
    """A call on an explicit stream, or with the caller's workspace, takes the
    checked Python path: the same bits as the common one, refusals alike."""
    s = torch.cuda.current_stream().cuda_stream
    rng = np.random.default_rng(970)
    f = synth.q4k_fields(rng, 256, 512)
    wp = bytes_to_device(qg.pack("q4k", synth.encode("q4k", f), 256, 512))
    x = to_device(synth.activations(rng, 7, 512, qg.F16), qg.F16) * 0.01
    res = torch.randn((7, 256), device="cuda").half()
    bias = torch.randn(256, device="cuda").half()
    for kw in (dict(), dict(bias=bias, act="gelu"), dict(residual=res), dict(out_layout=qg.X_FRAG),
               dict(gated=True, act="silu", bias=bias)):
        N = 128 if kw.get("gated") else 256
        if "residual" in kw:
            kw["residual"] = res[:, :N].contiguous()
        a = qg.linear("q4k", x, wp, N, **kw)
        assert torch.equal(a, qg.linear("q4k", x, wp, N, stream=s, **kw))
        assert torch.equal(a, qg.linear("q4k", x, wp, N, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **kw))
        xf = qg.x_to_xf(x)
        assert torch.equal(qg.linear_xf("q4k", xf, wp, 7, N, 512, **kw),
                           qg.linear_xf("q4k", xf, wp, 7, N, 512, stream=s, **kw))
    logits = torch.randn((9, 40), device="cuda")
    for a, b in zip(qg.moe_route(logits, 3), qg.moe_route(logits, 3, stream=s)):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)
    ids, w, offs, rows = qg.moe_route(logits[:, :2].contiguous(), 1)
    for a, b in zip(qg.moe_group(ids, 2), qg.moe_group(ids, 2, stream=s)):
        assert torch.equal(a, b)
    up = bytes_to_device(qg.pack("q4k", synth.encode("q4k", synth.q4k_fields(rng, 2 * 512, 512)), 2 * 512, 512))
    dn = bytes_to_device(qg.pack("q4k", synth.encode("q4k", synth.q4k_fields(rng, 2 * 512, 256)), 2 * 512, 256))
    x9 = torch.randn((9, 512), device="cuda").half() * 0.001
    a = qg.moe("q4k", "q4k", x9, up, dn, w, offs, rows, 256)
    ws = torch.empty(qg.moe_workspace_bytes(9, 1, 512, 256), dtype=torch.uint8, device="cuda")
    assert torch.equal(a, qg.moe("q4k", "q4k", x9, up, dn, w, offs, rows, 256, stream=s))
    assert torch.equal(a, qg.moe("q4k", "q4k", x9, up, dn, w, offs, rows, 256, workspace=ws))
    with pytest.raises(qg.QGemmError):
        qg.moe("q4k", "q4k", x9, up, dn, w, offs, rows, 256, workspace=ws[:-16])
    # no tokens
    e9 = torch.empty((0, 512), dtype=torch.float16, device="cuda")
    z = qg.moe("q4k", "q4k", e9, up, dn, w[:0], torch.zeros(3, dtype=torch.int32, device="cuda"), rows[:0], 256)
    assert z.shape == (0, 512)
    # what the common path leaves to the checks
    for bad in (lambda: qg.linear("q4k", x, wp, 256, bias=bias[:-1]), lambda: qg.linear("q4k", x.float(), wp, 256),
                lambda: qg.linear("q4k", torch.stack([x, x], 1)[:, 0], wp, 256), lambda: qg.linear("q4k", x, wp, 256, act="tanh"),
                lambda: qg.linear("q4k", x, wp[:-16], 256), lambda: qg.linear("q4k", x, wp, 256, residual=res.cpu()),
                lambda: qg.moe_route(logits.t(), 2), lambda: qg.moe_group(ids.long(), 2),
                lambda: qg.moe("q4k", "q4k", x9, up, dn, w, offs, rows[1:], 256),
                lambda: qg.moe("q4k", "q4k", x9, up, dn[:-16], w, offs, rows, 256)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad in (lambda: qg.linear("q4k", x, wp, 256, rung=99), lambda: qg.linear("q4k", x, wp, 100, out_layout=qg.X_FRAG),
                lambda: qg.moe_route(logits, 41), lambda: qg.moe_route(logits, 0), lambda: qg.moe_group(ids, 0),
                lambda: qg.moe_group(ids, 5000), lambda: qg.linear("q4k", x, wp, 24, gated=True),
                lambda: qg.linear("q4k", x, wp, 256, bias=torch.zeros(300, device="cuda").half()[4:260])):
        with pytest.raises(qg.QGemmError):
            bad()
