"""Mixture of experts: routing and grouping against exact host forms, the
few-token layer against its formula in 64 bits on the oracle's unpacked
weights, and the pieces run together as a model would run them."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
import quantized_weight_prefill_amd as qg
from quantized_weight_prefill_amd import synth
from tests.ffn_ref import (EPS32, HALF, SUB, act64, act_err, assert_within, bits, bits64, linear64, product)
from tests.helpers import bytes_to_device, to_device

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# routing and grouping
# ---------------------------------------------------------------------------

def group_ref(ids, E):
    by = [[] for _ in range(E)]
    flat = [int(v) for v in ids.reshape(-1)]
    for p, e in enumerate(flat):
        if 0 <= e < E:
            by[e].append(p)
    offs = np.concatenate([[0], np.cumsum([len(b) for b in by])])
    rows = [p for b in by for p in b]
    return offs.tolist(), rows + [-1] * (len(flat) - len(rows))


def route_ref(logits, k, score, renorm, scale):
    v = logits.double().cpu()
    v = torch.where(torch.isnan(v), torch.full_like(v, -math.inf), v).clamp(max=float(np.finfo(np.float32).max))
    ids = [sorted(range(v.shape[1]), key=lambda e, r=r: (-r[e], e))[:k] for r in v.tolist()]
    ids = torch.tensor(ids).reshape(v.shape[0], k)
    top = torch.gather(v, 1, ids)
    if score == "softmax":
        mx = v.max(1, keepdim=True)[0]
        safe = torch.where(torch.isinf(mx), torch.zeros_like(mx), mx)
        p = torch.exp(v - safe)
        w = torch.exp(top - safe) / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.sigmoid(top)
    if renorm:
        s = w.sum(1, keepdim=True)
        w = torch.where(s > 0, w / s, torch.zeros_like(w))
    return ids, w * scale


def check_route(logits, k, score, renorm, scale):
    E = logits.shape[1]
    ids, w, offs, rows = qg.moe_route(logits, k, score=score, renorm=renorm, scale=scale)
    rid, rw = route_ref(logits, k, score, renorm, scale)
    assert torch.equal(ids.cpu().long(), rid)
    # exp of a binary32 difference d is off by |d| 2^-24 and 1 ulp, a sum of n
    # positive terms by n 2^-24, the quotients by 2^-24 each; differences
    # beyond 100 have exps below 1e-43, whose subnormals are absolute
    tol = (100 + E + 8) * 2.0 ** -24 * rw.abs() + 2e-38 * max(1.0, scale)
    if renorm:  # quotients of scores as small as the subnormals carry their grid
        tol = tol + 1e-6 * rw.abs()
    assert bool(((w.cpu().double() - rw).abs() <= tol).all()), (w.cpu(), rw)
    ro, rr = group_ref(rid.numpy(), E)
    assert offs.tolist() == ro and rows.tolist() == rr


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 8, 2), (5, 64, 64), (64, 65, 6), (7, 200, 16), (2, 512, 9),
                                   (9, 1000, 8), (65, 128, 8), (200, 40, 8), (1024, 16, 1)])
def test_route(dtype, T, E, k):
    g = torch.Generator().manual_seed(T * 1000 + E)
    logits = (3 * torch.randn((T, E), generator=g)).to(dtype).cuda()
    for n, score in enumerate(("softmax", "sigmoid")):
        check_route(logits, k, score, bool(n), 1.0 + 1.5 * n)
        check_route(logits, k, score, not n, 1.0)


@pytest.mark.parametrize("T", [4, 100])
def test_route_ties_and_specials(T):
    """Equal logits go by index (signed zeros are equal); NaN counts as -inf,
    +inf as the largest float; a row of -inf has no weights."""
    E, k = 96, 8
    logits = torch.zeros((T, E))
    logits[0, 1::2] = -0.0
    logits[1] = torch.tensor([float(e // 7) for e in range(E)])
    logits[2] = -math.inf
    logits[3, :4] = torch.tensor([math.nan, math.inf, -math.inf, math.inf])
    logits[3, 4:] = torch.linspace(-200, 5, E - 4)
    for dt in (torch.float32, torch.bfloat16):
        for score in ("softmax", "sigmoid"):
            for renorm in (False, True):
                check_route(logits.to(dt).cuda(), k, score, renorm, 2.0)
    ids, w, _, _ = qg.moe_route(logits.cuda(), k)
    assert ids[0].tolist() == list(range(8)) and ids[2].tolist() == list(range(8))
    assert bool((w[2] == 0).all()) and bool(torch.isfinite(w).all())
    assert ids[3].tolist()[:2] == [1, 3]


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (7, 5, 3), (128, 1024, 8), (1023, 3, 1), (1024, 70, 1),
                                   (1025, 70, 1), (300, 33, 7), (5000, 128, 8), (4097, 513, 3), (2050, 1, 1)])
def test_group(T, E, k):
    """Positions, order and the dropped pairs' tail, and nothing written
    outside; pairs of every size class."""
    rng = np.random.default_rng(T + E)
    for drop in (0.0, 0.4, 1.0):
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
        gone = rng.random((T, k)) < drop
        ids[gone] = rng.choice(np.array([-1, E, 2 ** 31 - 1, -2 ** 31], np.int64), gone.sum()).astype(np.int32)
        offs, rows = qg.moe_group(torch.from_numpy(ids).cuda(), E)
        ro, rr = group_ref(ids, E)
        assert offs.tolist() == ro and rows.tolist() == rr, drop


def test_group_of_no_tokens():
    offs, rows = qg.moe_group(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert offs.tolist() == [0] * 10 and rows.numel() == 0
    ids, w, offs, rows = qg.moe_route(torch.empty((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and offs.tolist() == [0] * 9


# ---------------------------------------------------------------------------
# the few-token layer
# ---------------------------------------------------------------------------

class Experts:
    """E experts' gate/up and down weights, packed, and their unpacked values."""

    def __init__(self, fu, fd, E, H, I, dtype, seed, group=64, zp=True):
        self.fu, self.fd, self.E, self.H, self.I, self.dtype = fu, fd, E, H, I, dtype
        w4 = "w4a16" in (fu, fd)
        self.group, self.zp = (group, zp) if w4 else (0, False)
        rs = synth.streams(seed, 2 * E)
        self.up64, self.dn64, up, dn = [], [], [], []
        for e in range(E):
            for fmt, N, K, rng, pk, w64 in ((fu, 2 * I, H, rs[2 * e], up, self.up64), (fd, H, I, rs[2 * e + 1], dn, self.dn64)):
                f = synth.weight_fields(fmt, rng, N, K, group, not zp)
                scale = 1.0 / (np.sqrt(K) * {"q4k": 1.5, "q6k": 7.0, "w4a16": 0.04}[fmt])
                for key in ("d", "dmin", "scales"):
                    if key in f:
                        f[key] = synth.f16_bits(f[key].view(np.float16).astype(np.float64) * scale)
                enc = synth.encode(fmt, f)
                pk.append(qg.pack(fmt, enc, N, K))
                w64.append(bits64(oracle.dequant(fmt, enc, N, K, dtype), dtype))
        self.up, self.dn = bytes_to_device(np.concatenate(up)), bytes_to_device(np.concatenate(dn))

    def run(self, x, weights, offs, rows, **kw):
        return qg.moe(self.fu, self.fd, x, self.up, self.dn, weights, offs, rows, self.I, group=self.group,
                      has_zp=self.zp, **kw)

    def want(self, x64, ids, weights, act, res=None):
        """(Y, its error before the store), from the definition with h rounded
        to the operand type wherever it falls within its error."""
        T, k = ids.shape
        y = torch.zeros((T, self.H), dtype=torch.float64)
        d = torch.zeros_like(y)
        mag = torch.zeros_like(y)
        for e in range(self.E):
            for t, j in torch.nonzero(ids == e).tolist():
                h, dh = linear64(x64[t:t + 1], self.up64[e], self.I, None, None, act, True)
                dh = dh + HALF[self.dtype] * (h.abs() + dh) + SUB[self.dtype]
                o, do = product(h, self.dn64[e])
                do = do + dh @ self.dn64[e].abs() * (1 + self.I * 2.0 ** -23)
                w = float(weights[t, j])
                y[t] += w * o[0]
                d[t] += abs(w) * do[0]
                mag[t] += abs(w) * (o[0].abs() + do[0])
        d = d + (k + 1) * EPS32 * mag
        if res is not None:
            y = y + res
            d = d + EPS32 * (y.abs() + d)
        return y, d


def check_moe(ex, T, k, ids, act, residual, seed, weights=None):
    rx, rr, rw = synth.streams(seed, 3)
    X, R = synth.activations(rx, T, ex.H, ex.dtype), synth.activations(rr, T, ex.H, ex.dtype)
    ids = torch.as_tensor(ids, dtype=torch.int32).reshape(T, k)
    if weights is None:
        weights = torch.from_numpy(rw.uniform(0.05, 1.0, (T, k)).astype(np.float32))
    x, r = to_device(X, ex.dtype), to_device(R, ex.dtype)
    offs, rows = qg.moe_group(ids.cuda(), ex.E)
    y = ex.run(x, weights.cuda(), offs, rows, act=act, residual=r if residual else None)
    want, d = ex.want(bits64(X, ex.dtype), ids, weights, act, bits64(R, ex.dtype) if residual else None)
    what = f"{ex.fu}/{ex.fd} E={ex.E} T={T} k={k} {act}"
    assert_within(y, want, d, ex.dtype, what)
    # two roundings to the type, h's and Y's, each at most eps/2 of its value
    # and of either sign: together within 2 * eps/2 of Y's norm
    err = (y.cpu().double() - want).norm() / want.norm().clamp(min=1e-30)
    assert float(err) <= 2 * HALF[ex.dtype] + 1e-5, (what, float(err))
    return x, r, weights.cuda(), offs, rows, y


FMTS = [("q4k", "q6k"), ("q6k", "q4k"), ("w4a16", "w4a16"), ("q4k", "w4a16")]


@pytest.mark.parametrize("dtype", [qg.F16, qg.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("fu,fd", FMTS)
def test_moe(fu, fd, dtype):
    """One token to a tile's worth and more per expert, every activation."""
    E, H, I = 5, 512, 256
    ex = Experts(fu, fd, E, H, I, dtype, 700)
    rng = np.random.default_rng(8)
    for n, (T, k) in enumerate(((1, 1), (1, 2), (2, 5), (7, 3), (17, 2), (40, 4), (150, 1))):
        ids = np.argsort(rng.random((T, E)), 1)[:, :k]
        check_moe(ex, T, k, ids, list(qg.ACTS)[n % 5], bool(n & 1), 710 + n)


@pytest.mark.parametrize("H,I,fu,fd", [(256, 256, "q4k", "q6k"), (128, 128, "w4a16", "w4a16"), (384, 640, "w4a16", "w4a16"),
                                       (1792, 768, "q6k", "q4k"), (2304, 1408, "q4k", "w4a16")])
def test_moe_sizes(H, I, fu, fd):
    """Widths whose chunks do not divide among the waves."""
    E = 3
    ex = Experts(fu, fd, E, H, I, qg.BF16, 720, group=128)
    rng = np.random.default_rng(9)
    for T, k in ((1, 2), (20, 2)):
        check_moe(ex, T, k, np.argsort(rng.random((T, E)), 1)[:, :k], "silu", True, 730)


@pytest.mark.parametrize("fu,fd,E,H,I,T,k", [("q4k", "w4a16", 31, 4096, 128, 40, 1), ("w4a16", "q6k", 3, 2048, 256, 512, 2)])
def test_moe_two_panels_per_workgroup(fu, fd, E, H, I, T, k):
    """Enough row tiles for the down product's waves to take two each: few rows
    to an expert, and the most pairs a call takes on few experts."""
    ex = Experts(fu, fd, E, H, I, qg.F16, 755)
    check_moe(ex, T, k, np.random.default_rng(11).integers(-1, E, (T, k)), "silu", True, 756)


def test_moe_skewed_and_dropped():
    """Every pair on one expert (several row tiles), experts without rows, a
    token that chose one expert twice, dropped pairs whose weights are not
    numbers, tokens with no pair left."""
    ex = Experts("q4k", "q6k", 6, 512, 256, qg.F16, 740)
    check_moe(ex, 90, 1, np.full((90, 1), 4), "silu", False, 741)
    check_moe(ex, 8, 3, np.tile([[2, 2, 5]], (8, 1)), "gelu", True, 742)
    ids = np.array([[0, -1], [-1, -1], [6, 3], [1, 2], [-7, 9]])
    w = torch.full((5, 2), 0.5)
    w[0, 1], w[1, 0], w[1, 1], w[2, 0], w[4, 1] = math.nan, math.inf, -math.inf, math.nan, math.nan
    clean = torch.where(torch.isfinite(w), w, torch.zeros_like(w))
    x, r, wc, offs, rows, y = check_moe(ex, 5, 2, ids, "silu", True, 743, weights=clean)
    y2 = ex.run(x, w.cuda(), offs, rows, act="silu", residual=r)
    assert torch.equal(bits(y2), bits(y))
    assert torch.equal(bits(y[1]), bits(r[1])) and torch.equal(bits(y[4]), bits(r[4]))
    y3 = ex.run(x, w.cuda(), offs, rows, act="silu")
    assert bool((y3[1] == 0).all()) and bool((y3[4] == 0).all())


def test_moe_largest_batch():
    """As many pairs as one call takes, and one more refused."""
    ex = Experts("w4a16", "w4a16", 9, 256, 128, qg.BF16, 750, zp=False)
    rng = np.random.default_rng(10)
    check_moe(ex, 128, 8, np.argsort(rng.random((128, 9)), 1)[:, :8], "silu", True, 751)
    x = torch.zeros((129, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(qg.QGemmError):
        ex.run(x, torch.zeros((129, 8), device="cuda"), torch.zeros(10, dtype=torch.int32, device="cuda"),
               torch.zeros(129 * 8, dtype=torch.int32, device="cuda"))


def test_moe_malformed_grouping_stays_inside():
    """Offsets and rows of any contents: nothing outside Y is written (their
    results mean nothing)."""
    ex = Experts("q4k", "q6k", 4, 256, 256, qg.F16, 760)
    T, k = 6, 2
    x = to_device(synth.activations(synth.streams(761, 1)[0], T, 256, qg.F16), qg.F16)
    w = torch.ones((T, k), device="cuda")
    big = 2 ** 31 - 1
    for offs, rows in (([0, big, -5, 3, big], [big] * 12), ([-9, -9, -9, -9, -9], [-1] * 12),
                       ([3, 2, 12, 1, 0], [-big, 11, 12, 13] * 3), ([big] * 5, list(range(12)))):
        buf = torch.full((T * 256 + 512,), 5.0, dtype=torch.float16, device="cuda")
        out = buf[:T * 256].view(T, 256)
        need = qg.moe_workspace_bytes(T, k, 256, 256) // 2
        ws = torch.full((need + 512,), 5.0, dtype=torch.float16, device="cuda")
        ex.run(x, w, torch.tensor(offs, dtype=torch.int32, device="cuda"), torch.tensor(rows, dtype=torch.int32, device="cuda"),
               out=out, workspace=ws[:need])
        torch.cuda.synchronize()
        assert bool((buf[T * 256:] == 5.0).all()) and bool((ws[need:] == 5.0).all())


def test_moe_in_place_stream_and_graph():
    ex = Experts("q4k", "q6k", 8, 512, 256, qg.BF16, 770)
    T, k = 9, 2
    rx, rl = synth.streams(771, 2)
    x = to_device(synth.activations(rx, T, 512, qg.BF16), qg.BF16)
    logits = torch.from_numpy(rl.standard_normal((T, 8)).astype(np.float32)).cuda()
    ids, w, offs, rows = qg.moe_route(logits, k)
    y = ex.run(x, w, offs, rows, residual=x)
    z = x.clone()
    assert ex.run(x, w, offs, rows, residual=z, out=z) is z and torch.equal(bits(z), bits(y))
    z = x.clone()
    assert torch.equal(bits(ex.run(z, w, offs, rows, residual=z, out=z)), bits(y))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ids2, w2, offs2, rows2 = qg.moe_route(logits, k)
        y2 = ex.run(x, w2, offs2, rows2, residual=x)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(bits(y2), bits(y))
    # routing and layer captured together, replayed on logits and x that change
    lg, xs = logits.clone(), x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, gw, go, gr = qg.moe_route(lg, k)
        gy = ex.run(xs, gw, go, gr, residual=xs)
    for i in range(4):
        lg.copy_(logits.roll(i, 1))
        xs.copy_(x.roll(i, 0))
        g.replay()
        torch.cuda.synchronize()
        _, w3, o3, r3 = qg.moe_route(lg, k)
        assert torch.equal(bits(gy), bits(ex.run(xs, w3, o3, r3, residual=xs))), i


def test_layers_side_by_side():
    """The same calls on two streams at once, then captured into two graphs
    that replay on two streams at once: each with the workspace that the
    allocator gave it, each with the bits of the call by itself."""
    ex = Experts("q4k", "q6k", 8, 512, 256, qg.BF16, 775)
    rx, rw = synth.streams(776, 2)
    f = synth.weight_fields("q4k", rw, 512, 4096)
    wp = bytes_to_device(qg.pack("q4k", synth.encode("q4k", f), 512, 4096))
    work = []
    for i, T in enumerate((9, 33)):
        logits = torch.from_numpy(rx.standard_normal((T, 8)).astype(np.float32)).cuda()
        x = to_device(synth.activations(rx, T, 512, qg.BF16), qg.BF16)
        wide = to_device(synth.activations(rx, T, 4096, qg.BF16), qg.BF16) * 0.01
        _, w, offs, rows = qg.moe_route(logits, 2)
        work.append((x, w, offs, rows, wide))

    def run(i):
        x, w, offs, rows, wide = work[i]
        # the linear layer's rung that splits K across workgroups has a workspace too
        return ex.run(x, w, offs, rows, residual=x), qg.linear("q4k", wide, wp, 512, act="silu", rung=11)

    assert qg.rung_name(11).endswith("-sk")
    want = [[bits(t) for t in run(i)] for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(i))
    torch.cuda.synchronize()
    assert all(torch.equal(bits(t), u) for i in range(2) for ts in got[i] for t, u in zip(ts, want[i]))
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(run(i))
    for _ in range(4):
        for t in outs[0] + outs[1]:
            t.zero_()
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(t), u) for i in range(2) for t, u in zip(outs[i], want[i]))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_layer_run_together():
    """A router product, the routing, the layer: against the same layer made
    of the routing, the grouped products and torch's own steps."""
    T, k, E, H, I = 12, 3, 16, 512, 256
    ex = Experts("q4k", "q6k", E, H, I, qg.F16, 780)
    rx, rw = synth.streams(781, 2)
    x = to_device(synth.activations(rx, T, H, qg.F16), qg.F16)
    f = synth.weight_fields("q6k", rw, E, H)
    f["d"] = synth.f16_bits(f["d"].view(np.float16).astype(np.float64) / (np.sqrt(H) * 7))
    router = bytes_to_device(qg.pack("q6k", synth.encode("q6k", f), E, H))
    logits = qg.linear("q6k", x, router, E)
    ids, w, offs, rows = qg.moe_route(logits, k)
    y = ex.run(x, w, offs, rows, residual=x)
    tok = (rows // k).long()
    gu = qg.grouped("q4k", x[tok].contiguous(), ex.up, 2 * I, offs, E).float()
    h = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).half()
    o = qg.grouped("q6k", h, ex.dn, H, offs, E).float() * w.reshape(-1)[rows.long()][:, None]
    ref = x.float().index_add_(0, tok, o)
    # the reference rounds gate, up, h and the experts' outputs to fp16: four
    # roundings of 2^-11 against the layer's two
    err = (y.float() - ref).norm() / ref.norm()
    assert float(err) <= 6 * 2.0 ** -11, float(err)


def test_dense_ffn_run_together():
    """Gate/up and down of a dense layer: the gated product hands the
    fragment-major activations to the down product, which adds the residual."""
    M, H, I = 70, 512, 768
    rx, r1, r2 = synth.streams(790, 3)
    x = to_device(synth.activations(rx, M, H, qg.F16), qg.F16)
    ws = []
    for fmt, N, K, rng in (("q4k", 2 * I, H, r1), ("q6k", H, I, r2)):
        f = synth.weight_fields(fmt, rng, N, K)
        for key in ("d", "dmin"):
            if key in f:
                f[key] = synth.f16_bits(f[key].view(np.float16).astype(np.float64) / (np.sqrt(K) * {"q4k": 1.5, "q6k": 7}[fmt]))
        ws.append(bytes_to_device(qg.pack(fmt, synth.encode(fmt, f), N, K)))
    hf = qg.linear_xf("q4k", qg.x_to_xf(x), ws[0], M, I, H, act="silu", gated=True, out_layout=qg.X_FRAG)
    y = qg.linear_xf("q6k", hf, ws[1], M, H, I, residual=x)
    gu = qg.gemm_xf("q4k", qg.x_to_xf(x), ws[0], M, 2 * I, H).float()
    h = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).half()
    ref = x.float() + qg.gemm_xf("q6k", qg.x_to_xf(h), ws[1], M, H, I).float()
    err = (y.float() - ref).norm() / ref.norm()
    assert float(err) <= 6 * 2.0 ** -11, float(err)
