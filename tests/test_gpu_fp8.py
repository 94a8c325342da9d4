"""GPU parity of the rounding to e4m3 with a scale for each group of 128 and of the
product of such values, against their FP64 oracle.

Tolerances:
- an 8-bit value is the nearest one of x / scale, except where that quotient lies
  within the fp32 arithmetic's error of the middle of two: the quotient 448 / m and
  the product, 2^-24 each, and 448's own product with m's scale: 2e-7 of the value;
- a scale is one fp32 division: 2^-24;
- the product: its values are exact in fp32 or wider, a group's 128 of them are
  summed by the tensor cores in at least 24 bits, each addition off by at most
  2^-23 of the partial sum where it cuts off: normwise 128 x 1.2e-7 = 1.5e-5 at the
  very worst, sqrt(128) x 1.2e-7 = 1.4e-6 where signs are random, and one rounding of
  2^-24 per group and for the scales; 1e-5 for fp32 outputs, and for bf16 ones a
  rounding of at most 2^-8 = 3.91e-3 more: 4e-3. (Over 8194 groups with random signs: the partial sum behind group g is
  sqrt(g / 8194) of the last one, so the roundings come to sqrt(8194 / 2) x 2^-24 = 3.9e-6 beside the 1.4e-6.)
"""

import numpy as np
import pytest
import torch

from oracle import layer
from tests.helpers import check_close, np64
from tests.test_gpu_layer import DT, gen_of

pytestmark = pytest.mark.gpu


def values(R, D, seed, io="bf16"):
    g = gen_of(seed)
    big = torch.where(torch.rand(D, generator=g) < 0.05, 30.0, 1.0)
    return (torch.randn(R, D, generator=g) * big).to(DT[io])


def check_q(q, scale, x, rows):
    """q the nearest values, scale to a rounding."""
    _, s, y = layer.quant8(np64(x), rows)
    assert np.all(np.abs(np64(scale) - s) <= 2.0 ** -23 * s)
    q = np64(q.float())
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    assert np.all(np.abs(q - y) <= step / 2 + 2e-7 * np.abs(y))


SHAPES = [(1, 1), (1, 128), (3, 5), (128, 128), (129, 127), (200, 300), (64, 4096), (1, 4096), (257, 16), (16, 257), (130, 1000)]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("R,D", SHAPES)
@pytest.mark.parametrize("blocks", [False, True])
def test_quant8_matches_oracle(io, R, D, blocks):
    import chunkwise_delta_rule_gb300 as kda
    x = values(R, D, 41, io)
    rows = 128 if blocks else 1
    both = kda.kda_quant8(kda.make_quant8_problem(x.cuda(), blocks=blocks, transposed=True))
    assert both.q.shape == (R, D) and both.qt.shape == (D, R) and both.q.dtype == torch.float8_e4m3fn
    assert both.q.stride(0) % 16 == 0 or R == 1
    check_q(both.q, both.scale, x, rows)
    check_q(both.qt, both.scale_t, x.t(), rows)
    for a, b in ((True, False), (False, True)):
        one = kda.kda_quant8(kda.make_quant8_problem(x.cuda(), blocks=blocks, rows=a, transposed=b))
        assert (one.q is None) == (not a) and (one.qt is None) == (not b)
        for s, t in zip(one, both):
            assert s is None or torch.equal(s.float(), t.float())


def test_quant8_of_strided_rows_and_more_axes():
    import chunkwise_delta_rule_gb300 as kda
    for io in ("bf16", "fp32"):
        x = values(150, 320, 42, io).cuda()
        want = kda.kda_quant8(kda.make_quant8_problem(x[:, 37:301].contiguous(), transposed=True))
        got = kda.kda_quant8(kda.make_quant8_problem(x[:, 37:301], transposed=True))
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(want, got))
        y = x[:, :256].unflatten(0, (2, 3, 25))
        r = kda.kda_quant8(kda.make_quant8_problem(y, transposed=True))
        want = kda.kda_quant8(kda.make_quant8_problem(x[:, :256], transposed=True))
        assert r.q.shape == y.shape and r.scale.shape == (2, 3, 25, 2)
        assert torch.equal(r.q.float().flatten(0, 2), want.q.float()) and torch.equal(r.scale.flatten(0, 2), want.scale)
        assert torch.equal(r.qt.float(), want.qt.float())
    with pytest.raises(ValueError, match="rows must be evenly spaced"):
        kda.make_quant8_problem(x[:, :256].unflatten(0, (2, 75))[:, :70])
    with pytest.raises(ValueError, match="rows must be dense"):
        kda.make_quant8_problem(x[:, ::2])
    with pytest.raises(ValueError, match="rows must be dense"):
        kda.make_quant8_problem(x[:1].expand(5, 320))
    with pytest.raises(ValueError, match="one of rows and transposed"):
        kda.make_quant8_problem(x, rows=False)
    for shape in ((0, 64), (3, 0, 64)):
        r = kda.kda_quant8(kda.make_quant8_problem(torch.zeros(shape, device="cuda"), transposed=True))
        assert r.q.shape == shape and r.qt.shape == (64, 0)


@pytest.mark.parametrize("blocks", [False, True])
def test_quant8_of_the_ends_of_the_range(blocks):
    """Groups of zeros, of the smallest and of the largest values, and of NaN and infinities beside ordinary ones."""
    import chunkwise_delta_rule_gb300 as kda
    x = torch.linspace(-1, 1, 128).repeat(128, 8)
    for i, f in enumerate((0.0, 1e-45, 1e-38, 1e-30, 1e30, 3e38)):
        x[:, 128 * i:128 * (i + 1)] *= f
    clean = x.clone()
    x[5, 128 * 6 + 3], x[7, 128 * 7 + 4] = float("nan"), float("inf")
    r = kda.kda_quant8(kda.make_quant8_problem(x.cuda(), blocks=blocks, transposed=not blocks))
    q, s = np64(r.q.float()), np64(r.scale)
    assert not q[:, :128].any() and not s[:, 0].any()
    rows = 128 if blocks else 1
    for i in range(2, 6):       # (at 1e-45 the values themselves are 0 and 2^-149)
        part = clean[:, 128 * i:128 * (i + 1)]
        want = np.repeat(layer.quant8(np64(part), rows)[1], rows, 0)
        back = q[:, 128 * i:128 * (i + 1)] * s.repeat(rows, 0)[:, i:i + 1]
        assert np.all(np.abs(back - np64(part)) <= np.maximum(np.abs(np64(part)) / 16, want / 1024) * (1 + 1e-5) + 1e-45)
    if blocks:
        assert np.isnan(s[0, 6]) and np.isinf(s[0, 7]) and np.all(np.isfinite(s[0, :6]))
    else:
        assert np.isnan(s[5, 6]) and np.isinf(s[7, 7]) and np.sum(~np.isfinite(s)) == 2
        st = np64(r.scale_t)
        assert np.isnan(st[128 * 6 + 3, 0]) and np.isinf(st[128 * 7 + 4, 0]) and np.sum(~np.isfinite(st)) == 2


# ------------------------------------------------------------------ the product

def mm_case(M, N, K, b, seed):
    g = gen_of(seed)
    a = (torch.randn(M, K, generator=g) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
    w = (torch.randn(N, K, generator=g) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
    G = -(-K // 128)
    sa = torch.exp2(4 * torch.rand(M, G, generator=g) - 8)
    sb = torch.exp2(4 * torch.rand(N if b == "rows" else -(-N // 128), G, generator=g) - 8)
    return a, sa, w, sb


def mm_ref(a, sa, w, sb):
    return layer.mm8(np64(a.float()), np64(sa), np64(w.float()), np64(sb))


def cuda(*t):
    return [x.cuda() for x in t]


MM = [(1, 1, 1), (1, 128, 128), (2, 16, 16), (3, 5, 7), (64, 128, 256), (1, 4096, 512), (7, 1000, 1111), (16, 256, 2048), (17, 129, 130),
      (64, 512, 4096), (65, 257, 384), (128, 128, 128), (129, 255, 640), (200, 384, 100), (300, 1000, 1040), (777, 130, 272),
      (256, 512, 1024), (1030, 16, 4096), (128, 1, 128),
      (2000, 1300, 300), (1537, 1793, 140), (4100, 770, 1100), (3, 5, (1 << 20) + 200)]


@pytest.mark.parametrize("M,N,K", MM)
@pytest.mark.parametrize("b", ["blocks", "rows"])
def test_mm8_matches_oracle(M, N, K, b):
    import chunkwise_delta_rule_gb300 as kda
    c = mm_case(M, N, K, b, 43)
    ref = mm_ref(*c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out, tol in (("fp32", 1e-5), ("bf16", 4e-3)):
        y = kda.kda_mm8(kda.make_mm8_problem(*cuda(*c), out=out), err=err)
        assert y.shape == (M, N) and y.dtype == DT[out]
        check_close(out, np64(y), ref, tol)
        assert torch.equal(y, kda.kda_mm8(kda.make_mm8_problem(*cuda(*c), out=out)))
    assert int(err) == 0


@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (300, 384, 1024)])
def test_mm8_adds_up_whole_numbers_exactly(M, N, K):
    """Small whole numbers and scales that are powers of two: every partial sum fits 24 bits."""
    import chunkwise_delta_rule_gb300 as kda
    g = gen_of(44)
    a = torch.randint(-8, 9, (M, K), generator=g).float().to(torch.float8_e4m3fn)
    w = torch.randint(-8, 9, (N, K), generator=g).float().to(torch.float8_e4m3fn)
    sa = torch.exp2(torch.randint(-2, 3, (M, K // 128), generator=g).float())
    sb = torch.exp2(torch.randint(-2, 3, (N // 128, K // 128), generator=g).float())
    y = kda.kda_mm8(kda.make_mm8_problem(*cuda(a, sa, w, sb), out="fp32"))
    assert np.array_equal(np64(y), mm_ref(a, sa, w, sb))


def test_mm8_of_strided_rows_and_more_axes():
    """Rows that start on any address, and a's leading axes."""
    import chunkwise_delta_rule_gb300 as kda
    for M, N, K, off in ((40, 140, 272, 16), (40, 140, 272, 1), (200, 300, 257, 3), (3, 260, 512, 48)):
        a, sa, w, sb = mm_case(M, N, K, "blocks", 45)
        ref = mm_ref(a, sa, w, sb)
        wide = [torch.full((t.shape[0], K + 64), 448.0).to(torch.float8_e4m3fn) for t in (a, w)]
        for x, t in zip(wide, (a, w)):
            x[:, off:off + K] = t
        x, z = (t.cuda()[:, off:off + K] for t in wide)
        sac, sbc = cuda(sa, sb)
        y = kda.kda_mm8(kda.make_mm8_problem(x, sac, z, sbc, out="fp32"))
        check_close("y", np64(y), ref, 1e-5)
        mixed = kda.kda_mm8(kda.make_mm8_problem(x, sac, w.cuda(), sbc, out="fp32"))
        check_close("y", np64(mixed), ref, 1e-5)
    a, sa, w, sb = mm_case(24, 130, 256, "blocks", 46)
    y = kda.kda_mm8(kda.make_mm8_problem(a.cuda().unflatten(0, (2, 3, 4)), sa.cuda().unflatten(0, (2, 3, 4)), *cuda(w, sb), out="fp32"))
    assert y.shape == (2, 3, 4, 130)
    check_close("y", np64(y).reshape(24, 130), mm_ref(a, sa, w, sb), 1e-5)
    none = kda.kda_mm8(kda.make_mm8_problem(a.cuda()[:0], sa.cuda()[:0], *cuda(w, sb)))
    assert none.shape == (0, 130)


@pytest.mark.parametrize("M", [2, 200])
def test_mm8_keeps_rows_apart(M):
    """A NaN or an infinity, in a value or a scale, reaches its row or column of y and no other."""
    import chunkwise_delta_rule_gb300 as kda
    a, sa, w, sb = mm_case(M, 300, 300, "rows", 47)
    ref = mm_ref(a, sa, w, sb)
    a[1, 17], sa[0, 2], w[5, 299], sb[129, 0] = float("nan"), float("inf"), float("nan"), float("nan")
    y = np64(kda.kda_mm8(kda.make_mm8_problem(*cuda(a, sa, w, sb), out="fp32")))
    rows, cols = np.arange(M) > 1, ~np.isin(np.arange(300), (5, 129))
    assert not np.isfinite(y[:2]).any() and not np.isfinite(y[:, ~cols]).any()
    if M > 2:
        check_close("y", y[rows][:, cols], ref[rows][:, cols], 1e-5)


def test_mm8_into_a_given_output_and_its_refusals():
    import chunkwise_delta_rule_gb300 as kda
    c = cuda(*mm_case(33, 64, 256, "blocks", 48))
    p = kda.make_mm8_problem(*c, out="fp32")
    y = torch.empty(33, 64, device="cuda")
    assert kda.kda_mm8(p, y=y).data_ptr() == y.data_ptr() and torch.equal(y, kda.kda_mm8(p))
    for match, call in (("y must be", lambda: kda.kda_mm8(p, y=y.bfloat16())), ("y must be", lambda: kda.kda_mm8(p, y=y[:32])),
                        ("err must be", lambda: kda.kda_mm8(p, err=torch.zeros(1, dtype=torch.int32))),
                        ("scale_a must be", lambda: kda.make_mm8_problem(c[0], c[1][:, :1].contiguous(), c[2], c[3])),
                        ("scale_a must be", lambda: kda.make_mm8_problem(c[0], c[1].double(), c[2], c[3])),
                        ("scale_b must be", lambda: kda.make_mm8_problem(c[0], c[1], c[2], c[1])),
                        ("b must be", lambda: kda.make_mm8_problem(c[0], c[1], c[2][:, :128], c[3])),
                        ("b must be", lambda: kda.make_mm8_problem(c[0], c[1], c[2].cpu(), c[3])),
                        ("a's rows must be dense", lambda: kda.make_mm8_problem(c[0][:, ::2], c[1][:, :1].contiguous(), c[2][:, :128], c[3]))):
        with pytest.raises(ValueError, match=match):
            call()


def test_the_norms_rows_go_into_the_product():
    """The residual stream's norm with 8-bit rows, and the projection that reads them."""
    import chunkwise_delta_rule_gb300 as kda
    for R, D, N in ((5, 512, 384), (300, 640, 256)):
        x, w, g = values(R, D, 49).cuda(), values(N, D, 50, "fp32").cuda() * 0.02, torch.ones(D, device="cuda")
        q, s, _ = kda.kda_norm_fwd(kda.make_norm_problem(x, g, out="e4m3", group=128))
        b = kda.kda_quant8(kda.make_quant8_problem(w, blocks=True))
        y = kda.kda_mm8(kda.make_mm8_problem(q, s, b.q, b.scale))
        check_close("y", np64(y), mm_ref(q.cpu(), s.cpu(), b.q.cpu(), b.scale.cpu()), 4e-3)
        # against the unrounded values: 2^-4 of each value at most, 2^-4 sqrt(2) / sqrt(3) of a sum's norm for
        # roundings that are spread evenly and independent
        want = layer.norm(np64(x), np64(g), None, 1e-6)["y"] @ np64(w).T
        check_close("y", np64(y), want, 2.0 ** -4 * (2 / 3) ** 0.5)


@pytest.mark.parametrize("io,wio", [("bf16", "fp32"), ("fp32", "bf16"), ("bf16", "bf16")])
def test_linear8_gradients(io, wio):
    """y, dx and dweight are the products of the values that the roundings stand for."""
    import chunkwise_delta_rule_gb300 as kda
    x, w, dy = values(150, 264, 51, io), values(200, 264, 52, wio), values(150, 200, 53, io)
    xl, wl = x.cuda().unflatten(0, (3, 50)).requires_grad_(), w.cuda().requires_grad_()
    y = kda.linear8(xl, wl)
    assert y.shape == (3, 50, 200) and y.dtype == DT[io]
    y.backward(dy.cuda().unflatten(0, (3, 50)))

    def held(t, rows, transposed=False):
        r = kda.kda_quant8(kda.make_quant8_problem(t.cuda(), blocks=rows == 128, rows=not transposed, transposed=transposed))
        q, s = (r.qt, r.scale_t) if transposed else (r.q, r.scale)
        q, s = np64(q.float()), np64(s)
        return q * np.repeat(np.repeat(s, rows, 0)[:q.shape[0]], 128, 1)[:, :q.shape[1]]

    hw = held(w, 128)
    for name, got, want in (("y", y, held(x, 1) @ hw.T), ("dx", xl.grad, held(dy, 1) @ hw),
                            ("dw", wl.grad, held(dy, 1, True) @ held(x, 1, True).T)):
        check_close(name, np64(got).reshape(want.shape), want, 4e-3 if got.dtype == torch.bfloat16 else 1e-5)
    # one of the two alone
    w2 = w.cuda().requires_grad_()
    kda.linear8(x.cuda(), w2).backward(dy.cuda())
    assert torch.equal(w2.grad, wl.grad)
    x2 = x.cuda().requires_grad_()
    kda.linear8(x2, w.cuda()).backward(dy.cuda())
    assert torch.equal(x2.grad, xl.grad.flatten(0, 1))
    with torch.no_grad():
        assert torch.equal(kda.linear8(x.cuda(), w.cuda()), y.flatten(0, 1))


def test_linear8_of_more_than_2_20_tokens():
    """The weight's gradient sums over all that the forward takes."""
    import chunkwise_delta_rule_gb300 as kda
    n = (1 << 20) + 40
    x, w, dy = values(n, 16, 61), values(8, 16, 62), values(n, 8, 63)
    wl = w.cuda().float().requires_grad_()
    kda.linear8(x.cuda(), wl).backward(dy.cuda())

    def held(t):
        r = kda.kda_quant8(kda.make_quant8_problem(t.cuda(), rows=False, transposed=True))
        return np64(r.qt.float()) * np.repeat(np64(r.scale_t), 128, 1)[:, :n]

    check_close("dw", np64(wl.grad), held(dy) @ held(x).T, 1e-5)


def test_linear8_without_tokens():
    import chunkwise_delta_rule_gb300 as kda
    x = torch.zeros(2, 0, 64, device="cuda", requires_grad=True)
    w = torch.ones(32, 64, device="cuda", requires_grad=True)
    y = kda.linear8(x, w)
    y.sum().backward()
    assert y.shape == (2, 0, 32) and x.grad.shape == x.shape and w.grad.shape == w.shape and not w.grad.any()


def test_graph_and_streams():
    """A captured product replays on new values; products on two streams at once keep theirs."""
    import chunkwise_delta_rule_gb300 as kda
    for M, N, K in ((1, 512, 1024), (300, 300, 1000)):
        c = cuda(*mm_case(M, N, K, "blocks", 54))
        p = kda.make_mm8_problem(*c, out="fp32")
        kda.kda_mm8(p)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = kda.kda_mm8(p)
        for seed in (55, 56):
            for t, new in zip(c, mm_case(M, N, K, "blocks", seed)):
                t.copy_(new)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, kda.kda_mm8(p))
        cases = [kda.make_mm8_problem(*cuda(*mm_case(M, N, K, "blocks", s)), out="fp32") for s in (57, 58)]
        want = [kda.kda_mm8(q) for q in cases]
        streams = [torch.cuda.Stream() for _ in cases]
        torch.cuda.synchronize()
        got = [[kda.kda_mm8(q, stream=s) for q, s in zip(cases, streams)] for _ in range(6)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for row in got for a, b in zip(row, want))
