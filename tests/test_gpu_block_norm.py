"""The norms around a block, and their gradients, against the 64-bit formulas."""
import pytest
import torch

import norms_common as plain
from block_common import assert_close, matrix
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu

BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6

# T, d, type, weights' type, gate, (post norm, pre norm), scale, row stride
CASES = [
    (1, 1, F32, F32, "row", (1, 1), 1.0, None), (3, 2, BF, BF, None, (1, 1), 1.0, None),
    (5, 7, FP16, F32, "full", (1, 1), 0.5, None), (4, 8, BF, F32, "full", (1, 1), 1.0, None),
    (33, 31, F32, F32, "row", (1, 1), -2.0, 33), (70, 33, BF, BF, "full", (1, 1), 1.0, None),
    (9, 255, FP16, FP16, None, (1, 1), 2.5, 258), (300, 256, BF, BF, "full", (1, 1), 1.0, None),
    (300, 520, FP16, F32, "row", (1, 1), 1.0, 528), (2000, 64, BF, F32, "full", (1, 1), 1.0, None),
    (64, 1000, BF, BF, "full", (1, 0), 1.0, None), (64, 1000, FP16, FP16, "row", (0, 1), 0.7, None),
    (40, 1000, BF, F32, None, (0, 0), 1.0, None), (40, 96, F32, F32, "full", (0, 1), 1.0, 100),
    (257, 1023, F32, F32, "row", (1, 1), 0.5, None), (31, 1536, BF, BF, "full", (1, 1), 1.0, 1600),
    (5, 2047, BF, BF, "row", (1, 1), 1.0, 2049), (5, 2049, FP16, F32, "full", (1, 1), 1.0, None),
    (170, 4096, BF, BF, "row", (1, 1), 1.0, None), (4, 4096, F32, F32, "full", (1, 1), 1.0, None),
    (160, 7168, BF, BF, "full", (1, 1), 1.0, None), (160, 7168, FP16, F32, "full", (1, 1), 1.0, None),
    (3, 7167, BF, BF, "full", (1, 1), 1.0, None), (310, 8192, BF, F32, "row", (1, 1), 1.0, None),
    # rows that start anywhere: every place of 16 bytes, whole warps of vectors and one more
    (41, 512, BF, F32, "full", (1, 1), 1.0, 513), (23, 1024, FP16, FP16, "row", (1, 1), 1.0, 1027),
    (19, 256, F32, F32, "full", (1, 1), 0.5, 257), (30, 9, BF, BF, "full", (1, 1), 1.0, 10),
    (700, 515, BF, BF, "full", (1, 1), 1.0, None), (333, 4099, FP16, F32, "full", (1, 1), 1.0, 4101),
    (7, 130, BF, BF, "full", (0, 1), 1.0, 131), (7, 1, BF, BF, "full", (1, 0), 1.0, 3),
    (2, 16384, F32, F32, "full", (1, 1), 1.0, None), (2, 16384, BF, BF, "full", (1, 1), 1.0, None),
    (2, 16381, BF, F32, "row", (1, 1), 1.0, None), (3, 12000, BF, BF, "full", (1, 1), 1.0, None),
    # long rows: halves of them, of the same and of different sizes
    (400, 14336, BF, BF, "row", (1, 1), 1.0, None), (170, 8200, FP16, F32, "full", (1, 1), 0.5, 8216),
    (1, 8196, F32, F32, None, (1, 1), 1.0, None), (79, 16384, F32, F32, None, (1, 1), 1.0, None),
    (160, 10248, BF, BF, "full", (1, 0), 1.0, None), (77, 16376, FP16, FP16, "row", (0, 1), 1.0, None),
    (333, 14335, BF, BF, "row", (1, 1), 1.0, None), (40, 9001, FP16, F32, "full", (1, 1), 1.0, 9003),
    (20, 12301, F32, F32, None, (1, 1), 1.0, None), (18, 9217, BF, BF, None, (1, 1), 1.0, 9218),
]
IDS = [f"T{c[0]}d{c[1]}-{str(c[2])[6:]}-{c[4]}-{c[5][0]}{c[5][1]}-ld{c[7] or c[1]}" for c in CASES]


def inputs(case):
    T, d, dt, wt, gate, _, _, ld = case
    gen = torch.Generator().manual_seed(T * 100003 + d)
    m = {k: matrix(T, d, dt, gen, ld, scale=s) for k, s in (("x", 2.0), ("b", 0.7), ("dy", 1.0), ("du", 1.0))}
    m["gate"] = None
    if gate == "full":
        m["gate"] = matrix(T, d, dt, gen, ld, scale=2.0)
    elif gate == "row":
        m["gate"] = matrix(T, 1, F32, gen, scale=2.0)[:, 0].contiguous()
    m["post"], m["pre"] = ((1 + 0.3 * torch.randn(d, generator=gen)).to(wt).cuda() for _ in range(2))
    return m


def cpu(m, *names):
    return [None if m[k] is None else m[k].cpu() for k in names]


def check(got, ref, T, zmax, what=""):
    for name, value in got.items():
        if value is None:
            assert name not in ref, name
            continue
        want, size = ref[name]
        c = plain.C[name] + 2 * zmax + (T if name in ("dpost", "dpre") else 0)
        assert_close(value, want, size, c, what + name)


def steepest(gate):
    """|z| of the gates: what an approximate 2^(z log2 e) may be off by."""
    return 0.0 if gate is None or gate.numel() == 0 else float(gate.float().abs().max())


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_backward(case):
    T, d, dt, wt, _, (post_norm, pre_norm), scale, _ = case
    m = inputs(case)
    kw = dict(gate=m["gate"], scale=scale)
    y, u, r_post, r_pre = moe.moe_block_norm(m["x"], m["b"], m["post"], m["pre"] if pre_norm else None, eps=EPS,
                                             post_norm=bool(post_norm), pre_norm=bool(pre_norm), stats=True, **kw)
    x, b, post, pre, gate, dy, du = cpu(m, "x", "b", "post", "pre", "gate", "dy", "du")
    args = (x, b, post, pre, gate, scale, EPS, post_norm, pre_norm)
    o, z = plain.forward(*args), steepest(gate)
    assert_close(y, o["y"], o["Y"], plain.C["y"] + 2 * z, "y")
    assert (r_post is None) == (not post_norm) and (u is None) == (r_pre is None) == (not pre_norm)
    if post_norm:
        assert_close(r_post, o["r_post"][:, 0], o["r_post"][:, 0], 20, "rstd_post")
    if pre_norm:
        assert_close(u, o["u"], o["U"], plain.C["u"] + 2 * z, "u")
        assert_close(r_pre, o["r_pre"][:, 0], (o["r_pre"] * o["rho"])[:, 0], plain.C["u"] + 2 * z, "rstd_pre")
    y2, u2 = moe.moe_block_norm(m["x"], m["b"], m["post"], m["pre"] if pre_norm else None, eps=EPS,
                                post_norm=bool(post_norm), pre_norm=bool(pre_norm), **kw)
    assert torch.equal(y2, y) and (u is None or torch.equal(u2, u))
    names = ("dx", "db", "dgate", "dpost", "dpre")
    got = moe.moe_block_norm_backward(m["dy"], m["du"] if pre_norm else None, m["x"], m["b"], m["post"],
                                      m["pre"] if pre_norm else None, r_post, r_pre, **kw)
    assert got[3].dtype == wt and (got[4] is None or got[4].dtype == wt)
    check(dict(zip(names, got)), plain.backward(dy, du, *args), T, z)
    if pre_norm:  # no gradient by the stream
        alone = moe.moe_block_norm_backward(None, m["du"], m["x"], m["b"], m["post"], m["pre"], r_post, r_pre, **kw)
        check(dict(zip(names, alone)), plain.backward(None, du, *args), T, z, "alone ")
    # results in the places of inputs
    again = moe.moe_block_norm_backward(m["dy"], m["du"] if pre_norm else None, m["x"], m["b"], m["post"],
                                        m["pre"] if pre_norm else None, r_post, r_pre, dx=m["dy"], db=m["b"], **kw)
    # (the order of sums may go with where the first output's rows start)
    check(dict(zip(names, again)), plain.backward(dy, du, *args), T, z, "in place ")
    assert again[0].data_ptr() == m["dy"].data_ptr() and again[1].data_ptr() == m["b"].data_ptr()
    m = inputs(case)
    y2, u2 = moe.moe_block_norm(m["x"], m["b"], m["post"], m["pre"] if pre_norm else None, eps=EPS, y=m["x"],
                                post_norm=bool(post_norm), pre_norm=bool(pre_norm), gate=m["gate"], scale=scale,
                                u=m["b"] if pre_norm else None)
    assert y2.data_ptr() == m["x"].data_ptr()
    assert_close(y2, o["y"], o["Y"], plain.C["y"] + 2 * z, "y in place")
    if pre_norm:
        assert_close(u2, o["u"], o["U"], plain.C["u"] + 2 * z, "u in place")


@pytest.mark.parametrize("case", [c for c in CASES if c[4] is None or c[1] in (1, 7, 1023, 2049, 7168, 16384)], ids=str)
def test_rmsnorm(case):
    T, d, dt, wt = case[:4]
    m = inputs(case)
    x, pre, dy, du = cpu(m, "x", "pre", "dy", "du")
    u, rstd = moe.moe_rmsnorm(m["x"], m["pre"], EPS, stats=True)
    o = plain.forward(x, None, None, pre, None, 1.0, EPS)
    assert_close(u, o["u"], o["U"], plain.C["u"], "y")
    assert_close(rstd, o["r_pre"][:, 0], o["r_pre"][:, 0], 20, "rstd")
    assert torch.equal(moe.moe_rmsnorm(m["x"], m["pre"], EPS), u)
    for res in (None, dy):
        dx, dgamma = moe.moe_rmsnorm_backward(m["du"], m["x"], m["pre"], rstd, dres=None if res is None else m["dy"])
        check({"dx": dx, "dpre": dgamma}, plain.backward(res, du, x, None, None, pre, None, 1.0, EPS), T, 0)
    ref = plain.backward(dy, du, x, None, None, pre, None, 1.0, EPS)
    again, _ = moe.moe_rmsnorm_backward(m["du"], m["x"], m["pre"], rstd, dres=m["dy"], dx=m["du"])
    check({"dx": again, "dpre": dgamma}, ref, T, 0, "in place ")
    assert_close(moe.moe_rmsnorm(m["x"], m["pre"], EPS, y=m["x"]), o["u"], o["U"], plain.C["u"], "y in place")


def test_without_weights():
    T, d = 37, 200
    gen = torch.Generator().manual_seed(4)
    x, b, dy, du = (matrix(T, d, BF, gen) for _ in range(4))
    y, u, rp, rq = moe.moe_block_norm(x, b, stats=True)
    o = plain.forward(x.cpu(), b.cpu(), None, None, None, 1.0, EPS)
    assert_close(y, o["y"], o["Y"], plain.C["y"], "y")
    assert_close(u, o["u"], o["U"], plain.C["u"], "u")
    ref = plain.backward(dy.cpu(), du.cpu(), x.cpu(), b.cpu(), None, None, None, 1.0, EPS)
    for wdtype in (None, BF):
        dx, db, dgate, dpost, dpre = moe.moe_block_norm_backward(dy, du, x, b, None, None, rp, rq, wdtype=wdtype)
        assert dpost.dtype == dpre.dtype == (wdtype or F32)
        check(dict(dx=dx, db=db, dgate=dgate, dpost=dpost, dpre=dpre), ref, T, 0)


@pytest.mark.parametrize("d,ld", [(256, 256), (1023, 1023), (7168, 7168)])
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_zero_rows_and_steep_gates(d, ld, dt):
    """Rows of zeros (the root of eps alone), gates that are shut, open or infinite."""
    T = 8
    gen = torch.Generator().manual_seed(d)
    x, b, dy, du = (matrix(T, d, dt, gen) for _ in range(4))
    b[0], x[1], b[2], x[2] = 0, 0, 0, 0
    z = torch.zeros(T, device="cuda")
    z[3], z[4], z[5], z[6] = float("-inf"), float("inf"), -200.0, 90.0
    for gate in (z, z[:, None].expand(T, d).to(dt).contiguous()):
        y, u, rp, rq = moe.moe_block_norm(x, b, gate=gate, eps=EPS, stats=True)
        got = moe.moe_block_norm_backward(dy, du, x, b, None, None, rp, rq, gate=gate)
        args = (x.cpu(), b.cpu(), None, None, gate.cpu(), 1.0, EPS)
        o = plain.forward(*args)
        assert_close(y, o["y"], o["Y"], 250, "y")
        assert_close(u, o["u"], o["U"], 300, "u")
        check(dict(zip(("dx", "db", "dgate", "dpost", "dpre"), got)), plain.backward(dy.cpu(), du.cpu(), *args), T, 200)


@pytest.mark.parametrize("T,d,dt", [(45, 300, BF), (45, 300, F32), (91, 9000, BF), (20, 8501, F32)], ids=str)
def test_operands_that_start_at_different_places(T, d, dt):
    """Each operand in a buffer of its own stride and start."""
    gen = torch.Generator().manual_seed(17)

    def mat(ld, start):
        v = torch.randn(T * ld + start + d, generator=gen).to(dt).cuda()
        return torch.as_strided(v, (T, d), (ld, 1), start)

    x, b, gate, dy, du = mat(d + 1, 0), mat(d + 3, 1), mat(d, 3), mat(d + 7, 2), mat(d + 2, 5)
    y, u, dx, db = mat(d + 5, 4), mat(d, 0), mat(d + 9, 7), mat(d + 4, 1)
    w = torch.randn(d, generator=gen).to(dt).cuda()
    _, _, rp, rq = moe.moe_block_norm(x, b, w, w, gate=gate, stats=True, y=y, u=u)
    args = (x.cpu(), b.cpu(), w.cpu(), w.cpu(), gate.cpu(), 1.0, EPS)
    o, z = plain.forward(*args), steepest(gate)
    assert_close(y, o["y"], o["Y"], plain.C["y"] + 2 * z, "y")
    assert_close(u, o["u"], o["U"], plain.C["u"] + 2 * z, "u")
    got = moe.moe_block_norm_backward(dy, du, x, b, w, w, rp, rq, gate=gate, dx=dx, db=db)
    check(dict(zip(("dx", "db", "dgate", "dpost", "dpre"), got)), plain.backward(dy.cpu(), du.cpu(), *args), T, z)


@pytest.mark.parametrize("d", [203, 9003])
def test_writes_nothing_else(d):
    """What lies around the rows of the outputs stays as it was."""
    T, ld = 37, d + 7
    gen = torch.Generator().manual_seed(18)
    x, b, gate, dy, du = (matrix(T, d, BF, gen, d + 2) for _ in range(5))
    bufs = [torch.full((T + 2, ld), 7.0, device="cuda", dtype=BF) for _ in range(4)]
    y, u, dx, db = (v[1:-1, 3:3 + d] for v in bufs)
    _, _, rp, rq = moe.moe_block_norm(x, b, gate=gate, stats=True, y=y, u=u)
    moe.moe_block_norm_backward(dy, du, x, b, None, None, rp, rq, gate=gate, dx=dx, db=db)
    for v, inner in zip(bufs, (y, u, dx, db)):
        assert not (inner == 7.0).all()
        inner.fill_(7.0)
        assert (v == 7.0).all()


@pytest.mark.parametrize("T,d,ld", [(1, 7, 7), (3, 1001, 1001), (9, 130, 131), (17, 64, 64), (40, 7, 9), (500, 33, 33)])
def test_scratch_of_the_stated_size(T, d, ld):
    """The partial weight sums stay inside moe_block_norm_scratch_bytes."""
    gen = torch.Generator().manual_seed(T)
    x, b, dy, du = (matrix(T, d, BF, gen, ld) for _ in range(4))
    _, _, rp, rq = moe.moe_block_norm(x, b, stats=True)
    want = moe.moe_block_norm_backward(dy, du, x, b, None, None, rp, rq)
    nbytes = int(moe.lib().moe_block_norm_scratch_bytes(T, d))
    buf = torch.full((nbytes + (1 << 20),), 113, dtype=torch.uint8, device="cuda")
    got = moe.moe_block_norm_backward(dy, du, x, b, None, None, rp, rq, scratch=buf[:nbytes])
    assert (buf[nbytes:] == 113).all()
    assert all(p is q is None or torch.equal(p, q) for p, q in zip(got, want))


def test_not_a_number_stays_in_its_row():
    T, d = 40, 512
    gen = torch.Generator().manual_seed(2)
    x, b, gate, dy, du = (matrix(T, d, BF, gen) for _ in range(5))
    clean = moe.moe_block_norm(x, b, gate=gate)
    for t, m in ((3, x), (5, b), (7, gate)):
        m[t, 100] = float("nan")
    b[9, 0] = float("inf")
    y, u, rp, rq = moe.moe_block_norm(x, b, gate=gate, stats=True)
    rows = torch.ones(T, dtype=torch.bool)
    rows[[3, 5, 7, 9]] = False
    assert torch.equal(y[rows], clean[0][rows]) and torch.equal(u[rows], clean[1][rows])
    for t in (3, 5, 7, 9):
        assert u[t].isnan().all() and y[t].isnan().any()
    dx, db, dgate, _, _ = moe.moe_block_norm_backward(dy, du, x, b, None, None, rp, rq, gate=gate)
    for g in (dx, db, dgate):
        assert g[rows].isfinite().all() and g[3].isnan().all() and g[9].isnan().any()


def test_gradients_by_differences():
    T, d = 6, 72
    gen = torch.Generator().manual_seed(8)
    v = {k: torch.randn(T, d, generator=gen).cuda() for k in ("x", "b", "gate")}
    v |= {k: 1 + 0.2 * torch.randn(d, generator=gen).cuda() for k in ("post", "pre")}
    dy, du = (torch.randn(T, d, generator=gen).cuda() for _ in range(2))

    def loss(v):
        y, u = moe.moe_block_norm(**v, scale=0.5)
        return float((y.double() * dy.double()).sum() + (u.double() * du.double()).sum())

    _, _, rp, rq = moe.moe_block_norm(**v, scale=0.5, stats=True)
    dx, db, dgate, dpost, dpre = moe.moe_block_norm_backward(dy, du, v["x"], v["b"], v["post"], v["pre"], rp, rq,
                                                             gate=v["gate"], scale=0.5)
    for name, grad in dict(x=dx, b=db, gate=dgate, post=dpost, pre=dpre).items():
        step = torch.randn(grad.shape, generator=gen).cuda()
        step /= step.norm()
        h = 2.0 ** -6
        plus, minus = (loss(v | {name: v[name] + s * step}) for s in (h, -h))
        want = float((grad.double() * step.double()).sum())
        # the difference's own error: h^2 / 6 times a third derivative of order 10 per unit
        # step and output (2 T d outputs of order 1), and fp32 roundings of the outputs over h
        slack = h * h / 6 * 10 * (2 * T * d) ** 0.5 + 2.0 ** -20 * (2 * T * d) ** 0.5 / h
        assert abs((plus - minus) / (2 * h) - want) <= slack, (name, (plus - minus) / (2 * h), want)


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    y, u, rp, rq = moe.moe_block_norm(x, x, gate=x, stats=True)
    assert y.shape == u.shape == (0, 64) and rp.shape == (0,)
    out = moe.moe_block_norm_backward(x, x, x, x, None, None, rp, rq, gate=x)
    assert out[0].shape == out[1].shape == out[2].shape == (0, 64)
    assert not out[3].any() and not out[4].any() and out[3].shape == (64,)


def test_leading_dimensions():
    gen = torch.Generator().manual_seed(1)
    x, b = (torch.randn(3, 5, 72, generator=gen).cuda() for _ in range(2))
    gate = torch.randn(3, 5, generator=gen).cuda()
    y, u, rp, rq = moe.moe_block_norm(x, b, gate=gate, stats=True)
    assert y.shape == x.shape and rp.shape == (3, 5)
    flat = moe.moe_block_norm(x.view(15, 72), b.view(15, 72), gate=gate.view(15))
    assert torch.equal(y.view(15, 72), flat[0]) and torch.equal(u.view(15, 72), flat[1])
    dx, db, dgate, _, _ = moe.moe_block_norm_backward(y, u, x, b, None, None, rp, rq, gate=gate)
    assert dx.shape == db.shape == x.shape and dgate.shape == (3, 5)
    one = moe.moe_block_norm(x[0, 0], b[0, 0])
    assert one[0].shape == (72,)


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements into their buffers."""
    T, d, ld = 35, 64, 1 << 26
    gen = torch.Generator().manual_seed(6)
    x, b = (torch.empty(T * ld, dtype=FP16, device="cuda").view(T, ld)[:, :d] for _ in range(2))
    x.copy_(torch.randn(T, d, generator=gen)), b.copy_(torch.randn(T, d, generator=gen))
    want = moe.moe_block_norm(x.contiguous(), b.contiguous(), gate=b.contiguous(), stats=True)
    y, u, rp, rq = moe.moe_block_norm(x, b, gate=b, stats=True, y=torch.empty_like(want[0]))
    assert torch.equal(y, want[0]) and torch.equal(u, want[1])
    want = moe.moe_block_norm_backward(y, u, x.contiguous(), b.contiguous(), None, None, rp, rq, gate=b.contiguous())
    got = moe.moe_block_norm_backward(y, u, x, b, None, None, rp, rq, gate=b, dx=x)  # (all rows start on 16 bytes)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("T,d", [(300, 1024), (200, 9000), (90, 9001)])
def test_captured_calls_and_streams(T, d):
    gen = torch.Generator().manual_seed(11)
    x, b, gate, dy = (matrix(T, d, BF, gen) for _ in range(4))

    def step():
        y, u, rp, rq = moe.moe_block_norm(x, b, gate=gate, stats=True)
        return y, u, *moe.moe_block_norm_backward(dy, u, x, b, None, None, rp, rq, gate=gate)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        x.copy_(torch.randn(T, d, generator=gen))
        graph.replay()
        for p, q in zip(out, step()):
            assert torch.equal(p, q)
    want = moe.moe_block_norm(x, b, gate=gate)
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_block_norm(x, b, gate=gate, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_backward_passes_at_once():
    """Calls on two streams, whose kernels run side by side."""
    gen = torch.Generator().manual_seed(12)
    sets = [[matrix(T, d, BF, gen) for _ in range(4)] for T, d in ((600, 12000), (700, 8960))]
    stats = [moe.moe_block_norm(x, b, stats=True)[2:] for x, b, _, _ in sets]

    def back(k):
        x, b, dy, du = sets[k]
        return moe.moe_block_norm_backward(dy, du, x, b, None, None, *stats[k])

    want = [back(0), back(1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((k, back(k)))
    torch.cuda.synchronize()
    assert all(p is q is None or torch.equal(p, q) for k, out in got for p, q in zip(out, want[k]))
