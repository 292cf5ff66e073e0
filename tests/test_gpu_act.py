"""GPU parity of the layer with its epilogue (tq_linear_act) against the fp64 reference, through the C ABI: every
element of Y within the bound of act_testutil.act_rows, which counts the roundings of the kernels."""

from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import rank_augmented_quantized_amd as tq  # noqa: E402
from act_testutil import ACTS, act_rows, assert_within  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tq.load()


def make(n, d, m, r, seed, x="bf16", bias=True, res=None, gated=False, scale=1.0):
    """Inputs on the CPU (fp32 values already rounded to their type)."""
    g = torch.Generator().manual_seed(seed)
    X = (torch.randn((n, d), generator=g) * scale).to(DT[x])
    X[:, d // 3] *= 8
    codes = torch.randint(0, 256, (m, d // 2), generator=g, dtype=torch.uint8)
    s_w = (0.5 + torch.rand(m, generator=g)) * (0.25 / d ** 0.5)
    l1 = l2 = None
    if r:
        l1 = (torch.randn((d, r), generator=g) / d ** 0.5).bfloat16()
        l2 = (torch.randn((r, m), generator=g) / r ** 0.5).bfloat16()
    b = torch.randn(m, generator=g) if bias else None
    mo = m // 2 if gated else m
    rs = torch.randn((n, mo), generator=g).to(DT[res]) if res else None
    return X, codes, s_w, l1, l2, b, rs


def reference(X, codes, s_w, l1, l2, b, rs, act, gated, y):
    f = lambda t: None if t is None else t.float().numpy()  # noqa: E731
    return act_rows(f(X), codes.numpy(), f(s_w), f(l1), f(l2), f(b), act, gated, f(rs), y)


def call(X, codes, s_w, l1, l2, b, rs, act, gated, y, ws=None, Y=None):
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    m, r = codes.shape[0], 0 if l1 is None else l1.shape[1]
    lr = tq.tq_pack_lowrank(dev(l1), dev(l2)) if r else None
    return tq.tq_linear_act(dev(X), dev(codes), dev(s_w), lr, m, r, bias=dev(b), act=ACTS[act], gated=gated, residual=dev(rs),
                            y_dtype=DT[y], ws=ws, Y=Y)


CASES = [
    # n, d, m, r, x, y, act, gated, bias, residual
    (1, 32, 1, 0, "f32", "f32", "none", False, True, None),  # one value; a row shorter than a load step
    (1, 96, 17, 1, "bf16", "f32", "relu", False, True, "f32"),
    (2, 64, 16, 8, "bf16", "bf16", "silu", True, False, None),
    (3, 512, 1001, 16, "f32", "f32", "gelu", False, True, "f32"),
    (5, 1056, 50, 256, "bf16", "f32", "gelu_tanh", True, True, "bf16"),
    (15, 4096, 258, 64, "bf16", "bf16", "silu", True, True, "bf16"),
    (16, 544, 300, 32, "f32", "bf16", "gelu", False, True, None),
    (17, 2048, 129, 100, "bf16", "f32", "none", False, False, "bf16"),
    (31, 8192, 70, 64, "bf16", "f32", "silu", True, False, "f32"),
    (33, 256, 514, 32, "bf16", "bf16", "gelu_tanh", True, True, "bf16"),
    (47, 160, 333, 48, "f32", "f32", "silu", False, True, "f32"),
    (130, 1024, 520, 128, "bf16", "f32", "gelu", True, True, "f32"),
    (200, 512, 1000, 0, "bf16", "bf16", "relu", True, True, None),
    (300, 2080, 640, 64, "f32", "f32", "none", False, True, "bf16"),
    (1030, 512, 514, 32, "bf16", "f32", "silu", True, False, None),
    (1100, 4096, 260, 200, "bf16", "bf16", "none", False, False, "bf16"),
    # few rows: every kernel by row length, the longest rows, all ranks
    (2, 16416, 40, 32, "bf16", "f32", "silu", True, True, "f32"),
    (3, 65536, 24, 200, "bf16", "bf16", "none", False, True, None),
    (8, 14336, 77, 64, "f32", "f32", "gelu_tanh", False, True, "f32"),
    (9, 5120, 66, 200, "bf16", "f32", "relu", True, True, "bf16"),
    (20, 3968, 130, 256, "bf16", "f32", "none", False, False, None),
    (12, 2048, 5000, 0, "bf16", "bf16", "silu", True, False, None),
    # many rows: 256 x 256 and 256 x 128 tiles, whole and ragged, each residual and its absence
    (40, 64, 57400, 16, "bf16", "bf16", "silu", False, True, "bf16"),
    (270, 160, 57344, 32, "bf16", "bf16", "none", False, False, "bf16"),
    (70, 96, 57402, 40, "f32", "f32", "silu", True, True, "f32"),
    (33, 288, 57600, 64, "bf16", "bf16", "silu", True, False, "bf16"),
    (200, 96, 28700, 100, "bf16", "f32", "relu", False, True, "f32"),
    (129, 512, 28672, 32, "bf16", "bf16", "silu", True, True, None),
    (250, 64, 28673, 8, "bf16", "bf16", "none", False, True, "bf16"),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_linear_act(case):
    n, d, m, r, x, y, act, gated, bias, res = case
    args = make(n, d, m, r, 40 + n, x, bias, res, gated)
    out = call(*args, act, gated, y)
    torch.cuda.synchronize()
    assert_within(out.float().cpu().numpy(), *reference(*args, act, gated, y), what=str(case))


@pytest.mark.parametrize("n", [4, 40])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", sorted(ACTS))
def test_every_activation_over_its_whole_range(n, gated, act):
    """Large pre-activations of both signs: saturated sigmoids, exp past its range, the far tails of gelu."""
    args = list(make(n, 128, 96, 8, 7, "f32", True, None, gated))
    args[5] = torch.linspace(-200.0, 200.0, 96)[torch.randperm(96, generator=torch.Generator().manual_seed(3))]
    for y in ("f32", "bf16"):
        out = call(*args, act, gated, y)
        assert_within(out.float().cpu().numpy(), *reference(*args, act, gated, y), what=f"{act} {y}")


def test_zero_rows_and_zero_weights():
    for n in (3, 50):
        args = list(make(n, 256, 64, 16, 9, "bf16", True, "bf16", True))
        args[0][1] = 0  # s_x = 0: only the bias remains
        args[1][5] = 0
        args[2][6] = 0.0
        out = call(*args, "silu", True, "f32")
        assert_within(out.float().cpu().numpy(), *reference(*args, "silu", True, "f32"), what=f"n={n}")


def test_no_epilogue_equals_the_plain_layer():
    """act none, no bias, no residual: tq_linear's Y up to its rounding of T to one bf16 value."""
    for n in (1, 9, 30, 64, 1500):
        args = make(n, 1024, 256, 0, 11, "bf16", False, None, False)
        out = call(*args, "none", False, "f32")
        plain = tq.tq_linear(args[0].to(DEV), args[1].to(DEV), args[2].to(DEV), None, 256, 0, y_dtype=torch.float32)
        assert torch.equal(out, plain), n


@pytest.mark.parametrize("n,d,m", [(2, 512, 390), (20, 512, 390), (20, 2048, 390), (40, 512, 390), (300, 512, 390), (40, 64, 28702), (300, 64, 57344)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_residual_in_place(n, d, m, gated, dt):
    args = make(n, d, m, 32, 13, "bf16", True, dt, gated)
    want = call(*args, "gelu", gated, dt)
    Y = args[6].to(DEV).clone()
    lr = tq.tq_pack_lowrank(args[3].to(DEV), args[4].to(DEV))
    tq.tq_linear_act(args[0].to(DEV), args[1].to(DEV), args[2].to(DEV), lr, m, 32, bias=args[5].to(DEV), act=ACTS["gelu"], gated=gated, residual=Y, Y=Y)
    assert torch.equal(Y, want)


@pytest.mark.parametrize("n,d,m,r", [(1, 2048, 96, 32), (5, 512, 99, 8), (40, 512, 99, 0), (70, 64, 57400, 16)])
def test_nothing_is_written_beside_y(n, d, m, r):
    args = make(n, d, m, r, 23, "bf16", True, None, False)
    for y in ("bf16", "f32"):
        guard = torch.full((n + 32, m), 5.0, dtype=DT[y], device=DEV)
        off = 16  # rows, a multiple of 16 bytes for every m
        call(*args, "silu", False, y, Y=guard[off: off + n])
        torch.cuda.synchronize()
        assert (guard[:off] == 5.0).all() and (guard[off + n:] == 5.0).all()
        assert_within(guard[off: off + n].float().cpu().numpy(), *reference(*args, "silu", False, y), what=y)


def test_no_rows():
    X = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    out = tq.tq_linear_act(X, torch.zeros((32, 32), dtype=torch.uint8, device=DEV), torch.ones(32, device=DEV), None, 32, 0)
    assert out.shape == (0, 32)


def test_two_streams_at_once():
    """Two calls in flight on two streams, each with its own workspace."""
    a, b = make(64, 2048, 1024, 32, 5, "bf16", True, None, False), make(3, 4096, 2048, 64, 6, "bf16", True, None, True)
    want = [call(*a, "silu", False, "f32"), call(*b, "gelu", True, "f32")]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(6):
        with torch.cuda.stream(s1):
            got[0].append(call(*a, "silu", False, "f32"))
        with torch.cuda.stream(s2):
            got[1].append(call(*b, "gelu", True, "f32"))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


def test_one_workspace_for_every_shape():
    """A workspace zero-filled once serves calls of any shape in turn, on every path, and again."""
    shapes = [(1, 4096, 512, 64, True), (40, 512, 300, 32, False), (8, 1024, 260, 0, True), (1200, 256, 130, 16, False),
              (24, 2048, 128, 128, True)]
    need = max(tq.load().tq_linear_act_workspace_bytes(n, d, m, r) for n, d, m, r, _ in shapes)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for n, d, m, r, gated in shapes:
            args = make(n, d, m, r, n + d, "bf16", True, None, gated)
            out = call(*args, "silu", gated, "f32", ws=ws)
            fresh = call(*args, "silu", gated, "f32")
            assert torch.equal(out, fresh), (n, d, m, r)


@pytest.mark.parametrize("n", [1, 12, 40, 1100])
def test_graph_replay(n):
    args = make(n, 1024, 512, 32, 17, "bf16", True, "bf16", True)
    dev = [None if t is None else t.to(DEV) for t in args]
    X, codes, s_w, l1, l2, b, rs = dev
    lr = tq.tq_pack_lowrank(l1, l2)
    ws = tq.linear_act_workspace(n, 1024, 512, 32, DEV)
    Y = torch.zeros((n, 256), dtype=torch.bfloat16, device=DEV)

    def go():
        tq.tq_linear_act(X, codes, s_w, lr, 512, 32, bias=b, act=ACTS["silu"], gated=True, residual=rs, Y=Y, ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for i in range(4):
        X.copy_(make(n, 1024, 512, 32, 100 + i, "bf16", True, "bf16", True)[0])
        eager = tq.tq_linear_act(X, codes, s_w, lr, 512, 32, bias=b, act=ACTS["silu"], gated=True, residual=rs)
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, eager), i


def test_other_stream():
    args = make(25, 512, 256, 32, 19, "bf16", True, None, False)
    want = call(*args, "relu", False, "bf16")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(*args, "relu", False, "bf16")
    s.synchronize()
    assert torch.equal(got, want)


def test_binding_refuses_wrong_shapes():
    X, codes, s_w, l1, l2, b, rs = [None if t is None else t.to(DEV) for t in make(4, 64, 32, 8, 1, res="bf16")]
    lr = tq.tq_pack_lowrank(l1, l2)
    ok = dict(bias=b, residual=rs)
    tq.tq_linear_act(X, codes, s_w, lr, 32, 8, **ok)
    for bad in (dict(bias=b[:31]), dict(residual=rs[:3]), dict(Y=torch.empty((4, 16), dtype=torch.bfloat16, device=DEV)), dict(bias=b.half())):
        with pytest.raises((ValueError, TypeError)):
            tq.tq_linear_act(X, codes, s_w, lr, 32, 8, **{**ok, **bad})
    both = torch.zeros((5, 32), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):  # overlapping, not the same
        tq.tq_linear_act(X, codes, s_w, lr, 32, 8, residual=both[:4], Y=both[1:])
    with pytest.raises(ValueError):
        tq.tq_linear_act(X, codes[:30], s_w, lr, 32, 8)
    with pytest.raises(ValueError):
        tq.tq_linear_act(X, codes, s_w, lr[:100], 32, 8)
    with pytest.raises(tq.TQError):
        tq.tq_linear_act(X, codes, s_w, lr, 32, 8, act=77)
    with pytest.raises(ValueError):
        tq.tq_linear_act(X, codes, s_w, lr, 32, 8, gated=True, residual=rs)
