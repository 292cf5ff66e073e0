"""GPU parity of the routing plan, the experts' layers and the combination, alone and as they are used together:
integers exact, sums within bounds counted from their roundings (act_testutil.act_rows)."""

from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import rank_augmented_quantized_amd as tq  # noqa: E402
from act_testutil import ACTS, U, act_rows, assert_within  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tq.load()


def plan_ref(ids, E):
    flat = ids.reshape(-1).astype(np.int64)
    keep = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(keep, flat, E), kind="stable")[: int(keep.sum())]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[keep], minlength=E))])
    pos = np.full(flat.shape, -1, dtype=np.int64)
    pos[order] = np.arange(order.size)
    return offsets, order, pos.reshape(ids.shape)


def draw_ids(n, k, E, seed, kind="mixed"):
    rng = np.random.default_rng(seed)
    if kind == "one":  # every pair on one expert
        return np.full((n, k), E // 2, dtype=np.int64)
    if kind == "none":
        return np.full((n, k), -1, dtype=np.int64)
    if kind == "same":  # a token's choices repeat an expert
        return np.repeat(rng.integers(0, E, size=(n, 1)), k, axis=1)
    ids = np.minimum((E * rng.random((n, k)) ** 2.0).astype(np.int64), E - 1)
    if kind == "dropped":
        ids[rng.random((n, k)) < 0.3] = -1
        ids[rng.random((n, k)) < 0.05] = E
        ids[rng.random((n, k)) < 0.05] = -(2 ** 31)
    return ids


PLANS = [(0, 2, 4, "mixed"), (1, 1, 1, "mixed"), (1, 8, 8, "mixed"), (3, 2, 1, "one"), (7, 3, 5, "dropped"), (16, 8, 128, "mixed"),
         (63, 1, 64, "mixed"), (64, 1, 63, "same"), (65, 3, 1024, "mixed"), (1000, 8, 257, "dropped"), (1024, 8, 16, "one"),
         (1025, 8, 33, "mixed"), (4097, 6, 1024, "dropped"), (9001, 8, 100, "none"), (33333, 8, 256, "mixed"), (20000, 5, 3, "one"), (32768, 8, 1024, "dropped"),
         (66000, 4, 300, "mixed"), (70001, 8, 8, "dropped")]
PLANS += [(512, 8, 40, "mixed"), (513, 8, 1000, "dropped"), (66001, 8, 130, "dropped"), (131100, 8, 1024, "mixed")]  # either side of each block size


@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("case", PLANS, ids=["-".join(map(str, c)) for c in PLANS])
def test_expert_plan(case, bits):
    n, k, E, kind = case
    ids = draw_ids(n, k, E, n + E, kind)
    t = torch.from_numpy(ids.astype(np.int32 if bits == 32 else np.int64)).to(DEV)
    order = torch.full((n * k,), -7, dtype=torch.int32, device=DEV)
    offsets, order, pos = tq.tq_expert_plan(t, E, order=order)
    torch.cuda.synchronize()
    ro, rr, rp = plan_ref(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    got = order.cpu().numpy()
    assert np.array_equal(got[: rr.size], rr)
    assert (got[rr.size:] == -7).all()  # behind the last kept pair: left as it was
    assert np.array_equal(pos.cpu().numpy(), rp)


def test_plan_ids_past_32_bits_are_dropped():
    ids = torch.tensor([[1, 2 ** 32 + 1], [-(2 ** 40), 0]], device=DEV)
    offsets, order, pos = tq.tq_expert_plan(ids, 2)
    assert offsets.tolist() == [0, 1, 2] and pos.tolist() == [[1, -1], [-1, 0]] and order[:2].tolist() == [3, 0]


def layers(E, d, m, r, seed, bias):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (E * m, d // 2), generator=g, dtype=torch.uint8)
    s_w = (0.5 + torch.rand(E * m, generator=g)) * (0.25 / d ** 0.5)
    l1 = [(torch.randn((d, r), generator=g) / d ** 0.5).bfloat16() for _ in range(E)] if r else None
    l2 = [(torch.randn((r, m), generator=g) / r ** 0.5).bfloat16() for _ in range(E)] if r else None
    return codes, s_w, l1, l2, torch.randn(E * m, generator=g) if bias else None


def pack(l1, l2):
    return torch.cat([tq.tq_pack_lowrank(a.to(DEV), b.to(DEV)) for a, b in zip(l1, l2)]) if l1 else None


def experts_ref(X, order, offsets, k, lay, m, act, gated, y):
    """Rows of every expert, concatenated in sorted order, with their bounds."""
    codes, s_w, l1, l2, bias = lay
    f = lambda t: None if t is None else t.float().numpy()  # noqa: E731
    ys, bs = [], []
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        x = f(X)[order[a:b] // k] if order is not None else f(X)[a:b]
        c = slice(e * m, (e + 1) * m)
        v, bound = act_rows(x, codes[c].numpy(), f(s_w[c]), f(l1[e]) if l1 else None, f(l2[e]) if l2 else None,
                            f(bias[c]) if bias is not None else None, act, gated, None, y)
        ys.append(v)
        bs.append(bound)
    mo = m // 2 if gated else m
    return (np.concatenate(ys), np.concatenate(bs)) if ys else (np.zeros((0, mo)), np.ones((0, mo)))


ECASES = [
    # n, topk, E, d, m, r, x, y, act, gated, bias, ids, gather
    (1, 1, 1, 32, 1, 0, "f32", "f32", "none", False, True, "mixed", True),
    (1, 2, 8, 128, 34, 16, "bf16", "bf16", "silu", True, False, "mixed", True),
    (4, 2, 8, 4096, 130, 64, "bf16", "f32", "silu", True, True, "mixed", True),
    (5, 3, 7, 96, 65, 8, "f32", "bf16", "gelu", False, True, "dropped", True),
    (9, 4, 4, 512, 48, 256, "bf16", "f32", "relu", False, False, "same", True),
    (16, 1, 3, 288, 100, 32, "bf16", "f32", "gelu_tanh", True, True, "one", False),
    (24, 6, 64, 1408, 70, 32, "bf16", "f32", "none", False, False, "mixed", False),
    (40, 2, 5, 256, 260, 100, "f32", "f32", "silu", False, True, "dropped", True),
    (100, 8, 130, 64, 33, 8, "bf16", "bf16", "none", False, True, "mixed", True),
    (150, 2, 4, 512, 516, 32, "bf16", "f32", "silu", True, False, "mixed", True),
    (333, 4, 6, 320, 130, 64, "bf16", "bf16", "gelu", True, True, "dropped", True),
    (700, 1, 3, 1024, 300, 32, "f32", "f32", "none", False, False, "one", False),
    (900, 2, 4, 544, 520, 48, "bf16", "f32", "gelu", True, True, "mixed", True),
    (12, 2, 5, 64, 32, 8, "bf16", "bf16", "none", False, False, "none", True),
    # few rows per expert: each kernel by row length, all ranks, many experts
    (6, 2, 3, 16416, 20, 16, "bf16", "f32", "none", False, True, "mixed", True),
    (5, 2, 4, 14336, 40, 64, "f32", "bf16", "silu", True, False, "dropped", False),
    (7, 2, 4, 5120, 34, 200, "bf16", "f32", "none", False, True, "mixed", True),
    (30, 3, 9, 2048, 130, 128, "bf16", "f32", "gelu", True, True, "dropped", True),
    (20, 4, 1000, 64, 16, 8, "bf16", "f32", "none", False, True, "mixed", True),
    # many: tiles of 128 and 256 rows, k split over blocks and not
    (300, 2, 4, 256, 300, 32, "bf16", "bf16", "silu", True, True, "mixed", True),
    (310, 2, 4, 96, 513, 0, "f32", "f32", "relu", False, True, "dropped", True),
    (2600, 4, 9, 64, 80, 200, "bf16", "f32", "none", False, False, "mixed", True),
    (60, 2, 2, 16416, 36, 32, "bf16", "bf16", "none", False, False, "mixed", True),
]


@pytest.mark.parametrize("case", ECASES, ids=["-".join(map(str, c)) for c in ECASES])
def test_linear_experts(case):
    n, k, E, d, m, r, x, y, act, gated, bias, kind, gather = case
    g = torch.Generator().manual_seed(n * 7 + E)
    ids = draw_ids(n, k, E, n + E, kind)
    nx = n if gather else n * k
    X = torch.randn((nx, d), generator=g).to(DT[x])
    X[:, d // 3] *= 8
    lay = layers(E, d, m, r, 5 + n, bias)
    offsets, order, pos = tq.tq_expert_plan(torch.from_numpy(ids).to(DEV), E)
    mo = m // 2 if gated else m
    Y = torch.full((n * k, mo), 7.0, dtype=DT[y], device=DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    tq.tq_linear_experts(X.to(DEV), dev(lay[0]), dev(lay[1]), pack(lay[2], lay[3]), m, r, offsets, order=order if gather else None,
                         topk=k if gather else 1, bias=dev(lay[4]), act=ACTS[act], gated=gated, Y=Y)
    torch.cuda.synchronize()
    ro, rr, _ = plan_ref(ids, E)
    ref, bound = experts_ref(X, rr if gather else None, ro, k, lay, m, act, gated, y)
    kept = int(ro[-1])
    got = Y.float().cpu().numpy()
    assert (got[kept:] == 7.0).all()  # rows behind the last expert: left as they were
    assert_within(got[:kept], ref, bound, what=str(case))


def test_every_expert_is_the_layer_alone():
    """An expert's rows are tq_linear_act's on those tokens, whatever the others do (same integer sums and epilogue)."""
    n, k, E, d, m, r = 130, 2, 4, 512, 256, 0
    ids = draw_ids(n, k, E, 3)
    X = torch.randn((n, d), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    codes, s_w, _, _, bias = [t.to(DEV) if torch.is_tensor(t) else t for t in layers(E, d, m, r, 3, True)]
    offsets, order, _ = tq.tq_expert_plan(torch.from_numpy(ids).to(DEV), E)
    Y = tq.tq_linear_experts(X, codes, s_w, None, m, r, offsets, order=order, topk=k, bias=bias, act=2, gated=True, y_dtype=torch.float32)
    off = offsets.tolist()
    for e in range(E):
        rows = (order[off[e]: off[e + 1]] // k).long()
        alone = tq.tq_linear_act(X[rows].contiguous(), codes[e * m: (e + 1) * m], s_w[e * m: (e + 1) * m], None, m, r,
                                 bias=bias[e * m: (e + 1) * m], act=2, gated=True, y_dtype=torch.float32)
        assert torch.equal(Y[off[e]: off[e + 1]], alone), e


@pytest.mark.parametrize("offsets", [[0, 5, 3, 40], [-9, 2, 10 ** 9, 2 ** 31 - 1], [6, 6, 6, 6], [12, 0, 0, 12], [-5, -4, -3, -2]])
@pytest.mark.parametrize("gather", [False, True])
def test_bad_offsets_and_orders_stay_inside(offsets, gather):
    """Offsets and orders that no plan makes are clamped: the call ends, and memory beside Y keeps its contents."""
    n, d, m = 12, 128, 64
    X = torch.randn((n, d), device=DEV).bfloat16()
    codes, s_w, _, _, _ = layers(3, d, m, 0, 1, False)
    guard = torch.full((n + 64, m), 3.0, dtype=torch.bfloat16, device=DEV)
    order = torch.tensor([2 ** 31 - 1, -1, 5, -(2 ** 31), 0, 1, 2, 3, 10 ** 6, 7, 8, 9], dtype=torch.int32, device=DEV)
    tq.tq_linear_experts(X, codes.to(DEV), s_w.to(DEV), None, m, 0, torch.tensor(offsets, dtype=torch.int32, device=DEV),
                         order=order if gather else None, Y=guard[32: 32 + n])
    torch.cuda.synchronize()
    assert (guard[:32] == 3.0).all() and (guard[32 + n:] == 3.0).all()


def combine_ref(Z, pos, w, res):
    Z, w = Z.double().numpy(), w.double().numpy()
    n, k = pos.shape
    y = res.double().numpy().copy() if res is not None else np.zeros((n, Z.shape[1]))
    mag = np.abs(y)
    for t in range(n):
        for j in range(k):
            if 0 <= pos[t, j] < Z.shape[0]:
                y[t] += w[t, j] * Z[pos[t, j]]
                mag[t] += np.abs(w[t, j] * Z[pos[t, j]])
    return y, mag


@pytest.mark.parametrize("case", [
    (1, 1, 1, "f32", "f32", "f32", None, 0.0), (3, 2, 64, "bf16", "bf16", "f32", "bf16", 0.0), (5, 8, 100, "bf16", "f32", "f32", "f32", 0.3),
    (7, 9, 2056, "f32", "f32", "bf16", "bf16", 0.2), (2, 64, 257, "bf16", "bf16", "bf16", None, 0.5), (300, 3, 72, "bf16", "bf16", "f32", "bf16", 0.1),
    (4, 6, 4096, "f32", "bf16", "f32", "f32", 1.0)], ids=str)
def test_expert_combine(case):
    n, k, m, z, y, w, res, drop = case
    g = torch.Generator().manual_seed(n + m)
    Z = torch.randn((n * k, m), generator=g).to(DT[z])
    pos = torch.randperm(n * k, generator=g).int().reshape(n, k)
    pos[torch.rand((n, k), generator=g) < drop] = -1
    wt = torch.randn((n, k), generator=g).to(DT[w])
    wt[pos < 0] = float("nan")  # a dropped pair's weight counts for nothing
    rs = torch.randn((n, m), generator=g).to(DT[res]) if res else None
    out = tq.tq_expert_combine(Z.to(DEV), pos.to(DEV), wt.to(DEV), residual=None if rs is None else rs.to(DEV), y_dtype=DT[y])
    ref, mag = combine_ref(Z, pos.numpy(), torch.nan_to_num(wt), rs)
    bound = k * U / (1 - k * U) * mag * 1.01
    bound = bound + (2.0 ** -8 if y == "bf16" else U) * (np.abs(ref) + bound) + 2.0 ** -126
    assert_within(out.float().cpu().numpy(), ref, bound, what=str(case))


def test_combine_in_place_and_out_of_range_positions():
    Z = torch.randn((6, 40), device=DEV)
    Z[5] = float("inf")
    pos = torch.tensor([[0, 6], [2 ** 31 - 1, 1], [-(2 ** 31), -1]], dtype=torch.int32, device=DEV)
    w = torch.ones((3, 2), device=DEV)
    Y = torch.randn((3, 40), device=DEV)
    want = Y.clone()
    want[0] += Z[0]
    want[1] += Z[1]
    tq.tq_expert_combine(Z, pos, w, residual=Y, Y=Y)
    assert torch.equal(Y, want)
    none = tq.tq_expert_combine(torch.empty((0, 40), device=DEV), pos, w, residual=Y)
    assert torch.equal(none, Y.bfloat16())


def test_combine_of_the_most_tokens():
    """2^24 tokens of one expert each, Y[t] = 2 Z[n - 1 - t] exactly, the last blocks' rows among them."""
    n = 1 << 24
    Z = torch.arange(n, dtype=torch.float32, device=DEV).view(n, 1)
    pos = torch.arange(n - 1, -1, -1, dtype=torch.int32, device=DEV).view(n, 1)
    w = torch.full((n, 1), 2.0, device=DEV)
    Y = tq.tq_expert_combine(Z, pos, w, y_dtype=torch.float32)
    assert torch.equal(Y, 2 * Z.flip(0))


def mlp(X, ids, wt, E, gu, dn, m1, m2, r, bufs=None):
    """The experts' MLP as a model calls it: plan, gate and up, down on the sorted rows, combination on the residual."""
    b = bufs or {}
    offsets, order, pos = tq.tq_expert_plan(ids, E, *b.get("plan", ()))
    H = tq.tq_linear_experts(X, gu[0], gu[1], gu[2], m1, r, offsets, order=order, topk=ids.shape[1], act=2, gated=True, Y=b.get("H"), ws=b.get("ws1"))
    Z = tq.tq_linear_experts(H, dn[0], dn[1], dn[2], m2, r, offsets, Y=b.get("Z"), ws=b.get("ws2"))
    return tq.tq_expert_combine(Z, pos, wt, residual=X, Y=b.get("Y")), (offsets, order, pos, H, Z)


@pytest.mark.parametrize("n,k,E", [(1, 2, 8), (6, 2, 4), (70, 4, 16), (600, 2, 4)])
def test_mixture_of_experts_together(n, k, E):
    """Each step against the reference on the step before it, with tokens dropped."""
    d, f, r = 256, 192, 32
    g = torch.Generator().manual_seed(n)
    X = torch.randn((n, d), generator=g).bfloat16()
    ids = draw_ids(n, k, E, n, "dropped" if n > 1 else "mixed")
    wt = torch.softmax(torch.randn((n, k), generator=g), 1)
    gu, dn = layers(E, d, 2 * f, r, 1, False), layers(E, f, d, r, 2, False)
    dev = lambda lay: (lay[0].to(DEV), lay[1].to(DEV), pack(lay[2], lay[3]))  # noqa: E731
    Y, (offsets, order, pos, H, Z) = mlp(X.to(DEV), torch.from_numpy(ids).to(DEV), wt.to(DEV), E, dev(gu), dev(dn), 2 * f, d, r)
    ro, rr, rp = plan_ref(ids, E)
    kept = int(ro[-1])
    assert np.array_equal(offsets.cpu().numpy(), ro) and np.array_equal(pos.cpu().numpy(), rp)
    H, Z = H.cpu()[:kept], Z.cpu()[:kept]
    assert_within(H.float().numpy(), *experts_ref(X, rr, ro, k, gu, 2 * f, "silu", True, "bf16"), what="gate/up")
    assert_within(Z.float().numpy(), *experts_ref(H, None, ro, 1, dn, d, "none", False, "bf16"), what="down")
    ref, mag = combine_ref(Z, rp, wt, X)
    bound = k * U * 1.01 * mag
    assert_within(Y.float().cpu().numpy(), ref, bound + 2.0 ** -8 * (np.abs(ref) + bound) + 2.0 ** -126, what="combine")


@pytest.mark.parametrize("n", [3, 90])
def test_graph_replay_with_new_routing(n):
    """One captured graph serves every routing: ids, activations and weights change between replays, the plan follows."""
    k, E, d, f, r = 2, 6, 256, 128, 16
    gu, dn = layers(E, d, 2 * f, r, 1, False), layers(E, f, d, r, 2, False)
    dev = lambda lay: (lay[0].to(DEV), lay[1].to(DEV), pack(lay[2], lay[3]))  # noqa: E731
    gu, dn = dev(gu), dev(dn)
    X = torch.zeros((n, d), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros((n, k), dtype=torch.int64, device=DEV)
    wt = torch.full((n, k), 0.5, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    bufs = dict(plan=(torch.zeros(E + 1, **i32), torch.zeros(n * k, **i32), torch.zeros((n, k), **i32)),
                H=torch.zeros((n * k, f), dtype=torch.bfloat16, device=DEV), Z=torch.zeros((n * k, d), dtype=torch.bfloat16, device=DEV),
                Y=torch.zeros((n, d), dtype=torch.bfloat16, device=DEV), ws1=tq.linear_experts_workspace(n, k, d, 2 * f, r, E, DEV),
                ws2=tq.linear_experts_workspace(n * k, 1, f, d, r, E, DEV))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mlp(X, ids, wt, E, gu, dn, 2 * f, d, r, bufs)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlp(X, ids, wt, E, gu, dn, 2 * f, d, r, bufs)
    for i, kind in enumerate(("mixed", "dropped", "one", "none", "mixed")):
        X.copy_(torch.randn((n, d), generator=torch.Generator().manual_seed(i)))
        ids.copy_(torch.from_numpy(draw_ids(n, k, E, i, kind)))
        eager, _ = mlp(X, ids, wt, E, gu, dn, 2 * f, d, r)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs["Y"], eager), kind


def test_two_graphs_share_a_workspace():
    """Graphs of different shapes captured with one workspace and one set of outputs, replayed in turn with eager work
    between: a launch leaves nothing in the workspace that the next one reads."""
    E, d, m, r = 8, 2048, 96, 64
    lay = layers(E, d, m, r, 41, True)
    dev = (lay[0].to(DEV), lay[1].to(DEV), pack(lay[2], lay[3]), lay[4].to(DEV))
    runs, need = [], 0
    for n, k in ((6, 2), (150, 2), (40, 4)):  # the rows product; the tile product, T split over k
        g = torch.Generator().manual_seed(n)
        X = torch.randn((n, d), generator=g).bfloat16().to(DEV)
        ids = torch.from_numpy(draw_ids(n, k, E, n, "mixed")).to(DEV)
        plan = tq.tq_expert_plan(ids, E)
        runs.append((X, k, plan))
        need = max(need, tq.linear_experts_workspace(n, k, d, m, r, E, DEV).numel())
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    out = [torch.empty((X.shape[0] * k, m), dtype=torch.bfloat16, device=DEV) for X, k, _ in runs]

    def once(i):
        X, k, (offsets, order, _) = runs[i]
        tq.tq_linear_experts(X, dev[0], dev[1], dev[2], m, r, offsets, order=order, topk=k, bias=dev[3], act=2, Y=out[i], ws=ws)

    want = []
    for i in range(3):
        once(i)
        want.append(out[i].clone())
    torch.cuda.synchronize()
    graphs = []
    for i in range(3):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            once(i)
        graphs.append(graph)
    for i in (0, 1, 2, 1, 0, 2, 2, 1):
        out[i].zero_()
        graphs[i].replay()
        once((i + 1) % 3)
        torch.cuda.synchronize()
        assert torch.equal(out[i], want[i]), i


def test_binding_refuses_wrong_shapes():
    codes, s_w, _, _, _ = layers(3, 64, 32, 0, 1, False)
    codes, s_w = codes.to(DEV), s_w.to(DEV)
    X = torch.randn((4, 64), device=DEV).bfloat16()
    offsets, order, pos = tq.tq_expert_plan(torch.zeros((4, 2), dtype=torch.int64, device=DEV), 3)
    tq.tq_linear_experts(X, codes, s_w, None, 32, 0, offsets, order=order, topk=2)
    with pytest.raises(ValueError):
        tq.tq_linear_experts(X, codes, s_w, None, 32, 0, offsets, order=order, topk=1)
    with pytest.raises(ValueError):
        tq.tq_linear_experts(X, codes, s_w, None, 32, 0, offsets, topk=2)
    with pytest.raises(ValueError):
        tq.tq_linear_experts(X, codes[:64], s_w, None, 32, 0, offsets, order=order, topk=2)
    with pytest.raises(TypeError):
        tq.tq_linear_experts(X, codes, s_w, None, 32, 0, offsets.long(), order=order, topk=2)
    with pytest.raises(TypeError):
        tq.tq_expert_plan(torch.zeros((4, 2), device=DEV), 3)
    with pytest.raises(ValueError):
        tq.tq_expert_combine(torch.zeros((8, 16), device=DEV), pos, torch.ones((4, 3), device=DEV))
