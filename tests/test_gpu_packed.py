"""Activations in 8 bits on the GPU: the format bit for bit, and the products
and gradients that write or read it against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import block_ref as ref
import expert_routing_ffn_gb300 as moe
import train_ref
from test_gpu_train import TYPES, clean, dev, empty, host, ints, rnd, routing, workspace
from train_ref import STEP, check, rounded

pytestmark = pytest.mark.gpu


def nb(cols):
    return (cols + 31) // 32


def buffers(rows, cols):
    """Packed rows full of 0x55: every byte has to be written."""
    q, e = moe.packed_rows(rows, cols)
    return q.fill_(0x55), e.fill_(0x55)


def given(q, E):
    """A reference's packed rows on the GPU."""
    return dev(ref.kept(q)), dev(E.astype(np.uint8))


def values(q, e, cols):
    """What packed rows on the GPU stand for, in 64 bits."""
    return ref.unpack(ref.columns(ints(q).astype(np.int64), nb(cols)), ints(e).astype(np.int64), cols)


SIZES = [(1, 1, "bf16"), (1, 31, "f32"), (3, 32, "bf16"), (2, 33, "bf16"), (5, 40, "f32"), (17, 256, "bf16"), (4, 257, "f32"),
         (700, 72, "bf16"), (9, 1001, "bf16"), (3, 4096, "f32"), (1, 65536, "bf16"), (2, 65535, "f32"), (3000, 8, "bf16")]


@pytest.mark.parametrize("rows,cols,kind", SIZES)
def test_pack_and_unpack_bit_for_bit(rows, cols, kind):
    rng = np.random.default_rng(rows + cols)
    t = (torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)) * 10.0 ** torch.from_numpy(rng.integers(-12, 12, (rows, 1)))).to(TYPES[kind])
    x, xh = t.cuda(), t.double().numpy()
    q, e = buffers(rows, cols)
    moe.moe_pack_rows(x, q, e)
    rq, rE = ref.pack(xh)
    assert np.array_equal(ints(e), rE)
    assert np.array_equal(ints(q), ref.kept(rq))
    for okind in ("bf16", "f32"):  # either type holds the values exactly
        out = empty((rows, cols), okind)
        moe.moe_unpack_rows(q, e, None, 1, out)
        assert np.array_equal(host(out), ref.unpack(rq, rE, cols))
    # rows of a wider tensor, in and out
    wide = torch.zeros((rows, cols + 5), dtype=TYPES[kind], device="cuda")
    wide[:, 3:3 + cols] = x
    q2, e2 = buffers(rows, cols)
    moe.moe_pack_rows(wide[:, 3:3 + cols], q2, e2)
    assert torch.equal(q2, q) and torch.equal(e2, e)
    out = empty((rows, cols + 5), "f32")
    moe.moe_unpack_rows(q, e, None, 1, out[:, 3:3 + cols])
    assert np.array_equal(host(out[:, 3:3 + cols]), ref.unpack(rq, rE, cols))
    assert bool(out[:, :3].isnan().all()) and bool(out[:, 3 + cols:].isnan().all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_values_where_the_format_turns(kind):
    """Ties, the border to the next power, the largest and smallest values, zeros of both signs, infinities, NaN."""
    big, tiny = float(torch.finfo(TYPES[kind]).max), 2.0 ** -133 if kind == "bf16" else 2.0 ** -149
    rows = [[127.0, 0.5, 1.5, -2.5, -0.5], [127.5, 1.0], [127.49, 3.0], [-127.5], [128.0, 1.0], [63.75, 0.25], [64.0], [big, -big, 1.0], [tiny],
            [-tiny, 2.0 ** -128], [2.0 ** -126, 2.0 ** -127], [2.0 ** -120, 2.0 ** -121 * 1.9921875], [0.0, -0.0], [float("inf"), 1.0],
            [float("nan"), 1.0], [-float("inf"), float("nan"), big], [2.0 ** -121 * 1.9921875], [2.0 ** -121 * 1.984375, 2.0 ** -128]]
    x = torch.zeros(len(rows), 70)
    for i, r in enumerate(rows):
        for at in (0, 37):  # the second block holds them too, the last one is empty
            x[i, at:at + len(r)] = torch.tensor(r)
    x = x.to(TYPES[kind])
    rq, rE = ref.pack(x.double().numpy())
    q, e = buffers(len(rows), 70)
    moe.moe_pack_rows(x.cuda(), q, e)
    assert np.array_equal(ints(e), rE) and np.array_equal(ints(q), ref.kept(rq))
    out = empty((len(rows), 70), kind)
    moe.moe_unpack_rows(q, e, None, 1, out)
    assert np.array_equal(host(out), ref.unpack(rq, rE, 70), equal_nan=True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_what_was_restored_packs_to_the_same_bytes(kind):
    x = torch.from_numpy(np.random.default_rng(3).standard_normal((300, 500)).astype(np.float32)).to(TYPES[kind]).cuda()
    (q, e), (q2, e2) = buffers(300, 500), buffers(300, 500)
    moe.moe_pack_rows(x, q, e)
    moe.moe_unpack_rows(q, e, None, 1, x)
    moe.moe_pack_rows(x, q2, e2)
    assert torch.equal(q, q2) and torch.equal(e, e2)


def test_gather_with_indices_that_name_no_row():
    rng = np.random.default_rng(2)
    x, xh = rnd(rng, (6, 100), "bf16")
    q, e = buffers(6, 100)
    moe.moe_pack_rows(x, q, e)
    v = ref.unpack(*ref.pack(xh), 100)
    index = np.array([0, 11, 5, -1, 3, 12, 1 << 30, -(1 << 31), 2, 2], np.int32)
    out = empty((10, 100), "bf16")
    moe.moe_unpack_rows(q, e, dev(index), 2, out)
    exact = np.stack([v[i // 2] if 0 <= i < 12 else np.zeros(100) for i in index.tolist()])
    assert np.array_equal(host(out), exact)
    none = empty((3, 100), "bf16")
    moe.moe_unpack_rows(q[:0], e[:0], dev(np.array([0, 1, -1], np.int32)), 1, none)
    assert not none.any()
    moe.moe_pack_rows(x[:0], q, e)
    moe.moe_unpack_rows(q, e, None, 1, none[:0])


def test_offsets_past_32_bits():
    """More than 2^32 packed values: the last rows are their own."""
    rows, cols = (1 << 16) + 3, 65536
    q = torch.zeros((rows, cols), dtype=torch.int8, device="cuda")
    e = torch.zeros((rows, cols // 32), dtype=torch.uint8, device="cuda")
    q[-1], e[-1] = 3, 127
    out = empty((2, cols), "bf16")
    moe.moe_unpack_rows(q, e, dev(np.array([rows - 1, rows - 2], np.int32)), 1, out)
    assert bool((out[0] == 3).all()) and not out[1].any()
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-1] = 5.0
    moe.moe_pack_rows(x, q, e)
    assert bool((q[-1] == 80).all()) and bool((e[-1] == 123).all()) and not q[-2].any()


# ---------------------------------------------------------------- combine, gradient

COMBINE = [(1, 2048, 64, 6, "all", "bf16"), (1, 7, 3, 1, "none", "f32"), (33, 250, 40, 8, "some", "bf16"), (33, 251, 40, 8, "some", "f32"),
           (257, 1000, 40, 8, "skew", "f32"), (64, 40, 300, 16, "all", "f32"), (700, 33, 512, 16, "skew", "bf16"), (129, 3584, 64, 8, "all", "bf16"),
           (40, 1024, 8, 2, "one", "bf16"), (12, 1032, 16, 9, "some", "bf16"), (2000, 264, 8, 2, "some", "f32"),
           (1900, 768, 40, 8, "some", "bf16"), (5, 12000, 8, 2, "all", "bf16")]


@pytest.mark.parametrize("T,d,N,k,how,kind", COMBINE)
@pytest.mark.parametrize("gated", [True, False])
def test_combine_gradient(T, d, N, k, how, kind, gated):
    rng = np.random.default_rng(T + d)
    D = moe.make_dims(T, d, N, k, 64, wtype=kind)
    _, _, inv = train_ref.sort_slots(routing(rng, T, N, k, how), N, 0)
    rq, rE = ref.pack(rng.standard_normal((T * k, d)).astype(np.float32).astype(np.float64))
    y = ref.unpack(rq, rE, d)
    q, e = given(rq, rE)
    dout, doh = rnd(rng, (T, d + 8), kind)
    dout, doh = dout[:, :d], doh[:, :d]
    gate, gh = rnd(rng, (T, k), "f32") if gated else (None, None)
    dy, dgate = empty((T * k, d), kind), empty((T, k), "f32")
    moe.moe_combine_rows_grad_packed(D, dout, q, e, gate, dev(inv), dy, dgate)
    edy, edg, mag = train_ref.combine_grad(doh, y, gh, inv)
    check(host(dy), edy, rounded(edy, 4 * STEP * np.abs(edy), kind), "dy")
    check(host(dgate), edg, train_ref.bound(edg, d, mag, "f32"), "dgate")
    dy2, dgate2 = empty((T * k, d), kind), empty((T, k), "f32")
    moe.moe_combine_rows_grad_packed(D, dout, None, None, gate, dev(inv), dy2, None)
    moe.moe_combine_rows_grad_packed(D, dout, q, e, gate, dev(inv), None, dgate2)
    assert torch.equal(dy2, dy) and torch.equal(dgate2, dgate)


# ---------------------------------------------------------------- products

PRODUCTS = [  # T, d, I, N, k, routing, type
    (1, 64, 64, 8, 2, "all", "bf16"), (3, 7, 5, 4, 2, "all", "f32"), (9, 40, 33, 8, 2, "some", "bf16"), (16, 256, 512, 8, 2, "all", "f32"),
    (40, 72, 200, 5, 3, "some", "bf16"), (100, 128, 96, 4, 2, "one", "bf16"), (70, 100, 60, 3, 1, "skew", "f32"), (300, 64, 104, 4, 2, "skew", "f32"),
    (200, 264, 136, 9, 4, "some", "bf16"), (513, 192, 72, 2, 1, "all", "bf16"), (700, 128, 320, 16, 4, "skew", "bf16"), (6, 512, 256, 64, 6, "all", "bf16"),
    (20, 64, 64, 8, 2, "none", "bf16"), (260, 511, 301, 4, 2, "all", "bf16"), (1100, 96, 448, 3, 2, "all", "bf16"), (90, 65, 1000, 2, 1, "some", "f32"),
]


def _layer(rng, T, d, I, N, k, how, kind, sd):
    D = moe.make_dims(T, d, N, k, I, wtype=kind)
    off, _, _ = train_ref.sort_slots(routing(rng, T, N, k, how), N, 0)
    w = [rnd(rng, (N, I, d), kind, sd) for _ in range(2)]
    return D, off, w


@pytest.mark.parametrize("T,d,I,N,k,how,kind", PRODUCTS)
def test_up_products_keep_g_and_u(T, d, I, N, k, how, kind):
    rng = np.random.default_rng(T + d + I)
    D, off, ((wg, wgh), (wu, wuh)) = _layer(rng, T, d, I, N, k, how, kind, 1.5 / np.sqrt(d))
    M = T * k
    x, xh = rnd(rng, (M, d), kind)
    xh[off[-1]:] = 0
    ws = workspace(D)
    (gq, gs), (uq, us), h = buffers(M, I), buffers(M, I), empty((M, I), kind)
    moe.moe_experts_up_packed(D, x, dev(off), wg, wu, gq, gs, uq, us, h, ws)
    clean(ws)
    g, u, eh, mg, mu = train_ref.experts_up(xh, off, wgh, wuh)
    check(host(h), eh, train_ref.up_h_limit(g, u, eh, mg, mu, d, kind), "h")
    for q, s, exact, mag, name in ((gq, gs, g, mg, "g"), (uq, us, u, mu, "u")):
        raw, E = ref.columns(ints(q).astype(np.int64), nb(I)), ints(s).astype(np.int64)
        assert not raw.reshape(M, -1)[:, I:].any()
        off_ = (d + 8) * STEP * mag  # of the float32 sum
        # E is that of a sum within the error of the exact one
        pad = np.zeros((2, M, nb(I) * 32))
        pad[0, :, :I], pad[1, :, :I] = np.abs(exact) - off_, np.abs(exact) + off_
        low, high = np.maximum(pad, 0).reshape(2, M, -1, 32).max(3)
        for m, ok in ((low, np.less_equal), (high, np.greater_equal)):
            assert ok(ref.pack(np.repeat(m.reshape(-1, 1), 2, 1))[1].reshape(E.shape), E).all(), name
        check(ref.unpack(raw, E, I), exact, off_ + np.repeat(0.5 * 2.0 ** (E - 127.0), 32, 1)[:, :I] + 2.0 ** -126, name)
    assert not gq[int(off[-1]):].any() and not us[int(off[-1]):].any() and not h[int(off[-1]):].any()


@pytest.mark.parametrize("T,d,I,N,k,how,kind", PRODUCTS)
@pytest.mark.parametrize("gtype", ["layer", "f32"])
def test_down_gradient_reads_g_and_u(T, d, I, N, k, how, kind, gtype):
    rng = np.random.default_rng(T + d + I + 1)
    D, off, ((wd, wdh), _) = _layer(rng, T, d, I, N, k, how, kind, 1.5 / np.sqrt(d))
    M, gk = T * k, kind if gtype == "layer" else "f32"
    live = int(off[-1])
    dy, dyh = rnd(rng, (M, d), kind)
    dyh[live:] = 0
    packs = []
    for _ in range(2):
        v = rng.standard_normal((M, I)).astype(np.float32).astype(np.float64) * 2.0
        v[live:] = 0
        packs.append(ref.pack(v))
    (gq, gs), (uq, us) = (given(*p) for p in packs)
    g, u = (ref.unpack(*p, I) for p in packs)
    ws = workspace(D)
    h, dg, du, dw = empty((M, I), kind), empty((M, I), kind), empty((M, I), kind), empty((N, I, d), gk)
    moe.moe_experts_down_grad_packed(D, dy, gq, gs, uq, us, dev(off), wd, h, dg, du, dw, False, ws)
    clean(ws)
    eh = g * train_ref.sigmoid(g) * u
    check(host(h), eh, rounded(eh, 16 * STEP * np.abs(eh), kind), "h")
    edg, edu, og, ou = train_ref.experts_dh(dyh, g, u, off, wdh)
    check(host(dg), edg, rounded(edg, og, kind), "dg")
    check(host(du), edu, rounded(edu, ou, kind), "du")
    edw, mag, terms = train_ref.experts_dw(host(h), dyh, off, N)  # of h as it is rounded
    check(host(dw), edw, train_ref.bound(edw, terms, mag, gk), "dw")
    if gk == "f32":
        moe.moe_experts_down_grad_packed(D, dy, gq, gs, uq, us, dev(off), wd, h, dg, du, dw, True, ws)
        check(host(dw), 2 * edw, 2 * train_ref.bound(edw, terms, mag, gk) + 4 * STEP * np.abs(edw), "dw twice")
    h2, dg2, du2 = empty((M, I), kind), empty((M, I), kind), empty((M, I), kind)
    moe.moe_experts_down_grad_packed(D, dy, gq, gs, uq, us, dev(off), wd, h2, dg2, du2, None, False, ws)
    assert torch.equal(h2, h) and torch.equal(dg2, dg) and torch.equal(du2, du)


@pytest.mark.parametrize("kind,d,I", [("bf16", 64, 96), ("f32", 40, 50)])
def test_a_block_that_is_not_finite_reads_as_nan(kind, d, I):
    rng = np.random.default_rng(6)
    T, N = 40, 2
    D, off, ((wg, _), (wu, _)) = _layer(rng, T, d, I, N, 1, "all", kind, 0.2)
    x, _ = rnd(rng, (T, d), kind)
    x[0, 3], x[1, 5] = float("inf"), float("nan")
    ws = workspace(D)
    (gq, gs), (uq, us), h = buffers(T, I), buffers(T, I), empty((T, I), kind)
    moe.moe_experts_up_packed(D, x, dev(off), wg, wu, gq, gs, uq, us, h, ws)
    assert bool((gs[:2] == 255).all()) and bool((us[:2] == 255).all()) and not gq[:2].any()
    assert not bool((gs[2:] == 255).any())
    dy, _ = rnd(rng, (T, d), kind)
    dg, du = empty((T, I), kind), empty((T, I), kind)
    moe.moe_experts_down_grad_packed(D, dy, gq, gs, uq, us, dev(off), wg, h, dg, du, None, False, ws)
    clean(ws)
    for t in (h, dg, du):
        assert bool(t[:2].isnan().all()) and bool(t[2:].isfinite().all())


def test_empty_batch():
    D = moe.make_dims(0, 64, 4, 2, 64)
    ws = workspace(D)
    z, off = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    q, e = moe.packed_rows(0, 64)
    w = torch.ones((4, 64, 64), dtype=torch.bfloat16, device="cuda")
    moe.moe_experts_up_packed(D, z, off, w, w, q, e, q, e, z, ws)
    dw = torch.full((4, 64, 64), float("nan"), device="cuda")
    moe.moe_experts_down_grad_packed(D, z, q, e, q, e, off, w, z, z, z, dw, False, ws)
    assert not dw.any()
    moe.moe_combine_rows_grad_packed(D, z, q, e, None, torch.zeros(0, dtype=torch.int32, device="cuda"), z, None)
    clean(ws)


def test_repeats_bit_for_bit_and_in_a_graph():
    rng = np.random.default_rng(7)
    T, d, I, N, k = 300, 256, 192, 8, 2
    D, off, ((wg, _), (wu, _)) = _layer(rng, T, d, I, N, k, "skew", "bf16", 0.1)
    x, _ = rnd(rng, (T * k, d), "bf16")
    dy, _ = rnd(rng, (T * k, d), "bf16")
    ws, o = workspace(D), dev(off)
    t = [*buffers(T * k, I), *buffers(T * k, I), *(empty((T * k, I), "bf16") for _ in range(4)), empty((N, I, d), "f32")]

    def both():
        moe.moe_experts_up_packed(D, x, o, wg, wu, *t[:4], t[4], ws)
        moe.moe_experts_down_grad_packed(D, dy, *t[:4], o, wg, t[5], t[6], t[7], t[8], False, ws)

    both()
    first = [v.clone() for v in t]
    for v in t:
        v.fill_(0x11)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, t))
    clean(ws)
