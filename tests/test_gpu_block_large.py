"""Norms, block ends and the packed combine's gradient on tensors of more than
2^32 values: the last rows are what a call on them alone gives, bit for bit."""
import pytest
import torch

import expert_routing_ffn_gb300 as moe
from test_gpu_train import clean, workspace

pytestmark = pytest.mark.gpu

T, d, TAIL = (1 << 20) + 50000, 4096, 5000  # the tail alone goes through shared memory too
assert T * d > 1 << 32


def _tail(gen, rows=T, dtype=torch.bfloat16):
    """Zeros, and ordinary values in the last rows."""
    x = torch.zeros((rows, d), dtype=dtype, device="cuda")
    x[-TAIL:] = torch.randn(TAIL, d, device="cuda", generator=gen).to(dtype)
    return x


def _dims(n, k=1):
    return moe.make_dims(n, d, 8, k, 64)


def test_norm_and_its_gradient():
    gen = torch.Generator("cuda").manual_seed(1)
    x, dn = _tail(gen), _tail(gen)
    w = torch.randn(d, device="cuda", generator=gen).bfloat16()
    got = []
    for n in (T, TAIL):
        D, ws = _dims(n), workspace(_dims(n))
        o, dx, r = torch.full_like(x[-n:], 3.0), torch.full_like(x[-n:], 3.0), torch.zeros(n, device="cuda")
        moe.moe_norm_rows(D, x[-n:], w, 1e-6, 0.0, o, r)
        moe.moe_norm_rows_grad(D, dn[-n:], x[-n:], r, w, 0.0, None, dx, None, False, ws)
        clean(ws)
        assert not o[:-TAIL].any() and not dx[:-TAIL].any()
        got.append([t[-TAIL:].clone() for t in (o, dx, r)])
        del o, dx
    assert all(torch.equal(a, b) for a, b in zip(*got)) and bool(got[0][0].any())


def test_block_and_its_gradient():
    gen = torch.Generator("cuda").manual_seed(2)
    y, res, dnext = _tail(gen), _tail(gen), _tail(gen)
    w = torch.randn(d, device="cuda", generator=gen).bfloat16()
    gate = torch.randn(T, device="cuda", generator=gen)
    B = moe.make_block(gate=moe.MOE_GATE_TOKEN)
    got = []
    for n in (T, TAIL):
        D, ws = _dims(n), workspace(_dims(n))
        out, nxt, dres, dy = (torch.full_like(y[-n:], 3.0) for _ in range(4))
        ra, rb, dg = (torch.zeros(n, device="cuda") for _ in range(3))
        moe.moe_block_out(D, B, y[-n:], res[-n:], gate[-n:], w, w, out, nxt, ra, rb)
        moe.moe_block_out_grad(D, B, None, dnext[-n:], y[-n:], out, gate[-n:], w, w, ra, rb, dres, dy, dg, None, None, False, ws)
        clean(ws)
        assert not any(bool(t[:-TAIL].any()) for t in (out, nxt, dres, dy, dg))
        got.append([t[-TAIL:].clone() for t in (out, nxt, ra, rb, dres, dy, dg)])
        del out, nxt, dres, dy
    assert all(torch.equal(a, b) for a, b in zip(*got)) and bool(got[0][0].any())


def test_combine_gradient_from_packed_rows():
    gen = torch.Generator("cuda").manual_seed(3)
    k, n = 2, T // 2
    y = _tail(gen, n * k)
    q, e = moe.packed_rows(n * k, d)
    moe.moe_pack_rows(y, q, e)
    del y
    dout = _tail(gen, n)
    gate = torch.randn(n, k, device="cuda", generator=gen)
    got = []
    for tokens in (n, TAIL):
        rows = tokens * k
        inv = torch.arange(rows, dtype=torch.int32, device="cuda").view(tokens, k)
        dy, dgate = torch.full((rows, d), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((tokens, k), 3.0, device="cuda")
        moe.moe_combine_rows_grad_packed(_dims(tokens, k), dout[-tokens:], q[-rows:], e[-rows:], gate[-tokens:], inv, dy, dgate)
        assert not dy[:-TAIL * k].any() and not dgate[:-TAIL].any()
        got.append([dy[-TAIL * k:].clone(), dgate[-TAIL:].clone()])
        del dy
    assert all(torch.equal(a, b) for a, b in zip(*got)) and bool(got[0][0].any()) and bool(got[0][1].any())
