"""The paged operators at the ends of their ranges: caches of more than 2^32
bytes, batches of thousands of sequences, positions near the end of int32, one
workspace for calls in turn, and calls at once on two streams."""
import numpy as np
import pytest
import torch

from helpers import new_workspace, to64
from oracle import paged as op
from test_paged_gpu import (BF16, F16, Pages, check_attention, check_prompt, gen, i32, randn, run_attention, run_prompt,
                            starts, status_ok, table_of)
from transformer_layer_gb300 import ds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,u4,page,pages", [(BF16, False, 64, 70000), (F16, True, 64, 270000)])
def test_pages_past_32_bit_offsets(dtype, u4, page, pages):
    """The same calls on a cache of over 2^32 bytes, whose last pages are used, and
    on a small one: equal bits everywhere."""
    nk, nh, d, lens, step = 4, 8, 128, [150, 1, 70], 2
    row = d // 2 if u4 else d
    need = [-(-(n + step) // page) for n in lens]
    g = gen(3)
    n = sum(lens)
    q, k, v = (randn((n, h, d), g, dtype) for h in (nh, nk, nk))
    q1, k1, v1 = (randn((3 * step, h, d), g, dtype) for h in (nh, nk, nk))
    results = []
    for total in (pages, sum(need)):
        ks, vs = (torch.empty((total, nk, page, row), dtype=torch.uint8 if u4 else dtype, device="cuda") for _ in range(2))
        assert total != pages or ks.numel() * ks.element_size() > 1 << 32
        sc = [torch.empty((total, nk, page, 2), dtype=F16, device="cuda") for _ in range(2)] if u4 else [None, None]
        table, at = np.full((3, max(need)), -1), total
        for b, m in enumerate(need):
            at -= m
            table[b, :m] = np.arange(at, at + m)
        c = ds.paged_cache(ks, vs, i32(table), dtype, *sc)
        nb = ds.ds_paged_attention_workspace_bytes(c, nh, 3, step)
        ws, rot = new_workspace(nb), ds.rotary(table_of(256, d))
        qr, q1r, out = torch.empty_like(q), torch.empty_like(q1), torch.empty_like(q1)
        ds.ds_paged_append(c, q, k, v, qr, i32(starts(lens)), i32([0, 0, 0]), 3, rot, ws)
        ds.ds_paged_append(c, q1, k1, v1, q1r, i32([0, step, 2 * step, 3 * step]), i32(lens), 3, rot, ws)
        ds.ds_paged_attention(c, q1r, out, i32(lens), 3, step, ws, nb)
        kg, vg = torch.empty_like(k), torch.empty_like(v)
        ds.ds_paged_gather(c, kg, vg, i32(starts(lens)), i32([0, 0, 0]), 3, ws)
        status_ok(ws)
        results.append((qr, q1r, out, kg, vg))
        del ks, vs, sc, c
    for a, b in zip(*results):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    if not u4:
        assert torch.equal(results[0][4], v)


@pytest.mark.parametrize("u4", [False, True])
def test_thousands_of_sequences(u4):
    """3000 sequences, most without rows or idle: append, attention and prompts."""
    rng = np.random.default_rng(5)
    B, page, nk, nh, d = 3000, 16, 1, 2, 64
    lens = np.where(rng.random(B) < 0.3, rng.integers(1, 20, B), 0)
    lens[1234], lens[B - 1] = 400, 33
    c = Pages([int(n) for n in lens], page, nk, d, F16, u4, 71)
    q = randn((B, nh, d), gen(1), F16)
    out, ws = run_attention(c, q, [int(n) for n in lens], 1)
    status_ok(ws)
    check_attention(c, q, out, [int(n) for n in lens], 1, d ** -0.5)
    cu = starts(lens)
    n = int(cu[-1])
    qp, k, v = (randn((n, h, d), gen(2), F16) for h in (nh, nk, nk))
    out, ws = run_prompt(qp, k, v, i32(cu), i32(cu), B)
    status_ok(ws)
    check_prompt(qp, k, v, out, cu, cu, d ** -0.5)
    ws = new_workspace(256)
    ds.ds_paged_append(c.handle, None, k, v, None, i32(cu), i32(np.zeros(B)), B, None, ws)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    ds.ds_paged_gather(c.handle, ko, vo, i32(cu), i32(np.zeros(B)), B, ws)
    status_ok(ws)
    for x, y in ((k, ko), (v, vo)):
        if u4:  # half a step of the row's range over 15, the scale's and minimum's rounding, and the result's
            x64 = to64(x)
            s = (x64.max(-1, keepdims=True) - x64.min(-1, keepdims=True)) / 15
            mag = np.abs(x64).max(-1, keepdims=True)
            assert np.all(np.abs(to64(y) - x64) <= s / 2 * (1 + 2.0 ** -10) + (2 * mag + 16 * s) * 2.0 ** -10)
        else:
            assert torch.equal(x, y)


def test_positions_at_the_end_of_int32():
    """A length at int32's end lies past every cache: flagged, its rows nowhere written, and no other sequence's."""
    page, nk, d, big = 16, 2, 64, 2 ** 31 - 1
    c = Pages([48, 40], page, nk, d, F16, False, 4)  # the first: full pages
    k, v = (randn((6, nk, d), gen(2), F16) for _ in range(2))
    kc, vc = c.k.clone(), c.v.clone()
    ws = new_workspace(256)
    ds.ds_paged_append(c.handle, None, k, v, None, i32([0, 3, 6]), i32([big, 7]), 2, None, ws)
    assert ds.ds_workspace_status(ws)[1] == ds.DS_DEVFLAG_CACHE_OVERFLOW
    for t in range(3):
        pg, r = op.place(c.table, page, 1, 7 + t)
        kc[pg, :, r], vc[pg, :, r] = k[3 + t], v[3 + t]
    assert torch.equal(c.k.view(torch.int16), kc.view(torch.int16)) and torch.equal(c.v.view(torch.int16), vc.view(torch.int16))
    ko, vo = torch.full_like(k, 5), torch.full_like(v, 5)
    ws = new_workspace(256)
    ds.ds_paged_gather(c.handle, ko, vo, i32([0, 3, 6]), i32([big, 7]), 2, ws)
    assert ds.ds_workspace_status(ws)[1] == ds.DS_DEVFLAG_CACHE_OVERFLOW
    assert (ko[:3] == 0).all() and (vo[:3] == 0).all() and torch.equal(ko[3:], k[3:]) and torch.equal(vo[3:], v[3:])
    q = randn((6, nk, d), gen(6), F16)
    nb = ds.ds_paged_attention_workspace_bytes(c.handle, nk, 2, 3)
    ws, out, ref = new_workspace(nb), torch.empty_like(q), torch.empty_like(q)
    full = c.table.shape[1] * page  # as many rows as the table can hold: what such a length attends
    for past, o in ((big, out), (full, ref)):
        ds.ds_paged_attention(c.handle, q, o, i32([past, 7]), 2, 3, ws, nb)
    code, flags = ds.ds_workspace_status(ws)
    assert flags & ds.DS_DEVFLAG_CACHE_OVERFLOW
    assert torch.isfinite(out).all() and torch.equal(out, ref)


def test_one_workspace_for_calls_in_turn():
    """Calls of every kind that join parts, one after the other in one workspace, give the bits of fresh ones."""
    g = gen(7)
    lens = [3000, 1, 900]
    c = Pages(lens, 16, 2, 128, F16, False, 5)
    c4 = Pages(lens, 32, 2, 64, BF16, True, 6)
    cu_q, cu_k, many = starts([3, 300]), starts([20000, 900]), starts([2000] * 4)
    q, q4 = randn((3, 8, 128), g, F16), randn((6, 4, 64), g, BF16)
    pq, pk, pv = randn((303, 2, 64), g, BF16), randn((20900, 1, 64), g, BF16), randn((20900, 1, 64), g, BF16)
    mq, mk, mv = (randn((8000, 30, 64), g, BF16) for _ in range(3))
    calls = [
        lambda ws: run_attention(c, q, lens, 1, ws=ws)[0],
        lambda ws: run_prompt(pq, pk, pv, i32(cu_q), i32(cu_k), 2, ws=ws)[0],
        lambda ws: run_attention(c4, q4, lens, 2, ws=ws)[0],
        lambda ws: run_prompt(mq, mk, mv, i32(many), i32(many), 4, ws=ws)[0],
    ]
    fresh = [f(None) for f in calls]
    ws = new_workspace(max(ds.ds_paged_attention_workspace_bytes(c.handle, 8, 3, 1),
                           ds.ds_paged_attention_workspace_bytes(c4.handle, 4, 3, 2),
                           ds.ds_prompt_attention_workspace_bytes(2, 2, 303),
                           ds.ds_prompt_attention_workspace_bytes(30, 4, 8000)))
    for i in (0, 1, 2, 3, 1, 0, 3, 3, 2, 1, 1, 0):
        assert torch.equal(calls[i](ws), fresh[i]), i
    status_ok(ws)


def test_two_streams_at_once():
    """Prompts and new tokens at the same time on two streams, a workspace each, again and again."""
    g = gen(9)
    lens = [2500, 80, 700]
    c = Pages(lens, 16, 2, 128, BF16, False, 8)
    q = randn((3, 8, 128), g, BF16)
    cu_q, cu_k = starts([700, 40]), starts([9000, 40])
    pq, pk, pv = randn((740, 4, 128), g, BF16), randn((9040, 2, 128), g, BF16), randn((9040, 2, 128), g, BF16)
    tq, tk = i32(cu_q), i32(cu_k)
    ref, ref_p = run_attention(c, q, lens, 1)[0], run_prompt(pq, pk, pv, tq, tk, 2)[0]
    torch.cuda.synchronize()
    check_prompt(pq, pk, pv, ref_p, cu_q, cu_k, 128 ** -0.5)
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, run_attention(c, q, lens, 1)[0] if i == 2 else run_prompt(pq, pk, pv, tq, tk, 2)[0]))
    torch.cuda.synchronize()
    for i, x in got:
        assert torch.equal(x, ref if i == 2 else ref_p)


def test_u4_values_that_average_out_over_a_long_cache():
    """200 thousand 4-bit rows around zero: the sums over codes and over minima are
    hundreds of times their difference, the result.  What is left of it is the rounding of
    the output and of each weight (fp16, acting on scale * (code - 8)): independent, each
    at most half a step and so 2^-11 / sqrt(3) of its value in the root mean square.
    A tenth is allowed for the fp32 sums."""
    N, nk, G, d, page = 200000, 8, 2, 128, 64
    n_pages = -(-N // page)
    g = gen(13)
    k, v = (torch.randint(0, 256, (n_pages, nk, page, d // 2), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    scale = torch.rand((n_pages, nk, page, 1), generator=g, device="cuda") * 0.1 + 0.3
    sc = torch.cat([scale, -7.5 * scale], -1).half()
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3))
    c = ds.paged_cache(k, v, table.int().cuda()[None].contiguous(), F16, sc, sc)
    q = randn((1, nk * G, d), g, F16) * 0.3
    nb = ds.ds_paged_attention_workspace_bytes(c, nk * G, 1, 1)
    ws, out = new_workspace(nb), torch.empty_like(q)
    ds.ds_paged_attention(c, q, out, i32([N - 1]), 1, 1, ws, nb)
    status_ok(ws)
    order = table.cuda()

    def rows(codes, h):  # codes, scales and minima of a head's positions, in 64 bits
        x = codes[order, h].reshape(-1, d // 2)[:N]
        s = sc[order, h].reshape(-1, 2)[:N].double()
        return torch.stack([x & 15, x >> 4], -1).reshape(N, d).double(), s[:, :1], s[:, 1:]

    err, allowed = 0.0, 0.0
    for h in range(nk):
        kc, ks, km = rows(k, h)
        vc, vs, vm = rows(v, h)
        for i in range(G):
            p = torch.softmax((kc * ks + km) @ q[0, h * G + i].double() * d ** -0.5, 0)
            ref = p @ (vc * vs + vm)
            weights = (p * p) @ (vs * (vc - 8)) ** 2
            err += ((out[0, h * G + i].double() - ref) ** 2).sum().item()
            allowed += (2.0 ** -22 / 3 * (ref ** 2 + weights)).sum().item()
    assert err <= 1.1 ** 2 * allowed, (err / allowed) ** 0.5
