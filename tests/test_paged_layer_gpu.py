"""GPU parity of the layer over a paged cache (ds_layer_forward_paged): packed
prompts enter the pages, then new tokens are decoded over them, as a server
would call it.  The oracle is fed the device's input and, for the attention,
the rows that the device's pages hold after the call (the new rows are checked
against the oracle's keys and values, to the pages' rounding)."""
import numpy as np
import pytest
import torch

import oracle
from helpers import DeviceLayer, check_close, new_workspace, to64
from oracle import paged as op
from test_paged_gpu import BF16, F16, Pages, i32, starts, table_of
from transformer_layer_gb300 import ds, inputs

pytestmark = pytest.mark.gpu


def reference(x, p, heads, attend):
    """The layer in float64 with region 2 given: attend(q [N, nh, d], k, v)."""
    N, H = x.shape
    h1 = oracle.layer_norm(x, p["ln1_g"], p["ln1_b"])
    q, k, v = np.split(oracle.linear(h1, p["w_qkv"], p["b_qkv"]).reshape(N, 3 * heads, H // heads), 3, axis=1)
    x1 = x + oracle.linear(attend(q, k, v).reshape(N, H), p["w_o"], p["b_o"])
    g = oracle.gelu_tanh(oracle.linear(oracle.layer_norm(x1, p["ln2_g"], p["ln2_b"]), p["w_fc1"], p["b_fc1"]))
    return x1 + oracle.linear(g, p["w_fc2"], p["b_fc2"])


@pytest.mark.parametrize("act,weight,H,nh,F,u4,page,first,new", [
    (F16, F16, 512, 8, 2048, False, 16, [5, 40, 1], [1, 1, 3]),
    (BF16, BF16, 512, 4, 1024, True, 32, [33, 0, 17, 130], [1, 2]),
    (F16, torch.int8, 1024, 8, 2048, True, 16, [20, 3], [1, 4]),
    (BF16, BF16, 512, 4, 1024, False, 64, [70, 64], [1]),
    (F16, F16, 256, 4, 1024, True, 16, [4], [1, 1]),
])
def test_layer_over_pages(act, weight, H, nh, F, u4, page, first, new):
    L = DeviceLayer(H, nh, F, seed=1700, act_dtype=act, weight_dtype=weight)
    try:
        p, d, B = L.oracle_params(), H // nh, len(first)
        cap = [n + sum(new) for n in first]
        c = Pages(cap, page, nh, d, act, u4, 81)
        tab = table_of(256, d)
        rot, tab64 = ds.rotary(tab), to64(tab)
        past, step = np.zeros(B, np.int64), 0
        ws = None
        for T in [0] + new:
            count = np.array(first) if T == 0 else np.full(B, T)
            cu, N = starts(count), int(count.sum())
            pad = 2 if T == 0 else 0
            x = inputs.hidden(N + pad, 1, H, 1700, step=step, dtype=act, device="cuda").reshape(N + pad, H)
            y = torch.full_like(x, float("nan"))
            nb = ds.ds_layer_paged_workspace_bytes(L.handle, c.handle, N + pad, B, T)
            assert nb > 0
            if ws is None or ws.numel() < nb:
                ws = new_workspace(nb)
                ws[256:].fill_(0xff)           # only the status word has to be zero
            n0 = ds.ds_launch_count()
            ds.ds_layer_forward_paged(L.handle, x, y, c.handle, rot, i32(cu), i32(past), B, T, ws, nb)
            assert 5 + 2 <= ds.ds_launch_count() - n0 <= 7 + 4
            code, flags = ds.ds_workspace_status(ws)
            assert code == ds.DS_OK and flags == 0
            kv = c.values()

            def attend(q, k, v):
                out = np.zeros_like(q)
                for b in range(B):
                    r = slice(int(cu[b]), int(cu[b + 1]))
                    n = int(past[b]) + r.stop - r.start
                    at = [op.rotate(z[r.start + i], tab64[int(past[b]) + i]) for z in (q, k) for i in range(r.stop - r.start)]
                    qr, kr = np.array(at[:len(at) // 2]), np.array(at[len(at) // 2:])
                    ks, vs = (op.sequence_rows(z, c.table, page, b, n) for z in kv)
                    for want, got in ((kr, ks[int(past[b]):]), (v[r], vs[int(past[b]):])):
                        if len(want):
                            err = np.abs(got - want)
                            spread = want.max(-1, keepdims=True) - want.min(-1, keepdims=True)
                            # two roundings of the type, the projection's own error; a 4-bit step
                            assert np.all(err <= (spread / 15 * 0.55 if u4 else 0) + 2e-2)
                    if len(qr):
                        out[r] = op.attend(qr, ks, vs, int(past[b]) + 1, d ** -0.5)[0]
                return out

            ref = reference(to64(x)[:N], p, nh, attend)
            check_close(y[:N], ref, act, what=f"T={T} past={past.tolist()}")
            past = past + count
            step += 1
    finally:
        L.close()


def test_layer_over_pages_refusals_and_graph():
    H, nh = 256, 4
    L = DeviceLayer(H, nh, 1024, seed=1701)
    try:
        c = Pages([40, 40], 16, nh, 64, F16, False, 82)
        x = inputs.hidden(2, 1, H, 1701, device="cuda").reshape(2, H)
        y = torch.empty_like(x)
        past = i32([3, 17])
        nb = ds.ds_layer_paged_workspace_bytes(L.handle, c.handle, 2, 2, 1)
        ws = new_workspace(nb)
        other = Pages([40], 16, 2, 64, F16, False, 83)   # another number of key heads
        n0 = ds.ds_launch_count()
        for call, code in (
                (lambda: ds.ds_layer_forward_paged(L.handle, x, y, other.handle, None, None, past[:1], 1, 2, ws, nb), ds.DS_ERR_INVALID_ARG),
                (lambda: ds.ds_layer_forward_paged(L.handle, x, x, c.handle, None, None, past, 2, 1, ws, nb), ds.DS_ERR_INVALID_ARG),
                (lambda: ds.ds_layer_forward_paged(L.handle, x, y, c.handle, None, None, past, 2, 17, ws, nb), ds.DS_ERR_INVALID_ARG),
                (lambda: ds.ds_layer_forward_paged(L.handle, x, y, c.handle, None, None, past, 2, 3, ws, nb), ds.DS_ERR_INVALID_ARG),
                (lambda: ds.ds_layer_forward_paged(L.handle, x, y, c.handle, None, None, past, 2, 1, ws, nb - 256), ds.DS_ERR_WORKSPACE)):
            with pytest.raises(ds.DSError) as e:
                call()
            assert e.value.code == code
        assert ds.ds_layer_paged_workspace_bytes(L.handle, other.handle, 2, 2, 1) == 0
        assert ds.ds_launch_count() == n0
        k0 = c.k.clone()
        ds.ds_layer_forward_paged(L.handle, x, y, c.handle, None, None, past, 2, 1, ws, nb)
        torch.cuda.synchronize()
        ref, k1 = y.clone(), c.k.clone()
        c.k.copy_(k0)
        y.fill_(0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ds.ds_layer_forward_paged(L.handle, x, y, c.handle, None, None, past, 2, 1, ws, nb)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(torch.nan_to_num(c.k), torch.nan_to_num(k1))
    finally:
        L.close()
