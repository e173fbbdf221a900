"""Streaming attention without a GPU: bad arguments are refused on the host, before any CUDA call, by
the C entry points and by the binding."""
import ctypes

import pytest
import torch

from block_sparse_linear_router_b200 import build as B
from block_sparse_linear_router_b200 import sla2

P = 1 << 20        # a token address: 256-byte aligned, never read


@pytest.fixture(scope="module")
def lib():
    B.build()
    return sla2.load_library()


def _wdesc(**kw):
    d = dict(B=2, Hq=4, Hkv=2, N=100, d=64, window=8, sinks=2, causal=1, dtype=0, scale=0.125, workspace=P,
             workspace_bytes=1 << 30)
    d.update(kw)
    return sla2.WindowDesc(**d)


def _wview(i=0, H=4, d=64, **kw):
    v = dict(data=P + 4096 * (i + 1), stride_b=100 * H * d, stride_h=100 * d, stride_n=d)
    v.update(kw)
    return sla2.View(**v)


def _wfwd(lib, desc, q=None, k=None, v=None, out=None):
    return lib.sla2_window_forward(desc, q or _wview(0), k or _wview(1, 2), v or _wview(2, 2), out or _wview(3), None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(N=0), 1), (dict(Hkv=3), 1), (dict(window=0), 1),
    (dict(window=-5), 1), (dict(sinks=-1), 1), (dict(causal=2), 1), (dict(dtype=2), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(d=96), 2), (dict(d=256), 2),
    (dict(B=1 << 16, Hq=1 << 10, Hkv=1), 2), (dict(B=1, Hq=64, Hkv=1, N=1 << 26), 2)])
def test_window_description_is_checked(lib, bad, code):
    d = _wdesc(**bad)
    assert _wfwd(lib, d) == code
    assert lib.sla2_window_backward_workspace_size(d) == 0
    views = [_wview(i, 4) for i in range(8)]
    assert lib.sla2_window_backward(d, *views[:4], P, *views[4:], None) == code


def test_window_of_many_sequences_and_heads(lib):
    """B * Hq * N < 2^31 is the only limit on them."""
    for ok in (dict(B=1024, Hq=64, Hkv=2), dict(B=70000, Hq=4, Hkv=1), dict(B=1, Hq=1, Hkv=1, N=1 << 30)):
        assert lib.sla2_window_backward_workspace_size(_wdesc(**ok)) > 0
    for bad in (dict(B=1 << 20, Hq=1 << 11, Hkv=1, N=1), dict(B=2, Hq=1, Hkv=1, N=1 << 30)):
        assert lib.sla2_window_backward_workspace_size(_wdesc(**bad)) == 0 and _wfwd(lib, _wdesc(**bad)) == 2


@pytest.mark.parametrize("bad", [dict(data=None), dict(data=P + 8), dict(stride_n=32), dict(stride_n=0), dict(stride_n=68),
                                 dict(stride_h=-64), dict(stride_b=0), dict(stride_b=1 << 39)])
def test_window_views_are_checked(lib, bad):
    for i, H in enumerate((4, 2, 2, 4)):
        views = [None] * 4
        views[i] = _wview(i, H, **bad)
        assert _wfwd(lib, _wdesc(), *views) == 1
    for i in range(8):
        views = [_wview(j) for j in range(8)]
        views[i] = _wview(i, **bad)
        assert lib.sla2_window_backward(_wdesc(), *views[:4], P, *views[4:], None) == 1
    assert lib.sla2_window_forward(None, _wview(0), _wview(1), _wview(2), _wview(3), None, None) == 1


def test_window_outputs_may_not_be_inputs(lib):
    for i in range(3):
        assert _wfwd(lib, _wdesc(), out=_wview(i)) == 1
    base = [_wview(j) for j in range(8)]      # q k v out | dout dq dk dv
    for o in (5, 6, 7):
        for i in range(8):
            if i != o:
                views = list(base)
                views[o] = base[i]
                assert lib.sla2_window_backward(_wdesc(), *views[:4], P, *views[4:], None) == 1
    assert lib.sla2_window_backward(_wdesc(), *base[:4], None, *base[4:], None) == 1     # no lse


def test_window_backward_workspace(lib):
    base = [_wview(j) for j in range(8)]
    n = lib.sla2_window_backward_workspace_size(_wdesc())
    assert n > 0 and n % 256 == 0
    for bad in (dict(workspace=None), dict(workspace=P + 16), dict(workspace_bytes=n - 1)):
        assert lib.sla2_window_backward(_wdesc(**bad), *base[:4], P, *base[4:], None) == 3


def _cache(**kw):
    d = dict(num_pages=10, Hkv=2, page=64, d=64, k_codes=P, v_codes=P, k_scale=P, v_scale=P)
    d.update(kw)
    return sla2.CacheDesc(**d)


def _step(**kw):
    d = dict(B=3, T=3, Hq=4, max_pages=5, dtype=0, page_table=P, kv_lens=P, cu_new=P)
    d.update(kw)
    return sla2.StepDesc(**d)


def _tview(i=0, **kw):
    v = dict(data=P + 4096 * (i + 1), stride_b=0, stride_h=64, stride_n=256)
    v.update(kw)
    return sla2.View(**v)


def _append(lib, c=None, s=None, views=None, cos=P, sin=P, rows=8, dim=64, inter=0):
    v = views or [_tview(i) for i in range(5)]
    return lib.sla2_cache_append(c or _cache(), s or _step(), *v, cos, sin, rows, dim, inter, None)


def _attend(lib, c=None, s=None, q=None, out=None, window=8, sinks=0, scale=0.1, ws=P, n=1 << 30):
    return lib.sla2_cache_attention(c or _cache(), s or _step(), q or _tview(0), out or _tview(1), window, sinks, scale, ws,
                                    n, None)


@pytest.mark.parametrize("cache,step,code", [
    (dict(num_pages=0), {}, 1), (dict(Hkv=0), {}, 1), (dict(Hkv=3), {}, 1), (dict(page=48), {}, 2), (dict(page=8), {}, 2),
    (dict(page=256), {}, 2), (dict(d=80), {}, 2), (dict(k_codes=None), {}, 1), (dict(v_codes=P + 4), {}, 1),
    (dict(k_scale=None), {}, 1), (dict(v_scale=None), {}, 1), ({}, dict(B=0), 1), ({}, dict(T=0), 1), ({}, dict(T=-1), 1),
    ({}, dict(Hq=0), 1), ({}, dict(Hq=5), 1), ({}, dict(max_pages=0), 1), ({}, dict(dtype=3), 1),
    ({}, dict(page_table=None), 1), ({}, dict(kv_lens=None), 1), ({}, dict(cu_new=None), 1)])
def test_cache_and_step_are_checked(lib, cache, step, code):
    c, s = _cache(**cache), _step(**step)
    assert _append(lib, c, s) == code
    assert _attend(lib, c, s) == code
    assert lib.sla2_cache_attention_workspace_size(c, s) == 0
    assert lib.sla2_cache_attention_workspace_size(None, _step()) == 0


def test_append_arguments_are_checked(lib):
    for bad in (dict(data=None), dict(data=P + 8), dict(stride_n=32), dict(stride_h=0), dict(stride_n=260), dict(stride_n=-256)):
        for i in range(5):
            v = [_tview(j) for j in range(5)]
            v[i] = _tview(i, **bad)
            assert _append(lib, views=v) == 1
    v = [_tview(j) for j in range(5)]
    for out, src in ((3, 0), (3, 1), (3, 2), (4, 0), (4, 1), (4, 2), (3, 4)):
        w = list(v)
        w[out] = v[src]
        assert _append(lib, views=w) == 1
    assert _append(lib, views=[v[0], v[1], None, v[3], None]) == 1      # q_out without q
    assert _append(lib, views=[v[0], v[1], v[2], None, None]) == 1      # q without q_out
    for kw in (dict(dim=24), dict(dim=80), dict(dim=-16), dict(dim=0), dict(rows=0), dict(cos=None), dict(sin=None),
               dict(cos=None, sin=None), dict(inter=2), dict(cos=P + 4)):
        assert _append(lib, **kw) == 1, kw


def test_cache_attention_arguments_are_checked(lib):
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0),
               dict(out=_tview(0)), dict(q=_tview(0, stride_n=8)), dict(out=_tview(1, data=P + 2))):
        assert _attend(lib, **kw) == 1, kw
    n = lib.sla2_cache_attention_workspace_size(_cache(), _step())
    assert n > 0
    for kw in (dict(ws=None), dict(ws=P + 16), dict(n=n - 1)):
        assert _attend(lib, **kw) == 3, kw


def test_the_status_code_has_a_name(lib):
    assert b"page" in lib.sla2_status_string(6)
    assert str(sla2.Sla2Error(6, "x")).endswith("position)")


def _q(H=4, N=10, d=64, dt=torch.bfloat16):
    return torch.zeros(2, H, N, d, dtype=dt)


@pytest.mark.parametrize("change,match", [
    (dict(k=_q(2, 9)), "k and v"), (dict(v=_q(1)), "k and v"), (dict(k=_q(3), v=_q(3)), "multiple"),
    (dict(q=_q(dt=torch.float32)), "bf16"), (dict(v=_q(2, dt=torch.float16)), "bf16"), (dict(window=0), "window"),
    (dict(sinks=-1), "sinks"), (dict(lens=torch.zeros(2, dtype=torch.int64)), "lens"),
    (dict(lens=torch.zeros(3, dtype=torch.int32)), "lens"), (dict(out=_q(2)), "outputs"), (dict(q=torch.zeros(4, 10, 64)), "q, k, v"),
    (dict(q=torch.zeros(2, 4, 64, 10, dtype=torch.bfloat16).transpose(2, 3)), "contiguous"),
    (dict(status=torch.zeros(2, dtype=torch.int32)), "status"), ({}, "CUDA device")])
def test_window_binding_refuses(change, match):
    a = dict(q=_q(), k=_q(2), v=_q(2), window=4)
    a.update(change)
    with pytest.raises(ValueError, match=match):
        sla2.window_forward(**a)


def test_window_backward_binding_refuses():
    q, k = _q(), _q(2)
    lse = torch.zeros(2, 4, 10)
    for a, match in (((q, k, k, q, lse, _q(2), 4), "outputs"), ((q, k, k, q, lse.double(), q, 4), "lse"),
                     ((q, k, k, q, lse[:, :2], q, 4), "lse"), ((q, k, k, q.float(), lse, q, 4), "outputs"),
                     ((q, k, k, q, lse, q, 4), "CUDA device")):
        with pytest.raises(ValueError, match=match):
            sla2.window_backward(*a)


def test_cache_binding_refuses():
    c = sla2.KVCache.empty(4, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        sla2.KVCache(c.k_codes, c.v_codes[:2], c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        sla2.KVCache(c.k_codes, c.v_codes, c.k_scale.double(), c.v_scale)
    with pytest.raises(ValueError):
        sla2.KVCache(c.k_codes.transpose(0, 1), c.v_codes.transpose(0, 1), c.k_scale.T, c.v_scale.T)
    k = torch.zeros(3, 2, 64, dtype=torch.float16)
    table, lens, cu = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    rope = (torch.zeros(5, 16), torch.zeros(5, 16))
    good = dict(k=k, v=k, page_table=table, kv_lens=lens, cu_new=cu)
    for change, match in ((dict(k=k[..., :32]), "token arrays"), (dict(v=k[:2]), "k and v"), (dict(v=k.bfloat16()), "k and v"),
                          (dict(page_table=table.long()), "page_table"), (dict(kv_lens=lens[:2]), "kv_lens"),
                          (dict(cu_new=lens), "cu_new"), (dict(q=torch.zeros(3, 3, 64, dtype=torch.float16)), "multiple"),
                          (dict(q=torch.zeros(3, 4, 64)), "q must be"), (dict(q_out=k), "q_out"), (dict(k_out=k[:1]), "k_out"),
                          (dict(rope=(rope[0], rope[1].double())), "rope"), (dict(rope=(rope[0][:, :12],) * 2), "rope"),
                          (dict(rope=(torch.zeros(5, 40),) * 2), "rope_dim"), ({}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            sla2.cache_append(c, **{**good, **change})
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    good = dict(q=q, page_table=table, kv_lens=lens, cu_new=cu)
    for change, match in ((dict(q=q.float()), "token arrays"), (dict(q=q[:, :3]), "multiple"), (dict(window=0), "window"),
                          (dict(sinks=-1), "sinks"), (dict(out=q.bfloat16()), "out"), ({}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            sla2.cache_attention(c, **{**good, **change})
