"""Host-side checks of the 4-bit cache's entry points: sizes, and refusals before any launch
(fake device addresses that are never dereferenced)."""
import pytest
import torch

from dequant_gemv_amd import binding as B

A = 0x10000
OK, ARG, UNS, MIS, WS = (B.DQG_OK, B.DQG_ERR_INVALID_ARG, B.DQG_ERR_UNSUPPORTED,
                         B.DQG_ERR_MISALIGNED, B.DQG_ERR_WORKSPACE)


def test_page_bytes():
    assert B.kv4_page_bytes(4, 128, 64, 32) == 4 * 64 * 144
    assert B.kv4_page_bytes(1, 64, 32, 32) == 32 * 72
    assert B.kv4_page_bytes(8, 256, 128, 128) == 8 * 128 * 264
    for bad in ((0, 128, 64, 32), (4, 96, 64, 32), (4, 64, 64, 128), (4, 128, 48, 32),
                (4, 128, 16, 32), (4, 128, 64, 64), (4, 128, 1 << 17, 32), (2000, 128, 64, 32)):
        assert B.kv4_page_bytes(*bad) == 0, bad


def test_workspace_bytes():
    f = B.kv4_attention_workspace_bytes
    assert f(1, 1, 32, 4, 128, 256) == 0          # one split
    assert f(1, 1, 32, 4, 128, 100000) > 0
    for bad in ((0, 1, 32, 4, 128, 4096), (1, 0, 32, 4, 128, 4096), (1, 1, 30, 4, 128, 4096),
                (1, 1, 32, 4, 96, 4096), (1, 1, 32, 4, 128, 0), (1, 1, 32, 4, 128, -5)):
        assert f(*bad) == 0, bad


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 4, 128), (8, 8, 64), (14, 2, 256), (7, 1, 128)])
def test_workspace_grows_with_each_size(Hq, Hkv, D):
    f = B.kv4_attention_workspace_bytes
    lens = [1, 255, 256, 511, 512, 4096, 4097, 131072, 1 << 30]
    for axis in range(3):
        for fixed in ((1, 1, 4096), (17, 5, 100000), (300, 64, 1024)):
            prev = 0
            for x in (lens if axis == 2 else range(1, 1200, 7)):
                a = list(fixed)
                a[axis] = x
                n = f(a[0], a[1], Hq, Hkv, D, a[2])
                assert n >= prev and n % 256 == 0, (axis, a)
                prev = n


def _rows(fn, **kw):
    a = dict(k=A, v=A, T=4, ks=512, vs=512, B=2, cu=A, lens=A, table=A, mp=4, cache=A, pages=9,
             H=4, D=128, page=64, G=32, fmt=0, st=0)
    a.update(kw)
    return getattr(B.LIB, fn)(a["k"], a["v"], a["T"], a["ks"], a["vs"], a["B"], a["cu"], a["lens"],
                              a["table"], a["mp"], a["cache"], a["pages"], a["H"], a["D"],
                              a["page"], a["G"], a["fmt"], a["st"], None)


WHERE = [
    (dict(cu=0), ARG), (dict(lens=0), ARG), (dict(table=0), ARG), (dict(cache=0), ARG),
    (dict(T=0), ARG), (dict(B=0), ARG), (dict(mp=0), ARG), (dict(pages=0), ARG), (dict(H=0), ARG),
    (dict(fmt=2), UNS), (dict(fmt=0x100), UNS), (dict(D=96), UNS), (dict(G=64), UNS),
    (dict(page=48), UNS), (dict(page=16), UNS), (dict(mp=1 << 25), UNS), (dict(B=1 << 17), UNS),
    (dict(T=1 << 23), UNS), (dict(H=2000), UNS),
    (dict(cache=A + 8), MIS), (dict(cu=A + 2), MIS), (dict(lens=A + 1), MIS),
    (dict(table=A + 2), MIS), (dict(st=A + 2), MIS),
]


@pytest.mark.parametrize("fn", ["kv4_write", "kv4_read"])
@pytest.mark.parametrize("kw,status", WHERE + [
    (dict(k=0), ARG), (dict(v=0), ARG), (dict(ks=511), ARG), (dict(vs=0), ARG), (dict(ks=-8), ARG),
    (dict(ks=516), MIS), (dict(vs=513), MIS), (dict(k=A + 8), MIS), (dict(v=A + 2), MIS)])
def test_rows_are_refused(fn, kw, status):
    assert _rows(fn, **kw) == status


def _attend(**kw):
    a = dict(q=A, T=4, qs=4096, B=2, cu=A, lens=A, table=A, mp=4, cache=A, pages=9, Hq=32, H=4,
             D=128, page=64, G=32, fmt=0, scale=0.1, window=0, sinks=0, rows=0, kv=0, out=A,
             os=4096, lse=0, st=0, ws=0, wsb=0)
    a.update(kw)
    return B.LIB.kv4_attention(a["q"], a["T"], a["qs"], a["B"], a["cu"], a["lens"], a["table"],
                               a["mp"], a["cache"], a["pages"], a["Hq"], a["H"], a["D"],
                               a["page"], a["G"], a["fmt"], a["scale"], a["window"], a["sinks"],
                               a["rows"], a["kv"], a["out"], a["os"], a["lse"], a["st"], a["ws"],
                               a["wsb"], None)


@pytest.mark.parametrize("kw,status", WHERE + [
    (dict(fmt=B.KV4_FORCE_FEW | B.KV4_FORCE_MANY), ARG), (dict(fmt=B.KV4_FORCE_FEW | 2), UNS),
    (dict(q=0), ARG), (dict(out=0), ARG), (dict(Hq=0), ARG), (dict(Hq=30), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(window=-1), ARG),
    (dict(sinks=-1), ARG), (dict(rows=-1), ARG), (dict(kv=-1), ARG), (dict(qs=4088), ARG),
    (dict(os=4000), ARG), (dict(qs=4100), MIS), (dict(os=4097), MIS), (dict(q=A + 8), MIS),
    (dict(out=A + 2), MIS), (dict(lse=A + 2), MIS), (dict(ws=A + 8, wsb=1 << 30), MIS),
    (dict(mp=64, ws=A, wsb=1024), WS), (dict(T=1 << 22, Hq=1024, qs=1 << 18, os=1 << 18), UNS),
])
def test_attention_is_refused(kw, status):
    assert _attend(**kw) == status


@pytest.mark.parametrize("fn", ["kv4_write", "kv4_read"])
@pytest.mark.parametrize("T,B_,H", [(1 << 22, 1, 1024), (1, 65536, 256), (1 << 22, 65536, 52)])
def test_rows_beyond_a_grid_are_refused(fn, T, B_, H):
    assert _rows(fn, T=T, B=B_, H=H, ks=H * 128, vs=H * 128) == UNS


@pytest.mark.parametrize("T,B_,Hq,H,path", [
    (65536, 65536, 128, 128, 0), (1 << 18, 65536, 1024, 128, B.KV4_FORCE_FEW),
    (1 << 16, 65536, 1024, 1024, B.KV4_FORCE_MANY), (1 << 16, 1 << 16, 128, 128, B.KV4_FORCE_FEW)])
def test_tiles_beyond_a_grid_are_refused(T, B_, Hq, H, path):
    assert _attend(T=T, B=B_, Hq=Hq, H=H, qs=Hq * 128, os=Hq * 128, fmt=path) == UNS


def test_binding_refuses():
    c = torch.zeros(3, B.kv4_page_bytes(2, 64, 32, 32), dtype=torch.uint8)
    cu, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 3, dtype=torch.int32)
    rows = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # host tensors
        B.kv4_write(rows, rows, cu, lens, table, c, 32, 32, B.FMT_INT4)
    with pytest.raises(ValueError):
        B.kv4_attention(rows, cu, lens, table, c, 2, 32, 32, B.FMT_INT4, 0.1)
    with pytest.raises(ValueError):
        B.kv4_read(1, 2, 64, cu, lens, table, c, 32, 32, B.FMT_INT4)
    with pytest.raises(ValueError):
        B.kv4_write(rows[0], rows, cu, lens, table, c, 32, 32, B.FMT_INT4)
    with pytest.raises(ValueError):
        B.kv4_cache(3, 2, 96, 32, 32, "cpu")
    assert B.kv4_cache(3, 2, 64, 32, 32, "cpu").shape == c.shape
    assert B.kv4_workspace(1, 1, 2, 2, 64, 100, "cpu") is None
