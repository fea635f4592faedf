"""Refusals of the entry points for rotary positions, pages and shared prefixes, on the host, before
any launch."""
import os

import pytest
import torch

from exact_io_aware_28_gb300 import fa

from test_paged_latent_boundary import A, I32, INV, UNS, X, _call, _z

pytestmark = pytest.mark.skipif(not os.path.exists(fa.LIB_PATH),
                                reason="libfa_gb300.so not built")

ROPE = dict(x=X[0], y=X[1], xb=2 * 10 * 64, xh=10 * 64, xn=64, yb=2 * 10 * 64, yh=10 * 64, yn=64,
            pos=X[2], pa=30, pb=10, axes=2, turns=X[3], axis=X[4], B=3, H=2, N=10, d=64, rot=64,
            inter=0, inv=0, dtype=fa.FA_BF16)
BYTES = 3 * 2 * 10 * 64 * 2


@pytest.mark.parametrize("kw,code", [
    ({"x": None}, INV), ({"x": A + 8}, INV), ({"y": None}, INV), ({"y": X[1] + 4}, INV),
    ({"pos": None}, INV), ({"pos": A + 2}, INV), ({"turns": None}, INV), ({"turns": X[3] + 4}, INV),
    ({"axis": None}, INV), ({"axis": X[4] + 1}, INV), ({"axes": 0}, INV), ({"B": 0}, INV),
    ({"H": 0}, INV), ({"N": -1}, INV), ({"dtype": 2}, INV), ({"d": 60}, UNS), ({"d": 8, "rot": 8}, UNS),
    ({"d": 2048, "rot": 64}, UNS), ({"rot": 24}, UNS), ({"rot": 0}, UNS), ({"rot": 80}, UNS),
    ({"B": 70000}, UNS), ({"H": 70000}, UNS), ({"N": (1 << 30) + 1}, UNS),
    ({"xn": 60}, INV), ({"yh": 644}, INV), ({"xb": -64}, INV), ({"pa": -1}, INV), ({"pb": -10}, INV),
    ({"dtype": fa.FA_FP32, "xn": 66, "x": X[5]}, INV),
    # y's elements over one another
    ({"yn": 56}, INV), ({"yn": 0}, INV), ({"yh": 9 * 64}, INV), ({"yb": 0}, INV),
    ({"yn": 128, "yh": 64, "yb": 10 * 128 - 8}, INV),
    # y over an input, in part or with other strides
    ({"y": X[0] + 128}, INV), ({"y": X[0], "yn": 128, "yh": 64}, INV), ({"y": X[0] - 16}, INV),
    ({"y": X[0] + BYTES - 16}, INV), ({"y": X[2]}, INV), ({"y": X[3] + 240}, INV),
    ({"y": X[4] - BYTES + 16}, INV),
])
def test_rope_rejects(kw, code):
    assert _call("fa_rope", ROPE, kw) == code


QE, KE, PAGE = 4 * 64, 2 * 64, 2 * 16 * 64
RAPPEND = dict(q=X[0], k=X[1], v=X[2], qs=QE, ks=KE, vs=KE, qo=X[3], qos=QE, kc=X[4], vc=X[5], ps=PAGE,
               slots=X[6], pos=X[7], pa=5, axes=1, turns=X[8], axis=X[9], T=5, Hq=4, Hkv=2, P=8, page=16,
               d=64, rot=64, inter=0)
FUSED = 8 * 64    # q, k, v as slices of one projection


@pytest.mark.parametrize("kw,code", [
    ({"q": None}, INV), ({"k": A + 8}, INV), ({"v": None}, INV), ({"qo": X[3] + 2}, INV),
    ({"kc": None}, INV), ({"vc": X[5] + 4}, INV), ({"slots": X[6] + 2}, INV), ({"pos": None}, INV),
    ({"turns": X[8] + 4}, INV), ({"axis": None}, INV), ({"axes": 0}, INV), ({"T": -1}, INV),
    ({"Hq": 0}, INV), ({"Hkv": 0}, INV), ({"qs": QE - 8}, INV), ({"ks": KE + 4}, INV),
    ({"vs": 0}, INV), ({"qos": QE - 8}, INV), ({"ps": PAGE - 8}, INV), ({"P": 0}, INV),
    ({"page": 24}, UNS), ({"d": 96}, UNS), ({"rot": 72}, UNS), ({"rot": 128}, UNS),
    ({"T": (1 << 26) + 1}, UNS), ({"T": 0}, fa.FA_OK),
    ({"axes": 2, "pa": -5}, INV),
    # what may share memory and what not
    ({"qo": X[0] + 16}, INV), ({"qo": X[0], "qos": QE + 64}, INV), ({"qo": X[1]}, INV),
    ({"qo": X[2] + 32}, INV), ({"qo": X[4]}, INV), ({"qo": X[5] + 64}, INV), ({"qo": X[6]}, INV),
    ({"qo": X[8]}, INV), ({"kc": X[0]}, INV), ({"vc": X[1]}, INV), ({"kc": X[2] + 64}, INV),
    ({"vc": X[4]}, INV), ({"vc": X[4] + 2 * PAGE}, INV), ({"kc": X[7]}, INV), ({"vc": X[9]}, INV),
    # rows of one projection: in place of the queries, but not over the keys' or values' rows
    ({"q": X[0], "k": X[0] + 2 * QE, "v": X[0] + 2 * (QE + KE), "qs": FUSED, "ks": FUSED, "vs": FUSED,
      "qo": X[0] + 2 * KE, "qos": FUSED}, INV),
    ({"q": X[0], "k": X[0] + 2 * (QE - 8), "v": X[0] + 2 * (QE + KE), "qs": FUSED, "ks": FUSED,
      "vs": FUSED, "qo": X[0], "qos": FUSED}, INV),
])
def test_rope_append_rejects(kw, code):
    assert _call("fa_rope_append", RAPPEND, kw) == code


FORK = dict(cl=X[0], table=X[1], stride=16, M=16, free=X[2], n_free=8, src=X[3], dst=X[4], n=3, cs=X[5],
            cd=X[6], cr=X[7], taken=X[8], B=4, page=16, P=64)


@pytest.mark.parametrize("kw,code", [
    ({"cl": None}, INV), ({"table": A + 2}, INV), ({"free": None}, INV), ({"src": None}, INV),
    ({"dst": X[4] + 1}, INV), ({"cs": None}, INV), ({"cd": None}, INV), ({"cr": X[7] + 2}, INV),
    ({"taken": None}, INV), ({"n": -1}, INV), ({"n_free": -1}, INV), ({"B": 0}, INV), ({"M": 0}, INV),
    ({"stride": 15}, INV), ({"P": 0}, INV), ({"page": 8}, UNS), ({"P": 1 << 27}, UNS),
    ({"B": 8193}, UNS), ({"n": 8193}, UNS), ({"B": 8192, "M": 16385, "stride": 16385}, UNS),
    ({"cs": X[3]}, INV), ({"cd": X[5] + 8}, INV), ({"taken": X[2] + 28}, INV), ({"cl": X[4]}, INV),
    ({"table": X[2] - 64}, INV), ({"cr": X[1] + 12}, INV),
])
def test_fork_rejects(kw, code):
    assert _call("fa_paged_fork", FORK, kw) == code


FREE = dict(cl=X[0], table=X[1], stride=16, M=16, rows=X[2], n=3, refs=X[3], free=X[4], n_free=X[5], B=4,
            page=16, P=64)


@pytest.mark.parametrize("kw,code", [
    ({"cl": A + 2}, INV), ({"table": None}, INV), ({"rows": None}, INV), ({"refs": None}, INV),
    ({"free": X[4] + 2}, INV), ({"n_free": None}, INV), ({"n": -2}, INV), ({"B": 0}, INV),
    ({"stride": 3}, INV), ({"page": 17}, UNS), ({"B": 8193}, UNS), ({"P": 0}, INV),
    ({"refs": X[2]}, INV), ({"free": X[3] + 4 * 63}, INV), ({"n_free": X[0] + 4}, INV),
    ({"refs": X[1]}, INV), ({"n_free": X[4]}, INV),
])
def test_free_rejects(kw, code):
    assert _call("fa_paged_free", FREE, kw) == code


COMPACT = dict(cl=X[0], table=X[1], stride=16, M=16, moved=X[2], cs=X[3], cd=X[4], n=32, used=X[5], B=4,
               page=16, P=64)


@pytest.mark.parametrize("kw,code", [
    ({"cl": None}, INV), ({"table": A + 1}, INV), ({"moved": None}, INV), ({"cs": None}, INV),
    ({"cd": X[4] + 2}, INV), ({"used": None}, INV), ({"n": 31}, INV), ({"B": -1}, INV),
    ({"page": 0}, UNS), ({"B": 9000}, UNS), ({"M": 17}, INV), ({"P": 1 << 27, "n": 1 << 26}, UNS),
    ({"moved": X[0]}, INV), ({"cs": X[2] + 16}, INV), ({"cd": X[3]}, INV), ({"used": X[1] + 8}, INV),
    ({"table": X[0] - 32}, INV),
])
def test_compact_rejects(kw, code):
    assert _call("fa_paged_compact", COMPACT, kw) == code


COPY = dict(kc=X[0], vc=X[1], ps=8 * 16 * 64, src=X[2], dst=X[3], rows=X[4], n=5, P=16, Hkv=8, page=16,
            d=64)


@pytest.mark.parametrize("kw,code", [
    ({"kc": None}, INV), ({"vc": X[1] + 8}, INV), ({"src": None}, INV), ({"dst": X[3] + 2}, INV),
    ({"rows": X[4] + 1}, INV), ({"n": -1}, INV), ({"Hkv": 0}, INV), ({"ps": 8 * 16 * 64 - 8}, INV),
    ({"P": 0}, INV), ({"d": 96}, UNS), ({"page": 24}, UNS), ({"Hkv": 70000}, UNS),
    ({"n": 0, "kc": None}, fa.FA_OK),
    ({"vc": X[0]}, INV), ({"vc": X[0] + 2 * 8 * 16 * 64}, INV), ({"src": X[0] + 16}, INV),
    ({"dst": X[1] + 8}, INV), ({"rows": X[0] - 8}, INV),
])
def test_copy_rejects(kw, code):
    assert _call("fa_paged_copy", COPY, kw) == code


SHARED = dict(q=X[0], k=X[1], v=X[2], ps=8 * 16 * 64, table=X[3], stride=16, M=16, cl=X[4], start=X[8],
              len=X[9], groups=2, o=X[5], lse=X[6], B=4, Hq=16, Hkv=8, P=16, page=16, d=64, scale=0.125,
              ws=X[7], wsb=1 << 30)


@pytest.mark.parametrize("kw,code", [
    ({"q": None}, INV), ({"k": A + 8}, INV), ({"v": None}, INV), ({"o": X[5] + 2}, INV),
    ({"lse": X[6] + 2}, INV), ({"cl": None}, INV), ({"table": X[3] + 2}, INV), ({"ws": None}, INV),
    ({"ws": X[7] + 8}, INV), ({"wsb": 4096}, INV), ({"start": None}, INV), ({"start": X[8] + 1}, INV),
    ({"len": None}, INV), ({"len": X[9] + 2}, INV), ({"groups": 0}, INV), ({"groups": 5}, INV),
    ({"groups": -1}, INV), ({"B": 0, "groups": 0}, INV), ({"Hq": 12}, INV), ({"Hq": 8 * 17}, UNS),
    ({"d": 96}, UNS), ({"page": 24}, UNS), ({"P": 0}, INV), ({"stride": 3}, INV),
    ({"ps": 8 * 16 * 64 - 8}, INV), ({"scale": 0.0}, INV), ({"scale": float("nan")}, INV),
    ({"B": 8192, "Hq": 8}, UNS),
    ({"B": 4096, "M": 1 << 17, "stride": 1 << 17, "Hq": 8, "Hkv": 8}, UNS),
    ({"o": X[0]}, INV), ({"o": X[1] + 64}, INV), ({"lse": X[4]}, INV), ({"lse": X[5] + 16}, INV),
    ({"ws": X[3] + 112}, INV), ({"ws": X[8] - 16}, INV), ({"lse": X[9] + 4}, INV), ({"o": X[8]}, INV),
])
def test_shared_rejects(kw, code):
    assert _call("fa_decode_shared", SHARED, kw) == code


def test_shared_workspace_bytes():
    assert fa.fa_decode_shared_workspace_bytes(4, 16, 8, 64) > 0
    assert fa.fa_decode_shared_workspace_bytes(4, 16, 8, 96) == 0
    assert fa.fa_decode_shared_workspace_bytes(4, 12, 8, 64) == 0
    assert fa.fa_decode_shared_workspace_bytes(0, 16, 8, 64) == 0
    # rows grow it by at most three results each
    a, b = (fa.fa_decode_shared_workspace_bytes(n, 16, 8, 64) for n in (4, 104))
    assert 0 < b - a <= 100 * (16 * 3 * 68 * 4 + 20) + 512


# ------------------------------------------------------------------ the binding's own checks

def _plan(rot=64):
    return fa.rope_table(rot, device="cpu")


def test_rope_binding_checks():
    x, pos = _z(2, 3, 5, 64), _z(1, 2, 5, dtype=I32)
    good = dict(x=x, y=_z(2, 3, 5, 64), pos=pos, table=_plan())

    def bad(err, **kw):
        with pytest.raises(err):
            fa.fa_rope(**{**good, **kw})
    bad(ValueError, x=_z(2, 3, 64))
    bad(TypeError, x=x.half())
    bad(ValueError, y=_z(2, 3, 5, 128))
    bad(ValueError, y=_z(2, 3, 5, 64, dtype=torch.float32))
    bad(ValueError, x=_z(2, 3, 5, 128)[..., ::2])
    bad(ValueError, y=_z(2, 3, 64, 5).transpose(2, 3))
    bad(TypeError, pos=pos.long())
    bad(ValueError, pos=_z(2, 5, dtype=I32))
    bad(ValueError, pos=_z(1, 2, 6, dtype=I32))
    bad(ValueError, pos=_z(1, 2, 10, dtype=I32)[..., ::2])
    bad(TypeError, table=(_plan()[0].int(), _plan()[1]))
    bad(ValueError, table=(_plan()[0], _plan(32)[1]))
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.fa_rope(**good)
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.rope(x, pos, _plan())


def test_rope_append_binding_checks():
    good = dict(q=_z(5, 4, 64), k=_z(5, 2, 64), v=_z(5, 2, 64), pos=_z(1, 5, dtype=I32), table=_plan(),
                q_out=_z(5, 4, 64), k_cache=_z(3, 2, 16, 64), v_cache=_z(3, 2, 16, 64),
                slots=_z(5, dtype=I32))

    def bad(err, **kw):
        with pytest.raises(err):
            fa.fa_rope_append(**{**good, **kw})
    bad(ValueError, q=_z(4, 4, 64))
    bad(ValueError, v=_z(5, 1, 64))
    bad(TypeError, v=_z(5, 2, 64, dtype=torch.float32))
    bad(ValueError, q_out=_z(5, 3, 64))
    bad(ValueError, v_cache=_z(6, 2, 16, 64)[::2])
    bad(ValueError, pos=_z(5, dtype=I32))
    bad(TypeError, pos=_z(1, 5))
    bad(TypeError, slots=_z(5, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.fa_rope_append(**good)


def test_pages_binding_checks():
    i = lambda *s: _z(*s, dtype=I32)                                      # noqa: E731
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.paged_fork(i(4), i(4, 3), i(2), i(2), i(2), 16, 8)
    with pytest.raises(ValueError):
        fa.paged_fork(i(4), i(4, 3), i(2), i(2), i(3), 16, 8)
    with pytest.raises(TypeError):
        fa.paged_fork(i(4).long(), i(4, 3), i(2), i(2), i(2), 16, 8)
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.paged_free(i(4), i(4, 3), i(1), 16, 8)
    with pytest.raises(ValueError):
        fa.fa_paged_free(i(4), i(4, 3), i(1), i(7), i(8), i(1), 16, 8)
    with pytest.raises(ValueError):
        fa.paged_free(i(4), i(3, 3), i(1), 16, 8)
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.paged_compact(i(4), i(4, 3), 16, 8)
    with pytest.raises(ValueError):
        fa.fa_paged_compact(i(4), i(4, 3), i(8), i(4), i(5), i(1), 16, 8)
    k, v = _z(4, 2, 16, 64), _z(4, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.paged_copy(k, v, i(2), i(2))
    with pytest.raises(ValueError):
        fa.paged_copy(k, _z(8, 2, 16, 64)[::2], i(2), i(2))
    with pytest.raises(ValueError):
        fa.paged_copy(k[0, 0], None, i(2), i(2))
    with pytest.raises(ValueError):
        fa.paged_copy(_z(4, 16, 500), None, i(2), i(2))
    with pytest.raises(ValueError):
        fa.paged_copy(k, v, i(2), i(2), i(3))


def test_shared_binding_checks():
    q, pool = _z(3, 4, 64), _z(5, 2, 16, 64)
    good = dict(q=q, k=pool, v=pool, block_table=_z(3, 4, dtype=I32), cache_len=_z(3, dtype=I32),
                group_start=_z(3, dtype=I32), shared_len=_z(2, dtype=I32), o=_z(3, 4, 64),
                lse=_z(3, 4, dtype=torch.float32), workspace=_z(64, dtype=torch.uint8))

    def bad(err, **kw):
        with pytest.raises(err):
            fa.fa_decode_shared(**{**good, **kw})
    bad(TypeError, q=q.float())
    bad(ValueError, group_start=_z(2, dtype=I32))
    bad(TypeError, group_start=_z(3, dtype=torch.int64))
    bad(TypeError, shared_len=_z(2, dtype=torch.int64))
    bad(ValueError, cache_len=_z(2, dtype=I32))
    bad(ValueError, v=_z(10, 2, 16, 64)[::2])
    bad(ValueError, workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 26))
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.fa_decode_shared(**good)
