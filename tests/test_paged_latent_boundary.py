"""Refusals of the paged-cache and latent entry points, on the host, before any launch."""
import os

import pytest
import torch

from exact_io_aware_28_gb300 import fa

pytestmark = pytest.mark.skipif(not os.path.exists(fa.LIB_PATH),
                                reason="libfa_gb300.so not built")

A = 0x100000  # a fake, aligned address: never dereferenced on the host
X = [A + (i << 40) for i in range(16)]   # more of them, far apart
INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


def _call(name, defaults, kw):
    args = dict(defaults)
    assert set(kw) <= set(args)
    args.update(kw)
    return getattr(fa.load(), name)(*args.values(), None)


TABLES = dict(cl=A, nl=A + 0x1000, free=A + 0x2000, n_free=8, table=A + 0x3000, stride=16, M=16,
              total=A + 0x4000, start=A + 0x5000, slots=A + 0x6000, n_slots=64, taken=A + 0x7000,
              B=4, page=16, P=64)


@pytest.mark.parametrize("kw,code", [
    ({"cl": None}, INV), ({"nl": A + 2}, INV), ({"table": None}, INV), ({"total": None}, INV),
    ({"start": A + 1}, INV), ({"taken": None}, INV), ({"slots": None}, INV),
    ({"free": None}, INV), ({"B": 0}, INV), ({"P": 0}, INV), ({"M": 0}, INV),
    ({"stride": 15}, INV), ({"n_slots": -1}, INV), ({"n_free": -1}, INV),
    ({"page": 8}, UNS), ({"page": 48}, UNS), ({"page": 512}, UNS), ({"page": 0}, UNS),
    ({"B": 8193}, UNS), ({"B": 8192, "M": 16385, "stride": 16385}, UNS),
    ({"P": 1 << 27}, UNS),
    ({"total": A}, INV),                    # in place over an input that other blocks still read
    ({"start": A + 0x1000 - 16}, INV), ({"slots": A + 0x2010}, INV), ({"taken": A + 12}, INV),
    ({"table": A + 0x2000 - 4 * (3 * 16 + 15)}, INV),
    ({"slots": A + 0x4008}, INV), ({"taken": A + 0x3000}, INV),   # outputs over one another
    ({"n_slots": (1 << 30) + 1, "slots": A + (1 << 33)}, UNS),
])
def test_tables_rejects(kw, code):
    assert _call("fa_paged_tables", TABLES, kw) == code


APPEND = dict(k=A, v=A, ks=512, vs=512, kc=A, vc=A, ps=8 * 16 * 64, slots=A, T=4, P=16, Hkv=8,
              page=16, d=64)


@pytest.mark.parametrize("kw,code", [
    ({"k": None}, INV), ({"v": A + 8}, INV), ({"kc": A + 4}, INV), ({"vc": None}, INV),
    ({"slots": A + 2}, INV), ({"T": -1}, INV), ({"Hkv": 0}, INV), ({"ks": 504}, INV),
    ({"vs": 516}, INV), ({"ps": 8 * 16 * 64 - 8}, INV), ({"ps": 8 * 16 * 64 + 4}, INV),
    ({"d": 96}, UNS), ({"page": 12}, UNS), ({"P": 1 << 27}, UNS), ({"P": 0}, INV),
    ({"T": 0}, fa.FA_OK),                                        # nothing to do, nothing launched
])
def test_append_rejects(kw, code):
    assert _call("fa_paged_append", APPEND, kw) == code


LAPPEND = dict(c=A, r=A, cs=512, rs=64, cache=A, ps=16 * 576, slots=A, T=4, P=16, page=16)


@pytest.mark.parametrize("kw,code", [
    ({"c": None}, INV), ({"r": A + 4}, INV), ({"cache": None}, INV), ({"slots": None}, INV),
    ({"cs": 504}, INV), ({"rs": 68}, INV), ({"ps": 16 * 576 - 8}, INV), ({"page": 20}, UNS),
    ({"T": -3}, INV), ({"T": 0}, fa.FA_OK),
])
def test_latent_append_rejects(kw, code):
    assert _call("fa_latent_append", LAPPEND, kw) == code


DECODE = dict(q=X[0], k=X[1], v=X[2], ps=8 * 16 * 64, table=X[3], stride=16, M=16, cl=X[4], o=X[5],
              lse=X[6], B=2, Hq=16, Hkv=8, P=16, page=16, d=64, scale=0.125, ws=X[7], wsb=1 << 30)


@pytest.mark.parametrize("kw,code", [
    ({"q": None}, INV), ({"k": A + 8}, INV), ({"v": None}, INV), ({"o": A + 2}, INV),
    ({"lse": A + 2}, INV), ({"cl": None}, INV), ({"table": A + 2}, INV), ({"ws": None}, INV),
    ({"ws": A + 8}, INV), ({"wsb": 64}, INV), ({"B": 0}, INV), ({"Hq": 12}, INV),
    ({"Hq": 8 * 17}, UNS), ({"d": 96}, UNS), ({"page": 24}, UNS), ({"P": 0}, INV),
    ({"stride": 3}, INV), ({"M": -1}, INV), ({"ps": 8 * 16 * 64 - 8}, INV),
    ({"scale": 0.0}, INV), ({"scale": float("nan")}, INV), ({"scale": -1.0}, INV),
    ({"B": 8192, "Hq": 8, "Hkv": 8}, UNS), ({"M": (1 << 26) + 1, "stride": 1 << 27}, UNS),
    ({"ps": 1 << 39}, UNS),
    # outputs over inputs or one another
    ({"o": X[0]}, INV), ({"o": X[1] + 64}, INV), ({"o": X[2] + 16 * 8 * 16 * 64 * 2 - 16}, INV),
    ({"lse": X[4]}, INV), ({"lse": X[5] + 16}, INV), ({"ws": X[3] + 112}, INV), ({"ws": X[6]}, INV),
])
def test_decode_paged_rejects(kw, code):
    assert _call("fa_decode_paged", DECODE, kw) == code


LDECODE = dict(q=X[0], cache=X[1], ps=16 * 576, table=X[2], stride=16, M=16, cl=X[3], o=X[4],
               lse=X[5], B=2, H=16, P=16, page=16, scale=0.07, ws=X[6], wsb=1 << 30)


@pytest.mark.parametrize("kw,code", [
    ({"q": A + 8}, INV), ({"cache": None}, INV), ({"o": None}, INV), ({"lse": None}, INV),
    ({"cl": A + 3}, INV), ({"table": None}, INV), ({"ws": None}, INV), ({"wsb": 1000}, INV),
    ({"B": 0}, INV), ({"H": 0}, INV), ({"H": 129}, UNS), ({"B": 70000}, UNS),
    ({"page": 1}, UNS), ({"ps": 100}, INV), ({"scale": float("inf")}, INV),
    # outputs over inputs or one another
    ({"o": X[0]}, INV), ({"o": X[1] + 16 * 16 * 576 * 2 - 16}, INV), ({"lse": X[3] + 4}, INV),
    ({"ws": X[0] - 16}, INV), ({"lse": X[4] + 2 * 16 * 512 * 2 - 4}, INV),
    ({"ws": X[2] + 64}, INV),
])
def test_latent_decode_rejects(kw, code):
    assert _call("fa_latent_decode", LDECODE, kw) == code


LFWD = dict(q=X[0], kn=X[1], kr=X[2], v=X[3], o=X[4], oa=None, lse=X[5], B=1, H=2, N=100, causal=1,
            kv=None, scale=0.07, dtype=fa.FA_BF16)


@pytest.mark.parametrize("kw,code", [
    ({"q": None}, INV), ({"kn": A + 8}, INV), ({"kr": None}, INV), ({"v": A + 2}, INV),
    ({"o": None}, INV), ({"oa": A + 4}, INV), ({"lse": A + 1}, INV), ({"kv": A + 2}, INV),
    ({"N": 0}, INV), ({"B": -1}, INV), ({"dtype": 3}, INV), ({"scale": 0.0}, INV),
    ({"B": 256, "H": 256}, UNS), ({"N": 1 << 25}, UNS),
    ({"o": X[3]}, INV), ({"o": X[0] + 2 * 100 * 192 * 2 - 16}, INV), ({"oa": X[4]}, INV),
    ({"lse": X[4] + 32}, INV), ({"oa": X[1]}, INV), ({"kv": X[5]}, INV),
])
def test_latent_fwd_rejects(kw, code):
    assert _call("fa_latent_fwd", LFWD, kw) == code


LBWD = dict(q=X[0], kn=X[1], kr=X[2], v=X[3], oa=X[4], lse=X[5], do=X[6], dq=X[7], dkn=X[8], dkr=X[9],
            dv=X[10], B=1, H=2, N=100, causal=1, kv=None, scale=0.07, dtype=fa.FA_BF16, ws=X[11],
            wsb=1 << 30)


@pytest.mark.parametrize("kw,code", [
    ({"oa": None}, INV), ({"do": A + 8}, INV), ({"dq": None}, INV), ({"dkn": A + 4}, INV),
    ({"dkr": None}, INV), ({"dv": None}, INV), ({"lse": None}, INV), ({"ws": None}, INV),
    ({"ws": A + 128}, INV), ({"wsb": 100 * 2 * 64 * 4}, INV), ({"N": 0}, INV),
    ({"dtype": 2}, INV), ({"scale": float("nan")}, INV), ({"H": 70000}, UNS),
    ({"dq": X[0]}, INV), ({"dv": X[6]}, INV), ({"dkn": X[1]}, INV), ({"dkr": X[2] + 16}, INV),
    ({"dv": X[8]}, INV), ({"ws": X[5]}, INV), ({"ws": X[10]}, INV), ({"dq": X[4]}, INV),
])
def test_latent_bwd_rejects(kw, code):
    assert _call("fa_latent_bwd", LBWD, kw) == code


def test_workspace_bytes():
    assert fa.fa_decode_paged_workspace_bytes(2, 16, 8, 64) > 0
    assert fa.fa_decode_paged_workspace_bytes(2, 16, 8, 96) == 0
    assert fa.fa_decode_paged_workspace_bytes(2, 12, 8, 64) == 0
    # a few results a CTA, whatever the batch is: only the prefix sums grow with it
    more = fa.fa_decode_paged_workspace_bytes(502, 16, 8, 64)
    assert more - fa.fa_decode_paged_workspace_bytes(2, 16, 8, 64) == 500 * 8
    assert fa.fa_latent_decode_workspace_bytes(4, 129) == 0
    assert fa.fa_latent_decode_workspace_bytes(4, 128) > 0
    assert fa.fa_latent_bwd_workspace_bytes(1, 2, 100) == 1024 + 200 * 64 * 4
    assert fa.fa_latent_bwd_workspace_bytes(1, 2, 0) == 0


# ------------------------------------------------------------------ the binding's own checks

def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


I32 = torch.int32


def test_binding_checks_shapes_and_types():
    q, pool = _z(2, 4, 64), _z(5, 2, 16, 64)
    table, lens = _z(2, 3, dtype=I32), _z(2, dtype=I32)
    o, lse, ws = _z(2, 4, 64), _z(2, 4, dtype=torch.float32), _z(64, dtype=torch.uint8)
    good = dict(q=q, k=pool, v=pool, block_table=table, cache_len=lens, o=o, lse=lse, workspace=ws)

    def bad(err, **kw):
        with pytest.raises(err):
            fa.fa_decode_paged(**{**good, **kw})
    bad(TypeError, q=q.float())
    bad(TypeError, block_table=table.long())
    bad(TypeError, cache_len=lens.long())
    bad(ValueError, cache_len=_z(3, dtype=I32))
    bad(ValueError, block_table=_z(3, 3, dtype=I32))
    bad(ValueError, block_table=_z(2, 6, dtype=I32)[:, ::2])
    bad(ValueError, v=_z(5, 2, 32, 64))
    bad(ValueError, k=_z(5, 16, 2, 64).transpose(1, 2), v=_z(5, 16, 2, 64).transpose(1, 2))
    bad(ValueError, k=_z(10, 2, 16, 64)[::2])          # another page stride than v's
    bad(ValueError, o=_z(2, 4, 128))
    bad(ValueError, q=_z(4, 2, 64).transpose(0, 1))
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.fa_decode_paged(**good)


def test_binding_refuses_host_tensors_and_wrong_latents():
    c, r, cache, slots = _z(3, 512), _z(3, 64), _z(4, 16, 576), _z(3, dtype=I32)
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.latent_append(c, r, cache, slots)
    with pytest.raises(ValueError):
        fa.latent_append(_z(3, 500), r, cache, slots)
    with pytest.raises(TypeError):
        fa.latent_append(c, r, cache, slots.long())
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.paged_append(_z(3, 2, 64), _z(3, 2, 64), _z(4, 2, 16, 64), _z(4, 2, 16, 64), slots)
    with pytest.raises(ValueError):
        fa.paged_append(_z(3, 2, 64), _z(3, 1, 64), _z(4, 2, 16, 64), _z(4, 2, 16, 64), slots)
    x = _z(1, 2, 8, 192), _z(1, 2, 8, 128), _z(1, 8, 64), _z(1, 2, 8, 128)
    lse = _z(1, 2, 8, dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA tensors"):
        fa.fa_latent_fwd(*x, _z(1, 2, 8, 128), None, lse)
    with pytest.raises(ValueError):
        fa.fa_latent_fwd(x[0], x[1], _z(1, 2, 8, 64), x[3], _z(1, 2, 8, 128), None, lse)
    with pytest.raises(TypeError):
        fa.fa_latent_fwd(x[0], x[1].float(), x[2], x[3], _z(1, 2, 8, 128), None, lse)
    with pytest.raises(ValueError):
        fa.fa_latent_decode(_z(2, 4, 512), cache, _z(2, 3, dtype=I32), _z(2, dtype=I32),
                            _z(2, 4, 512), _z(2, 4, dtype=torch.float32), _z(8))


def test_binding_refuses_workspaces_that_repeat_their_bytes():
    # an expanded tensor counts bytes that it does not have
    ws = torch.zeros(1, dtype=torch.uint8).expand(1 << 24)
    table, lens = _z(2, 3, dtype=I32), _z(2, dtype=I32)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        fa.fa_decode_paged(_z(2, 4, 64), _z(5, 2, 16, 64), _z(5, 2, 16, 64), table, lens,
                           _z(2, 4, 64), _z(2, 4, dtype=torch.float32), ws)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        fa.fa_latent_decode(_z(2, 4, 576), _z(4, 16, 576), table, lens, _z(2, 4, 512),
                            _z(2, 4, dtype=torch.float32), ws)
    x = _z(1, 2, 8, 192), _z(1, 2, 8, 128), _z(1, 8, 64), _z(1, 2, 8, 128)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        fa.fa_latent_bwd(*x, _z(1, 2, 8, 128, dtype=torch.float32),
                         _z(1, 2, 8, dtype=torch.float32), x[3], *x, ws)
    # strides that leave room, or another order of the dimensions, do no harm
    for ws in (torch.zeros(1 << 14, dtype=torch.uint8)[::2], _z(64, 8).t(), _z(4, 8)[:, :0],
               torch.zeros(200, dtype=torch.uint8).as_strided((2, 4), (100, 0))):
        with pytest.raises(ValueError, match="CUDA tensors"):
            fa.fa_latent_bwd(*x, _z(1, 2, 8, 128, dtype=torch.float32),
                             _z(1, 2, 8, dtype=torch.float32), x[3], *x, ws)


PAGE = 8 * 16 * 64                          # elements of a page of APPEND's pools


@pytest.mark.parametrize("kw,code", [
    ({"vc": X[0]}, INV),                                          # one pool for both
    ({"vc": X[0] + 2 * (PAGE - 8)}, INV),                         # the last piece of a page
    ({"vc": X[0] + 2 * PAGE}, INV),                               # the pool a page on
    ({"kc": X[0] + 2 * 5 * PAGE, "vc": X[0]}, INV),
    ({"vc": X[0] + 2 * (15 * PAGE + 8)}, INV),                    # its last page
    ({"ps": 2 * PAGE, "vc": X[0] + 2 * (PAGE - 8)}, INV),         # side by side, but too close
    ({"ps": 2 * PAGE, "vc": X[0] + 2 * (31 * PAGE - 8)}, INV),
    ({"ps": 2 * PAGE, "kc": X[0] + 2 * (PAGE + 8), "vc": X[0]}, INV),   # over the next page
    ({"T": 0, "vc": X[0]}, fa.FA_OK),                             # no rows, nothing to disturb
    # and the other refusals with pools apart
    ({"k": None}, INV), ({"v": X[2] + 8}, INV), ({"kc": X[0] + 4}, INV), ({"vc": None}, INV),
    ({"slots": X[4] + 2}, INV), ({"ks": 504}, INV), ({"vs": 516}, INV), ({"ps": PAGE + 4}, INV),
])
def test_append_refuses_pools_that_share_memory(kw, code):
    base = dict(APPEND, k=X[1], v=X[2], kc=X[0], vc=X[3], slots=X[4])
    assert _call("fa_paged_append", base, kw) == code
