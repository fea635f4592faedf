"""The bf16 forward where none of a CTA's 256 query rows sees a key, again and again over many more
CTAs than run at once: such rows are zero (their queries are being loaded into the memory that O is
staged in), every other row is what it was, and every element of the outputs is written."""
import pytest
import torch

from exact_io_aware_28_gb300 import fa

pytestmark = pytest.mark.gpu

B, H, N = 48, 16, 600     # three CTAs a head, the last with one tile
RUNS = 40


def _run(x, drop, kw):
    q, k, v = x
    o = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    if drop:
        fa.fa_fwd_dropout(q, k, v, o, lse, drop, seed=5, **kw)
    else:
        fa.fa_fwd(q, k, v, o, lse, **kw)
    return o, lse


@pytest.mark.parametrize("drop", [0, 26])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("mask", ["length", "blocks", "tail"])
def test_rows_of_ctas_without_keys_are_zero_every_time(mask, causal, d, drop):
    g = torch.Generator(device="cuda").manual_seed(d + drop)
    x = [torch.randn(B, H, N, d, generator=g, device="cuda").bfloat16() for _ in range(3)]
    dead = torch.zeros(B, N, dtype=torch.bool, device="cuda")
    kw = {"causal": causal}
    if mask == "length":
        kw["kv_len"] = torch.tensor([0, N], dtype=torch.int32, device="cuda").repeat(B // 2)
        dead[::2] = True
    else:
        bm = torch.ones(5, 5, dtype=torch.uint8, device="cuda")
        rows = slice(1, 4) if mask == "blocks" else slice(4, 5)     # rows of 128; 256 and more: a CTA's
        bm[rows] = 0
        kw["blockmask"] = bm
        dead[:, 128 * rows.start:128 * rows.stop] = True
    dead = dead[:, None].expand(B, H, N)
    first = _run(x, drop, kw)
    torch.cuda.synchronize()
    assert fa.fa_device_error() == fa.FA_OK
    assert torch.isfinite(first[0].float()).all() and torch.isfinite(first[1][~dead]).all()
    if not drop:
        assert (first[0][~dead] != 0).any(-1).all()
    for _ in range(RUNS):
        o, lse = _run(x, drop, kw)
        assert (o[dead] == 0).all(), "rows that see no key are not zero"
        assert torch.isneginf(lse[dead]).all()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    assert fa.fa_device_error() == fa.FA_OK
