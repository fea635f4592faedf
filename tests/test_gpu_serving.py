"""The paged-cache and latent operators as a program uses them: tables, appends and decode step
after step, captured in a CUDA graph, on streams of their own; the expanded and absorbed forms of
latent attention on the same weights; a training step captured and replayed."""
import numpy as np
import pytest
import torch

from exact_io_aware_28_gb300 import fa
from oracle import latent, paged

from _latent_bound import G, U, check_grads, check_lse, check_o
from test_gpu_paged import _gen, _i32, _np, _ok

pytestmark = pytest.mark.gpu
I32 = torch.int32
BF = torch.bfloat16


class Server:
    """A pool, a block table and the requests' lengths, kept on the GPU."""

    def __init__(self, B, M, page, P, Hkv, d, seed):
        g = _gen(seed)
        self.B, self.page, self.P = B, page, P
        self.k = torch.full((P, Hkv, page, d), float("nan"), dtype=BF, device="cuda")
        self.v = torch.full_like(self.k, float("nan"))
        self.table = torch.full((B, M), -1, dtype=I32, device="cuda")
        self.lens = torch.zeros(B, dtype=I32, device="cuda")
        self.free = torch.randperm(P, generator=g).int().cuda()
        self.ws = fa.alloc_decode_paged_workspace(B, 2 * Hkv, Hkv, d)

    def step(self, new_len, k, v, q):
        total, _, slots, taken = fa.paged_tables(self.lens, new_len, self.free, self.table,
                                                 self.page, self.P, k.shape[0])
        fa.paged_append(k, v, self.k, self.v, slots)
        o, lse = fa.decode_paged(q, self.k, self.v, self.table, total, workspace=self.ws)
        self.lens.copy_(total)
        return o, lse, taken

    def check(self, q, o, lse, scale):
        ro, rlse, spread = paged.decode(_np(q), _np(self.k), _np(self.v), self.table.cpu().numpy(),
                                        self.lens.tolist(), scale)
        check_o(_np(o), ro, spread)
        check_lse(_np(lse), rlse)


def test_prompts_then_tokens():
    B, Hkv, d, page = 4, 2, 64, 16
    s = Server(B, 8, page, 40, Hkv, d, seed=1)
    g = _gen(2)
    held = [([], []) for _ in range(B)]
    news = [[37, 0, 16, 1]] + [[1, 1, 1, 0]] * 3 + [[0, 20, 1, 15]] + [[1, 1, 1, 1]] * 2
    for new in news:
        T = sum(new) + 2                                     # two rows of padding
        k, v = (torch.randn(T, Hkv, d, generator=g).bfloat16() for _ in range(2))
        q = torch.randn(B, 2 * Hkv, d, generator=g).bfloat16().cuda()
        o, lse, taken = s.step(_i32(new), k.cuda(), v.cuda(), q)
        _ok()
        s.free = s.free[taken.item():].contiguous()
        at = 0
        for b, n in enumerate(new):
            held[b][0].append(k[at:at + n])
            held[b][1].append(v[at:at + n])
            at += n
        s.check(q, o, lse, 0.125)
        # and against the rows themselves, not the pool
        for b in range(B):
            kk, vv = (torch.cat(x).transpose(0, 1)[None] for x in held[b])
            assert s.lens[b].item() == kk.shape[2]
            if kk.shape[2]:
                pool = [np.pad(_np(x), ((0, 0), (0, 0), (0, 256 - x.shape[2]), (0, 0)))
                        for x in (kk, vv)]
                ro, rl, sp = paged.decode(_np(q[b:b + 1]), *pool, np.array([[0]]), [kk.shape[2]],
                                          0.125)
                check_o(_np(o[b:b + 1]), ro, sp)
                check_lse(_np(lse[b:b + 1]), rl)


def test_a_captured_step_replayed_on_new_inputs():
    B, Hkv, d, page = 3, 2, 128, 16
    s = Server(B, 6, page, 30, Hkv, d, seed=3)
    g = _gen(4)
    k, v = (torch.randn(40, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(B, 2 * Hkv, d, generator=g).bfloat16().cuda()
    s.step(_i32([20, 0, 15]), k[:35], v[:35], q)             # a prompt, before the capture
    s.free = s.free[3:].contiguous()
    new, kn, vn, qn = _i32([0] * B), k[:4].clone(), v[:4].clone(), q.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step(new, kn, vn, qn)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse, taken = s.step(new, kn, vn, qn)
    for i in range(4):                                       # padded batches: row 3 has no token
        new.copy_(_i32([1, i % 2, 1]))
        for t in (kn, vn, qn):
            t.copy_(torch.randn(t.shape, generator=g).bfloat16())
        graph.replay()
        _ok()
        n = taken.item()
        s.free[:s.free.numel() - n] = s.free[n:].clone()
        s.check(qn, o, lse, d ** -0.5)


def test_two_streams_with_a_workspace_each():
    g = _gen(5)
    cases = []
    for H in (4, 20):
        cache = torch.randn(20, 32, 576, generator=g).bfloat16().cuda()
        q = torch.randn(2, H, 576, generator=g).bfloat16().cuda()
        cases.append((q, cache, torch.arange(20, dtype=I32, device="cuda").view(2, 10),
                      _i32([300, 111])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[] for _ in cases]
    for _ in range(5):
        for i, x in enumerate(cases):
            # once with a stream object, once with its handle
            outs[i].append(fa.latent_decode(*x, stream=streams[i]))
            outs[i].append(fa.latent_decode(*x, stream=streams[i].cuda_stream))
    _ok()
    for x, got in zip(cases, outs):
        ro, rlse, sp = latent.decode(*(_np(t) for t in x[:2]), x[2].cpu().numpy(), x[3].tolist(),
                                     192 ** -0.5, 512)
        for o, lse in got:
            check_o(_np(o), ro, sp)
            check_lse(_np(lse), rlse)


def test_inputs_of_another_stream_may_be_dropped():
    # the default stream by its handle; the helper keeps its inputs' memory until the named stream's work is done
    side = torch.cuda.Stream()
    g = _gen(6)
    base = torch.randn(1, 4, 700, 192, generator=g).bfloat16().cuda()
    ref = None
    for _ in range(3):
        x = [t.clone() for t in (base, base[..., :128], base[:, 0, :, :64], base[..., 64:])]
        x = [t.contiguous() for t in x]
        side.wait_stream(torch.cuda.current_stream())
        o, lse = fa.latent_forward(*x, True, stream=side)
        del x
        for _ in range(4):       # would take the freed memory over
            torch.full((1, 4, 700, 192), 7.0, dtype=BF, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
        ref = (o, lse) if ref is None else ref
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    x = [t.contiguous() for t in (base, base[..., :128], base[:, 0, :, :64], base[..., 64:])]
    o, lse = fa.latent_forward(*x, True, stream=0)
    _ok()
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_expanded_and_absorbed_forms_agree():
    # Projections that select columns of the latent vector are exact in bf16, so both forms are
    # the same function of the same numbers: a prompt in the expanded form, its rows into the
    # latent cache, and the last token once more in the absorbed form.
    H, N, page = 6, 150, 32
    g = _gen(7)
    c, r = torch.randn(N, 512, generator=g).bfloat16(), torch.randn(N, 64, generator=g).bfloat16()
    pick_k = torch.stack([torch.randperm(512, generator=g)[:128] for _ in range(H)])
    pick_v = torch.stack([torch.randperm(512, generator=g)[:128] for _ in range(H)])
    q = torch.randn(1, H, N, 192, generator=g).bfloat16()
    kn = torch.stack([c[:, i] for i in pick_k])[None].contiguous()
    v = torch.stack([c[:, i] for i in pick_v])[None].contiguous()
    o, lse = fa.latent_forward(q.cuda(), kn.cuda(), r[None].cuda(), v.cuda(), True)
    qa = torch.zeros(1, H, 576)
    for h in range(H):
        qa[0, h, pick_k[h]] = q[0, h, -1, :128].float()
        qa[0, h, 512:] = q[0, h, -1, 128:].float()
    P = 7
    cache = torch.zeros(P, page, 576, dtype=BF, device="cuda")
    table = torch.full((1, 5), -1, dtype=I32, device="cuda")
    total, _, slots, _ = fa.paged_tables(_i32([0]), _i32([N]), _i32([6, 1, 4, 0, 3]), table, page,
                                         P, N)
    fa.latent_append(c.cuda(), r.cuda(), cache, slots)
    oa, lsea = fa.latent_decode(qa.bfloat16().cuda(), cache, table, total)
    _ok()
    ref, rlse, sp = latent.forward(*(_np(t) for t in (q, kn, r[None], v)), 192 ** -0.5, True)
    got = np.stack([_np(oa)[0, h, pick_v[h].numpy()] for h in range(H)])
    for x, l in ((_np(o)[0, :, -1], _np(lse)[0, :, -1]), (got, _np(lsea)[0])):
        check_o(x, ref[0, :, -1], sp[0, :, -1])
        check_lse(l, rlse[0, :, -1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_captured_training_step_replayed_on_new_inputs(dtype):
    B, H, N = 2, 2, 200
    name = "bf16" if dtype == BF else "fp32"
    g = _gen(8)
    shapes = (B, H, N, 192), (B, H, N, 128), (B, N, 64), (B, H, N, 128), (B, H, N, 128)
    x = [torch.randn(*s, generator=g).to(dtype).cuda() for s in shapes]
    kv = _i32([200, 131])
    ws = fa.alloc_latent_workspace(B, H, N)

    def step():
        o, lse, acc = fa.latent_forward(*x[:4], True, kv, need_grad=True)
        return (o, lse) + fa.latent_backward(*x[:4], acc, lse, x[4], True, kv, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        for t in x:
            t.copy_(torch.randn(t.shape, generator=g).to(dtype))
        kv.copy_(_i32([77, 200]))
        graph.replay()
        _ok()
        host = [_np(t) for t in x]
        ro, rlse, sp = latent.forward(*host[:4], 192 ** -0.5, True, [77, 200])
        check_o(_np(out[0]), ro, sp, name)
        check_lse(_np(out[1]), rlse, name)
        ref, err = latent.backward(*host, 192 ** -0.5, True, [77, 200],
                                   U[name] if name == "bf16" else 0.0, G[name])
        check_grads([_np(t) for t in out[2:]], ref, err, name)


def test_gradients_against_differences():
    # fp32: the derivative along a random direction against (L(x + e t) - L(x - e t)) / 2e.  The
    # difference of two losses of size |L| is good to about 2 gamma |L| / 2e, gamma the fp32 error
    # of the outputs' sum (G), and e^2 of the third derivative on top; e = 2^-5 balances the two
    # for these sizes, so 1% of the terms' absolute sum is allowed.
    B, H, N = 1, 2, 70
    g = _gen(9)
    shapes = (B, H, N, 192), (B, H, N, 128), (B, N, 64), (B, H, N, 128)
    x = [torch.randn(*s, generator=g).cuda() for s in shapes]
    do = torch.randn(B, H, N, 128, generator=g).cuda()
    o, lse, acc = fa.latent_forward(*x, True, need_grad=True)
    grads = fa.latent_backward(*x, acc, lse, do, True)
    e = 2.0 ** -5
    for i in range(4):
        t = torch.randn(x[i].shape, generator=g).cuda()
        t /= t.double().square().mean().sqrt() * x[i].numel() ** 0.5 / 8   # a short step
        lo, hi = list(x), list(x)
        lo[i], hi[i] = x[i] - e * t, x[i] + e * t
        f = [(fa.latent_forward(*y, True)[0].double() * do.double()).sum().item()
             for y in (lo, hi)]
        along = (grads[i].double() * t.double())
        assert abs((f[1] - f[0]) / (2 * e) - along.sum().item()) <= 0.01 * along.abs().sum().item()
    _ok()


@pytest.mark.parametrize("latent_rows", [False, True])
def test_appends_on_a_named_stream_keep_their_inputs(latent_rows):
    # The named stream is held up, so the rows are read after the caller has dropped them and filled
    # new tensors of their sizes.
    T, Hkv, d, page, P = 300, 4, 64, 32, 12
    g = _gen(10)
    if latent_rows:
        rows, pools = [(T, 512), (T, 64)], [torch.zeros(P, page, 576, dtype=BF, device="cuda")]
    else:
        rows = [(T, Hkv, d)] * 2
        pools = [torch.zeros(P, Hkv, page, d, dtype=BF, device="cuda") for _ in rows]
    append = fa.latent_append if latent_rows else fa.paged_append
    side = torch.cuda.Stream()
    for _ in range(3):
        host = [torch.randn(*s, generator=g).bfloat16() for s in rows]
        slots = torch.randperm(P * page, generator=g)[:T].int()
        before = [_np(p) for p in pools]
        x = [r.cuda() for r in host]
        at = slots.cuda()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        append(*x, *pools, at, stream=side)
        del x, at
        junk = [torch.full(s, 7.0, dtype=BF, device="cuda") for s in rows]
        junk.append(torch.full((T,), -1, dtype=I32, device="cuda"))
        torch.cuda.current_stream().wait_stream(side)
        _ok()
        if latent_rows:
            host = [torch.cat(host, 1)]
        for p, b, r in zip(pools, before, host):
            assert np.array_equal(_np(p), paged.append(b, _np(r), slots.tolist()))
        # a handle will do, and no stream is the current one
        append(*(r.cuda() for r in (host if not latent_rows else host[0].split((512, 64), 1))),
               *pools, slots.cuda(), stream=side.cuda_stream)
        side.synchronize()
        _ok()
