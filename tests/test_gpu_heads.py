"""Norm and rotation of heads, and the append to pages, against float64."""
import pytest
import torch

from tests import paged_reference as R
from verified_kv_cache_poissoncomp_gb300 import binding as B
from verified_kv_cache_poissoncomp_gb300 import inputs as I
from verified_kv_cache_poissoncomp_gb300.paged import PagedKV, Rope

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def freqs(rd, base=1e4):
    return torch.tensor([base ** (-2 * j / rd) for j in range(rd // 2)], dtype=torch.float64)


def check(got, x, pos, f, il, w, eps, what):
    y, tol = R.norm_rotate(x, pos, f, il, w, eps)
    R.close(got, y, tol, what)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("h,g,d,rd,il,norm,tokens", [
    (8, 4, 128, 128, False, True, 1), (8, 4, 128, 128, False, True, 257), (8, 4, 128, 64, True, False, 33),
    (2, 8, 64, 64, False, True, 5), (2, 8, 64, 32, True, True, 1000), (1, 1, 64, 16, False, False, 3),
    (1, 2, 128, 112, False, True, 7), (4, 1, 128, 16, True, True, 700), (1, 1, 64, 0, False, True, 2),
    (3, 2, 64, 48, False, True, 1333)])
def test_norm_rotate(dtype, h, g, d, rd, il, norm, tokens):
    qkv = randn((tokens, h * g + 2 * h, d), dtype, 1, 3.0)
    q, k = qkv[:, :h * g], qkv[:, h * g:h * g + h]
    pos = ((torch.arange(tokens, device="cuda") * 7919) % 131072).to(torch.int32)
    wq, wk = (randn((d,), dtype, 2), randn((d,), dtype, 3)) if norm else (None, None)
    c = PagedKV(h, g, d, dtype=dtype)
    f = freqs(rd) if rd else None
    rope = Rope(f, il) if rd else None
    qo, ko = c.norm_rotate(q, k, pos, rope, wq, wk, 1e-6)
    check(qo, q, pos, f, il, wq, 1e-6, "q")
    check(ko, k, pos, f, il, wk, 1e-6, "k")
    # one without the other, one normalised without the other
    q2, none = c.norm_rotate(q, None, pos, rope, wq)
    assert none is None and torch.equal(q2, qo)
    none, k2 = c.norm_rotate(None, k, pos, rope, None, wk)
    assert none is None and torch.equal(k2, ko)
    if norm:
        q3, k3 = c.norm_rotate(q, k, pos, rope, None, wk)
        check(q3, q, pos, f, il, None, 1e-6, "q as long as it is")
        assert torch.equal(k3, ko)
    # in place
    buf = qkv.clone()
    a, b = buf[:, :h * g], buf[:, h * g:h * g + h]
    c.norm_rotate(a, b, pos, rope, wq, wk, 1e-6, q_out=a, k_out=b)
    assert torch.equal(a, qo) and torch.equal(b, ko) and torch.equal(buf[:, h * g + h:], qkv[:, h * g + h:])
    c.sync()


@pytest.mark.parametrize("base", [1e4, 1e6])
def test_angles_of_far_and_negative_positions(base):
    pos = torch.tensor([0, 1, 4095, 131071, 1 << 20, (1 << 31) - 1, -1, -131072], dtype=torch.int32, device="cuda")
    x = randn((len(pos), 1, 128), torch.float16, 4)
    f = freqs(128, base)
    c = PagedKV(1, 1, 128, dtype=HF)
    y, _ = c.norm_rotate(x, None, pos, Rope(f))
    check(y, x, pos, f, False, None, 0, "far positions")


def test_small_heads_with_eps_and_zero_rows():
    x = randn((6, 1, 64), BF, 5, 1e-3)
    x[2] = 0
    w = randn((64,), BF, 6)
    c = PagedKV(1, 1, 64)
    for eps in (0.0, 1e-6, 1e-2):
        y, _ = c.norm_rotate(x, None, q_weight=w, eps=eps)
        keep = [0, 1, 3, 4, 5] if eps == 0 else list(range(6))  # 0 / 0 is not a number
        check(y[keep], x[keep], torch.zeros(len(keep), dtype=torch.int32), None, False, w, eps, f"eps {eps}")
        if eps:
            assert not y[2].any()


def test_keys_go_into_the_full_cache_layout():
    # k_out is the key half of [kv_heads][n][2][d]: the layout PoissonComp and the sketch read
    h, n, d = 2, 77, 128
    k, kv = randn((n, h, d), BF, 7), torch.full((h, n, 2, d), 9.0, dtype=BF, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    c, f = PagedKV(h, 4, d), freqs(128)
    c.norm_rotate(None, k, pos, Rope(f), k_out=kv[:, :, 0].transpose(0, 1))
    check(kv[:, :, 0].transpose(0, 1), k, pos, f, False, None, 0, "k half")
    assert bool((kv[:, :, 1] == 9).all())


@pytest.mark.parametrize("dtype,h,g,d,pt,tokens,with_q", [
    (BF, 8, 4, 128, 16, 8, True), (HF, 2, 8, 64, 32, 777, True), (BF, 8, 4, 128, 64, 300, False),
    (HF, 1, 1, 64, 256, 1, False), (BF, 4, 2, 128, 128, 1500, True)])
def test_append(dtype, h, g, d, pt, tokens, with_q):
    seqs, per = 5, max(2, -(-tokens // pt) + 1)
    kv = torch.full((2, seqs * per + 3, h, pt, 2, d), 7.0, dtype=dtype, device="cuda")
    before = kv.clone()
    table = torch.randperm(seqs * per + 3, device="cuda")[:seqs * per].to(torch.int32).view(seqs, per)
    qkv = randn((tokens, h * g + 2 * h, d), dtype, 8)
    q, k, v = qkv[:, :h * g], qkv[:, h * g:h * g + h], qkv[:, h * g + h:]
    seq = (torch.arange(tokens, device="cuda") % seqs).to(torch.int32)
    index = (torch.arange(tokens, device="cuda") // seqs + pt - 1).to(torch.int32)  # from a page's last slot on
    pad = torch.arange(tokens, device="cuda") % 7 == 3
    seq = torch.where(pad, -1, seq).to(torch.int32)
    pos = index + 1000
    wq, wk, f = randn((d,), dtype, 9), randn((d,), dtype, 10), freqs(d)
    c = PagedKV(h, g, d, kv=kv)
    qo = c.append(1, k, v, seq, index, table, pos, Rope(f), wk, 1e-5, q if with_q else None, wq)
    c.sync()
    if with_q:
        check(qo, q, pos, f, False, wq, 1e-5, "q")
    else:
        assert qo is None
    real = ~pad
    page, slot = table[seq[real].long(), (index[real] // pt).long()].long(), (index[real] % pt).long()
    check(kv[1, page, :, slot, 0], k[real], pos[real], f, False, wk, 1e-5, "k")
    assert torch.equal(kv[1, page, :, slot, 1], v[real])
    kv[1, page, :, slot] = 7.0
    assert torch.equal(kv, before)  # nothing else was written


def test_append_reports_bad_places_and_skips_them():
    h, d, pt = 2, 64, 16
    kv = torch.zeros((1, 4, h, pt, 2, d), dtype=BF, device="cuda")
    c = PagedKV(h, 1, d, kv=kv)
    k = torch.ones((1, h, d), dtype=BF, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = ints(0, 1, 2, 9).view(2, 2)
    for s, i, tab in [(2, 0, table), (-2, 0, table), (0, 32, table), (0, -1, table), (1, 16, table),
                      (1, 16, ints(0, 1, 2, -5).view(2, 2))]:
        c.append(0, k, k, ints(s), ints(i), tab)
        with pytest.raises(B.VerkvError) as e:
            c.sync()
        assert e.value.status == B.VERKV_EINVAL, (s, i)
        assert not kv.any()
    c.append(0, k, k, ints(-1), ints(-77), table)  # padding: its place is not looked at
    c.append(0, k, k, ints(1), ints(15), table)
    c.sync()
    assert bool((kv[0, 2, :, 15] == 1).all()) and int(kv.count_nonzero()) == h * 2 * d


def test_refusals():
    c = PagedKV(2, 2, 64, num_pages=2, page_tokens=16)
    q, k = randn((3, 4, 64), BF, 1), randn((3, 2, 64), BF, 2)
    pos, rope = torch.zeros(3, dtype=torch.int32, device="cuda"), Rope(freqs(64))
    n0 = B.verkv_launch_counts(c.ctx)
    bad = [lambda: c.norm_rotate(None, None), lambda: c.norm_rotate(q, k, None, rope), lambda: c.norm_rotate(q.half(), k),
           lambda: c.norm_rotate(q, k[:2]), lambda: c.norm_rotate(q.cpu(), None), lambda: c.norm_rotate(k, None),
           lambda: c.norm_rotate(q, k, pos.long(), rope), lambda: c.norm_rotate(q, k, pos[:2], rope),
           lambda: c.norm_rotate(q, None, k_out=k), lambda: c.norm_rotate(q, None, q_weight=q[0, 0, :32]),
           lambda: c.norm_rotate(q.transpose(1, 2).contiguous().transpose(1, 2), None),
           lambda: c.append(0, k, k, pos, pos, pos), lambda: c.append(1, k, k, pos, pos, pos.view(3, 1)),
           lambda: c.append(0, k, k[:1], pos, pos, pos.view(3, 1)), lambda: PagedKV(2, 2, 64).append(0, k, k, pos, pos, pos.view(3, 1)),
           lambda: PagedKV(2, 2, 64, dtype=torch.float32)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    # refused by the library: rows off 16 bytes, strides, weights, types, a rotation wider than a head
    flat = randn((1024,), BF, 3)
    rows = lambda t, a, b: B.verkv_rows(t.data_ptr(), a, b)  # noqa: E731
    L = B.lib()
    ok, out = rows(flat, 256, 64), rows(torch.empty_like(flat), 256, 64)
    rot = lambda q=ok, o=out, dt=B.VERKV_BF16, n=3, norm=None, rp=None, ps=pos.data_ptr(): (  # noqa: E731
        L.verkv_norm_rotate(c.ctx, dt, n, q, o, None, None, norm, rp, ps))
    assert rot(q=rows(flat[1:], 256, 64)) == B.VERKV_EINVAL
    assert rot(q=rows(flat, 257, 64)) == rot(q=rows(flat, 256, -64)) == B.VERKV_EINVAL
    assert rot(o=rows(flat, 64, 64)) == rot(o=rows(flat, 256, 32)) == rot(o=rows(flat, 256, 0)) == B.VERKV_EINVAL
    assert rot(o=None) == rot(dt=2) == rot(n=-1) == B.VERKV_EINVAL
    assert rot(norm=B.verkv_head_norm(flat.data_ptr() + 2, None, 1e-6)) == B.VERKV_EINVAL
    assert rot(norm=B.verkv_head_norm(None, None, -1.0)) == rot(norm=B.verkv_head_norm(None, None, float("nan"))) == B.VERKV_EINVAL
    t = rope.turns.data_ptr()
    for rp in (B.verkv_rope(80, 0, t), B.verkv_rope(24, 0, t), B.verkv_rope(-16, 0, t), B.verkv_rope(64, 0, None),
               B.verkv_rope(64, 0, t + 4)):
        assert rot(rp=rp) == B.VERKV_EINVAL
    assert rot(rp=B.verkv_rope(64, 0, t), ps=None) == B.VERKV_EINVAL
    span = B.verkv_span(pos.data_ptr(), 1, 3, None, 0)
    app = lambda pt=16, n=2, kv=None, sp=span: L.verkv_paged_append(  # noqa: E731
        c.ctx, B.verkv_pages(B.VERKV_BF16, pt, n, kv if kv is not None else c.kv.data_ptr()), 1, ok, ok, None, None, None, None, None,
        pos.data_ptr(), pos.data_ptr(), sp)
    assert app(pt=48) == app(pt=8) == app(pt=512) == app(n=0) == app(kv=c.kv.data_ptr() + 8) == B.VERKV_EINVAL
    assert app(n=1 << 27) == app(sp=None) == app(sp=B.verkv_span(pos.data_ptr(), 0, 3, None, 0)) == B.VERKV_EINVAL
    assert B.verkv_launch_counts(c.ctx) == n0  # nothing was launched
    assert c.norm_rotate(q[:0], k[:0], pos[:0], rope)[0].shape == (0, 4, 64)  # no tokens: nothing to do
    assert c.append(0, k[:0], k[:0], pos[:0], pos[:0], pos.view(3, 1)) is None
    assert B.verkv_launch_counts(c.ctx) == n0
    with torch.cuda.stream(torch.cuda.Stream()):
        with pytest.raises(ValueError):
            c.norm_rotate(q, k)


def test_keys_with_outlier_channels():
    # keys of the single-layer workload's shape, with its outlier channels: large squares, float32 sums
    w = I.tiny()
    k = torch.as_tensor(w.kv[0, 0, 0, :, 0].view("int16")).view(BF).cuda().view(-1, 1, w.d) * 30
    wk = randn((w.d,), BF, 11)
    c = PagedKV(1, 4, w.d)
    pos, f = torch.arange(w.n, dtype=torch.int32, device="cuda"), freqs(w.d, 1e6)
    _, y = c.norm_rotate(None, k, pos, Rope(f), None, wk, 1e-6)
    check(y, k, pos, f, False, wk, 1e-6, "workload keys")
