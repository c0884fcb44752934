"""Paged caches: refusals on the host (no GPU needed), and on the GPU the
block tables and slot maps against a plain allocator, the append against
indexed copies, and the attention against its definition in fp64.

Tolerances of the attention, per output element, fixed from the arithmetic
before the first run.  With w the exact weights, A = sum_j w_j |v_j| and
Z = max_j sum_i |q_i k_ji| / sqrt(d):
* a score is a d-term fp32 sum scaled once: off by at most (d + 4) 2^-24 Z, so
  a weight by twice that relative, plus 2^-20 for the exponential and its
  scaled argument; the sums over n keys add at most 2 n 2^-24;
* bf16 kernels may round a weight to bf16 (2^-8 A) and round the result once
  (2^-8 |o|)."""
import ctypes
import gc
import math
import threading
import time

import pytest
import torch

import token_sparse_attention_sm_b200 as sd

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ---- refusals (host only) -----------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    from token_sparse_attention_sm_b200 import build
    build.build()
    return sd.load()


def _pshape(**kw):
    from token_sparse_attention_sm_b200.paged import _PagedShape
    base = dict(B=2, T=8, Hq=8, Hkv=2, d=64, dtype=1, page_size=16, num_pages=10, max_blocks=4,
                max_new=0)
    base.update(kw)
    return _PagedShape(**base)


@pytest.mark.parametrize("kw,rc", [
    ({}, 0), (dict(T=0), 0), (dict(max_blocks=1, page_size=13), 0), (dict(d=128, dtype=0), 0),
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=7), 1), (dict(page_size=0), 1),
    (dict(num_pages=0), 1), (dict(max_blocks=0), 1), (dict(max_new=-1), 1),
    (dict(d=96), 2), (dict(dtype=2), 2), (dict(Hq=34), 2), (dict(B=4097), 2),
    (dict(page_size=24), 2), (dict(num_pages=1 << 27), 2), (dict(T=(1 << 24) + 1), 2),
    (dict(max_blocks=1 << 27), 2),
])
def test_paged_shapes(lib, kw, rc):
    n = ctypes.c_size_t(0)
    assert lib.sparse_paged_workspace_size(ctypes.byref(_pshape(**kw)), ctypes.byref(n)) == rc
    if rc == 0:
        assert n.value > 4096


def test_paged_calls_refuse_bad_pointers_and_sizes(lib):
    sh, F = _pshape(), 1 << 20  # F: an aligned address that is never used
    p = lambda x: ctypes.c_void_p(x)
    big = 1 << 32
    ok = [p(F)] * 4 + [10] + [p(F)] * 6
    def plan(i=None, v=None, ws=p(F), nb=big, s=sh):
        a = list(ok)
        if i is not None:
            a[i] = v
        return lib.sparse_paged_plan(ctypes.byref(s), *a, ws, nb, None)
    for i in (0, 1, 2, 3, 5, 6, 7, 8, 9, 10):
        assert plan(i, None) == 1
        assert plan(i, p(F + 2)) == 1
    assert plan(4, -1) == 1
    assert plan(ws=None) == 1 and plan(ws=p(F + 16)) == 1 and plan(nb=4095) == 3
    assert plan(s=_pshape(d=96)) == 2

    def append(K=F, V=F, k=F, ks=128, v=F, vs=128, slots=F, ws=F, nb=big, s=sh):
        return lib.sparse_paged_append(ctypes.byref(s), p(K), p(V), p(k), ks, p(v), vs, p(slots),
                                       p(ws), nb, None)
    for name in ("K", "V", "k", "v", "slots", "ws"):
        assert append(**{name: None}) == 1
        assert append(**{name: F + 2}) == 1
    assert append(ks=132) == 1 and append(vs=120) == 1 and append(s=_pshape(T=0)) == 1
    assert append(nb=16) == 3

    def attn(q=F, qs=512, K=F, V=F, t=F, st=F, kv=F, w=0, snk=0, out=F, lse=None, ws=F, nb=big,
             s=sh):
        return lib.sparse_paged_attn(ctypes.byref(s), p(q), qs, p(K), p(V), p(t), p(st), p(kv), w,
                                     snk, p(out), p(lse), p(ws), nb, None)
    for name in ("q", "K", "V", "t", "st", "kv", "out", "ws"):
        assert attn(**{name: None}) == 1
        assert attn(**{name: F + 2}) == 1
    assert attn(lse=F + 2) == 1 and attn(w=-1) == 1 and attn(snk=-1) == 1
    assert attn(qs=516) == 1 and attn(qs=504) == 1 and attn(s=_pshape(T=0)) == 1
    assert attn(nb=4096) == 3


def test_status_elsewhere_is_refused_like_the_rest(lib):
    sh, F = _pshape(), 1 << 20
    p = lambda x: ctypes.c_void_p(x)
    def attn(status, ws=F, nb=1 << 32):
        return lib.sparse_paged_attn_status(ctypes.byref(sh), p(F), 512, p(F << 1), p(F << 2),
                                            p(F), p(F), p(F), 0, 0, p(F << 3), None, p(ws), nb,
                                            p(status), None)
    assert attn(None) == 1 and attn(F + 2) == 1 and attn(F, ws=None) == 1 and attn(F, nb=16) == 3
    assert lib.sparse_paged_static_status(None) == 1


@pytest.mark.parametrize("T,stride", [(1, 512), (3, 512), (3, 1024)])
def test_attn_refuses_results_over_its_inputs(lib, T, stride):
    """Also where only the first or the last 16 bytes are shared."""
    sh = _pshape(T=T)
    es, n = (4, 2)[sh.dtype], ctypes.c_size_t(0)
    assert lib.sparse_paged_workspace_size(ctypes.byref(sh), ctypes.byref(n)) == 0
    row, A = sh.Hq * sh.d * es, 1 << 30
    cache = sh.num_pages * sh.Hkv * sh.page_size * sh.d * es
    p = lambda x: ctypes.c_void_p(x)
    def attn(out, lse):
        K, V, rest = A << 1, A << 2, A << 3
        return lib.sparse_paged_attn(ctypes.byref(sh), p(A), stride, p(K), p(V), p(rest), p(rest),
                                     p(rest), 0, 0, p(out), p(lse), p(rest), n.value, None)
    q = (T - 1) * stride * es + row
    for start, size in ((A, q), (A << 1, cache), (A << 2, cache)):
        for out in (start, start + size - 16, start - T * row + 16):
            assert attn(out, None) == 1
        for lse in (start, start + size - 16, start - T * sh.Hq * 4 + 16):
            assert attn(A << 4, lse) == 1
    assert attn(A << 4, (A << 4) + T * row - 16) == 1


def test_paged_python_refuses_host_tensors():
    K = torch.zeros(4, 2, 16, 64)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sd.paged_attn(torch.zeros(1, 4, 64), K, K, i[None], i, i)
    with pytest.raises(ValueError, match="CUDA"):
        sd.paged_append(K, K, torch.zeros(1, 2, 64), torch.zeros(1, 2, 64), i)
    with pytest.raises(ValueError, match="CUDA"):
        sd.paged_plan(i, i, i[None], i, i, 16, 1, 4)


BIG = 1 << 32


@pytest.mark.parametrize("kw", [dict(page_size=BIG + 16), dict(num_pages=BIG + 10),
                                dict(max_blocks=BIG + 4), dict(max_new=BIG + 1), dict(T=BIG + 8),
                                dict(B=BIG + 2), dict(d=BIG + 64), dict(page_size=16 - BIG),
                                dict(T=1 << 31)], ids=str)
def test_sizes_past_32_bits_are_refused(lib, kw):
    a = dict(B=2, T=8, Hq=8, Hkv=2, d=64, dtype=BF16, page_size=16, num_pages=10, max_blocks=4,
             max_new=8)
    assert sd.paged_workspace_bytes(**a) > 4096
    with pytest.raises((ValueError, sd.SparseDecodeError)):
        sd.paged_workspace_bytes(**{**a, **kw})


# ---- inputs and the plain forms ------------------------------------------------------

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _batch(new, kv, Hq, Hkv, d, page, dtype, seed=0, pad=0, extra_cols=1, q_pad=0, grow=None):
    """A ragged batch over shuffled pages.  Everything that no sequence owns
    (page tails, spare pages, unused table entries) holds NaN or rubbish."""
    g = torch.Generator().manual_seed(seed)
    nb = [max(0, -(-c // page)) for c in kv]
    pages = sum(nb) + 3
    perm = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(kv), max(nb + [1]) + extra_cols), 1 << 29, dtype=torch.int32)
    if extra_cols == 0 and max(nb + [1]) == 1:
        table = table[:, :1].contiguous()
    K = torch.full((pages, Hkv, page, d), float("nan"), dtype=dtype)
    V = torch.full((pages, Hkv, page, d), float("nan"), dtype=dtype)
    dense = []
    for b, c in enumerate(kv):
        k = torch.randn(Hkv, max(c, 0), d, generator=g)
        if grow is not None:
            k *= grow(torch.arange(max(c, 0)))[:, None]
        k = k.to(dtype)
        v = (torch.randn(Hkv, max(c, 0), d, generator=g) + 0.25).to(dtype)
        for j in range(nb[b]):
            pg = perm.pop()
            table[b, j] = pg
            m = min(page, c - j * page)
            K[pg, :, :m] = k[:, j * page:j * page + m]
            V[pg, :, :m] = v[:, j * page:j * page + m]
        dense.append((k, v))
    T = sum(new)
    q = torch.randn(T + pad, Hq * d + q_pad, generator=g).to(dtype)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    qc = q.cuda()[:, :Hq * d].unflatten(1, (Hq, d))
    return dict(new=new, kv=kv, starts=starts, dense=dense, q=q[:, :Hq * d].unflatten(1, (Hq, d)),
                Hq=Hq, Hkv=Hkv, d=d, dtype=dtype,
                args=(qc, K.cuda(), V.cuda(), table.cuda(), _i32(starts), _i32(kv)))


def _definition(x, window=0, sinks=0, hide=()):
    """out, lse, and the tolerances of both, in fp64 on the host; hide: (b, j)
    tokens that nobody sees."""
    Hq, Hkv, d = x["Hq"], x["Hkv"], x["d"]
    T = x["starts"][-1]
    out = torch.zeros(T, Hq, d, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros(T, Hq, dtype=torch.float64)
    for b, (n, c) in enumerate(zip(x["new"], x["kv"])):
        if n == 0:
            continue
        r = slice(x["starts"][b], x["starts"][b] + n)
        q = x["q"][r].double()
        k = x["dense"][b][0].double().repeat_interleave(Hq // Hkv, 0)
        v = x["dense"][b][1].double().repeat_interleave(Hq // Hkv, 0)
        z = torch.einsum("ihd,hjd->ihj", q, k) / math.sqrt(d)
        za = torch.einsum("ihd,hjd->ihj", q.abs(), k.abs()) / math.sqrt(d)
        p = torch.arange(c - n, c)[:, None]
        j = torch.arange(max(c, 0))[None]
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        for hb, hj in hide:
            if hb == b:
                see[:, hj] = False
        z = z.masked_fill(~see[:, None, :], -math.inf)
        l = torch.logsumexp(z, -1) if c > 0 else torch.full((n, Hq), -math.inf).double()
        w = torch.where(see[:, None, :], torch.exp(z - l[..., None]), torch.zeros(()).double())
        w = torch.nan_to_num(w)
        out[r] = torch.einsum("ihj,hjd->ihd", w, v)
        lse[r] = l
        a = torch.einsum("ihj,hjd->ihd", w, v.abs())
        Z = za.masked_fill(~see[:, None, :], 0).amax(-1) if c > 0 else torch.zeros(n, Hq).double()
        e = (d + 4) * 2.0 ** -24 * Z
        rel = 2 * e + 2.0 ** -20 + 2 * max(c, 1) * 2.0 ** -24
        tol[r] = rel[..., None] * a
        if x["dtype"] == BF16:
            tol[r] += 2.0 ** -8 * a + 2.0 ** -8 * out[r].abs()
        else:
            tol[r] += 2.0 ** -24 * out[r].abs()
        ltol[r] = rel + 2.0 ** -23 * l.abs().nan_to_num(posinf=0)
    return out, lse, tol + 1e-30, ltol


def _assert_attn(x, got, window=0, sinks=0, hide=()):
    out, lse, tol, ltol = _definition(x, window, sinks, hide)
    T = x["starts"][-1]
    o, l = got[0][:T].double().cpu(), got[1][:T].double().cpu()
    assert not torch.isnan(o).any()
    worst = ((o - out).abs() / tol).max().item() if T else 0
    assert worst <= 1, f"out off by {worst:.3g} tolerances"
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(l), empty) and (l[empty] < 0).all()
    d = ((l - lse).abs() / ltol)[~empty]
    assert d.numel() == 0 or d.max().item() <= 1, f"lse off by {d.max().item():.3g} tolerances"


# ---- attention -------------------------------------------------------------------------

HEADS = [(4, 4), (8, 2), (6, 2), (16, 1), (10, 2)]


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 3)])
def test_attn_ragged(lib, dtype, d, Hq, Hkv, window, sinks):
    new = [1, 70, 0, 5, 33, 1, 2]
    kv = [1, 70, 9, 133, 300, 260, 129]
    x = _batch(new, kv, Hq, Hkv, d, 16, dtype, seed=d + Hq, pad=3, q_pad=16)
    out = torch.full((sum(new) + 3, Hq, d), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((sum(new) + 3, Hq), 7.0, device="cuda")
    got = sd.paged_attn(*x["args"], window=window, sinks=sinks, out=out, lse=lse)
    _assert_attn(x, got, window, sinks)
    assert (out[-3:] == 7).all() and (lse[-3:] == 7).all()


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 272])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 0), (64, 130), (1 << 30, 5)])
def test_attn_decode(lib, dtype, page, window, sinks):
    kv = [1, 15, 16, 17, 128, 129, 640, 1500, 2, 1027]
    x = _batch([1] * len(kv), kv, 8, 2, 128, page, dtype, seed=page)
    got = sd.paged_attn(*x["args"], window=window, sinks=sinks, max_new=1)
    _assert_attn(x, got, window, sinks)
    # the kernels for more rows give the same answer within the same tolerances
    got = sd.paged_attn(*x["args"], window=window, sinks=sinks, max_new=9)
    _assert_attn(x, got, window, sinks)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,new", [(4, 4, 1), (4, 4, 11), (6, 2, 1), (10, 2, 1), (6, 2, 5),
                                        (16, 2, 2), (16, 1, 1), (14, 1, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 20)])
def test_attn_few_rows(lib, dtype, d, Hq, Hkv, new, window, sinks):
    """Every number of rows up to the 16 of the decode kernels, tokens and
    groups of heads mixed."""
    kv = [new, 31, 32, 33, 200, 1000]
    x = _batch([new, 1, 0, min(new, 2), new, new], kv, Hq, Hkv, d, 16, dtype, seed=Hq + new)
    _assert_attn(x, sd.paged_attn(*x["args"], window=window, sinks=sinks, max_new=new), window,
                 sinks)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B", [1000, 4096])
def test_attn_many_sequences(lib, dtype, B):
    """Runs over many short caches, some without new tokens, some empty."""
    new = [0 if i % 7 == 3 else 1 for i in range(B)]
    kv = [(i * 37) % 90 if i % 11 else 0 for i in range(B)]
    x = _batch(new, kv, 4, 2, 64, 16, dtype, seed=B)
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=1))
    if B == 1000:
        _assert_attn(x, sd.paged_attn(*x["args"], max_new=40))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_attn_padding_may_hold_anything(lib, dtype):
    """NaN in the padding rows of q and in the rows between two tokens' heads."""
    for new in ([1, 1, 1], [30, 1, 45]):
        x = _batch(new, [50, 20, 90], 8, 2, 64, 16, dtype, seed=3, pad=70, q_pad=8)
        T = sum(new)
        q = x["args"][0]
        q[T:] = float("nan")
        base = q._base if q._base is not None else q
        base.view(T + 70, -1)[:, 8 * 64:] = float("nan")
        out = torch.full(q.shape, 3.0, dtype=dtype, device="cuda")
        got = sd.paged_attn(*x["args"], max_new=max(new), out=out)
        _assert_attn(x, got)
        assert (out[T:] == 3).all()


@gpu
def test_a_workspace_shared_with_the_decode_step(lib):
    """Ordered calls of both kinds on one workspace leave each other alone."""
    g = torch.Generator().manual_seed(2)
    K, V = (torch.randn(1, 2, 5000, 128, generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn(1, 8, 128, generator=g).to(BF16).cuda()
    ref = sd.decode_step(q, q[None], K, V, k=100)
    x = _batch([1, 60], [3000, 700], 8, 2, 128, 16, BF16, seed=1)
    ws = sd.Workspace()
    for _ in range(3):
        got = sd.paged_attn(*x["args"], ws=ws)
        dec = sd.paged_attn(x["args"][0][:1], *x["args"][1:3], x["args"][3][:1].contiguous(),
                            x["args"][4][:2].contiguous(), x["args"][5][:1].contiguous(),
                            max_new=1, ws=ws)
        step = sd.decode_step(q, q[None], K, V, k=100, ws=ws)
        assert sd.read_device_flags(ws) == 0
        assert torch.equal(step["idx"], ref["idx"]) and torch.equal(step["out"], ref["out"])
        _assert_attn(x, got)
        assert torch.allclose(dec[1], got[1][:1], atol=1e-4)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,kv,window,sinks", [
    ([300], [300], 0, 0), ([300], [300], 128, 4), ([257], [1300], 0, 0), ([64], [4000], 0, 0),
    ([513], [900], 200, 129), ([129, 1, 400], [129, 2500, 401], 0, 0), ([9], [3100], 1000, 16),
    ([16] * 5, [700, 16, 255, 256, 257], 0, 0), ([700], [1100], 300, 0),
])
def test_attn_chunks(lib, dtype, new, kv, window, sinks):
    for (Hq, Hkv, d) in ((8, 2, 128), (12, 4, 64)):
        x = _batch(new, kv, Hq, Hkv, d, 32, dtype, seed=len(new) + d)
        got = sd.paged_attn(*x["args"], window=window, sinks=sinks)
        _assert_attn(x, got, window, sinks)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("max_new", [1, 3, None])
def test_attn_many_splits_and_steps(lib, dtype, max_new):
    """Long ranges over few heads (every worker takes a piece of one range),
    and rows of several tokens."""
    n = max_new or 40
    x = _batch([n], [9000], 4, 1, 128, 64, dtype, seed=n)
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=max_new))
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=max_new, window=5000, sinks=4), 5000, 4)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new", [1, 40])
def test_attn_long_runs(lib, dtype, d, page, new):
    """Runs of many tiles: every stage of a ring is reused several times."""
    x = _batch([new, 1], [30000, 17], 8, 8, d, page, dtype, seed=d + new)
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=new))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 150])
@pytest.mark.parametrize("grow", [
    lambda j: 0.02 * (j + 1.0),                # the maximum moves in every tile
    lambda j: 0.001 + 60.0 * (j // 200),       # by more than fp32's range between two tiles
    lambda j: 40.0 / (1 + j // 64),            # the first keys outweigh the rest
], ids=["grows", "jumps", "falls"])
def test_attn_scores_of_any_size(lib, dtype, d, new, grow):
    x = _batch([new, min(new, 2)], [900, 413], 8, 2, d, 16, dtype, seed=d + new, grow=grow)
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=new))
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=new, window=333, sinks=5), 333, 5)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [[1, 1], [2, 60]])
def test_attn_pages_in_several_places(lib, dtype, new):
    """Two sequences that share their first pages, and a page that stands twice
    in one sequence."""
    x = _batch(new, [300, 210], 8, 2, 128, 16, dtype, seed=5)
    table = x["args"][3]
    table[1, :6] = table[0, :6]
    table[0, 9] = table[0, 3]
    for (k0, k1) in zip(*x["dense"]):
        k1[:, :96] = k0[:, :96]
        k0[:, 144:160] = k0[:, 48:64]
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=max(new)))
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=max(new), window=150, sinks=20), 150, 20)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_attn_rows_that_see_nothing(lib, dtype):
    # more new tokens than cached ones: the first rows stand before the cache
    x = _batch([5, 3, 200, 1], [2, 0, 150, 0], 8, 2, 64, 16, dtype)
    got = sd.paged_attn(*x["args"])
    _assert_attn(x, got)
    assert (got[0][:3] == 0).all() and torch.isinf(got[1][:3]).all()
    x = _batch([1, 1], [0, 40], 8, 2, 64, 16, dtype)
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=1))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40])
def test_attn_bad_pages_hide_their_tokens(lib, dtype, new):
    kv = [200, 90]
    x = _batch([new] * 2, kv, 8, 2, 128, 16, dtype, seed=3)
    table = x["args"][3]
    table[0, 3] = -1
    table[1, 5] = x["args"][1].shape[0]
    hide = [(0, j) for j in range(48, 64)] + [(1, j) for j in range(80, 90)]
    ws = sd.Workspace()
    got = sd.paged_attn(*x["args"], max_new=new, ws=ws, check=False)
    _assert_attn(x, got, hide=hide)
    with pytest.raises(sd.SparseDecodeError, match="INDEX"):
        sd.read_device_status(ws)
    # outside the window an entry is not read
    q, K, V, _, qs, lens = x["args"]
    sd.paged_attn(q, K, V, table[:1].contiguous(), qs[:2].contiguous(), lens[:1].contiguous(),
                  window=16, sinks=7, max_new=new, ws=ws)


@gpu
def test_attn_bad_lengths_skip_the_sequence(lib):
    x = _batch([4, 4, 4], [40, 50, 60], 8, 2, 64, 16, BF16, seed=5)
    q, K, V, table, qs, kv = x["args"]
    ws = sd.Workspace()
    for lens, kw in (([40, -1, 60], {}), ([40, 1 << 30, 60], {}), ([40, 50, 60], {"max_new": 3})):
        out = torch.full_like(q, 7.0)
        sd.paged_attn(q, K, V, table, qs, _i32(lens), out=out, ws=ws, check=False, **kw)
        with pytest.raises(sd.SparseDecodeError, match="INDEX"):
            sd.read_device_status(ws)
        assert (out[4:8] == 7).all()
    out = torch.full_like(q, 7.0)
    sd.paged_attn(q, K, V, table, _i32([0, 13, 4, 12]), kv, out=out, ws=ws, check=False)
    with pytest.raises(sd.SparseDecodeError, match="INDEX"):
        sd.read_device_status(ws)


@gpu
@pytest.mark.parametrize("new", [1, 24])
def test_attn_offsets_past_32_bits(lib, new):
    """The sequence's pages lie beyond 2^31 elements of the pool."""
    Hq, Hkv, d, page = 8, 8, 128, 64
    pages = (1 << 31) // (Hkv * page * d) + 40
    x = _batch([new], [1000], Hq, Hkv, d, page, BF16, seed=9, extra_cols=0)
    q, K, V, table, qs, kv = x["args"]
    bigK = torch.empty(pages, Hkv, page, d, dtype=BF16, device="cuda")
    bigV = torch.empty_like(bigK)
    off = pages - K.shape[0]
    bigK[off:], bigV[off:] = K, V
    _assert_attn(x, sd.paged_attn(q, bigK, bigV, table + off, qs, kv, max_new=new))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_attn_on_a_dense_cache(lib, dtype):
    """A dense cache is one page per sequence, of any length; the decode step
    that selects every key gives the same single-token attention."""
    B, Hq, Hkv, d, ncap, n = 3, 8, 2, 64, 333, 301
    g = torch.Generator().manual_seed(1)
    K = torch.randn(B, Hkv, ncap, d, generator=g).to(dtype).cuda()
    V = torch.randn(B, Hkv, ncap, d, generator=g).to(dtype).cuda()
    q = torch.randn(B, Hq, d, generator=g).to(dtype).cuda()
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    out, lse = sd.paged_attn(q, K, V, table, _i32([0, 1, 2, 3]), _i32([n] * 3), max_new=1)
    ref = sd.decode_step(q, q[None], K, V, k=n, n=n)
    tol = 2.0 ** -5 if dtype == BF16 else 1e-5
    assert (out.float() - ref["out"][0].float()).abs().max() <= tol
    assert (lse - ref["lse"][0]).abs().max() <= 1e-3


# ---- plan and append -------------------------------------------------------------------

def _plain_plan(new, lens, table, free, page, T):
    """The allocator in plain Python."""
    table, free = [list(r) for r in table], list(free)
    starts, pos, slots = [0], [], []
    for b, (n, c) in enumerate(zip(new, lens)):
        for j in range(-(-c // page), -(-(c + n) // page)):
            table[b][j] = free.pop()
        for i in range(n):
            pos.append(c + i)
            slots.append(table[b][(c + i) // page] * page + (c + i) % page)
        starts.append(starts[-1] + n)
    pad = [-1] * (T - len(pos))
    return table, [c + n for n, c in zip(new, lens)], starts, pos + pad, slots + pad, free


PLANS = [([1], [0], 16, 1), ([1, 1, 1], [15, 16, 17], 16, 3), ([0, 0], [5, 0], 16, 0),
         ([40, 0, 7, 1], [0, 33, 16, 31], 16, 50), ([700, 1300, 1, 64], [3, 64, 127, 0], 64, 2100),
         ([1] * 300, [(7 * i) % 100 for i in range(300)], 16, 300),
         ([3] * 4096, [i % 50 for i in range(4096)], 16, 3 * 4096), ([5, 5], [2, 100], 48, 12)]


@gpu
@pytest.mark.parametrize("new,lens,page,T", PLANS)
def test_plan(lib, new, lens, page, T):
    B = len(new)
    cols = max(-(-(c + n) // page) for n, c in zip(new, lens)) + 2
    pages = sum(-(-(c + n) // page) for n, c in zip(new, lens)) + 5
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(B)).tolist()
    table = [[-1] * cols for _ in range(B)]
    for b, c in enumerate(lens):
        for j in range(-(-c // page)):
            table[b][j] = perm.pop()
    want = _plain_plan(new, lens, table, perm, page, T)
    tab, free = _i32(table), _i32(perm + [99999] * 3)
    nl, ln, fc = _i32(new), _i32(lens), _i32([len(perm)])
    for _ in range(2):  # repeatable while lens and free_count stay
        p = sd.paged_plan(nl, ln, tab, free, fc, page, T, pages)
        assert tab.tolist() == want[0]
        assert p["kv_lens"].tolist() == want[1] and p["q_start"].tolist() == want[2]
        assert p["positions"].tolist() == want[3] and p["slots"].tolist() == want[4]
        assert p["free_left"].tolist() == [len(want[5])]
    p = sd.paged_plan(nl, ln, tab, free, fc, page, T, pages, kv_lens=ln, free_left=fc)
    assert ln.tolist() == want[1] and fc.tolist() == [len(want[5])]
    assert p["slots"].tolist() == want[4]


@gpu
@pytest.mark.parametrize("T", [0, 3])
@pytest.mark.parametrize("free", [[], [4, 2]])
def test_plan_of_nothing(lib, T, free):
    """No new tokens, an empty free list, no rows."""
    table = _i32([[1, -1], [0, 3]])
    p = sd.paged_plan(_i32([0, 0]), _i32([16, 20]), table, _i32(free), _i32([len(free)]), 16, T, 5)
    assert p["kv_lens"].tolist() == [16, 20] and p["q_start"].tolist() == [0, 0, 0]
    assert p["positions"].tolist() == [-1] * T and p["slots"].tolist() == [-1] * T
    assert p["free_left"].tolist() == [len(free)] and table.tolist() == [[1, -1], [0, 3]]


@gpu
@pytest.mark.parametrize("new,lens,T,count,status", [
    ([2, 2], [0, 0], 3, 8, "CAPACITY"),       # more rows than T
    ([20, 20], [0, 0], 40, 3, "CAPACITY"),    # four pages, three free
    ([60, 1], [10, 0], 61, 8, "CAPACITY"),    # longer than the table row
    ([1, -1], [0, 5], 4, 8, "INDEX"), ([1, 1], [0, -5], 4, 8, "INDEX"),
    ([1, 1], [0, 0], 4, 9, "INDEX"), ([1, 1], [0, 0], 4, -1, "INDEX"),
])
def test_plan_refuses_a_batch_as_a_whole(lib, new, lens, T, count, status):
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    ws = sd.Workspace()
    p = sd.paged_plan(_i32(new), _i32(lens), table, _i32(list(range(8))), _i32([count]), 16, T, 8,
                      ws=ws, check=False)
    assert (table == -1).all() and p["kv_lens"].tolist() == lens
    assert p["q_start"].tolist() == [0, 0, 0] and p["free_left"].tolist() == [count]
    assert (p["positions"] == -1).all() and (p["slots"] == -1).all()
    with pytest.raises(sd.SparseDecodeError, match=status):
        sd.read_device_status(ws)
    with pytest.raises(sd.SparseDecodeError, match=status):
        sd.paged_plan(_i32(new), _i32(lens), table, _i32(list(range(8))), _i32([count]), 16, T, 8)


@gpu
def test_plan_bad_page_ids(lib):
    table = _i32([[3, 77, -1], [-1, -1, -1]])
    ws = sd.Workspace()
    # the tail page of sequence 0 is outside the pool, and so is the page sequence 1 takes
    p = sd.paged_plan(_i32([2, 1]), _i32([20, 0]), table, _i32([5, 8]), _i32([2]), 16, 4, 8, ws=ws,
                      check=False)
    assert p["slots"].tolist() == [-1, -1, -1, -1] and p["positions"].tolist() == [20, 21, 0, -1]
    with pytest.raises(sd.SparseDecodeError, match="INDEX"):
        sd.read_device_status(ws)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,Hkv,d,page", [(1, 1, 64, 16), (7, 2, 128, 16), (130, 8, 128, 64),
                                          (33, 3, 64, 48), (5, 40, 128, 16)])
def test_append(lib, dtype, T, Hkv, d, page):
    g = torch.Generator().manual_seed(T)
    pages = 20
    K = torch.randn(pages, Hkv, page, d, generator=g).to(dtype).cuda()
    V = torch.randn(pages, Hkv, page, d, generator=g).to(dtype).cuda()
    w = Hkv * d
    qkv = torch.randn(T, 3 * w, generator=g).to(dtype).cuda()
    k_new, v_new = (qkv[:, i * w:(i + 1) * w].unflatten(1, (Hkv, d)) for i in (1, 2))
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    slots[::5] = -1
    wantK, wantV = K.clone(), V.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            wantK[s // page, :, s % page] = k_new[t]
            wantV[s // page, :, s % page] = v_new[t]
    sd.paged_append(K, V, k_new, v_new, slots.cuda())
    assert torch.equal(K, wantK) and torch.equal(V, wantV)
    sd.paged_append(K, V, k_new.contiguous(), v_new.contiguous(), slots.cuda())
    assert torch.equal(K, wantK) and torch.equal(V, wantV)


@gpu
def test_append_bad_slots_write_nothing(lib):
    K = torch.zeros(4, 2, 16, 64, device="cuda")
    V = torch.zeros_like(K)
    new = torch.ones(4, 2, 64, device="cuda")
    with pytest.raises(sd.SparseDecodeError, match="INDEX"):
        sd.paged_append(K, V, new, new, _i32([64, -2, 1 << 30, 3]))
    assert K.sum() == 2 * 64 and (K[0, :, 3] == 1).all() and torch.equal(K, V)


@gpu
def test_python_refusals(lib):
    x = _batch([2], [20], 8, 2, 64, 16, BF16)
    q, K, V, table, qs, kv = x["args"]
    for bad in (lambda: sd.paged_attn(q.float(), K, V, table, qs, kv),
                lambda: sd.paged_attn(q, K, V[:1], table, qs, kv),
                lambda: sd.paged_attn(q, K, V, table.long(), qs, kv),
                lambda: sd.paged_attn(q, K, V, table, qs[:1], kv),
                lambda: sd.paged_attn(q, K, V, table, qs, kv, window=-1),
                lambda: sd.paged_attn(q, K, V, table, qs, kv, max_new=0),
                lambda: sd.paged_attn(q.transpose(0, 1), K, V, table, qs, kv),
                lambda: sd.paged_attn(q[:1].expand(2, 8, 64), K, V, table, qs, kv),
                lambda: sd.paged_attn(q, K, V, table, qs, kv, out=q.float()),
                lambda: sd.paged_append(K, V, q[:, :2].float(), q[:, :2], kv),
                lambda: sd.paged_append(K, V, q[:, :2], q[:, :2], kv),
                lambda: sd.paged_plan(kv, kv, table, kv, kv.long(), 16, 1, 4),
                lambda: sd.paged_plan(kv, kv, table, kv, kv, 16, -1, 4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sd.SparseDecodeError, match="UNSUPPORTED"):
        sd.paged_plan(kv, kv, table, kv, kv, 24, 1, 4)
    for t in (q, q.contiguous()):  # the results over the queries
        with pytest.raises((ValueError, sd.SparseDecodeError)):
            sd.paged_attn(t, K, V, table, qs, kv, out=t)
    out, lse = sd.paged_attn(q[:0], K, V, table, _i32([0, 0]), kv)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)


# ---- together ----------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_serving_steps(lib, dtype, window, sinks):
    """Prompts in chunks, then decode steps, over one pool: every step planned,
    appended and attended, against the definition on the whole history."""
    B, Hq, Hkv, d, page, pages = 3, 8, 2, 64, 16, 64
    g = torch.Generator().manual_seed(4)
    K = torch.full((pages, Hkv, page, d), float("nan"), dtype=dtype, device="cuda")
    V = K.clone()
    table = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
    count, lens = _i32([pages]), _i32([0] * B)
    hist = [(torch.zeros(Hkv, 0, d, dtype=dtype),) * 2 for _ in range(B)]
    total = [0] * B
    for new in ([50, 0, 3], [50, 70, 1], [1, 1, 1], [0, 1, 1], [1, 30, 1], [1, 1, 1]):
        T = sum(new) + 2
        qkv = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g).to(dtype)
        dq = qkv.cuda()
        q, k, v = (dq[:, a * d:b * d].unflatten(1, (b - a, d))
                   for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        p = sd.paged_plan(_i32(new), lens, table, free, count, page, T, pages, kv_lens=lens,
                          free_left=count)
        sd.paged_append(K, V, k, v, p["slots"])
        got = sd.paged_attn(q, K, V, table, p["q_start"], lens, window=window, sinks=sinks,
                            max_new=max(new))
        starts = p["q_start"].tolist()
        for b in range(B):
            r = slice(starts[b], starts[b + 1])
            hist[b] = (torch.cat([hist[b][0], k[r].cpu().transpose(0, 1)], 1),
                       torch.cat([hist[b][1], v[r].cpu().transpose(0, 1)], 1))
            total[b] += new[b]
        x = dict(new=new, kv=total, starts=starts, dense=hist, q=q.cpu(), Hq=Hq, Hkv=Hkv, d=d,
                 dtype=dtype)
        _assert_attn(x, got, window, sinks)
    assert count.tolist() == [pages - sum(-(-c // page) for c in total)]


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_captured_steps_follow_the_lengths(lib, dtype):
    """One captured decode step (plan, append, attention) replayed while the
    caches grow, a second graph with its own memory in between, on streams of
    their own."""
    B, Hq, Hkv, d, page, pages = 2, 8, 2, 64, 16, 40
    g = torch.Generator().manual_seed(6)
    x = _batch([1] * B, [30, 100], Hq, Hkv, d, page, dtype, seed=2, extra_cols=3)
    _, K0, V0, table, _, _ = x["args"]
    used = K0.shape[0]
    K = torch.full((pages, Hkv, page, d), float("nan"), dtype=dtype, device="cuda")
    V = K.clone()
    K[:used], V[:used] = K0, V0
    free = torch.arange(used, pages, dtype=torch.int32, device="cuda")
    count, lens, one = _i32([pages - used]), _i32([30, 100]), _i32([1, 1])
    q = torch.zeros(B, Hq, d, dtype=dtype, device="cuda")
    k = torch.zeros(B, Hkv, d, dtype=dtype, device="cuda")
    v = torch.zeros_like(k)
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            p = sd.paged_plan(one, lens, table, free, count, page, B, pages, check=False,
                              kv_lens=lens, free_left=count)
            sd.paged_append(K, V, k, v, p["slots"], check=False)
            outs.append(sd.paged_attn(q, K, V, table, p["q_start"], lens, max_new=1, check=False))
        graphs.append(gr)
    with pytest.raises(ValueError, match="capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            sd.paged_attn(q, K, V, table, p["q_start"], lens)
    hist, total = x["dense"], [30, 100]
    for step in range(6):
        qn = torch.randn(B, Hq, d, generator=g).to(dtype)
        kn, vn = (torch.randn(B, Hkv, d, generator=g).to(dtype) for _ in range(2))
        q.copy_(qn), k.copy_(kn), v.copy_(vn)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graphs[step % 2].replay()
        torch.cuda.current_stream().wait_stream(s)
        hist = [(torch.cat([hist[b][0], kn[b][:, None]], 1), torch.cat([hist[b][1], vn[b][:, None]], 1))
                for b in range(B)]
        total = [c + 1 for c in total]
        y = dict(new=[1, 1], kv=total, starts=[0, 1, 2], dense=hist, q=qn, Hq=Hq, Hkv=Hkv, d=d,
                 dtype=dtype)
        _assert_attn(y, outs[step % 2])


@gpu
def test_calls_on_two_streams(lib):
    """Calls on two streams at once do not share a workspace."""
    x = _batch([1, 20], [4000, 3000], 8, 2, 128, 16, BF16, seed=7)
    y = _batch([30], [2500], 8, 1, 128, 16, BF16, seed=8)
    torch.cuda.synchronize()
    sx, sy = torch.cuda.Stream(), torch.cuda.Stream()
    gx, gy = [], []
    for _ in range(10):
        with torch.cuda.stream(sx):
            gx.append(sd.paged_attn(*x["args"], check=False))
        with torch.cuda.stream(sy):
            gy.append(sd.paged_attn(*y["args"], check=False))
    torch.cuda.synchronize()
    _assert_attn(x, gx[-1])
    _assert_attn(y, gy[-1])
    for a in gx:
        assert torch.equal(a[0], gx[0][0]) and torch.equal(a[1], gx[0][1])
    for a in gy:
        assert torch.equal(a[0], gy[0][0]) and torch.equal(a[1], gy[0][1])


# ---- host threads that share a stream ------------------------------------------------------

class _HostPaged:
    """paged.py on host tensors, its C calls replaced by ones that note their
    launches and let other threads run in between."""

    def __init__(self, monkeypatch):
        from token_sparse_attention_sm_b200 import paged
        self.log, self.paged = [], paged
        monkeypatch.setattr(paged, "_stream_ws", {})
        monkeypatch.setattr(paged, "Workspace", lambda dev: sd.Workspace("cpu"))
        monkeypatch.setattr(paged, "_one_device", lambda *ts: 0)
        monkeypatch.setattr(paged, "_entry", lambda name: self.call)
        monkeypatch.setattr(paged, "_plain", lambda t: None)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
        monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False)

    def call(self, *a):
        me = threading.get_ident()
        for _ in range(3):  # a schedule, its items, the merge
            self.log.append(me)
            time.sleep(0.002)
        return 0

    def together(self, *calls):
        errors = []
        def run(f):
            try:
                for _ in range(5):
                    time.sleep(0.001)
                    f()
            except Exception as e:  # pragma: no cover
                errors.append(e)
        ts = [threading.Thread(target=run, args=(f,)) for f in calls]
        [t.start() for t in ts]
        [t.join() for t in ts]
        assert not errors
        assert len(self.log) == 15 * len(calls)
        for i in range(0, len(self.log), 3):
            assert len(set(self.log[i:i + 3])) == 1, "the launches of two calls are mixed"


def _host_attn(B, T):
    K = torch.zeros(4, 2, 16, 64)
    i = torch.zeros(B, dtype=torch.int32)
    return lambda: sd.paged_attn(torch.zeros(T, 8, 64), K, K, i[:, None].contiguous(),
                                 torch.zeros(B + 1, dtype=torch.int32), i, check=False)


def test_threads_on_one_stream_do_not_mix_their_launches(monkeypatch, lib):
    h = _HostPaged(monkeypatch)
    h.together(_host_attn(2, 40), _host_attn(3, 300), _host_attn(1, 1))  # it grows


@pytest.mark.parametrize("name", ["plan", "append", "attn"])
def test_c_calls_keep_the_global_lock(lib, name):
    """No other thread's launches can come between those of one call, the
    compiled calls' (which take no other lock) among them."""
    from token_sparse_attention_sm_b200 import paged
    fn = paged._entry(f"sparse_paged_{name}")
    assert fn._flags_ & 4  # ctypes' FUNCFLAG_PYTHONAPI
    assert fn.argtypes == getattr(lib, f"sparse_paged_{name}").argtypes


@gpu
def test_attn_from_threads_of_one_stream(lib):
    xs = [_batch([1, 20], [4000, 3000], 8, 2, 128, 16, BF16, seed=7),
          _batch([300, 2, 5], [2500, 70, 900], 8, 1, 128, 16, BF16, seed=8),
          _batch([1] * 9, [100 * i + 5 for i in range(9)], 8, 2, 128, 16, BF16, seed=9)]
    torch.cuda.synchronize()
    sd.paged._stream_ws.clear()  # the first calls make and grow it
    got, errors = [[] for _ in xs], []
    def run(i):
        try:
            for _ in range(20):
                got[i].append(sd.paged_attn(*xs[i]["args"], max_new=max(xs[i]["new"]),
                                            check=False))
        except Exception as e:  # pragma: no cover
            errors.append(e)
    ts = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    torch.cuda.synchronize()
    assert not errors
    for x, g in zip(xs, got):
        _assert_attn(x, g[0])
        assert all(torch.equal(a[0], g[0][0]) and torch.equal(a[1], g[0][1]) for a in g)


# ---- status -----------------------------------------------------------------------------

def test_a_workspace_that_grows_keeps_its_status():
    ws = sd.Workspace("cpu")
    ws.get(4096)[:4] = torch.tensor([2, 1, 0, 0], dtype=torch.uint8)
    ws.buf[4:64] = 7
    grown = ws.get(4 << 20)
    assert grown.numel() == 4 << 20 and grown[:4].tolist() == [2, 1, 0, 0]
    assert not grown[4:].any()
    assert ws.get(5) is grown


@gpu
@pytest.mark.parametrize("kept", [True, False])
def test_errors_before_a_growing_call_are_reported(lib, kept):
    """A batch that the plan refused, unread, then an attention that needs a
    larger workspace."""
    ws = None if kept else sd.Workspace()
    sd.paged._stream_ws.clear()
    x = _batch([300], [300], 8, 2, 128, 16, BF16)
    table = torch.full((1, 40), -1, dtype=torch.int32, device="cuda")
    p = sd.paged_plan(_i32([300]), _i32([0]), table, _i32([0, 1]), _i32([2]), 16, 300, 40, ws=ws,
                      check=False)
    q, K, V = x["args"][:3]
    with pytest.raises(sd.SparseDecodeError, match="CAPACITY"):
        sd.paged_attn(q, K, V, table, p["q_start"], p["kv_lens"], ws=ws)
    sd.paged_attn(*x["args"], ws=ws)  # read, and clear again


@gpu
@pytest.mark.parametrize("new", [1, 40])
def test_errors_of_a_replayed_graph_are_reported(lib, new):
    """A captured step without a workspace whose replays run out of pages, then
    one whose block table goes bad."""
    Hq, Hkv, d, page, pages = 8, 2, 64, 16, 12
    K = torch.zeros(pages, Hkv, page, d, dtype=BF16, device="cuda")
    V = torch.zeros_like(K)
    free = torch.arange(3, pages, dtype=torch.int32, device="cuda")
    table, count, lens, n = _i32([[0, 1, 2] + [-1] * 13]), _i32([1]), _i32([40]), _i32([new])
    q = torch.zeros(new, Hq, d, dtype=BF16, device="cuda")
    k = torch.zeros(new, Hkv, d, dtype=BF16, device="cuda")
    sd.paged_status(raise_on_error=False)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        p = sd.paged_plan(n, lens, table, free, count, page, new, pages, check=False,
                          kv_lens=lens, free_left=count)
        sd.paged_append(K, V, k, k, p["slots"], check=False)
        sd.paged_attn(q, K, V, table, p["q_start"], lens, max_new=new, check=False)
    assert sd.paged_status() == 0
    for _ in range(40):
        gr.replay()
    with pytest.raises(sd.SparseDecodeError, match="CAPACITY"):
        sd.paged_status()
    assert sd.paged_status() == 0
    table[0, 0] = pages
    lens.fill_(20), count.fill_(9)
    gr.replay()
    assert sd.paged_status(raise_on_error=False) == 8  # INDEX: the attention's


@gpu
def test_status_of_unchecked_calls(lib):
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    sd.paged_status(raise_on_error=False)
    sd.paged_plan(_i32([60]), _i32([10]), table, _i32([0]), _i32([1]), 16, 60, 8, check=False)
    with pytest.raises(sd.SparseDecodeError, match="CAPACITY"):
        sd.paged_status()
    assert sd.paged_status() == 0


@gpu
@pytest.mark.parametrize("checked", [True, False])
def test_a_wait_that_ran_out_costs_the_kept_workspace(lib, checked):
    x = _batch([1], [300], 8, 2, 64, 16, BF16)
    sd.paged_attn(*x["args"], max_new=1)
    stream = torch.cuda.current_stream().cuda_stream
    ws = sd.paged._stream_ws[torch.cuda.current_device(), stream]
    # a word that nothing increments, given up after a millisecond
    assert lib.sparse_selftest_bounded_wait(ws.buf.data_ptr(), ws.buf.numel(), 1000000,
                                            stream) == 0
    with pytest.raises(sd.SparseDecodeError, match="TIMEOUT"):
        sd.paged_attn(*x["args"], max_new=1) if checked else sd.paged_status()
    assert ws not in sd.paged._stream_ws.values()
    _assert_attn(x, sd.paged_attn(*x["args"], max_new=1))
    assert sd.paged._stream_ws[torch.cuda.current_device(), stream] is not ws


@gpu
def test_kept_workspaces_can_be_freed(lib):
    x = _batch([300], [300], 8, 2, 128, 16, BF16)
    sd.paged_release()
    gc.collect()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    got = sd.paged_attn(*x["args"])
    del got
    assert torch.cuda.memory_allocated() > before + (1 << 20)
    sd.paged_release()
    assert torch.cuda.memory_allocated() == before
    _assert_attn(x, sd.paged_attn(*x["args"]))


def test_status_is_not_read_inside_a_capture(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: True)
    with pytest.raises(ValueError, match="capture"):
        sd.paged_status()


@pytest.mark.parametrize("own,static,rc,left", [(0, 0, 0, 1), (0, 8, 8, 1), (4, 0, 4, 1),
                                                (7, 8, 7, 0), (8, 7, 8, 1), (7, 0, 7, 0)])
def test_status_of_both_words_is_read(monkeypatch, own, static, rc, left):
    from token_sparse_attention_sm_b200 import paged
    ws = sd.Workspace("cpu")
    ws.key = (0, 5)
    ws.get(4096)
    reads = {ws.buf.data_ptr(): own, 4096: static}
    class Library:
        @staticmethod
        def sparse_read_device_status(at, stream, flags):
            assert stream == 5
            return reads.pop(at)
    monkeypatch.setattr(paged, "_stream_ws", {(0, 5): ws})
    monkeypatch.setattr(paged, "load", lambda: Library)
    monkeypatch.setattr(paged, "_static_status", lambda dev: 4096)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 5)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False)
    assert sd.paged_status(raise_on_error=False) == rc
    assert not reads and len(paged._stream_ws) == left


def test_only_a_wait_that_ran_out_costs_the_kept_workspace(monkeypatch):
    from token_sparse_attention_sm_b200 import paged
    monkeypatch.setattr(paged, "_stream_ws", {})
    kept, own = sd.Workspace("cpu"), sd.Workspace("cpu")
    kept.key = (0, 0)
    for ws, status, left in ((kept, 8, 1), (own, 7, 1), (None, 7, 1), (kept, 7, 0)):
        paged._stream_ws[0, 0] = kept
        paged._drop_after(status, ws)
        assert len(paged._stream_ws) == left
    paged._stream_ws[0, 0] = kept
    sd.paged_release()
    assert not paged._stream_ws


# ---- values that are not finite -----------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,kv", [([1, 1], [700, 90]), ([1, 1], [20000, 90]),
                                    ([3, 2], [700, 90]), ([40, 7], [700, 90]),
                                    ([40, 1], [9000, 90]), ([300, 1], [300, 90])])
@pytest.mark.parametrize("what", ["key nan", "key inf", "query nan", "query inf"])
@pytest.mark.parametrize("window", [0, 30])
def test_attn_scores_that_are_not_finite(lib, dtype, d, new, kv, what, window):
    """A row with a score that is NaN or +inf has no softmax: out and lse are
    NaN, and lse is not the -inf of a row that sees nothing.  Rows that do not
    see the key, the other heads and the other sequence are as ever."""
    Hq, Hkv = 8, 2
    x = _batch(new, kv, Hq, Hkv, d, 16, dtype, seed=d)
    q, K, V, table = x["args"][:4]
    n, c = new[0], kv[0]
    value = float("nan") if what.endswith("nan") else float("inf")
    j = c - min(n, 2)       # the last or the last but one new token
    p = torch.arange(c - n, c)
    bad = torch.zeros(sum(new), Hq, dtype=torch.bool)
    sees = (p >= j) & ((p - window < j) if window else torch.ones_like(p, dtype=torch.bool))
    if what.startswith("key"):
        q[:n, 4:, 3] = q[:n, 4:, 3].abs() + 0.5     # of KV head 1
        x["q"][:n, 4:, 3] = x["q"][:n, 4:, 3].abs() + 0.5
        K[table[0, j // 16], 1, j % 16, 3] = value
        bad[:n, 4:] = sees[:, None]
    else:
        q[n - 1, 2, 5] = value
        bad[n - 1, 2] = True
    out, lse, tol, ltol = _definition(x, window, 0)
    got_out, got_lse = (t.double().cpu() for t in
                        sd.paged_attn(*x["args"], window=window, max_new=max(new)))
    assert torch.equal(torch.isnan(got_lse), bad)
    assert torch.equal(torch.isnan(got_out).all(-1), bad) and not torch.isnan(got_out[~bad]).any()
    assert ((got_out - out).abs() / tol)[~bad].max() <= 1
    assert ((got_lse - lse).abs() / ltol)[~bad].max() <= 1


@gpu
def test_calls_refuse_sizes_past_32_bits(lib):
    x = _batch([2], [20], 8, 2, 64, 16, BF16)
    q, K, V, table, qs, kv = x["args"]
    sd.paged_attn(*x["args"])  # the stream has a workspace: the compiled calls are asked first
    for bad in (lambda: sd.paged_plan(kv, kv, table, kv, kv, BIG + 16, 1, 4),
                lambda: sd.paged_plan(kv, kv, table, kv, kv, 16, BIG + 1, 4),
                lambda: sd.paged_plan(kv, kv, table, kv, kv, 16, 1, BIG + 4),
                lambda: sd.paged_plan(kv, kv, table, kv, kv, 16, (1 << 31) - 1, 4),
                lambda: sd.paged_attn(q, K, V, table, qs, kv, max_new=BIG + 1),
                lambda: sd.paged_attn(q, K, V, table, qs, kv, window=BIG + 1),
                lambda: sd.paged_attn(q, K, V, table, qs, kv, window=5, sinks=BIG)):
        with pytest.raises((ValueError, sd.SparseDecodeError)):
            bad()


# ---- the build of the compiled calls ---------------------------------------------------------

def test_compiled_calls_are_rebuilt_for_another_torch(monkeypatch, tmp_path, lib):
    """The module is compiled against torch and CPython: one that was built for
    others is not taken, however new the file."""
    from token_sparse_attention_sm_b200 import build, paged
    assert build.calls_current()
    ran = []
    def fake(cmd):
        ran.append(cmd)
        tag = next(c for c in cmd if c.startswith("-DPAGED_CALLS_TAG="))
        with open(cmd[-1], "wb") as f:
            f.write(b"x" + tag.split("=", 1)[1].strip('"').encode())
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "calls.so"))
    monkeypatch.setattr(build.subprocess, "check_call", fake)
    build.build_calls()
    assert len(ran) == 1 and build.calls_current()
    build.build_calls()
    assert len(ran) == 1
    monkeypatch.setattr(torch, "__version__", "2.99.0")
    assert not build.calls_current()
    paged._calls.cache_clear()
    with pytest.raises(RuntimeError, match="another torch"):
        paged._calls()
    build.build_calls()
    assert len(ran) == 2 and build.calls_current()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda n: "cpython-399")
    build.build_calls()
    assert len(ran) == 3


def test_the_library_is_built_before_the_compiled_calls(monkeypatch):
    from token_sparse_attention_sm_b200 import build
    order = []
    monkeypatch.setattr(build, "build_library", lambda *a: order.append("library"))
    monkeypatch.setattr(build, "build_calls", lambda *a: order.append("calls"))
    assert build.build() == build.LIB and order == ["library", "calls"]


# ---- one page per sequence: the decode step's caches -----------------------------------------

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,new,kv", [
    (333, [70, 1, 20], [333, 1, 300]), (13, [13, 5], [13, 13]), (1, [1, 1], [1, 1]),
    (200, [1, 1], [200, 129]), (2500, [40, 300], [2500, 2000]), (64, [64], [64]),
    (129, [33, 4], [129, 128]), (7, [1, 1], [7, 3]),
])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_attn_one_page_per_sequence(lib, dtype, d, page, new, kv, window, sinks):
    x = _batch(new, kv, 8, 2, d, page, dtype, seed=page, extra_cols=0)
    assert x["args"][3].shape[1] == 1
    _assert_attn(x, sd.paged_attn(*x["args"], window=window, sinks=sinks, max_new=max(new)),
                 window, sinks)
    _assert_attn(x, sd.paged_attn(*x["args"], window=window, sinks=sinks), window, sinks)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ncap", [90, 333])
def test_prefill_of_the_decode_steps_caches(lib, dtype, ncap):
    """Prompts in two chunks and a token through plan, append and attention on
    dense caches, which the decode step then reads."""
    B, Hq, Hkv, d = 2, 8, 2, 64
    g = torch.Generator().manual_seed(ncap)
    K = torch.full((B, Hkv, ncap, d), float("nan"), dtype=dtype, device="cuda")
    V = K.clone()
    table, lens = _i32([[-1], [-1]]), _i32([0, 0])
    free, count = _i32([1, 0]), _i32([2])  # sequence b gets page b
    hist = [(torch.zeros(Hkv, 0, d, dtype=dtype),) * 2 for _ in range(B)]
    total = [0, 0]
    for new in ([50, 30], [33, 53], [1, 1]):
        T = sum(new)
        q, k, v = (torch.randn(T, h, d, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
        p = sd.paged_plan(_i32(new), lens, table, free, count, ncap, T, B, kv_lens=lens,
                          free_left=count)
        assert table.tolist() == [[0], [1]]
        sd.paged_append(K, V, k.cuda(), v.cuda(), p["slots"])
        got = sd.paged_attn(q.cuda(), K, V, table, p["q_start"], lens, max_new=max(new))
        starts = p["q_start"].tolist()
        for b in range(B):
            r = slice(starts[b], starts[b + 1])
            hist[b] = (torch.cat([hist[b][0], k[r].transpose(0, 1)], 1),
                       torch.cat([hist[b][1], v[r].transpose(0, 1)], 1))
            total[b] += new[b]
            assert torch.equal(K[b, :, :total[b]].cpu(), hist[b][0])
            assert torch.equal(V[b, :, :total[b]].cpu(), hist[b][1])
        x = dict(new=new, kv=total, starts=starts, dense=hist, q=q, Hq=Hq, Hkv=Hkv, d=d,
                 dtype=dtype)
        _assert_attn(x, got)
    n = total[0]
    assert total == [n, n] and torch.isnan(K[:, :, n:]).all()
    K[:, :, n:], V[:, :, n:] = 0, 0
    step = sd.decode_step(q.cuda(), q.cuda()[None], K, V, k=n, n=n)
    tol = 2.0 ** -5 if dtype == BF16 else 1e-5
    assert (step["out"][0].float() - got[0].float()).abs().max() <= tol
    assert (step["lse"][0] - got[1]).abs().max() <= 1e-3


# ---- heads, pages ------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("G", range(1, 17))
def test_attn_chunks_of_every_group_size(lib, dtype, G):
    x = _batch([40, 300, 1], [200, 300, 77], 2 * G, 2, 64, 16, dtype, seed=G)
    _assert_attn(x, sd.paged_attn(*x["args"]))
    _assert_attn(x, sd.paged_attn(*x["args"], window=90, sinks=70), 90, 70)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 48, 80, 96, 128, 144, 256, 400])
def test_attn_chunks_of_every_page_size(lib, dtype, page):
    x = _batch([60, 5, 300], [700, 5, 401], 8, 2, 128, page, dtype, seed=page)
    _assert_attn(x, sd.paged_attn(*x["args"]))
    _assert_attn(x, sd.paged_attn(*x["args"], window=150, sinks=20), 150, 20)


# ---- weights in two parts ------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,n", [(1, 100), (8, 64), (2, 33)])
def test_attn_decode_keeps_16_bits_of_the_weights(lib, d, Hkv, n):
    """Values whose weighted sum almost cancels show the rounding of the
    weights.  q and k are small whole numbers, so scores are exact before they
    are scaled.  With w the weights and A = sum_j w_j |v_j|: scaled scores and
    their exponential are off by less than 2^-20 relative, sums over n keys by
    4 n 2^-24 (products that are cut, not rounded), a weight in two bf16 parts
    by 2^-16, the result by 2^-8 of itself."""
    g = torch.Generator().manual_seed(n + d)
    x = _batch([1], [n], Hkv, Hkv, d, 16, BF16, seed=n)
    q, K, V, table = x["args"][:4]
    qi = torch.randint(-1, 2, (1, Hkv, d), generator=g).to(BF16)
    ki = torch.randint(-1, 2, (Hkv, n, d), generator=g).to(BF16)
    z = torch.einsum("hd,hjd->hj", qi[0].double(), ki.double()) / math.sqrt(d)
    w = torch.softmax(z, -1)
    v = torch.randn(Hkv, n, d, generator=g).double()
    v = (v - torch.einsum("hj,hjd->hd", w, v)[:, None]).to(BF16)
    q.copy_(qi)
    for j in range(0, n, 16):
        m = min(16, n - j)
        K[table[0, j // 16], :, :m] = ki[:, j:j + m].cuda()
        V[table[0, j // 16], :, :m] = v[:, j:j + m].cuda()
    want = torch.einsum("hj,hjd->hd", w, v.double())
    A = torch.einsum("hj,hjd->hd", w, v.double().abs())
    tol = (2.0 ** -20 + 4 * n * 2.0 ** -24 + 2.0 ** -16) * A + 2.0 ** -8 * want.abs()
    got = sd.paged_attn(*x["args"], max_new=1)[0][0].double().cpu()
    assert ((got - want).abs() / tol).max() <= 1
    # one bf16 part alone would be far outside
    p = torch.exp(z - z.amax(-1, keepdim=True))
    one = torch.einsum("hj,hjd->hd", p.to(BF16).double(), v.double()) / p.sum(-1, keepdim=True)
    assert ((one - want).abs() / tol).max() > 4


# ---- graphs and streams that overlap ---------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_captured_chunks_follow_the_lengths(lib, dtype):
    """One captured step of up to 40 new tokens per sequence, replayed with
    other lengths: the schedule, the claim counter and the pieces of long
    ranges are made anew each time, in two graphs in turn."""
    B, Hq, Hkv, d, page, T = 2, 8, 1, 64, 16, 64
    g = torch.Generator().manual_seed(6)
    x = _batch([1] * B, [5000, 100], Hq, Hkv, d, page, dtype, seed=2, extra_cols=20)
    _, K0, V0, table, _, _ = x["args"]
    used, pages = K0.shape[0], K0.shape[0] + 40
    K = torch.full((pages, Hkv, page, d), float("nan"), dtype=dtype, device="cuda")
    V = K.clone()
    K[:used], V[:used] = K0, V0
    free = torch.arange(used, pages, dtype=torch.int32, device="cuda")
    count, lens, new = _i32([pages - used]), _i32([5000, 100]), _i32([1, 1])
    q = torch.zeros(T, Hq, d, dtype=dtype, device="cuda")
    k = torch.zeros(T, Hkv, d, dtype=dtype, device="cuda")
    v = torch.zeros_like(k)
    graphs, outs, starts = [], [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            p = sd.paged_plan(new, lens, table, free, count, page, T, pages, check=False,
                              kv_lens=lens, free_left=count)
            sd.paged_append(K, V, k, v, p["slots"], check=False)
            outs.append(sd.paged_attn(q, K, V, table, p["q_start"], lens, max_new=40,
                                      check=False))
        graphs.append(gr)
        starts.append(p["q_start"])
    hist, total = x["dense"], [5000, 100]
    for step, ns in enumerate(([40, 3], [1, 40], [0, 17], [30, 0], [1, 1], [39, 25])):
        n = sum(ns)
        qn = torch.randn(n, Hq, d, generator=g).to(dtype)
        kn, vn = (torch.randn(n, Hkv, d, generator=g).to(dtype) for _ in range(2))
        new.copy_(_i32(ns)), q[:n].copy_(qn), k[:n].copy_(kn), v[:n].copy_(vn)
        for o in outs[step % 2]:
            o.fill_(7)
        graphs[step % 2].replay()
        at = starts[step % 2].tolist()
        assert at == [0, ns[0], n]
        hist = [tuple(torch.cat([old, t[at[b]:at[b + 1]].transpose(0, 1)], 1)
                      for old, t in zip(hist[b], (kn, vn))) for b in range(B)]
        total = [c + m for c, m in zip(total, ns)]
        y = dict(new=ns, kv=total, starts=at, dense=hist, q=qn, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype)
        _assert_attn(y, outs[step % 2])
        assert all((o[n:] == 7).all() for o in outs[step % 2])
    assert sd.paged_status() == 0


@gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40])
def test_calls_that_overlap_keep_their_scratch_apart(lib, captured, dtype, new):
    """Calls whose ranges are cut for all SMs, on two streams (or in two graphs
    replayed there) with no order between them."""
    xs = [_batch([new], [20000], 8, 2, 128, 16, dtype, seed=7),
          _batch([new, new], [9000, 7000], 4, 1, 128, 16, dtype, seed=8)]
    alone = [sd.paged_attn(*x["args"], max_new=new) for x in xs]
    for x, a in zip(xs, alone):
        _assert_attn(x, a)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    calls = [lambda x=x: sd.paged_attn(*x["args"], max_new=new, check=False) for x in xs]
    if captured:
        graphs = [torch.cuda.CUDAGraph() for _ in xs]
        outs = []
        for gr, f in zip(graphs, calls):
            with torch.cuda.graph(gr):
                outs.append(f())
        def replay(i):
            graphs[i].replay()
            return tuple(o.clone() for o in outs[i])
        calls = [lambda: replay(0), lambda: replay(1)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(25):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    for a, each in zip(alone, got):
        for o in each:
            assert torch.equal(o[0], a[0]) and torch.equal(o[1], a[1])
    for s in streams:
        with torch.cuda.stream(s):
            assert sd.paged_status() == 0
