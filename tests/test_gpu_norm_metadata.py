"""Layer norm with its gradients, and the paged metadata, on the GPU."""
from __future__ import annotations

import pytest
import torch

import depthwise_causal_conv1d_amd as lib
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAN = float("nan")
DIMS = [1, 2, 7, 64, 255, 512, 1001, 1024, 2048, 4096, 4100, 8192, 8200, 16384, 20001]


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    t = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale
    return t.to(dtype)


def rows_on_gpu(t, odd):
    """[rows, dim] in rows of aligned length, or from an odd element on; NaN around."""
    rows, dim = t.shape
    ld = dim + 1 if odd else (dim + 15) // 8 * 8
    buf = torch.full((rows * ld + 8,), NAN, dtype=t.dtype, device="cuda")
    return buf[1 if odd else 0:].as_strided((rows, dim), (ld, 1)).copy_(t)


def reference(s, w, b, eps):
    """out and its bound: the mean is off by (dim / 64 + 10) EPS of the mean of
    |s|, so a difference d by that and half a step; the variance's mean adds
    its own additions (halved by the root) and twice the differences'."""
    dim = s.shape[1]
    mean = s.mean(1, keepdim=True)
    d = s - mean
    rstd = 1 / torch.sqrt(d.square().mean(1, keepdim=True) + eps)
    chain = (dim / 64 + 10) * R.EPS
    emean = chain * s.abs().mean(1, keepdim=True) + 2 * R.EPS * mean.abs()
    ed = emean + 2 * R.EPS * (d.abs() + s.abs())
    # a shifted mean enters the variance squared, a rounded difference as its product with d
    var = d.square().mean(1, keepdim=True)
    evar = 2 * (ed * d.abs()).mean(1, keepdim=True) + ed.square().mean(1, keepdim=True) + chain * var
    erel = (evar / (var + eps)) + 8 * R.EPS
    y = d * rstd * w + b
    ey = (d * rstd * w).abs() * (erel + 4 * R.EPS) + ed * (rstd * w).abs() + 2 * R.EPS * y.abs()
    return y, ey, d, rstd, ed, erel, chain


def grads(g, s, w, eps, dres):
    y, _, d, rstd, ed, erel, chain = reference(s, w, torch.zeros_like(w), eps)
    hat, wg = d * rstd, g * w
    ehat = hat.abs() * (erel + 2 * R.EPS) + ed * rstd
    flat, proj = wg.mean(1, keepdim=True), (wg * hat).mean(1, keepdim=True)
    eflat = (chain + 2 * R.EPS) * wg.abs().mean(1, keepdim=True)
    eproj = (wg.abs() * ehat).mean(1, keepdim=True) + (chain + 4 * R.EPS) * (wg * hat).abs().mean(1, keepdim=True)
    inner = wg - flat - hat * proj
    einner = 4 * R.EPS * (wg.abs() + flat.abs() + (hat * proj).abs()) + eflat + ehat * proj.abs() + hat.abs() * eproj
    dx, edx = rstd * inner, rstd * (einner + inner.abs() * (erel + 2 * R.EPS))
    if dres is not None:
        dx, edx = dx + dres, edx + 2 * R.EPS * (dx.abs() + dres.abs())
    n = s.shape[0]
    dw, edw = (g * hat).sum(0), (g.abs() * ehat).sum(0) + n * R.EPS * (g * hat).abs().sum(0)
    return dict(dx=(dx, edx), dweight=(dw, edw), dbias=(g.sum(0), n * R.EPS * g.abs().sum(0)))


def check_norm(x, res, w, b, eps, odd):
    s = R.f64(x) + (R.f64(res) if res is not None else 0)
    zero = torch.zeros(x.shape[1], dtype=torch.float64)
    y, ey = reference(s, R.f64(w), R.f64(b) if b is not None else zero, eps)[:2]
    xd = rows_on_gpu(x, odd)
    rd = rows_on_gpu(res, odd) if res is not None else None
    bd = b.cuda() if b is not None else None
    out = lib.layer_norm_fwd(xd, w.cuda(), bd, eps, residual=rd, out=rows_on_gpu(x, odd))
    R.check(out, y, ey, "out")
    if res is not None:
        R.check(rd, s, R.EPS * s.abs(), "sum")
    at = rd if res is not None else xd
    g, dres = rand(91, *x.shape, dtype=x.dtype), rand(92, *x.shape, dtype=x.dtype)
    for dr in (None, dres):
        ref = grads(R.f64(g), R.f64(at), R.f64(w), eps, R.f64(dr) if dr is not None else None)
        got = lib.layer_norm_bwd(rows_on_gpu(g, odd), at, w.cuda(), eps,
                                 dresidual=rows_on_gpu(dr, odd) if dr is not None else None,
                                 dx=rows_on_gpu(x, odd))
        for n, t in zip(("dx", "dweight", "dbias"), got):
            R.check(t, *ref[n], n)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_and_gradients(dim, dtype):
    dt, rows = DT[dtype], 9
    x, res = rand(1, rows, dim, dtype=dt), rand(2, rows, dim, dtype=dt, scale=2.0)
    x[3], res[3] = 0, 0
    w, b = (rand(3, dim) * 0.2 + 1).to(dt), rand(4, dim, dtype=dt)
    for odd in (False, True):
        check_norm(x, res, w, b, 1e-5, odd)
    check_norm(x, None, w, None, 1e-3, False)


@pytest.mark.parametrize("rows,dim", [(4100, 136), (4100, 2056), (2051, 8193)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_many_rows(rows, dim, dtype):
    """The counts of workgroups that share a call's rows, one row left over."""
    dt = DT[dtype]
    x, g = rand(1, rows, dim, dtype=dt), rand(2, rows, dim, dtype=dt)
    w = (rand(3, dim) * 0.2 + 1).to(dt)
    ref = grads(R.f64(g), R.f64(x), R.f64(w), 1e-5, None)
    for n, t in zip(ref, lib.layer_norm_bwd(g.cuda(), x.cuda(), w.cuda(), 1e-5)):
        R.check(t, *ref[n], n)


@pytest.mark.parametrize("rows", [0, 1, 2, 513, 1500])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_row_counts(rows, dtype):
    dt = DT[dtype]
    w, b = (rand(3, 96) * 0.2 + 1).to(dt), rand(4, 96, dtype=dt)
    if rows:
        check_norm(rand(1, rows, 96, dtype=dt), rand(2, rows, 96, dtype=dt), w, b, 1e-5, False)
        return
    e = torch.empty(0, 96, dtype=dt, device="cuda")
    assert lib.layer_norm_fwd(e, w.cuda(), b.cuda()).shape == (0, 96)
    _, dw, db = lib.layer_norm_bwd(e, e, w.cuda())
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_norm_of_rows_far_from_zero():
    """A mean of 2^12 against differences of one: the variance is theirs."""
    x = rand(1, 8, 1000) + 4096.0
    check_norm(x, None, torch.ones(1000), torch.zeros(1000), 1e-5, False)
    check_norm(torch.full((4, 512), 3.0), None, torch.ones(512), rand(2, 512), 1e-5, False)


def test_norm_in_place_and_nan():
    x, w, b = rand(1, 7, 256), torch.ones(256), torch.zeros(256)
    want = lib.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    xd = x.cuda()
    assert torch.equal(lib.layer_norm_fwd(xd, w.cuda(), b.cuda(), out=xd), want)
    x[2, 9] = NAN
    out = lib.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    assert bool(out[2].isnan().all()) and torch.equal(out[[0, 1, 3, 4, 5, 6]], want[[0, 1, 3, 4, 5, 6]])


# ---------------------------------------------------------------- metadata

def tables(query, context, free, table, bs, padded):
    """The same by hand, request by request."""
    table, qsl, used = table.clone(), [0], 0
    n = max(padded, 1)
    seq, start, pos, slot = ([0] * n for _ in range(4))
    slot = [-1] * n
    width = table.shape[1]
    for r, (m, c) in enumerate(zip(query, context)):
        m, c = max(m, 0), max(c, 0)
        for j in range(-(-c // bs), -(-(c + m) // bs)):
            if j < width:
                table[r, j] = free[used] if used < len(free) else -1
            used += 1
        for i in range(m):
            t, p = qsl[-1] + i, c + i
            if t < padded:
                seq[t], start[t], pos[t] = r, qsl[-1], p
                if p // bs < width and table[r, p // bs] >= 0:
                    slot[t] = int(table[r, p // bs]) * bs + p % bs
        qsl.append(qsl[-1] + m)
    return dict(table=table, qsl=qsl, seq=seq[:padded], start=start[:padded], pos=pos[:padded],
                slot=slot[:padded], used=[used])


def run_metadata(query, context, nfree, width, bs, padded, seed=0, extra=0, optional=True):
    gen = torch.Generator().manual_seed(seed)
    R_ = len(query)
    free = torch.randperm(nfree + 5, generator=gen)[:nfree].to(torch.int32)
    table = torch.randint(0, 1000, (R_, width), generator=gen, dtype=torch.int32)
    want = tables(query, context, free.tolist(), table, bs, padded)
    wide = torch.full((R_, width + extra), -9, dtype=torch.int32)
    wide[:, :width] = table
    dev = wide.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    q, c = torch.tensor(query, **i32), torch.tensor(context, **i32)
    qsl = torch.full((R_ + 3,), -9, **i32)
    seq, start = (torch.full((padded,), -9, **i32) for _ in range(2))
    pos, slot = (torch.full((padded,), -9, dtype=torch.int64, device="cuda") for _ in range(2))
    used = torch.full((1,), -9, **i32)
    lib.sconv_paged_metadata(q, c, free.cuda(), dev[:, :width], bs, qsl, seq if optional else None,
                             start if optional else None, pos, slot, used if optional else None)
    assert torch.equal(dev[:, :width].cpu(), want["table"])
    assert bool((dev[:, width:] == -9).all()) and bool((qsl[R_ + 1:] == -9).all())
    assert qsl[:R_ + 1].tolist() == want["qsl"]
    assert pos.tolist() == want["pos"] and slot.tolist() == want["slot"]
    if optional:
        assert seq.tolist() == want["seq"] and start.tolist() == want["start"]
        assert used.tolist() == want["used"]


def lens(seed, n, hi):
    return torch.randint(0, hi + 1, (n,), generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("bs", [1, 16, 24])
@pytest.mark.parametrize("n,q,c", [(1, 1, 0), (1, 700, 33), (7, 40, 100), (256, 1, 500), (300, 9, 70),
                                   (4096, 2, 20), (4097, 2, 20), (5003, 3, 9)])
def test_metadata(n, q, c, bs):
    query, context = lens(n, n, q), lens(n + 1, n, c)
    total = sum(query)
    for padded in {0, total, total + 77, max(total - 3, 0)}:
        run_metadata(query, context, total + n, (q + c) // bs + 2, bs, padded, extra=3)


def test_metadata_edges():
    run_metadata([], [], 4, 3, 16, 10)                          # no requests
    run_metadata([0, 0, 0], [0, 16, 17], 4, 3, 16, 5)           # nothing new
    run_metadata([5, 40, 3], [0, 8, 31], 2, 4, 16, 60)          # the free list ends
    run_metadata([5, 40, 3], [0, 8, 31], 0, 4, 16, 60)          # nothing is free
    run_metadata([50, 20], [0, 40], 9, 2, 16, 80)               # tables too narrow
    run_metadata([50, 20], [0, 40], 9, 0, 16, 80)               # no tables
    run_metadata([-4, 6], [3, -9], 9, 2, 16, 9)                 # negative lengths count as zero
    run_metadata([3] * 5, [2] * 5, 9, 2, 16, 20, optional=False)
    run_metadata([1] * 5000, [3] * 5000, 100, 2, 4, 5000)       # the two-launch form, list ends
    run_metadata([1] * 5000, [3] * 5000, 9000, 1, 4, 5000)
    # a negative entry that is already in the table
    i32 = dict(dtype=torch.int32, device="cuda")
    z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    slot, pos = z(2, torch.int64), z(2, torch.int64)
    lib.sconv_paged_metadata(torch.tensor([2], **i32), torch.tensor([5], **i32), z(1),
                             torch.tensor([[-1]], **i32), 16, z(2), None, None, pos, slot)
    assert slot.tolist() == [-1, -1] and pos.tolist() == [5, 6]


def test_metadata_drives_the_paged_conv():
    """A prompt in two steps and decoded tokens, with metadata from lengths
    alone, against the conv over the whole sequence; graph replays in between."""
    H, D, W, bs, T = 2, 16, 4, 8, 45
    C = H * D
    x, w = rand(1, T, C, dtype=torch.bfloat16).cuda(), rand(2, C, W, dtype=torch.bfloat16).cuda()
    z = torch.zeros(W - 1 + T, C, dtype=torch.float64)
    z[W - 1:] = R.f64(x)
    want = sum(R.f64(w)[:, j] * z[j:j + T] for j in range(W))
    cache = torch.full((16, H, bs, D), NAN, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ids = torch.tensor([11, 3, 7, 14, 2, 9, 0, 5], **i32)
    table = torch.full((2, 8), -1, **i32)
    most = 24
    seq, start = (torch.zeros(most, **i32) for _ in range(2))
    pos, slot = (torch.zeros(most, dtype=torch.int64, device="cuda") for _ in range(2))
    qsl, used = torch.zeros(3, **i32), torch.zeros(1, **i32)
    out = torch.zeros(T, C, dtype=torch.float32)
    q, c = torch.zeros(2, **i32), torch.zeros(2, **i32)
    xin = torch.zeros(most, C, dtype=torch.bfloat16, device="cuda")
    free = torch.zeros(8, **i32)

    def step():
        lib.sconv_paged_metadata(q, c, free, table, bs, qsl, seq, start, pos, slot, used)
        return lib.sconv_fused_insert_conv(xin, w, cache, pos, table, seq, slot, start, 0, D, bs,
                                           use_residual=False)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    done = taken = 0
    for n in (20, 19, 1, 1, 1, 1, 1, 1):
        q.copy_(torch.tensor([n, 0]))
        c.copy_(torch.tensor([done, 0]))
        free[:8 - taken].copy_(ids[taken:])
        xin.zero_()
        xin[:n].copy_(x[done:done + n])
        graph.replay()
        torch.cuda.synchronize()
        taken += int(used)
        out[done:done + n] = held[:n].float().cpu()
        done += n
    assert done == T and taken == -(-T // bs)
    assert table[0, :6].tolist() == ids[:6].tolist()
    # W products in fp32, one rounding to bf16
    lim = 2.0 ** -8 * want.abs() + 8 * R.EPS * sum((R.f64(w)[:, j] * z[j:j + T]).abs() for j in range(W))
    assert bool(((out.double() - want).abs() <= lim * (1 + 1e-6)).all())
