"""Token-model operators on the GPU against plain 64-bit implementations of their
formulas: embedding lookup and gradient, products grouped by expert, preference and
policy losses.

Tolerances.  Every operator sums in FP32 and rounds once, so each output element v may be
off by u * |v| (u: half a unit in the last place of its type, doubled for the rounding of
a value that is itself off) plus the FP32 sum's error: n adds of terms whose magnitudes
sum to A are off by at most n * 2^-23 * A in any order, truncating adders included.
"""
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8, "f16": 2.0 ** -10}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}
E32 = 2.0 ** -23


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=gen(seed), device="cuda").to(dtype)


def pitched(rows, cols, dtype, pad=0, shift=0, fill=7.0):
    """A rows x cols view of a larger buffer (row pitch cols + pad, first element at
    shift), and the buffer."""
    buf = torch.full((shift + rows * (cols + pad) + 64,), fill, device="cuda", dtype=dtype)
    view = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    return view, buf


def outside_untouched(view, buf, fill=7.0):
    seen = torch.zeros_like(buf, dtype=torch.bool)
    seen.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    return bool((buf[~seen] == fill).all())


def close(got, want, tol):
    err = (got.double() - want.double()).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, worst {err[bad].max():.3e} "
                           f"against {tol.expand_as(err)[bad].min():.3e}")


# ---------------------------------------------------------------------------- embedding
@pytest.mark.parametrize("tdt,odt", list(itertools.product(DT, DT)))
def test_embed_types(gpu_lib, tdt, odt):
    table = randn(97, 72, seed=1, dtype=DT[tdt])
    ids = torch.randint(0, 97, (53,), generator=gen(2), device="cuda")
    out = torch.empty(53, 72, device="cuda", dtype=DT[odt])
    ws = gpu_lib.embed_workspace(53, 97, 72)
    gpu_lib.embed(table, ids, out, ws, scale=1.7)
    want = table[ids].double() * float(np.float32(1.7))
    close(out, want, ULP[odt] * want.abs() + E32 * want.abs() + TINY[odt])
    assert gpu_lib.get_status(ws) == 0


@pytest.mark.parametrize("rows", [0, 1, 3, 4, 5, 31, 1000])
@pytest.mark.parametrize("dim", [1, 7, 8, 64, 129, 2048, 2050])
def test_embed_sizes(gpu_lib, rows, dim):
    table = randn(33, dim, seed=3, dtype=torch.bfloat16)
    ids = torch.randint(0, 33, (rows,), generator=gen(4), device="cuda", dtype=torch.int32)
    out, buf = pitched(rows, dim, torch.bfloat16, pad=5, shift=3)
    ws = gpu_lib.embed_workspace(rows, 33, dim)
    gpu_lib.embed(table, ids, out, ws)
    assert torch.equal(out, table[ids.long()])          # scale 1: the same bits
    assert outside_untouched(out, buf)


def test_embed_padding_and_bad_tokens(gpu_lib):
    table = randn(10, 40, seed=5)
    table[3] = float("nan")                              # padding rows are not read
    ids = torch.tensor([1, 3, 9, 10, -1, -7, 2 ** 40, 0, 3], device="cuda")
    out = torch.full((9, 40), 5.0, device="cuda")
    ws = gpu_lib.embed_workspace(9, 10, 40)
    gpu_lib.embed(table, ids, out, ws, padding_id=3)
    ok = torch.tensor([1, 0, 1, 0, 0, 0, 0, 1, 0], device="cuda").bool()
    assert torch.equal(out[ok], table[ids[ok]])
    assert (out[~ok] == 0).all()
    assert gpu_lib.get_status(ws) == 6 and gpu_lib.get_status(ws) == 0
    gpu_lib.embed(table, ids[:2], out[:2], ws, padding_id=3)
    assert gpu_lib.get_status(ws) == 0                   # padding alone is no error
    dout, grad = randn(9, 40, seed=6), torch.full((10, 40), 5.0, device="cuda")
    gpu_lib.embed_grad(dout, ids, grad, ws, padding_id=3)
    want = torch.zeros(10, 40, device="cuda").index_put_((ids[ok],), dout[ok])
    assert torch.equal(grad, want)
    assert gpu_lib.get_status(ws) == 6


def test_embed_long_offsets(gpu_lib):
    """Element offsets past 2^31 in the table and in the gradient."""
    vocab, dim = 70001, 32768
    table = torch.zeros(vocab, dim, device="cuda", dtype=torch.bfloat16)
    table[-1] = 1.5
    table[65536] = 2.5
    ids = torch.tensor([vocab - 1, 65536, 5], device="cuda")
    out = torch.empty(3, dim, device="cuda", dtype=torch.bfloat16)
    ws = gpu_lib.embed_workspace(3, vocab, dim)
    gpu_lib.embed(table, ids, out, ws)
    assert [float(r.min()) for r in out] == [1.5, 2.5, 0.0] == [float(r.max()) for r in out]
    gpu_lib.embed_grad(out, ids, table, ws, scale=2.0)
    assert float(table[-1].min()) == 3.0 and float(table[65536].max()) == 5.0
    assert float(table.float().sum()) == 8.0 * dim


def embed_grad_want(dout, ids, vocab, scale):
    want = torch.zeros(vocab, dout.shape[1], device="cuda", dtype=torch.float64)
    mag = torch.zeros_like(want)
    want.index_put_((ids.long(),), dout.double() * scale, accumulate=True)
    mag.index_put_((ids.long(),), dout.double().abs() * scale, accumulate=True)
    cnt = torch.bincount(ids.long(), minlength=vocab)[:, None].double()
    return want, (cnt + 2) * E32 * mag


@pytest.mark.parametrize("ddt,gdt", list(itertools.product(DT, DT)))
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_types(gpu_lib, ddt, gdt, accumulate):
    vocab, dim, rows = 61, 72, 400
    dout = randn(rows, dim, seed=1, dtype=DT[ddt])
    ids = torch.randint(0, 50, (rows,), generator=gen(2), device="cuda")   # 50..60 absent
    grad = randn(vocab, dim, seed=3, dtype=DT[gdt])
    old = grad.clone()
    ws = gpu_lib.embed_workspace(rows, vocab, dim)
    gpu_lib.embed_grad(dout, ids, grad, ws, scale=0.75, accumulate=accumulate)
    want, tol = embed_grad_want(dout, ids, vocab, 0.75)
    if accumulate:
        want += old.double()
        assert torch.equal(grad[50:], old[50:])
    close(grad, want, tol + 2 * ULP[gdt] * want.abs() + E32 * old.double().abs() + TINY[gdt])
    assert gpu_lib.get_status(ws) == 0


# rows: within one sorting tile, several tiles; vocabularies of one, two and three digits;
# all tokens equal (one run through every chunk), all different, frequencies falling with
# the rank, runs that end on chunk borders
@pytest.mark.parametrize("rows", [0, 1, 2, 8, 9, 2047, 2049, 8193, 20000, 65536, 65537, 150000])
@pytest.mark.parametrize("vocab,kind", [(1, "same"), (7, "uniform"), (600, "same"),
                                        (600, "blocks"), (30000, "falling"),
                                        (300000, "uniform"), (300000, "last")])
def test_embed_grad_runs(gpu_lib, rows, vocab, kind):
    dim = 24 if vocab < 100000 else 3
    g = gen(rows + vocab)
    ids = {
        "same": lambda: torch.full((rows,), vocab // 2, device="cuda"),
        "last": lambda: torch.full((rows,), vocab - 1, device="cuda"),
        "uniform": lambda: torch.randint(0, vocab, (rows,), generator=g, device="cuda"),
        "blocks": lambda: torch.arange(rows, device="cuda") // 8 % vocab,
        "falling": lambda: (vocab ** torch.rand(rows, generator=g, device="cuda")).long() - 1,
    }[kind]().int()
    dout = randn(rows, dim, seed=9, dtype=torch.bfloat16)
    grad, buf = pitched(vocab, dim, torch.float32, pad=8)
    ws = gpu_lib.embed_workspace(rows, vocab, dim)
    gpu_lib.embed_grad(dout, ids, grad, ws, scale=1.0)
    want, tol = embed_grad_want(dout, ids, vocab, 1.0)
    close(grad, want, tol + ULP["f32"] * want.abs())
    assert outside_untouched(grad, buf)
    first = grad.clone()
    gpu_lib.embed_grad(dout, ids, grad, ws, scale=1.0)   # a used workspace, the same bits
    assert torch.equal(first, grad)


@pytest.mark.parametrize("dim,shift", [(1, 0), (5, 1), (1001, 0), (1024, 3), (4100, 0)])
def test_embed_grad_alignment(gpu_lib, dim, shift):
    rows, vocab = 700, 90
    src, _ = pitched(rows, dim, torch.float16, pad=3, shift=shift)
    src.copy_(randn(rows, dim, seed=4))
    ids = torch.randint(0, vocab, (rows,), generator=gen(5), device="cuda")
    grad, buf = pitched(vocab, dim, torch.float32, pad=1, shift=shift)
    ws = gpu_lib.embed_workspace(rows, vocab, dim)
    gpu_lib.embed_grad(src, ids, grad, ws)
    want, tol = embed_grad_want(src, ids, vocab, 1.0)
    close(grad, want, tol + ULP["f32"] * want.abs())
    assert outside_untouched(grad, buf)


# ------------------------------------------------------------------------------ experts
def offsets_of(counts):
    off = np.zeros(len(counts) + 1, np.int32)
    np.cumsum(counts, out=off[1:])
    return torch.from_numpy(off).cuda()


def group_case(counts, k, n, dtype, seed=0, rest=0):
    rows = int(sum(counts)) + rest
    x = randn(rows, k, seed=seed, dtype=dtype)
    w = randn(len(counts), n, k, seed=seed + 1, dtype=dtype)
    dy = randn(rows, n, seed=seed + 2, dtype=dtype)
    return x, w, dy, offsets_of(counts)


def group_want(x, w, dy, off):
    """The three products and the magnitudes of their sums, in 64 bits."""
    o = off.tolist()
    xd, wd, yd = x.double(), w.double(), dy.double()
    y, ym = torch.zeros(len(x), w.shape[1], device="cuda", dtype=torch.float64), None
    ym = torch.zeros_like(y)
    dx = torch.zeros_like(xd)
    dxm = torch.zeros_like(xd)
    dw, dwm = torch.zeros_like(wd), torch.zeros_like(wd)
    for e in range(len(o) - 1):
        a, b = o[e], o[e + 1]
        y[a:b], ym[a:b] = xd[a:b] @ wd[e].T, xd[a:b].abs() @ wd[e].abs().T
        dx[a:b], dxm[a:b] = yd[a:b] @ wd[e], yd[a:b].abs() @ wd[e].abs()
        dw[e], dwm[e] = yd[a:b].T @ xd[a:b], yd[a:b].abs().T @ xd[a:b].abs()
    return (y, ym), (dx, dxm), (dw, dwm)


def check_group(casgd, x, w, dy, off, dt):
    (y, ym), (dx, dxm), (dw, dwm) = group_want(x, w, dy, off)
    counts = (off[1:] - off[:-1]).double()
    k, n = x.shape[1], dy.shape[1]
    ws = casgd.group_workspace(x, w, dy)
    got = torch.full_like(dy, 9.0)
    casgd.group_product(x, w, off, got, ws)
    close(got, y, ULP[dt] * y.abs() + (k + 2) * E32 * ym + TINY[dt])
    got = torch.full_like(x, 9.0)
    casgd.group_product_dx(dy, w, off, got, ws)
    close(got, dx, ULP[dt] * dx.abs() + (n + 2) * E32 * dxm + TINY[dt])
    got = torch.full_like(w, 9.0)
    casgd.group_product_dw(dy, x, off, got, ws)
    close(got, dw, ULP[dt] * dw.abs() + (counts[:, None, None] + 2) * E32 * dwm + TINY[dt])
    assert casgd.get_status(ws) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("counts", [[1], [0], [5, 0, 3], [128, 127, 129, 1], [0, 0, 300, 0],
                                    [15, 16, 17, 31, 33, 63, 65], [257, 640]])
@pytest.mark.parametrize("k,n", [(64, 64), (72, 40), (200, 264), (512, 136)])
def test_group_sizes(gpu_lib, dt, counts, k, n):
    check_group(gpu_lib, *group_case(counts, k, n, DT[dt]), dt)


@pytest.mark.parametrize("k,n", [(1, 1), (3, 5), (7, 64), (64, 9), (65, 130), (301, 8)])
def test_group_odd_widths(gpu_lib, k, n):
    check_group(gpu_lib, *group_case([3, 0, 70, 140], k, n, torch.bfloat16), "bf16")


@pytest.mark.parametrize("groups,rows", [(64, 40), (128, 3), (200, 900), (1024, 2000), (7, 5000)])
def test_group_many(gpu_lib, groups, rows):
    rng = np.random.default_rng(groups)
    p = rng.gamma(0.5, size=groups)
    check_group(gpu_lib, *group_case(rng.multinomial(rows, p / p.sum()), 88, 120,
                                     torch.bfloat16), "bf16")


@pytest.mark.parametrize("counts", [[700, 0, 1500], [3000]])
def test_group_deep(gpu_lib, counts):
    check_group(gpu_lib, *group_case(counts, 1416, 1160, torch.bfloat16), "bf16")


@pytest.mark.parametrize("pads", [(8, 16, 24), (1, 0, 3), (0, 8, 5)])
def test_group_pitches(gpu_lib, pads):
    k, n, counts = 104, 72, [30, 0, 140]
    x, w, dy, off = group_case(counts, k, n, torch.bfloat16, rest=6)
    xs, xb = pitched(len(x), k, torch.bfloat16, pad=pads[0], shift=8 * (pads[0] % 2))
    ys, yb = pitched(len(x), n, torch.bfloat16, pad=pads[2])
    wbuf = torch.full((3, n + 2, k + pads[1]), 7.0, device="cuda", dtype=torch.bfloat16)
    wv = wbuf[:, :n, :k]
    (y, ym), (dx, dxm), (dw, dwm) = group_want(x, w, dy, off)
    ws = gpu_lib.group_workspace(xs, wv, ys)
    xs.copy_(x), wv.copy_(w)
    gpu_lib.group_product(xs, wv, off, ys, ws)
    close(ys, y, ULP["bf16"] * y.abs() + (k + 2) * E32 * ym)   # rows after the groups: zeros
    assert outside_untouched(ys, yb)
    ys.copy_(dy)
    gpu_lib.group_product_dx(ys, wv, off, xs, ws)
    close(xs, dx, ULP["bf16"] * dx.abs() + (n + 2) * E32 * dxm)
    assert outside_untouched(xs, xb)
    xs.copy_(x)
    gpu_lib.group_product_dw(ys, xs, off, wv, ws)
    close(wv, dw, ULP["bf16"] * dw.abs() + 150 * E32 * dwm)
    assert (wbuf[:, n:] == 7.0).all() and (wbuf[:, :, k:] == 7.0).all()


def test_group_long_offsets(gpu_lib):
    """Element offsets past 2^31 in the weights, read and written."""
    e, n, k = 40, 8192, 8192
    w = torch.zeros(e, n, k, device="cuda", dtype=torch.bfloat16)
    w[39] = 0.5
    x = torch.ones(40, k, device="cuda", dtype=torch.bfloat16)
    y = torch.empty(40, n, device="cuda", dtype=torch.bfloat16)
    off = offsets_of([1] * 40)
    ws = gpu_lib.group_workspace(x, w, y)
    gpu_lib.group_product(x, w, off, y, ws)
    assert (y[:39] == 0).all() and (y[39] == k / 2).all()
    y.fill_(2)
    gpu_lib.group_product_dw(y, x, off, w, ws)
    assert (w[39] == 2).all() and (w[0] == 2).all()
    gpu_lib.group_product_dx(y, w, off, x, ws)
    assert (x == 4 * n).all()


def test_group_infinities_stay_in_their_rows(gpu_lib):
    """Inf and NaN in one expert's rows, or in rows of no expert, reach no other result."""
    counts = [37, 21, 0, 50]
    x, w, dy, off = group_case(counts, 128, 96, torch.bfloat16, rest=9)
    (y, _), (dx, _), (dw, _) = group_want(x, w, dy, off)
    x[40], x[110], dy[45], dy[109] = float("inf"), float("nan"), float("nan"), float("inf")
    ws = gpu_lib.group_workspace(x, w, dy)
    got = torch.empty_like(dy)
    gpu_lib.group_product(x, w, off, got, ws)
    ok = torch.ones(len(x), dtype=torch.bool, device="cuda")
    ok[40] = False
    assert torch.isfinite(got[ok]).all() and not torch.isfinite(got[40]).any()
    assert (got[108:] == 0).all()
    got = torch.empty_like(x)
    gpu_lib.group_product_dx(dy, w, off, got, ws)
    assert torch.isfinite(got[:45]).all() and torch.isfinite(got[46:]).all()
    got = torch.empty_like(w)
    gpu_lib.group_product_dw(dy, x, off, got, ws)
    assert torch.isfinite(got[[0, 2, 3]]).all() and not torch.isfinite(got[1]).any()
    assert (got[2] == 0).all()


def test_group_bad_offsets(gpu_lib):
    """Descending, negative or too large offsets touch nothing outside and are reported."""
    x, w, dy, _ = group_case([40, 40], 64, 64, torch.bfloat16)
    for bad in ([0, 60, 20], [0, 40, 90], [-5, 40, 80], [3, 40, 80], [0, 2 ** 31 - 1, -2 ** 31]):
        off = torch.tensor(bad, device="cuda", dtype=torch.int64).int()
        ws = gpu_lib.group_workspace(x, w, dy)
        y, buf = pitched(80, 64, torch.bfloat16, pad=8)
        gpu_lib.group_product(x, w, off, y, ws)
        assert gpu_lib.get_status(ws) == 6
        assert outside_untouched(y, buf)
        gpu_lib.group_product_dw(dy, x, off, torch.empty_like(w), ws)
        assert gpu_lib.get_status(ws) == 6


def test_group_gradients_are_differences(gpu_lib):
    """dx and dw against central differences of sum(dy * y); y is linear in each, so a
    difference is off by rounding alone: 2^-9 of each y, twice, over the step."""
    x, w, dy, off = group_case([20, 0, 44], 64, 48, torch.float16, seed=11)
    ws = gpu_lib.group_workspace(x, w, dy)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    gpu_lib.group_product_dx(dy, w, off, dx, ws)
    gpu_lib.group_product_dw(dy, x, off, dw, ws)

    def f(xx, ww):
        y = torch.empty_like(dy)
        gpu_lib.group_product(xx, ww, off, y, ws)
        return float((y.double() * dy.double()).sum()), \
            float((y.double().abs() * dy.double().abs()).sum())

    # steps of 0, +-1 on values rounded to 1/256, exact in 16 bits
    x8, w8 = (x * 64).round() / 64, (w * 64).round() / 64
    for which, grad in (("x", dx), ("w", dw)):
        if which == "x":
            gpu_lib.group_product_dx(dy, w8, off, grad, ws)
        else:
            gpu_lib.group_product_dw(dy, x8, off, grad, ws)
        step = torch.randint(-1, 2, grad.shape, generator=gen(3), device="cuda").half()
        args = [(x8 + s * step, w8) if which == "x" else (x8, w8 + s * step) for s in (1, -1)]
        (fp, mp), (fm, mm) = (f(*a) for a in args)
        want = float((grad.double() * step.double()).sum())
        mag = float((grad.double().abs() * step.double().abs()).sum())
        assert abs((fp - fm) / 2 - want) <= 2.0 ** -11 * (mp + mm + mag)


# ------------------------------------------------------------------------------- losses
def row_reference(x, targets, temperature=1.0):
    """64-bit log probabilities of the targets (0 in masked rows), softmax, and how far
    off an FP32 evaluation may be: the arguments' rounding (a few units of the largest
    |x|), the exponential (2 ulp) and the sum (at most vocab / 128 + 64 adds in a row)."""
    xd = x.double() / temperature
    keep = targets >= 0
    at = targets.clamp(min=0).long()
    lse = torch.logsumexp(xd, 1)
    lp = torch.where(keep, xd.gather(1, at[:, None])[:, 0] - lse, 0.0)
    p = torch.exp(xd - lse[:, None])
    top = torch.where(xd.isfinite(), xd.abs(), 0.0).amax(1)
    eps = E32 * (4 * top + x.shape[1] / 128 + 80)
    return lp, p, keep, at, eps


def grad_want(p, keep, at, coef):
    g = -coef[:, None] * p
    g[torch.arange(len(p), device=p.device), at] += coef
    g[~keep] = 0
    return g


def pref_reference(x, targets, off, ref, beta, kind, smoothing, mean):
    lp, p, keep, at, eps = row_reference(x, targets)
    o = off.tolist()
    ns = len(o) - 1
    logp = torch.zeros(ns, device="cuda", dtype=torch.float64)
    err = torch.zeros_like(logp)
    per = torch.ones_like(logp)
    for q in range(ns):
        m = keep[o[q]:o[q + 1]]
        if mean:
            per[q] = 1.0 / max(1, int(m.sum()))
        logp[q] = lp[o[q]:o[q + 1]][m].sum() * per[q]
        err[q] = (eps[o[q]:o[q + 1]] + 2 * E32 * lp[o[q]:o[q + 1]].abs())[m].sum() * per[q]
    d = logp - ref.double()
    z = beta * (d[0::2] - d[1::2])
    dz = beta * (err[0::2] + err[1::2]) + E32 * z.abs()
    if kind == 0:
        lpos, lneg = torch.nn.functional.softplus(-z), torch.nn.functional.softplus(z)
        gpos, gneg = -torch.sigmoid(-z), torch.sigmoid(z)
    else:
        lpos, lneg, gpos, gneg = (z - 1) ** 2 / 2, (z + 1) ** 2 / 2, z - 1, z + 1
    loss = ((1 - smoothing) * lpos + smoothing * lneg).mean()
    slope = (1 - smoothing) * gpos + smoothing * gneg
    g = slope * beta / len(z)
    dg = (dz + 8 * E32 * (1 + z.abs())) * abs(beta) / len(z)
    coef = torch.zeros(len(x), device="cuda", dtype=torch.float64)
    dcoef = torch.zeros_like(coef)
    for q in range(ns):
        sign = 1.0 if q % 2 == 0 else -1.0
        coef[o[q]:o[q + 1]] = sign * g[q // 2] * per[q]
        dcoef[o[q]:o[q + 1]] = dg[q // 2] * per[q]
    grad = grad_want(p, keep, at, coef)
    shape = grad_want(p, keep, at, torch.ones_like(coef)).abs()
    gtol = dcoef[:, None] * shape + coef.abs()[:, None] * p * (eps[:, None] + 8 * E32)
    dl = (dz * (1 + z.abs())).mean() + 8 * E32 * loss
    return dict(loss=loss, dl=dl, z=z, dz=dz, logp=logp, err=err, grad=grad, gtol=gtol)


def run_pref(casgd, x, t, off, ref, grad, **kw):
    pairs = (len(off) - 1) // 2
    out = casgd.PreferenceOut.alloc(pairs)
    ws = casgd.preference_workspace(len(x), pairs)
    casgd.preference_loss(x, t, off, ref, grad, out, ws, **kw)
    return out, ws


def check_pref(casgd, x, t, off, ref, dt, beta=0.3, kind=0, smoothing=0.1, mean=False, grad=None,
               **kw):
    grad = torch.full_like(x, 3.0) if grad is None else grad
    want = pref_reference(x, t, off, ref, beta, kind, smoothing, mean)
    out, ws = run_pref(casgd, x, t, off, ref, grad, beta=beta, kind=kind, smoothing=smoothing,
                       mean=mean, **kw)
    close(out.logp, want["logp"], want["err"] + E32 * want["logp"].abs())
    close(out.margin, want["z"], want["dz"])
    close(out.loss, want["loss"][None], want["dl"][None])
    s = kw.get("grad_scale", 1.0)
    close(grad, want["grad"] * s, ULP[dt] * (want["grad"] * s).abs() + want["gtol"] * s + TINY[dt])
    assert casgd.get_status(ws) == 0
    return out, grad


def loss_inputs(rows, vocab, dt, seed=0, spread=2.0, masked=0.2):
    x = (randn(rows, vocab, seed=seed) * spread).to(DT[dt])
    t = torch.randint(0, vocab, (rows,), generator=gen(seed + 1), device="cuda")
    t[torch.rand(rows, generator=gen(seed + 2), device="cuda") < masked] = -100
    return x, t


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("kind,mean", list(itertools.product([0, 1], [False, True])))
def test_preference_kinds(gpu_lib, dt, kind, mean):
    x, t = loss_inputs(60, 777, dt)
    off = offsets_of([7, 9, 0, 12, 20, 12])
    ref = torch.tensor([-40.0, -45, 0.5, -60, -90, -70], device="cuda")
    if mean:
        ref /= 9
    check_pref(gpu_lib, x, t, off, ref, dt, kind=kind, mean=mean, grad_scale=4.0)


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 100, 1000, 8191, 8192, 8193, 20011, 33000, 70001,
                                   131072, 262145])
@pytest.mark.parametrize("dt", DT)
def test_preference_vocabularies(gpu_lib, vocab, dt):
    x, t = loss_inputs(9, vocab, dt, seed=vocab)
    off = offsets_of([2, 3, 3, 1])
    check_pref(gpu_lib, x, t, off, torch.full((4,), -7.0, device="cuda"), dt)


@pytest.mark.parametrize("rows,pairs", [(1, 1), (2, 1), (700, 3), (5000, 40), (3000, 1500)])
def test_preference_lengths(gpu_lib, rows, pairs):
    x, t = loss_inputs(rows, 130, "bf16", seed=rows)
    rng = np.random.default_rng(rows)
    off = offsets_of(rng.multinomial(rows, np.full(2 * pairs, 0.5 / pairs)))
    logp = pref_reference(x, t, off, torch.zeros(2 * pairs, device="cuda"), 1.0, 0, 0.0,
                          False)["logp"]
    ref = (logp + torch.randn(2 * pairs, generator=gen(5), device="cuda")).float()
    check_pref(gpu_lib, x, t, off, ref, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,pad,shift", [(96, 8, 0), (97, 0, 0), (101, 3, 1), (12345, 2, 5),
                                             (40003, 1, 3)])
def test_preference_alignment_and_in_place(gpu_lib, dt, vocab, pad, shift):
    x0, t = loss_inputs(11, vocab, dt)
    off = offsets_of([6, 3])                            # rows 9 and 10: in no sequence
    ref = torch.tensor([-20.0, -21.0], device="cuda")
    x, xbuf = pitched(11, vocab, DT[dt], pad=pad, shift=shift)
    x.copy_(x0)
    grad, gbuf = pitched(11, vocab, DT[dt], pad=pad + 1, shift=shift + 2)
    _, g = check_pref(gpu_lib, x, t, off, ref, dt, grad=grad)
    assert outside_untouched(grad, gbuf) and (g[9:] == 0).all()
    first = grad.clone()
    run_pref(gpu_lib, x, t, off, ref, x, beta=0.3, smoothing=0.1)      # in place
    assert torch.equal(x, first) and outside_untouched(x, xbuf)


def test_preference_masked_rows_hide_everything(gpu_lib):
    """NaN and infinities in masked rows and in rows of no sequence reach nothing; entries
    of -inf (a masked vocabulary) and of the type's lowest value count for nothing."""
    x, t = loss_inputs(12, 300, "bf16", masked=0.0)
    x[:, 250:] = float("-inf")
    x[:, 240:250] = torch.finfo(torch.bfloat16).min
    t = t % 240
    off = offsets_of([5, 5])
    x[2], x[7, :100], x[11] = float("nan"), float("inf"), float("nan")
    t[2], t[7] = -1, -100
    ref = torch.tensor([-20.0, -21.0], device="cuda")
    clean = x.clone()
    clean[2], clean[7, :100], clean[11] = 0, 0, 0
    grad, grad_clean = torch.empty_like(x), torch.empty_like(x)
    a, _ = run_pref(gpu_lib, x, t, off, ref, grad)
    b, _ = run_pref(gpu_lib, clean, t, off, ref, grad_clean)
    for u, v in ((a.loss, b.loss), (a.margin, b.margin), (a.logp, b.logp), (grad, grad_clean)):
        assert torch.isfinite(u).all() and torch.equal(u, v)
    assert (grad[[2, 7, 10, 11]] == 0).all() and (grad[:, 240:] == 0).all()
    check_pref(gpu_lib, clean, t, off, ref, "bf16")
    # a target of probability zero: its log probability and the loss are infinite, the
    # gradient is finite
    t[0] = 299
    a, _ = run_pref(gpu_lib, clean, t, off, ref, grad)
    assert a.logp[0] == float("-inf") and a.loss[0] == float("inf")
    assert torch.isfinite(grad).all() and grad[0, 299] < 0
    # every row masked: log probabilities 0, the loss of the reference alone
    a, _ = run_pref(gpu_lib, x, torch.full_like(t, -100), off, ref, grad, beta=0.5)
    assert (a.logp == 0).all() and (grad == 0).all()
    assert abs(float(a.loss) - np.log1p(np.exp(0.5))) < 1e-6


def test_preference_loss_alone_and_bad_inputs(gpu_lib):
    x, t = loss_inputs(10, 50, "f32")
    off, ref = offsets_of([4, 6]), torch.zeros(2, device="cuda")
    grad = torch.empty_like(x)
    a, _ = run_pref(gpu_lib, x, t, off, ref, grad)
    b, _ = run_pref(gpu_lib, x, t, off, ref, None)
    assert torch.equal(a.loss, b.loss) and torch.equal(a.logp, b.logp)
    t2 = t.clone()
    t2[1] = 50
    grad.fill_(3)
    c, ws = run_pref(gpu_lib, x, t2, off, ref, grad)
    assert gpu_lib.get_status(ws) == 6 and (grad[1] == 0).all()
    t2[1] = -1
    d, _ = run_pref(gpu_lib, x, t2, off, ref, None)
    assert torch.equal(c.logp, d.logp)
    for bad in ([0, 8, 4], [0, 4, 11], [-3, 4, 10]):
        _, ws = run_pref(gpu_lib, x, t, torch.tensor(bad, device="cuda").int(), ref, grad)
        assert gpu_lib.get_status(ws) == 6
    empty = torch.empty(0, 50, device="cuda")
    e, ws = run_pref(gpu_lib, empty, t[:0], offsets_of([0, 0]), ref, torch.empty_like(empty))
    assert (e.logp == 0).all() and gpu_lib.get_status(ws) == 0
    assert abs(float(e.loss) - np.log(2)) < 1e-6


def test_preference_gradient_is_a_difference(gpu_lib):
    """Central differences of the loss along a direction d: off by h^2/6 of the third
    derivative (below 2 |d|_inf^3 (beta n)^3 here) and by the loss's rounding over h."""
    x, t = loss_inputs(24, 90, "f32", seed=8)
    off, ref = offsets_of([5, 7, 12, 0]), torch.tensor([-20.0, -27, -50, 1], device="cuda")
    grad = torch.empty_like(x)
    run_pref(gpu_lib, x, t, off, ref, grad, beta=0.1)
    d = randn(24, 90, seed=9)
    d /= d.norm()
    h = 0.02

    def f(s):
        return float(run_pref(gpu_lib, x + s * d, t, off, ref, None, beta=0.1)[0].loss)

    want = float((grad.double() * d.double()).sum())
    assert abs((f(h) - f(-h)) / (2 * h) - want) <= h * h + 64 * E32 / h


# policy
def policy_reference(x, t, w, old, adv, ref, kl, lo, hi, temp):
    lp, p, keep, at, eps = row_reference(x, t, temp)
    used = keep & (w != 0)
    wd = torch.where(used, w.double(), 0.0)
    q = torch.where(used, lp, 0.0)
    o = torch.where(used, old.double(), 0.0)
    a = torch.where(used, adv.double(), 0.0)
    r = torch.exp(q - o)
    c = r.clamp(1 - lo, 1 + hi)
    inside = torch.where(a >= 0, r <= 1 + hi, r >= 1 - lo)
    L = -torch.minimum(r * a, c * a)
    g = torch.where(inside, -r * a, 0.0)
    k = torch.zeros_like(L)
    if ref is not None:
        away = torch.where(used, ref.double(), 0.0) - q
        k = torch.exp(away) - away - 1
        L = L + kl * k
        g = g - kl * (torch.exp(away) - 1)
        away_abs = away.abs()
    else:
        away_abs = torch.zeros_like(L)
    dlp = eps + 4 * E32 * (lp.abs() + 1)
    amp = (r * a.abs() + kl * (torch.exp(away_abs) + 1)) * (dlp + 8 * E32)
    grad = grad_want(p, keep, at, wd * g / temp)
    shape = grad_want(p, keep, at, torch.ones_like(wd)).abs()
    gtol = (wd.abs() * amp / temp)[:, None] * shape + (wd * g / temp).abs()[:, None] * p * \
        (eps[:, None] + 8 * E32)
    # rows whose ratio lies within rounding of a clip border may fall on either side
    edge = torch.minimum((r - 1 - hi).abs(), (r - 1 + lo).abs()) <= r * (dlp + 8 * E32)
    return dict(stats=[(wd * L).sum(), (wd * k).sum(), (wd * (~inside & used)).sum()],
                dstats=[(wd.abs() * amp).sum() + E32 * (wd * L).abs().sum(),
                        (wd.abs() * (torch.exp(away_abs) + 1) * (dlp + 8 * E32)).sum(),
                        E32 * wd.abs().sum()],
                lp=lp, dlp=dlp, grad=grad, gtol=gtol, edge=edge & used)


def policy_inputs(rows, vocab, dt, seed=0, temp=1.0, masked=0.2):
    x, t = loss_inputs(rows, vocab, dt, seed=seed, masked=masked)
    lp = row_reference(x, t, temp)[0].float()
    return dict(x=x, t=t, old=lp + 0.2 * randn(rows, seed=seed + 5),
                ref=lp + 0.4 * randn(rows, seed=seed + 6), adv=randn(rows, seed=seed + 7),
                w=torch.rand(rows, generator=gen(seed + 8), device="cuda") / rows)


def run_policy(casgd, i, grad, ref=True, **kw):
    out = casgd.PolicyOut.alloc(len(i["x"]))
    ws = casgd.policy_workspace(len(i["x"]))
    casgd.policy_loss(i["x"], i["t"], i["w"], i["old"], i["adv"], grad, out, ws,
                      ref_logp=i["ref"] if ref else None, **kw)
    return out, ws


def check_policy(casgd, i, dt, grad=None, ref=True, kl=0.1, lo=0.2, hi=0.3, temp=1.0, scale=1.0):
    want = policy_reference(i["x"], i["t"], i["w"], i["old"], i["adv"],
                            i["ref"] if ref else None, kl if ref else 0.0, lo, hi, temp)
    assert not want["edge"].any()                       # the inputs keep clear of the borders
    grad = torch.full_like(i["x"], 3.0) if grad is None else grad
    out, ws = run_policy(casgd, i, grad, ref=ref, kl=kl, clip_low=lo, clip_high=hi,
                         temperature=temp, grad_scale=scale)
    close(out.logp, want["lp"], want["dlp"])
    for e in range(3):
        close(out.stats[e], want["stats"][e], want["dstats"][e] + E32 * want["stats"][e].abs())
    close(grad, want["grad"] * scale,
          ULP[dt] * (want["grad"] * scale).abs() + want["gtol"] * scale + TINY[dt])
    assert casgd.get_status(ws) == 0
    return out, grad


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("ref,temp", list(itertools.product([True, False], [1.0, 0.7])))
def test_policy_kinds(gpu_lib, dt, ref, temp):
    check_policy(gpu_lib, policy_inputs(200, 501, dt, temp=temp), dt, ref=ref, temp=temp,
                 scale=16.0)


@pytest.mark.parametrize("vocab", [1, 2, 3, 33, 1000, 8191, 8193, 16385, 32768, 50001, 65537,
                                   131071, 262144, 300001, 600011])
@pytest.mark.parametrize("dt", DT)
def test_policy_vocabularies(gpu_lib, vocab, dt):
    check_policy(gpu_lib, policy_inputs(7, vocab, dt, seed=vocab), dt, scale=8.0)


@pytest.mark.parametrize("rows", [0, 1, 2, 151, 153, 4000])
def test_policy_rows(gpu_lib, rows):
    check_policy(gpu_lib, policy_inputs(rows, 320, "bf16", seed=rows), "bf16")


# many rows for each group of threads that takes them in turn, masked ones between
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,vocab", [(3000, 2100), (2500, 4097), (1500, 9001), (700, 33000),
                                        (500, 128000)])
def test_policy_many_rows(gpu_lib, dt, rows, vocab):
    i = policy_inputs(rows, vocab, dt, seed=rows, masked=0.3)
    ws, out = gpu_lib.policy_workspace(rows), gpu_lib.PolicyOut.alloc(rows)
    grad = torch.empty_like(i["x"])
    for _ in range(3):
        t0 = torch.cuda.Event(enable_timing=True)
        t1 = torch.cuda.Event(enable_timing=True)
        t0.record()
        gpu_lib.policy_loss(i["x"], i["t"], i["w"], i["old"], i["adv"], grad, out, ws,
                            ref_logp=i["ref"], kl=0.1, clip_low=0.2, clip_high=0.3)
        t1.record()
    assert gpu_lib.get_status(ws) == 0
    assert t0.elapsed_time(t1) < 200                    # no wait ran into its bound (1 s)
    stats, logp, first = out.stats.clone(), out.logp.clone(), grad.clone()
    lp, p, keep, at, eps = row_reference(i["x"], i["t"])
    close(logp, lp, eps + 4 * E32 * (lp.abs() + 1))
    # rows of the gradient sum to zero up to their rounding, and none is left unwritten
    assert torch.isfinite(first).all() and (first[~keep] == 0).all()
    mag = first.double().abs().sum(1)
    bound = (ULP[dt] + eps + 8 * E32) * mag + vocab * TINY[dt]
    assert (first.double().sum(1).abs() <= bound).all()
    again, _ = run_policy(gpu_lib, i, grad.zero_(), kl=0.1, clip_low=0.2, clip_high=0.3)
    assert torch.equal(grad, first) and torch.equal(again.logp, logp)   # the same bits
    assert torch.equal(again.stats, stats)
    run_policy(gpu_lib, i, i["x"], kl=0.1, clip_low=0.2, clip_high=0.3)        # in place
    assert torch.equal(i["x"], first)
    assert torch.isfinite(stats).all()


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("vocab,pad,shift", [(96, 8, 0), (97, 0, 0), (101, 3, 1), (12345, 2, 5),
                                             (70003, 1, 3)])
def test_policy_alignment_and_in_place(gpu_lib, dt, vocab, pad, shift):
    i = policy_inputs(11, vocab, dt)
    x, xbuf = pitched(11, vocab, DT[dt], pad=pad, shift=shift)
    x.copy_(i["x"])
    i["x"] = x
    grad, gbuf = pitched(11, vocab, DT[dt], pad=pad + 1, shift=shift + 2)
    check_policy(gpu_lib, i, dt, grad=grad)
    assert outside_untouched(grad, gbuf)
    run_policy(gpu_lib, i, x, kl=0.1, clip_low=0.2, clip_high=0.3)
    assert torch.equal(x, grad) and outside_untouched(x, xbuf)


def test_losses_long_offsets(gpu_lib):
    """Element offsets past 2^31 in the logits and the gradient: the last rows are those of
    a small call on them alone."""
    rows, vocab, few = 16500, 131072, 6
    i = policy_inputs(few, vocab, "bf16", seed=2, masked=0.0)
    x = torch.zeros(rows, vocab, device="cuda", dtype=torch.bfloat16)
    x[-few:] = i["x"]
    big = {"x": x, "t": torch.full((rows,), -1, device="cuda")}
    big["t"][-few:] = i["t"]
    for key in ("old", "ref", "adv", "w"):
        big[key] = torch.zeros(rows, device="cuda")
        big[key][-few:] = i[key]
    small = torch.empty_like(i["x"])
    a, _ = run_policy(gpu_lib, i, small, kl=0.1)
    b, _ = run_policy(gpu_lib, big, x, kl=0.1)                           # in place
    assert torch.equal(b.logp[-few:], a.logp) and torch.equal(b.stats, a.stats)
    assert torch.equal(x[-few:], small) and not x[:-few].any()
    x[-few:] = i["x"]
    off, ref = offsets_of([rows - few, few // 2, few - few // 2, 0]), torch.zeros(4, device="cuda")
    off_small = offsets_of([0, few // 2, few - few // 2, 0])
    c, _ = run_pref(gpu_lib, i["x"], i["t"], off_small, ref, small)
    d, _ = run_pref(gpu_lib, x, big["t"], off, ref, x)
    assert torch.equal(c.logp, d.logp) and torch.equal(c.loss, d.loss)
    assert torch.equal(x[-few:], small) and not x[:-few].any()


def test_policy_rows_of_weight_zero(gpu_lib):
    """A masked row is not read; a row of weight zero is, for its log probability, but
    nothing of it reaches the sums or the gradient."""
    i = policy_inputs(20, 400, "bf16", masked=0.0)
    i["t"][3], i["w"][5], i["w"][6] = -1, 0.0, 0.0
    clean = {k: v.clone() for k, v in i.items()}
    i["x"][3], i["old"][3], i["adv"][3] = float("nan"), float("nan"), float("inf")
    i["x"][5, 7], i["x"][6, :] = float("inf"), float("nan")
    i["old"][5], i["adv"][5], i["ref"][6] = float("nan"), float("inf"), float("nan")
    grad, grad_clean = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    a, _ = run_policy(gpu_lib, i, grad, kl=0.1)
    b, _ = run_policy(gpu_lib, clean, grad_clean, kl=0.1)
    assert torch.equal(a.stats, b.stats) and torch.equal(grad, grad_clean)
    assert torch.isfinite(grad).all() and (grad[[3, 5, 6]] == 0).all()
    assert a.logp[3] == 0
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[[5, 6]] = False
    assert torch.equal(a.logp[keep], b.logp[keep])
    c, _ = run_policy(gpu_lib, clean, None, kl=0.1)
    assert torch.equal(c.stats, b.stats) and torch.equal(c.logp, b.logp)
    clean["t"][0] = 400
    _, ws = run_policy(gpu_lib, clean, grad, kl=0.1)
    assert gpu_lib.get_status(ws) == 6 and (grad[0] == 0).all()


def test_policy_gradient_is_a_difference(gpu_lib):
    i = policy_inputs(30, 80, "f32", seed=4)
    grad = torch.empty_like(i["x"])
    run_policy(gpu_lib, i, grad, kl=0.1, clip_low=0.2, clip_high=0.3)
    d = randn(30, 80, seed=9)
    d /= d.norm()
    h = 0.002

    def f(s):
        j = dict(i, x=i["x"] + s * d)
        return float(run_policy(gpu_lib, j, None, kl=0.1, clip_low=0.2,
                                clip_high=0.3)[0].stats[0])

    # no row crosses a clip border within h: |d lp| <= 2 h, and the borders are further
    want = policy_reference(i["x"], i["t"], i["w"], i["old"], i["adv"], i["ref"], 0.1, 0.2, 0.3,
                            1.0)
    r = torch.exp(want["lp"] - i["old"].double())
    assert ((r - 0.8).abs() > 3 * h).all() and ((r - 1.3).abs() > 3 * h).all()
    slope = float((grad.double() * d.double()).sum())
    assert abs((f(h) - f(-h)) / (2 * h) - slope) <= h * h + 8 * E32 / h


# ------------------------------------------------------------------------------ streams
def test_another_stream(gpu_lib):
    s = torch.cuda.Stream()
    x, t = loss_inputs(64, 5000, "bf16")
    i = policy_inputs(64, 5000, "bf16")
    grad, g2 = torch.empty_like(x), torch.empty_like(x)
    a, _ = run_policy(gpu_lib, i, grad, kl=0.1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out = gpu_lib.PolicyOut.alloc(64)
        ws = gpu_lib.policy_workspace(64)
        gpu_lib.policy_loss(i["x"], i["t"], i["w"], i["old"], i["adv"], g2, out, ws,
                            ref_logp=i["ref"], kl=0.1)
    s.synchronize()
    assert torch.equal(grad, g2) and torch.equal(a.stats, out.stats)
    out2 = gpu_lib.PolicyOut.alloc(64)
    torch.cuda.synchronize()
    gpu_lib.policy_loss(i["x"], i["t"], i["w"], i["old"], i["adv"], g2.zero_(), out2, ws,
                        ref_logp=i["ref"], kl=0.1, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(grad, g2)


# rows whose scaled logits leave FP32
FAR_COLS = [1, 5, 2048, 2049, 33000]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("vocab", FAR_COLS)
def test_policy_rows_of_the_lowest_value(gpu_lib, dt, vocab):
    """Rows (0) of the type's lowest value, a vocabulary masked whole: uniform; (1) with one
    logit of the type's largest value, the target: certain; (2) whose target alone is
    lowest: its log probability is that value (to rounding) and its gradient zero.  Powers
    of two and exponentials of zero are exact, sums of ones too: what is left is the
    logarithm (2 ulp) and its product."""
    low, top = torch.finfo(DT[dt]).min, torch.finfo(DT[dt]).max
    x = randn(3, vocab, seed=5).to(DT[dt])
    x[0] = low
    t = torch.tensor([vocab // 2, vocab - 1, 0], device="cuda")
    x[1, vocab - 1], x[2, 0] = top, low
    one = torch.ones(3, device="cuda")
    logv = float(np.log(vocab))
    i = dict(x=x, t=t, w=one.clone(), old=torch.tensor([-logv, 0.0, 0.0], device="cuda"),
             adv=one)
    grad = torch.full_like(x, 3.0)
    out, ws = run_policy(gpu_lib, i, grad, ref=False)
    assert abs(float(out.logp[0]) + logv) <= 4 * E32 * (logv + 1)
    assert float(out.logp[1]) == 0
    if vocab > 1:
        lse = float(torch.logsumexp(x[2, 1:].double(), 0))
        want = low - lse
        assert abs(float(out.logp[2]) - want) <= 4 * E32 * abs(want) + 8 * E32 * (1 + abs(lse))
    want = torch.full((vocab,), 1.0 / vocab, device="cuda", dtype=torch.float64)
    want[vocab // 2] -= 1.0
    close(grad[0], want, ULP[dt] * want.abs() + 16 * E32 * (logv + 1) * want.abs() + TINY[dt] + E32)
    assert float(grad[1].float().abs().max()) == 0
    if vocab > 1:
        assert float(grad[2].float().abs().max()) == 0
    assert gpu_lib.get_status(ws) == 0


@pytest.mark.parametrize("vocab", FAR_COLS)
def test_policy_low_temperature(gpu_lib, vocab):
    """Logits over a temperature of 2e-38 leave FP32: equal ones are uniform still, and the
    larger of two is certain."""
    x = torch.full((2, vocab), 30.0, device="cuda")
    x[1] = 25.0
    x[1, vocab // 3] = 30.0
    t = torch.full((2,), vocab // 3, device="cuda")
    one = torch.ones(2, device="cuda")
    out, _ = run_policy(gpu_lib, dict(x=x, t=t, w=one, old=-one, adv=one), None, ref=False,
                        temperature=2e-38)
    logv = float(np.log(vocab))
    assert abs(float(out.logp[0]) + logv) <= 4 * E32 * (logv + 1)
    assert float(out.logp[1]) == 0


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("vocab", FAR_COLS)
def test_preference_rows_of_the_lowest_value(gpu_lib, dt, vocab):
    """Three uniform rows against one (all logits of the type's lowest value)."""
    x = torch.full((4, vocab), torch.finfo(DT[dt]).min, device="cuda", dtype=DT[dt])
    t = torch.full((4,), vocab - 1, device="cuda")
    off = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    ref = torch.zeros(2, device="cuda")
    grad = torch.full_like(x, 3.0)
    out, ws = run_pref(gpu_lib, x, t, off, ref, grad, beta=0.25, kind=0, smoothing=0.0)
    logv = float(np.log(vocab))
    tol = 16 * E32 * (logv + 1)
    assert abs(float(out.logp[0]) + 3 * logv) <= tol
    assert abs(float(out.logp[1]) + logv) <= tol
    assert abs(float(out.margin) + 0.5 * logv) <= tol
    g = -0.25 / (1 + np.exp(-0.5 * logv))               # d loss / d logp, z = -log(V) / 2
    shape = torch.full((4, vocab), -1.0 / vocab, device="cuda", dtype=torch.float64)
    shape[:, vocab - 1] += 1.0
    want = g * shape
    want[3] *= -1
    close(grad, want, (ULP[dt] + tol) * want.abs() + E32 + TINY[dt])
    assert gpu_lib.get_status(ws) == 0


@pytest.mark.parametrize("vocab", [40, 3000])
@pytest.mark.parametrize("adv", [1.0, -1.0])
def test_policy_keeps_nan(gpu_lib, vocab, adv):
    """A row whose ratio is no number (a NaN logit; -inf less -inf) shows in the sums and in
    its own gradient, and nowhere else."""
    i = policy_inputs(6, vocab, "f32", masked=0.0)
    i["adv"][:] = adv
    i["t"][4] = 1
    clean = torch.empty_like(i["x"])
    run_policy(gpu_lib, i, clean, ref=False)
    for row, set_ in ((2, lambda: i["x"][2].index_fill_(0, torch.tensor([7], device="cuda"),
                                                        float("nan"))),
                      (4, lambda: (i["x"][4, 1:2].fill_(float("-inf")),
                                   i["old"][4:5].fill_(float("-inf"))))):
        keep = {k: v.clone() for k, v in i.items()}
        set_()
        grad = torch.empty_like(clean)
        out, _ = run_policy(gpu_lib, i, grad, ref=False)
        assert out.stats[0].isnan() and grad[row].isnan().all()
        others = [r for r in range(6) if r != row]
        assert torch.equal(grad[others], clean[others])
        i = keep


def test_group_sums_of_long_depth(gpu_lib):
    """Tiles whose sums take longer than a wait between stages: one product 2^29 deep, and
    a weight gradient over 2^28 rows and a ragged end.  Few terms are not zero, so the sums
    are exact."""
    k = (1 << 29) + 8
    x = torch.zeros(1, k, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(1, 1, k, device="cuda", dtype=torch.bfloat16)
    y = torch.empty(1, 1, device="cuda", dtype=torch.bfloat16)
    for j, at in enumerate([0, 63, 64, 1 << 28, k - 9, k - 1]):
        x[0, at], w[0, 0, at] = 1.0, 2.0 ** j
    off = offsets_of([1])
    ws = gpu_lib.group_workspace(x, w, y)
    gpu_lib.group_product(x, w, off, y, ws)
    assert gpu_lib.get_status(ws) == 0
    assert float(y) == 63.0
    del x, w
    rows = (1 << 28) + 5
    x = torch.zeros(rows, 8, device="cuda", dtype=torch.bfloat16)
    dy = torch.zeros(rows, 8, device="cuda", dtype=torch.bfloat16)
    for j, at in enumerate([0, 63, 1 << 27, rows - 6, rows - 1]):
        x[at, 3], dy[at, 5] = 1.0, 2.0 ** j
    dw = torch.full((1, 8, 8), 9.0, device="cuda", dtype=torch.bfloat16)
    ws = gpu_lib.group_workspace(x, dw, dy)
    gpu_lib.group_product_dw(dy, x, offsets_of([rows]), dw, ws)
    assert gpu_lib.get_status(ws) == 0
    want = torch.zeros_like(dw)
    want[0, 5, 3] = 31.0
    assert torch.equal(dw, want)
