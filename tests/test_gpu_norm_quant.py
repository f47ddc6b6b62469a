"""idx_add_rmsnorm_quant against 64 bits: types, widths, groups, strides, empty and zero
rows, and the refusals of the binding."""
import pytest
import torch

import _serve_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def idx():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_indexer_tiles_gb300 as pkg
    return pkg


def inputs(rows, cols, dtype, residual, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * 3).to(dtype)
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(dtype)
    r = (torch.randn(rows, cols, generator=g) * 2).to(dtype) if residual else None
    return x, w, r


def run(idx, x, w, r=None, **kw):
    ro = torch.empty_like(r, device=DEV) if r is not None else None
    out, scale = idx.idx_add_rmsnorm_quant(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV),
                                           residual_out=ro, **kw)
    torch.cuda.synchronize()
    return out.cpu(), scale.cpu(), None if ro is None else ro.cpu()


@pytest.mark.parametrize("cols", [1, 7, 8, 64, 100, 128, 129, 250, 256, 1000, 1024, 1032, 2048, 4096,
                                  5000, 8192, 8200, 16384, 16392, 32768])
@pytest.mark.parametrize("dtype,residual", [(BF16, True), (FP16, False), (FP32, True)])
def test_widths(idx, cols, dtype, residual):
    x, w, r = inputs(5, cols, dtype, residual, seed=cols)
    out, scale, ro = run(idx, x, w, r)
    ref.check_norm(out, scale, x, w, r, ro)


@pytest.mark.parametrize("cols", [154, 926, 1500, 2052, 4500, 5003, 6146, 7999, 12345])
@pytest.mark.parametrize("dtype,residual", [(BF16, True), (FP16, True), (FP32, False)])
def test_many_rows_of_odd_widths(idx, cols, dtype, residual):
    """More row groups than blocks: every block takes several, one ahead."""
    rows = 3000 if cols < 3000 else 1300
    x, w, r = inputs(rows, cols, dtype, residual, seed=cols)
    out, scale, ro = run(idx, x, w, r)
    ref.check_norm(out, scale, x, w, r, ro)


@pytest.mark.parametrize("cols,group", [(128, 0), (256, 64), (1024, 32), (2048, 128), (4096, 0), (5120, 128), (6144, 0),
                                        (8192, 128), (16384, 32)])
def test_many_rows_in_vectors(idx, cols, group):
    rows = 30001 if cols < 512 else 2500
    x, w, r = inputs(rows, cols, BF16, True, seed=cols + group)
    out, scale, ro = run(idx, x, w, r, group=group)
    ref.check_norm(out, scale, x, w, r, ro, group=group)


@pytest.mark.parametrize("rows", [1, 2, 9, 131, 3001])
@pytest.mark.parametrize("cols,group", [(128, 0), (128, 128), (384, 128), (64, 64), (96, 32), (4096, 128), (7168, 64)])
def test_rows_and_groups(idx, rows, cols, group):
    x, w, r = inputs(rows, cols, BF16, rows % 2 == 1, seed=rows + cols)
    out, scale, ro = run(idx, x, w, r, group=group)
    ref.check_norm(out, scale, x, w, r, ro, group=group)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("start,cols,wide", [(0, 128, 576), (512, 64, 576), (3, 100, 259), (8, 2048, 2063)])
def test_column_slices(idx, dtype, start, cols, wide):
    """x is a slice of a wider projection, on and off the vector path's alignment."""
    x, _, _ = inputs(37, wide, dtype, False, seed=wide)
    _, w, _ = inputs(1, cols, dtype, False, seed=cols)
    d = x.to(DEV)[:, start:start + cols]
    out, scale = idx.idx_add_rmsnorm_quant(d, w.to(DEV))
    torch.cuda.synchronize()
    ref.check_norm(out.cpu(), scale.cpu(), x[:, start:start + cols], w)


def test_residual_in_place_and_no_residual_out(idx):
    x, w, r = inputs(33, 512, BF16, True, seed=1)
    d = r.to(DEV)
    a, sa = idx.idx_add_rmsnorm_quant(x.to(DEV), w.to(DEV), residual=d)
    assert torch.equal(d.cpu(), r)
    b, sb = idx.idx_add_rmsnorm_quant(x.to(DEV), w.to(DEV), residual=d, residual_out=d)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(sa, sb)
    ref.check_norm(b.cpu(), sb.cpu(), x, w, r, d.cpu())


def test_zero_rows_have_a_positive_scale(idx):
    x, w, _ = inputs(6, 256, BF16, False, seed=2)
    x[2] = 0
    x[4, 128:] = 0
    for group in (0, 128):
        out, scale, _ = run(idx, x, w, group=group)
        ref.check_norm(out, scale, x, w, group=group)
        assert (out[2].float() == 0).all()


def test_a_row_that_is_not_finite_leaves_the_others(idx):
    x, w, _ = inputs(64, 128, BF16, False, seed=3)
    clean = run(idx, x, w)
    for bad in (float("inf"), float("nan")):
        y = x.clone()
        y[7, 5] = bad
        out, scale, _ = run(idx, y, w)
        keep = torch.arange(64) != 7
        assert torch.equal(out.view(torch.uint8)[keep], clean[0].view(torch.uint8)[keep])
        assert torch.equal(scale[keep], clean[1][keep])


def test_eps_of_small_rows(idx):
    x, w, _ = inputs(4, 128, FP32, False, seed=4)
    x *= 1e-4
    for eps in (0.0, 1e-6, 1e-3):
        out, scale, _ = run(idx, x, w, eps=eps)
        ref.check_norm(out, scale, x, w, eps=eps)


def test_feeds_the_scorer(idx):
    """k and k_scale of normed index keys, as idx_score_materialise reads them."""
    import oracle
    import synth
    x, w, _ = inputs(500, 128, BF16, False, seed=5)
    k, k_scale, _ = run(idx, x, w)
    inp = synth.indexer_inputs(4, 500, 16, 128, 32, "fp8", seed=6)
    inp.k, inp.k_scale = k, k_scale
    got = idx.idx_score_materialise(*(getattr(inp, n).to(DEV) for n in ("q", "k", "k_scale", "w", "ks", "ke")))
    torch.cuda.synchronize()
    _, sc = oracle.score_topk(inp, want_scores=True)
    from _checks import check_scores
    for r in range(4):
        n = int(inp.ke[r] - inp.ks[r])
        check_scores(got[r, :n].cpu().numpy(), sc[r, :n])


def test_other_stream_and_no_rows(idx):
    x, w, r = inputs(64, 640, BF16, True, seed=7)
    want = run(idx, x, w, r)
    d = [t.to(DEV) for t in (x, w, r)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, scale = idx.idx_add_rmsnorm_quant(d[0], d[1], residual=d[2], stream=s)
    s.synchronize()
    assert torch.equal(out.cpu().view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(scale.cpu(), want[1])
    out, scale = idx.idx_add_rmsnorm_quant(d[0][:0], d[1], residual=d[2][:0])
    assert out.shape == (0, 640) and scale.shape == (0,)


def test_refusals(idx):
    x = torch.zeros(4, 64, dtype=BF16, device=DEV)
    w = torch.zeros(64, dtype=BF16, device=DEV)
    call = idx.idx_add_rmsnorm_quant
    for bad in (lambda: call(x, w.float()), lambda: call(x, w[:32]), lambda: call(x.t(), w),
                lambda: call(x, w, group=48), lambda: call(x, w, residual=x[:2]),
                lambda: call(x.cpu(), w), lambda: call(x.to(torch.float64), w.to(torch.float64)),
                lambda: call(x, w, out=torch.empty(4, 64, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(idx.IdxError) as e:
        call(x, w, eps=-1.0)
    assert e.value.code == 1
    with pytest.raises(idx.IdxError) as e:
        call(x, w, group=16)
    assert e.value.code == 1
    wide = torch.zeros(1, 32776, dtype=BF16, device=DEV)
    with pytest.raises(idx.IdxError) as e:
        call(wide, wide[0])
    assert e.value.code == 4
