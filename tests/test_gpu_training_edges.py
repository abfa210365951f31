"""Calls at the edges of what token statistics, orthogonalisation and the
momentum update allow: nothing to do, views of odd strides, one matrix read
twice, several calls at once, no learning rate."""

import pytest
import torch

import polar_reference as P
import training_reference as R
from conftest import gpu_available
from test_gpu_orthogonalize import make
from test_gpu_token_stats import check, dev
from test_gpu_token_stats import make as make_logits

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def test_lists_of_empty_matrices():
    import hash_table_cache_amd as H

    us = [torch.zeros(0, 5, device=dev()), torch.zeros(7, 0, device=dev(), dtype=torch.bfloat16)]
    got = H.orthogonalize(us)
    assert [tuple(g.shape) for g in got] == [(0, 5), (7, 0)]
    H.muon_update(us, us, [torch.zeros(u.shape, device=dev()) for u in us], 0.1)


def test_strides_that_do_not_matter():
    """A single row or column may have any stride across it."""
    import hash_table_cache_amd as H

    row = make(1, 50, torch.float32, 1)
    for u in (row.t()[:, :1] if row.t().stride(1) == 1 else row.t().as_strided((50, 1), (1, 50)),
              row.as_strided((1, 50), (3, 1)), make(9, 50, torch.float32, 2)[:, 7:8], make(9, 50, torch.float32, 2)[4:5]):
        P.assert_polar(H.orthogonalize([u])[0], R.f64(u), what=f"{tuple(u.shape)} {u.stride()}")


def test_one_matrix_read_twice():
    """The same input may appear again where no result goes into it, and gives the same bits."""
    import hash_table_cache_amd as H

    u = make(100, 200, torch.bfloat16, 3)
    a, b = H.orthogonalize([u, u])
    assert torch.equal(a, b)
    w = [make(100, 200, torch.float32, i) for i in (4, 5)]
    m = [torch.zeros(100, 200, device=dev()) for _ in w]
    alone = w[1].clone()
    H.muon_update(w, [u, u], m, [0.1, 0.2])
    H.muon_update([alone], [u], [torch.zeros(100, 200, device=dev())], 0.2)
    assert torch.equal(w[1], alone) and torch.equal(m[0], m[1])


def test_no_learning_rate():
    """lr = 0 moves the momentum and leaves the weights' bits."""
    import hash_table_cache_amd as H

    for shape in ((30, 40), (300, 500)):
        w, g, m = make(*shape, torch.bfloat16, 1), make(*shape, torch.bfloat16, 2), torch.zeros(shape, device=dev())
        before = w.clone()
        H.muon_update([w], [g], [m], 0.0, weight_decay=0.3)
        assert torch.equal(w, before) and bool(m.any())


def test_gradients_that_are_not_finite():
    """A bad gradient makes its own matrix NaN, none of the others of the call."""
    import hash_table_cache_amd as H

    shapes = [(40, 60), (50, 700), (300, 200), (40, 60), (300, 200)]
    w = [make(*s, torch.float32, i) for i, s in enumerate(shapes)]
    g = [make(*s, torch.float32, 10 + i) for i, s in enumerate(shapes)]
    keep = [x.clone() for x in w]
    for i, v in ((0, torch.nan), (1, torch.inf), (2, -torch.inf)):
        g[i][3, 4] = v
    m = [torch.zeros(s, device=dev()) for s in shapes]
    H.muon_update(w, g, m, 0.1)
    for i in range(3):
        assert bool(w[i].isnan().all())
    clean = [keep[3].clone(), keep[4].clone()]
    H.muon_update(clean, g[3:], [torch.zeros(s, device=dev()) for s in shapes[3:]], 0.1)
    for a, b in zip(clean, w[3:]):
        P.assert_close(a, R.f64(b), 1e-5 * float(b.norm()), "beside bad ones")


def test_many_calls_at_once():
    """Calls of every way on streams of their own, all under way together, each as alone."""
    import hash_table_cache_amd as H

    x, y = make_logits(90, 50021, torch.bfloat16, 6)
    z, v = make_logits(2000, 3001, torch.float32, 7)
    small, long = [make(60, 90, torch.bfloat16, 8)] * 3, [make(100, 4000, torch.float32, 9)]
    wide = [make(50, 5000, torch.float32, 10)]
    calls = [lambda s: H.token_stats(x, y, 12, stream=s), lambda s: H.orthogonalize(small, stream=s),
             lambda s: H.token_stats(z, v, 3, stream=s), lambda s: H.orthogonalize(long, stream=s),
             lambda s: H.orthogonalize(wide, stream=s)]
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = [c(s) for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for p, q in zip(a, b):
                assert torch.equal(p.nan_to_num(7.0), q.nan_to_num(7.0))


def test_labels_and_logits_of_one_column():
    import hash_table_cache_amd as H

    for dtype in (torch.float32, torch.float16):
        x, y = make_logits(25, 1, dtype, 3)
        check(x, y, 1.0, 64, "one column")
    with pytest.raises(ValueError, match="no columns"):
        H.token_stats(torch.zeros(3, 0, device=dev()), torch.zeros(3, dtype=torch.int64, device=dev()))


def test_refusals_of_views_and_types():
    import hash_table_cache_amd as H

    u = make(8, 9, torch.float32, 1)
    for bad, kind in ((u[0], ValueError), (u[:, ::2], ValueError), (u.double(), TypeError), (u[None], ValueError)):
        with pytest.raises(kind):
            H.orthogonalize([bad])
    with pytest.raises(H.HkvError):
        H.orthogonalize([u], out=[torch.empty(8, 9)])  # not the GPU's memory
    with pytest.raises(ValueError, match="is"):
        H.orthogonalize([u], out=[torch.empty(9, 8, device=dev())])
