"""Token statistics where calls change their team: rows and vocabularies around
the numbers at which a row goes to a wave, a workgroup of another size or to
several workgroups, and rows in which whole waves or workgroups find nothing.
Bounds as in test_gpu_token_stats.py, the formulas in 64 bits."""

import pytest
import torch

import training_reference as R
from conftest import gpu_available
from test_gpu_token_stats import Stats, backward_reference, check, dev, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

PER_VEC = {torch.float32: 4, torch.bfloat16: 8, torch.float16: 8}
TYPES = [torch.float32, torch.bfloat16, torch.float16]


# vectors of 16 bytes in a row: up to 256 a wave's, up to 1024 and 4096 a workgroup's of other sizes
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vecs", [(33, 256), (33, 257), (127, 1024), (127, 1025), (255, 1025), (256, 1025), (127, 4097),
                                       (128, 4096), (128, 4097), (255, 4097), (1023, 257), (1024, 256), (1025, 257),
                                       (1024, 1025)])
def test_where_the_team_changes(rows, vecs, dtype):
    vocab = vecs * PER_VEC[dtype] + vecs % 3
    x, y = make(rows, vocab, dtype, rows + vecs, pad=vecs % 5)
    check(x, y, 0.9, 20, f"{rows} {vocab}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(5, 3000), (3, 40000), (200, 40000), (1030, 9000)])
@pytest.mark.parametrize("k", [1, 6, 64])
def test_candidates_in_few_places(rows, vocab, k, dtype):
    """Rows masked but for a few elements: at the ends, together, far apart, and one alone."""
    gen = torch.Generator().manual_seed(rows + k)
    full = torch.randn(rows, vocab, generator=gen).to(dtype)
    x = torch.full((rows, vocab), -torch.inf, dtype=dtype)
    y = torch.zeros(rows, dtype=torch.int64)
    for r in range(rows):
        kind = r % 5
        if kind == 0:
            at = torch.tensor([0, vocab - 1])
        elif kind == 1:
            at = torch.arange(vocab - 9, vocab)
        elif kind == 2:
            at = torch.randperm(vocab, generator=gen)[:k + 1]
        elif kind == 3:
            at = torch.tensor([vocab // 2])
        else:
            at = torch.arange(vocab // 3, vocab // 3 + 100)
        x[r, at] = full[r, at]
        y[r] = at[r % len(at)]
    check(x.to(dev()), y.to(dev()), 1.0, k, f"{rows} {vocab}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [0, 1, 3, 7])
def test_views_that_begin_anywhere(offset, dtype):
    """Rows whose first element is not on 16 bytes, next to others' data that must not count."""
    rows, vocab = 70, 5003
    wide = torch.full((rows, vocab + 16), 99.0, dtype=dtype, device=dev())
    x, y = make(rows, vocab, dtype, offset)
    view = wide[:, offset:offset + vocab]
    view.copy_(x)
    st = check(view, y, 1.0, 9, f"offset {offset}")
    import hash_table_cache_amd as H

    apart = H.token_stats(x, y, 9)
    assert torch.equal(st.top_ids, apart.top_ids)
    g = torch.randn(rows, device=dev())
    grad = torch.full_like(wide, 5.0)
    H.token_stats_backward(view, y, st.lse, st.entropy, g, g, grad_out=grad[:, offset:offset + vocab])
    assert bool((grad[:, :offset] == 5.0).all()) and bool((grad[:, offset + vocab:] == 5.0).all())
    want = H.token_stats_backward(view.clone(), y, st.lse, st.entropy, g, g)
    assert torch.equal(grad[:, offset:offset + vocab].nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype,vocab", [(torch.float32, 257 * 4), (torch.bfloat16, 513 * 8), (torch.float16, 64 * 8 + 5),
                                         (torch.float16, 40009)])
def test_backward_where_the_team_changes(dtype, vocab):
    import hash_table_cache_amd as H

    gen = torch.Generator().manual_seed(vocab)
    x = (torch.randn(130, vocab, generator=gen) * 3).to(dtype).to(dev())
    y = torch.randint(0, vocab, (130,), generator=gen).to(dev())
    g, ge = torch.randn(130, generator=gen), torch.randn(130, generator=gen)
    st = H.token_stats(x, y, temperature=1.25)
    ref, tol = backward_reference(x, y, 1.25, st.lse, st.entropy, g, ge)
    got = H.token_stats_backward(x, y, st.lse, st.entropy, g.to(dev()), ge.to(dev()), temperature=1.25)
    R.assert_near(got, ref, tol, f"{vocab}")


def test_offsets_past_32_bits():
    """Rows that begin past 2^32 elements, in a buffer of wide rows."""
    import hash_table_cache_amd as H

    stride, rows, vocab = (1 << 31) + 8, 4, 1003
    if torch.cuda.mem_get_info()[0] < 3 * stride * 2 + (1 << 32):
        pytest.skip("not enough memory")
    buffer = torch.empty(3 * stride + vocab, dtype=torch.bfloat16, device=dev())
    view = buffer.as_strided((rows, vocab), (stride, 1))
    x, y = make(rows, vocab, torch.bfloat16, 3)
    view.copy_(x)
    st = check(view, y, 1.0, 5, "far")
    assert torch.equal(st.top_ids.cpu(), Stats(x, y, 1.0, 5).ids)
    g = torch.randn(rows, device=dev())
    want = H.token_stats_backward(x, y, st.lse, st.entropy, g, g)
    H.token_stats_backward(view, y, st.lse, st.entropy, g, g, grad_out=view)
    assert torch.equal(view, want)


def test_the_same_row_many_times():
    """A call gives the same bits again, and so do equal rows that begin alike: sums go by vectors from a
    row's first 16-byte boundary on, so that their order is another where that lies elsewhere in the row."""
    import hash_table_cache_amd as H

    for rows, vocab, dtype in ((64, 131072, torch.bfloat16), (300, 20011, torch.float32), (2000, 700, torch.float16)):
        x, y = make(1, vocab, dtype, 5)
        x, y = x.repeat(rows, 1), y.repeat(rows)
        a, b = H.token_stats(x, y, 30), H.token_stats(x, y, 30)
        alike = torch.arange(rows, device=dev()) * vocab * x.element_size() % 16 == 0
        for p, q in zip(a, b):
            assert torch.equal(p, q) and torch.equal(p[alike], p[:1].expand_as(p[alike]))
