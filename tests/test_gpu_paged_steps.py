"""Steps of a PagedCache that a server meets at its edges (needs a B200): without rows, idle, of many
sizes, on a stream beside the one that made the tensors."""
import pytest
import torch

import paged_util as U
from gpu_util import load_kivi
from test_gpu_paged import BF16, gen_of, ints, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kivi():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    return load_kivi()


def small_cache(K, **kw):
    return K.PagedCache(**{**dict(num_pages=64, page_size=16, num_layers=1, num_kv_heads=2,
                                  num_q_heads=4, head_dim=64, max_requests=3, max_tokens=256), **kw})


def step(cache, gen, new, pad=0, **kw):
    """One step of the given new tokens; what was appended, and the output's rows."""
    rows = sum(n for n in new if n > 0) + pad
    cache.assign(ints(new), rows, **kw)
    q, k, v = (randn(gen, rows, h, 64) for h in (4, 2, 2))
    cache.append(0, k, v)
    return q, k, v, cache.attend(0, q)


@pytest.mark.parametrize("largest", [False, True])
def test_steps_without_rows(kivi, largest):
    """Idle and release-only steps between others, with max_new given as the largest of the step's."""
    gen, cache = gen_of(51), small_cache(kivi)
    kw = lambda new: {"max_new": max(new)} if largest else {}  # noqa: E731
    first = step(cache, gen, [40, 9, 70], **kw([40, 9, 70]))
    for new, pad in (([0, 0, 0], 0), ([-1, 0, -1], 0), ([0, 0, 0], 3), ([-1, 0, -1], 2)):
        out = step(cache, gen, new, pad, **kw(new))[3]
        assert out.shape == (pad, 4, 64)
        assert cache.offsets.tolist() == [0] * 4
    assert cache.lengths.tolist() == [0, 9, 0] and cache.num_free.item() == 63
    q, k, v, out = step(cache, gen, [0, 1, 0], max_new=1)
    keys, values = (torch.cat([first[i][40:49], x]) for i, x in ((1, k), (2, v)))
    U.assert_close(out, *U.attend(q, keys, values), "the request that stayed")
    assert cache.check_device_status() == 0


def test_steps_of_many_sizes_hold_little_memory(kivi):
    """Slots and positions of every number of rows up to 200: few buffers, whose addresses stay."""
    cache, at, seen = small_cache(kivi), {}, set()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for rows in [*range(1, 201), *range(200, 0, -7), 0, 64]:
        cache.assign(ints([0, 0, 0]), rows)
        assert cache.slots.shape == cache.positions.shape == (rows,)
        assert cache.slots.tolist() == [-1] * rows and cache.positions.tolist() == [0] * rows
        if rows:
            where = cache.slots.data_ptr(), cache.positions.data_ptr()
            assert at.setdefault(rows, where) == where
            seen.add(where)
    assert len(seen) <= 9
    # nine sizes of 2 arrays of at most 512 bytes to 1 KB (the allocator's granule is 512 bytes)
    assert torch.cuda.memory_allocated() - before <= 9 * 2 * 1024
