"""Steps of a PagedCache that a server meets at its edges (needs a B200): without rows, idle, of many
sizes, on a stream beside the one that made the tensors."""
import pytest
import torch

import paged_util as U
from gpu_util import load_kivi
import test_gpu_paged
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


@pytest.mark.parametrize("op", ["packed", "paged", "append", "assign"])
def test_tensors_dropped_right_after_a_call_on_another_stream(kivi, op):
    """Inputs dropped while the call's stream is still busy: their memory is not handed out before
    the call has read them."""
    gen, stream = gen_of(61), torch.cuda.Stream()
    n, hkv, hq, dim, page = 4096, 2, 4, 64, 16
    ws = torch.zeros(kivi.kivi_attention_workspace_bytes(hkv, hq, dim), dtype=torch.uint8,
                     device="cuda")
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]

    def inputs():
        g = gen_of(62)
        q, k, v = (torch.randn(n, h, dim, generator=g, device="cuda").to(BF16)
                   for h in (hq, hkv, hkv))
        if op == "packed":
            return q, k, v, ints([0, n])
        if op == "append":
            return k, v, torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
        if op == "assign":
            return (ints([1] * 3000),)
        pages = [x.view(n // page, page, hkv, dim).transpose(1, 2).contiguous() for x in (k, v)]
        return q[-1:].clone(), *pages, table.clone(), ints([n]), ints([0, 1])

    def results():
        if op == "append":
            return [torch.zeros(n // page, hkv, page, dim, dtype=BF16, device="cuda")
                    for _ in range(2)]
        if op == "assign":
            z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
            return [z(3000), z(1), z(3001), z(3000), z(3000), z(1), z(3000, 1),
                    torch.arange(3000, dtype=torch.int32, device="cuda"), ints([3000])]
        return [torch.zeros(n if op == "packed" else 1, hq, dim, dtype=BF16, device="cuda")]

    def call(x, out, stream=None):
        if op == "packed":
            kivi.kivi_packed_attention(*x, ws, out=out[0], stream=stream)
        elif op == "paged":
            kivi.kivi_paged_attention(*x, ws, max_new=1, out=out[0], stream=stream)
        elif op == "append":
            kivi.kivi_paged_append(*x, *out, stream=stream)
        else:
            kv, nf, off, slots, pos, status, t, free, num_free = out
            kivi.kivi_paged_assign(torch.zeros_like(kv), x[0], t, free, num_free, page,
                                   kv_lengths=kv, num_free_out=nf, offsets=off, slots=slots,
                                   positions=pos, status=status, stream=stream)

    want, got = results(), results()
    call(inputs(), want)
    x = inputs()
    shapes = [(t.shape, t.dtype) for t in x]
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)  # about a tenth of a second
    call(x, got, stream)
    del x
    junk = [torch.empty(s, dtype=t, device="cuda").fill_(3) for s, t in shapes]
    torch.cuda.synchronize()
    assert len(junk) == len(shapes)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,page,width,rows", [(40, 64, 60, 16384), (40, 64, 60, 20000),
                                               (1, 16, 3000, 17001), (4096, 16, 8, 30000)])
def test_assign_of_many_rows(kivi, B, page, width, rows):
    """Around the number of rows from which a second kernel fills slots and positions."""
    test_gpu_paged.test_assign_over_steps(kivi, B, page, width, rows, 3)


@pytest.mark.parametrize("rows", [40, 3000, 20000])
def test_assign_reports_bad_page_ids(kivi, rows):
    """A table entry and a free page that are no page ids: their rows' slots are -1 and bit 2 is set,
    by the one kernel and by the rows' own; the other rows are as ever."""
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    for bad in (-3, 2 ** 31 - 1):
        table, free = z(3, 4), ints([7, bad, 9])
        table[0, 0], table[1, 0] = bad, 5
        lengths, status, slots, positions = ints([5, 15, 0]), z(1), z(rows) - 7, z(rows)
        kivi.kivi_paged_assign(lengths, ints([2, 3, 4]), table, free, ints([3]), 16,
                               kv_lengths=lengths, num_free_out=z(1), offsets=z(4), slots=slots,
                               positions=positions, status=status)
        # request 0 goes on in its bad page; 1 fills its page and pops 9; 2 pops the bad one
        assert slots[:9].tolist() == [-1, -1, 95, 144, 145, -1, -1, -1, -1]
        assert positions[:9].tolist() == [5, 6, 15, 16, 17, 0, 1, 2, 3]
        assert (slots[9:] == -1).all() and status.item() == 2
        assert lengths.tolist() == [7, 18, 4] and table[1:, :2].tolist() == [[5, 9], [bad, 0]]


def test_the_pages_hold_what_the_steps_appended(kivi):
    """Each request's tokens, read back by its table, over steps with releases between."""
    gen, cache = gen_of(71), small_cache(kivi, num_pages=20)
    keys, values = ([torch.empty(0, 2, 64, dtype=BF16, device="cuda")] * 3 for _ in range(2))
    for new in ([40, 9, 70], [1, 1, 1], [-1, 30, 1], [17, 1, 0], [1, -1, 60], [3, 100, 1]):
        k, v = step(cache, gen, new, pad=1)[1:3]
        off = cache.offsets.tolist()
        for b, n in enumerate(new):
            for held, x in ((keys, k), (values, v)):
                held[b] = torch.cat([held[b], x[off[b]:off[b + 1]]]) if n >= 0 else held[b][:0]
            length = keys[b].shape[0]
            assert cache.lengths[b].item() == length
            assert torch.equal(U.gather(cache.k_pages[0], cache.block_table[b], length), keys[b])
            assert torch.equal(U.gather(cache.v_pages[0], cache.block_table[b], length), values[b])
    assert cache.check_device_status() == 0
