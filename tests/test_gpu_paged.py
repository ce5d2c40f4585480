"""The paged 16-bit cache and attention over packed rows on the GPU (needs a B200), against the
plain 64-bit forms of paged_util (whose docstring derives the tolerance)."""
import random

import pytest
import torch

import paged_util as U
from gpu_util import load_kivi

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def kivi():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    return load_kivi()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(gen, *shape, dtype=BF16):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---- bookkeeping ----

class GpuBooks:
    def __init__(self, K, books, rows):
        self.K, self.page = K, books.page
        self.lengths, self.table = ints(books.lengths), ints(books.table)
        self.free, self.num_free = ints(books.free), ints([books.num_free])
        self.offsets = ints([-7] * (len(books.lengths) + 1))
        self.slots, self.positions = ints([-7] * rows), ints([-7] * rows)
        self.status = ints([0])

    def step(self, new, in_place=True):
        kv = self.lengths if in_place else torch.empty_like(self.lengths)
        nf = self.num_free if in_place else torch.empty_like(self.num_free)
        self.K.kivi_paged_assign(self.lengths, ints(new), self.table, self.free, self.num_free,
                                 self.page, kv_lengths=kv, num_free_out=nf, offsets=self.offsets,
                                 slots=self.slots, positions=self.positions, status=self.status)
        self.lengths, self.num_free = kv, nf
        code = int(self.status.item())
        self.status.zero_()
        return self.offsets.tolist(), self.slots.tolist(), self.positions.tolist(), code


def compare_books(gpu, books):
    assert gpu.lengths.tolist() == books.lengths
    assert gpu.num_free.tolist() == [books.num_free]
    assert gpu.free.tolist() == books.free
    assert gpu.table.tolist() == books.table


@pytest.mark.parametrize("B,page,width,rows,steps", [
    (1, 16, 1, 1, 4), (3, 16, 4, 40, 8), (17, 32, 8, 300, 8), (64, 128, 3, 1025, 6),
    (700, 16, 12, 5000, 5), (4096, 16, 4, 6000, 3)])
def test_assign_over_steps(kivi, B, page, width, rows, steps):
    """Random steps with prompts, single tokens, idle and released requests."""
    rng = random.Random(B * 31 + page)
    pages = B * width
    order = rng.sample(range(pages), pages)
    books = U.Books([0] * B, [[-1] * width for _ in range(B)], order, pages, page)
    gpu = GpuBooks(kivi, books, rows)
    for i in range(steps):
        new, left = [], rows
        for b in range(B):
            kind = rng.random()
            room = min(left, width * page - books.lengths[b])
            n = -1 if kind < 0.15 else 0 if kind < 0.3 else min(1, room) if kind < 0.7 else \
                rng.randint(0, min(room, 3 * rows // B + 1))
            new.append(n)
            left -= max(n, 0)
        want = books.step(new, rows)
        assert want[3] == 0
        assert gpu.step(new, in_place=i % 2 == 0) == want, f"step {i}"
        compare_books(gpu, books)


@pytest.mark.parametrize("new,lengths,num_free,code", [
    ([20, 0, 0], [0, 0, 0], 1, 8),            # two pages needed, one free
    ([0, 0, 65], [0, 0, 0], 12, 4),           # past the table's width
    ([30, 30, 10], [0, 0, 0], 12, 4),         # more rows than the buffers have
    ([1, 1, 1], [0, -5, 0], 12, 4),           # a negative length
    ([1, 1, 1], [0, 900, 0], 12, 4),          # a length past the table
    ([-1, -1, -1], [40, 64, 64], 12, 4),      # more pages given back than the pool has
    ([2**31 - 1, 2**31 - 1, 2], [0, 0, 0], 12, 4),
    ([-1, 17, 0], [16, 0, 0], 1, 0),          # the released page serves the next request
])
def test_assign_all_or_nothing(kivi, new, lengths, num_free, code):
    table = [[1, 2, 3, 4], [5, 6, 7, 8], [9, 10, 11, 0]]
    free = [7, 3, 2, 4, 5, 6, 8, 9, 10, 11, 0, 1]
    books = U.Books(lengths, table, free, num_free, 16)
    want = books.step(new, 64)
    assert want[3] == code
    gpu = GpuBooks(kivi, U.Books(lengths, table, free, num_free, 16), 64)
    assert gpu.step(new) == want
    compare_books(gpu, books)


# ---- append ----

@pytest.mark.parametrize("rows,hkv,dim,page,dtype", [
    (1, 1, 64, 16, BF16), (7, 3, 128, 32, FP16), (33, 8, 64, 256, BF16), (1000, 5, 128, 16, BF16)])
def test_append_writes_the_slots_and_nothing_else(kivi, rows, hkv, dim, page, dtype):
    gen = gen_of(rows)
    pages = rows // page + 4
    kp, vp = (randn(gen, pages, hkv, page, dim, dtype=dtype) for _ in range(2))
    # rows of a wider projection: strides other than heads * dim
    wide = randn(gen, rows, (2 * hkv + 1) * dim, dtype=dtype)
    k = wide[:, dim:dim * (hkv + 1)].view(rows, hkv, dim)
    v = wide[:, dim * (hkv + 1):].view(rows, hkv, dim)
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:rows].to(torch.int32)
    if rows > 5:
        slots[3] = -1
    want_k, want_v = kp.clone(), vp.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // page, :, s % page] = k[i]
            want_v[s // page, :, s % page] = v[i]
    status = ints([0])
    kivi.kivi_paged_append(k, v, slots, kp, vp, status)
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    assert status.item() == 0


def test_append_skips_slots_outside_the_pool(kivi):
    gen = gen_of(5)
    kp, vp = torch.zeros(2, 4, 1, 16, 64, dtype=BF16, device="cuda").unbind(0)
    k = randn(gen, 3, 1, 64)
    status = ints([0])
    kivi.kivi_paged_append(k, k, ints([64, 5, 2**31 - 1]), kp, vp, status)
    assert status.item() == 2
    assert torch.equal(kp[0, 0, 5], k[1, 0]) and kp.count_nonzero() == k[1].count_nonzero()


# ---- attention ----

class Pool:
    """Pages with NaN wherever no request has a token, and random page order."""

    def __init__(self, gen, lengths, hkv, dim, page, dtype, spare=2):
        have = [-(-n // page) for n in lengths]
        pages, width = sum(have) + spare, max(max(have), 1) + 1
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        self.table = torch.full((len(lengths), width), pages + 5, dtype=torch.int32, device="cuda")
        self.k, self.v = (torch.full((pages, hkv, page, dim), float("nan"), dtype=dtype,
                                     device="cuda") for _ in range(2))
        self.keys, self.values, first = [], [], 0
        for b, n in enumerate(lengths):
            self.table[b, :have[b]] = order[first:first + have[b]]
            first += have[b]
            k, v = (randn(gen, n, hkv, dim, dtype=dtype) for _ in range(2))
            j = torch.arange(n, device="cuda")
            ids = self.table[b].long()[j // page]
            self.k[ids, :, j % page] = k
            self.v[ids, :, j % page] = v
            self.keys.append(k)
            self.values.append(v)


def offsets_of(new):
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    return off


def workspace(K, hkv, hq, dim):
    return torch.zeros(K.kivi_attention_workspace_bytes(hkv, hq, dim), dtype=torch.uint8,
                       device="cuda")


def check_paged(K, requests, hkv, ratio, dim, page, dtype=BF16, seed=0, max_new=None,
                sm_scale=0.0, calls=1, pad=3):
    """requests: (keys, new rows) of each.  Rows of a wider projection in and out, NaN in the
    rows behind the last request's, which stay as they were."""
    gen = gen_of(seed)
    hq = hkv * ratio
    lengths, new = [r[0] for r in requests], [r[1] for r in requests]
    pool = Pool(gen, lengths, hkv, dim, page, dtype)
    off = offsets_of(new)
    ws = workspace(K, hkv, hq, dim)
    for c in range(calls):
        wide = torch.full((off[-1] + pad, hq * dim + 64), float("nan"), dtype=dtype, device="cuda")
        q = wide[:, 64:].view(-1, hq, dim)
        q[:off[-1]] = randn(gen, off[-1], hq, dim, dtype=dtype)
        out = torch.full((off[-1] + pad, hq * dim + 8), -5.0, dtype=dtype, device="cuda")
        K.kivi_paged_attention(q, pool.k, pool.v, pool.table, ints(lengths), ints(off), ws,
                               max_new=max_new, out=out[:, :hq * dim].view(-1, hq, dim),
                               sm_scale=sm_scale)
        assert (out[off[-1]:] == -5.0).all() and (out[:, hq * dim:] == -5.0).all()
        got = out[:, :hq * dim].view(-1, hq, dim)
        for b, n in enumerate(new):
            ref, mean = U.attend(q[off[b]:off[b] + n], pool.keys[b], pool.values[b], sm_scale)
            U.assert_close(got[off[b]:off[b] + n], ref, mean, f"request {b} of {requests[b]}")
    # no failure is reported unless some request has fewer keys than rows
    code = K.kivi_attention_status(ws)
    assert code == (4 if any(n > L for L, n in requests) else 0)


DECODE = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_page_sizes(kivi, page):
    check_paged(kivi, [(L, 1) for L in DECODE], 2, 4, 128, page, max_new=1, calls=2)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("hkv,ratio,dim", [(1, 1, 64), (3, 1, 128), (2, 2, 64), (2, 3, 128),
                                           (8, 4, 128), (1, 8, 64), (2, 7, 64), (1, 16, 128),
                                           (1, 24, 64), (1, 71, 64), (1, 128, 128)])
def test_decode_heads(kivi, hkv, ratio, dim, dtype):
    check_paged(kivi, [(L, 1) for L in (1, 40, 129, 517)], hkv, ratio, dim, 32, dtype, max_new=1)


def test_decode_long_and_short(kivi):
    check_paged(kivi, [(20000, 1), (1, 1), (4097, 1)], 2, 4, 128, 64, max_new=1, calls=2)


def test_decode_many_requests(kivi):
    check_paged(kivi, [(1 + 37 * b % 200, 1) for b in range(300)], 2, 2, 64, 16, max_new=1)


def test_decode_a_few_tokens_each(kivi):
    check_paged(kivi, [(100, 4), (5, 3), (700, 2), (64, 4), (0, 0), (64, 1)], 2, 4, 128, 16,
                max_new=4)


def test_rows_without_keys_are_zero(kivi):
    """Requests without keys, with fewer keys than rows, and without rows."""
    check_paged(kivi, [(0, 1), (50, 0), (33, 1), (0, 0), (2, 5), (0, 30)], 2, 4, 64, 16)
    check_paged(kivi, [(0, 1), (50, 0), (33, 1)], 2, 4, 64, 16, max_new=1)


@pytest.mark.parametrize("page", [16, 64, 256])
def test_chunk_page_sizes(kivi, page):
    check_paged(kivi, [(200, 200), (333, 77), (129, 5), (512, 64), (1, 1), (130, 129)], 2, 4, 128,
                page, calls=2)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("hkv,ratio,dim", [(2, 1, 64), (1, 1, 128), (2, 2, 128), (1, 3, 64),
                                           (2, 4, 128), (1, 8, 64), (1, 5, 128), (1, 16, 128),
                                           (1, 71, 64), (1, 128, 64)])
def test_chunk_heads(kivi, hkv, ratio, dim, dtype):
    check_paged(kivi, [(300, 300), (260, 31), (1000, 100)], hkv, ratio, dim, 32, dtype)


def test_chunk_of_long_context(kivi):
    check_paged(kivi, [(9000, 70)], 2, 4, 128, 128, calls=2)


def test_chunks_beside_decoding_requests(kivi):
    check_paged(kivi, [(700, 1), (1300, 300), (5, 1), (900, 1), (64, 64), (2000, 1)], 8, 4, 128,
                32, calls=2)


def test_sm_scale_and_peaked_rows(kivi):
    check_paged(kivi, [(500, 100), (400, 1)], 2, 2, 128, 32, sm_scale=0.02)
    check_paged(kivi, [(500, 100), (400, 1)], 2, 2, 64, 32, sm_scale=0.125 * 1.9)


def check_packed(K, lengths, hkv, ratio, dim, dtype=BF16, seed=0, pad=2, calls=1):
    gen = gen_of(seed)
    hq = hkv * ratio
    off = offsets_of(lengths)
    T = off[-1]
    ws = workspace(K, hkv, hq, dim)
    for c in range(calls):
        # one fused projection holds q, k and v side by side
        wide = torch.full((T + pad, (hq + 2 * hkv) * dim), float("nan"), dtype=dtype,
                          device="cuda")
        wide[:T] = randn(gen, T, wide.shape[1], dtype=dtype)
        q = wide[:, :hq * dim].view(-1, hq, dim)
        k = wide[:, hq * dim:(hq + hkv) * dim].view(-1, hkv, dim)
        v = wide[:, (hq + hkv) * dim:].view(-1, hkv, dim)
        out = torch.full((T + pad, hq, dim), -5.0, dtype=dtype, device="cuda")
        got = K.kivi_packed_attention(q, k, v, ints(off), ws, out=out)
        assert got is out and (out[T:] == -5.0).all()
        for b, n in enumerate(lengths):
            at = slice(off[b], off[b] + n)
            ref, mean = U.attend(q[at], k[at], v[at])
            U.assert_close(got[at], ref, mean, f"prompt {b} of {n}")
    assert K.kivi_attention_status(ws) == 0


@pytest.mark.parametrize("lengths", [[1], [2, 1, 3], [64], [127, 129], [128, 0, 256, 1],
                                     [255, 257], [1000], [33] * 40, [5, 700, 1, 1, 300, 64]])
def test_packed_lengths(kivi, lengths):
    check_packed(kivi, lengths, 2, 4, 128, calls=2)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("hkv,ratio,dim", [(1, 1, 64), (4, 1, 128), (2, 2, 64), (2, 3, 128),
                                           (1, 8, 128), (1, 6, 64), (2, 16, 64), (1, 71, 64),
                                           (1, 128, 128)])
def test_packed_heads(kivi, hkv, ratio, dim, dtype):
    check_packed(kivi, [70, 1, 300, 130], hkv, ratio, dim, dtype)


def test_packed_long(kivi):
    check_packed(kivi, [3000, 1500], 2, 2, 128)


def test_packed_many_requests(kivi):
    check_packed(kivi, [b % 5 for b in range(4096)], 1, 2, 64)


def test_neighbours_do_not_meet(kivi):
    """A prompt of NaN and infinities beside others leaves their rows alone."""
    gen = gen_of(3)
    off = offsets_of([100, 60, 131])
    q, k, v = (randn(gen, off[-1], h, 128) for h in (8, 2, 2))
    ref = [U.attend(q[a:b], k[a:b], v[a:b]) for a, b in ((0, 100), (160, 291))]
    for x in (q, k, v):
        x[100:130] = float("nan")
        x[130:160] = float("inf")
    ws = workspace(kivi, 2, 8, 128)
    got = kivi.kivi_packed_attention(q, k, v, ints(off), ws)
    U.assert_close(got[:100], *ref[0], "first")
    U.assert_close(got[160:], *ref[1], "last")


def test_bad_device_values_are_reported(kivi):
    """Page ids, lengths and offsets outside their buffers: a status bit, nothing else touched."""
    gen = gen_of(9)
    pool = Pool(gen, [100, 100], 2, 64, 16, BF16)
    ws = workspace(kivi, 2, 4, 64)
    for new, max_new in ((1, 1), (40, None)):
        q = randn(gen, 2 * new + 4, 4, 64)
        off = offsets_of([new, new])

        def call(table=pool.table, kv=(100, 100), off=off, max_new=max_new):
            out = torch.full_like(q, -5.0)
            kivi.kivi_paged_attention(q, pool.k, pool.v, table, ints(kv), ints(off), ws,
                                      max_new=max_new, out=out)
            code = kivi.kivi_attention_status(ws)
            assert (out[2 * new:] == -5.0).all()
            return out, code

        good, code = call()
        assert code == 0
        table = pool.table.clone()
        table[0, 2], table[0, 3] = -3, 2**31 - 1
        out, code = call(table=table)
        assert code == 2 and torch.equal(out[new:2 * new], good[new:2 * new])
        # a bad page reads as zero keys and values
        k, v = pool.keys[0].clone(), pool.values[0].clone()
        k[32:64], v[32:64] = 0, 0
        U.assert_close(out[:new], *U.attend(q[:new], k, v), "zero keys")
        out, code = call(kv=(-4, 100))
        assert code == 4 and (out[:new] == 0).all()
        assert torch.equal(out[new:2 * new], good[new:2 * new])
        out, code = call(kv=(100, 16 * pool.table.shape[1] + 1))
        assert code & 4 and torch.equal(out[:new], good[:new])
        out, code = call(off=[0, new, -9])
        assert code == 4 and torch.equal(out[:new], good[:new])
    # more new rows than promised: that request is left alone
    q = randn(gen, 42, 4, 64)
    out = torch.full_like(q, -5.0)
    kivi.kivi_paged_attention(q, pool.k, pool.v, pool.table, ints([100, 100]), ints([0, 41, 42]),
                              ws, max_new=1, out=out)
    assert kivi.kivi_attention_status(ws) == 4
    assert (out[:41] == -5.0).all() and not (out[41] == -5.0).any()


@pytest.mark.parametrize("hkv,ratio,dim,dtype", [(8, 1, 128, BF16), (4, 4, 64, FP16),
                                                 (2, 16, 128, BF16)])
def test_packed_items_cut_and_whole(kivi, hkv, ratio, dim, dtype):
    """Enough rows that cut items are joined by their last CTA (four items of 256 rows per SM)."""
    rows = 4 * 256 * 160 // (hkv * ratio)
    first = rows // 3
    check_packed(kivi, [first, 1, rows - first - 130, 0, 129], hkv, ratio, dim, dtype, calls=2)


def test_chunk_many_requests(kivi):
    check_paged(kivi, [(b % 90, b % 4) for b in range(4096)], 1, 8, 64, 16)


def test_growing_scores(kivi):
    """Row maxima that grow by more than the rescaling slack from tile to tile, and fall again."""
    gen = gen_of(21)
    for n, chunk, dtype in ((700, 700, BF16), (700, 90, FP16), (900, 1, BF16)):
        K, hkv, hq, dim = kivi, 2, 4, 64
        pool = Pool(gen, [n], hkv, dim, 32, dtype)
        # keys along one direction whose length changes: scores up to 60, in steps of 64 keys
        size = torch.tensor([0.1, 2.0, 0.5, 4.0, 1.0, 6.0, 7.5, 0.2], device="cuda")
        scale = size[(torch.arange(n, device="cuda") // 64) % 8]
        base = torch.ones(dim, device="cuda")
        keys = (scale[:, None, None] * base + 0.05 * torch.randn(n, hkv, dim, generator=gen,
                                                                 device="cuda")).to(dtype)
        pool.keys[0] = keys
        j = torch.arange(n, device="cuda")
        ids = pool.table[0].long()[j // 32]
        pool.k[ids, :, j % 32] = keys
        q = (1.0 + 0.05 * torch.randn(chunk, hq, dim, generator=gen, device="cuda")).to(dtype)
        got = K.kivi_paged_attention(q, pool.k, pool.v, pool.table, ints([n]), ints([0, chunk]),
                                     workspace(K, hkv, hq, dim), max_new=chunk)
        out, mean = U.attend(q, keys, pool.values[0])
        # scores reach 60: sum |q k| / sqrt(D) is 60 here, 4 times the bound of paged_util's
        # derivation, so the part of the scores' roundings grows by 4
        u = torch.finfo(dtype).eps / 2
        err = (got.double() - out).abs()
        assert (err <= (3 * u + 4 * 2.0 ** -11) * mean + 1e-6).all(), err.max().item()


@pytest.mark.parametrize("B", [31, 32, 33])
def test_request_counts_at_a_warp(kivi, B):
    """Both ways of forming the ranges (one warp, the whole block), requests without rows among them."""
    check_paged(kivi, [(5 + 61 * b % 400, b % 3 % 2) for b in range(B)], 2, 4, 128, 16, max_new=1)
    check_paged(kivi, [(5 + 61 * b % 400, (7 * b) % 6) for b in range(B)], 2, 8, 64, 32)
    check_packed(kivi, [(37 * b) % 150 for b in range(B)], 2, 2, 64)


def test_one_long_request_of_many_heads(kivi):
    check_paged(kivi, [(16000, 1)], 1, 16, 128, 64, max_new=1, calls=2)
    check_paged(kivi, [(16000, 3)], 1, 16, 128, 64, calls=2)


def test_calls_side_by_side(kivi):
    """Two streams with a workspace each, many calls at once: as one after the other."""
    gen = gen_of(23)
    pool = Pool(gen, [2500, 900, 300], 2, 128, 32, BF16)
    kv, steps = ints([2500, 900, 300]), []
    for new in ([300, 1, 90], [1, 1, 1]):
        off = offsets_of(new)
        q = randn(gen, off[-1], 8, 128)
        steps.append((q, ints(off), max(new)))

    def call(step, ws, **kw):
        q, off, max_new = step
        return kivi.kivi_paged_attention(q, pool.k, pool.v, pool.table, kv, off, ws,
                                         max_new=max_new, **kw)

    spaces = [workspace(kivi, 2, 8, 128) for _ in range(2)]
    want = [call(step, spaces[0]) for step in steps]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, (stream, ws) in enumerate(zip(streams, spaces)):
            for step in steps:
                got[i].append(call(step, ws, stream=stream))
    torch.cuda.synchronize()
    for outs in got:
        for j, out in enumerate(outs):
            assert torch.equal(out, want[j % 2])
    assert all(kivi.kivi_attention_status(ws) == 0 for ws in spaces)


def test_far_pages(kivi):
    """A pool of more than 2^31 elements, the requests' pages at its end and a prefix page shared."""
    gen = gen_of(31)
    hkv, hq, dim, page = 8, 16, 128, 64
    pages = (2 ** 31 // (hkv * dim * page)) + 40
    kp, vp = (torch.zeros(pages, hkv, page, dim, dtype=BF16, device="cuda") for _ in range(2))
    table = ints([[pages - 1, 3, pages - 2], [pages - 1, pages - 3, 5]])
    lengths, new = [150, 130], [1, 40]
    keys, values = ([randn(gen, n, hkv, dim) for n in lengths] for _ in range(2))
    keys[1][:64], values[1][:64] = keys[0][:64], values[0][:64]
    slots = torch.cat([table[b].long()[torch.arange(n, device="cuda") // page] * page
                       + torch.arange(n, device="cuda") % page
                       for b, n in enumerate(lengths)]).to(torch.int32)
    slots[lengths[0]:lengths[0] + 64] = -1  # the shared page is written once
    kivi.kivi_paged_append(torch.cat(keys), torch.cat(values), slots, kp, vp)
    ws = workspace(kivi, hkv, hq, dim)
    for new in ([1, 1], [1, 40]):
        q = randn(gen, sum(new), hq, dim)
        off = offsets_of(new)
        got = kivi.kivi_paged_attention(q, kp, vp, table, ints(lengths), ints(off), ws,
                                        max_new=max(new))
        for b in range(2):
            at = slice(off[b], off[b + 1])
            U.assert_close(got[at], *U.attend(q[at], keys[b], values[b]), f"request {b} of {new}")
    assert kivi.kivi_attention_status(ws) == 0


def test_more_tiles_than_a_call_counts(kivi):
    """Lengths whose tiles an int does not hold: refused on the device before any copy."""
    hkv, page, width = 128, 256, 2 ** 23 - 2
    kp = torch.zeros(1, hkv, page, 64, dtype=BF16, device="cuda")
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    ws = workspace(kivi, hkv, hkv, 64)
    for n in (1, 300):
        q = torch.zeros(n, hkv, 64, dtype=BF16, device="cuda")
        out = torch.full_like(q, -5.0)
        kivi.kivi_paged_attention(q, kp, kp, table, ints([page * width]), ints([0, n]), ws,
                                  max_new=n, out=out)
        assert kivi.kivi_attention_status(ws) == 4
        assert (out == -5.0).all()


# ---- together ----

def run_steps(K, prompts, chunk, decode, hkv, hq, dim, page, dtype, layers=2, seed=1):
    """Prompts in chunks, then single tokens, through assign, append and attend of a PagedCache;
    the last request is released half way and its place taken again."""
    gen = gen_of(seed)
    total = [n + decode for n in prompts]
    qkv = [[[randn(gen, t, h, dim, dtype=dtype) for h in (hq, hkv, hkv)] for t in total]
           for _ in range(layers)]
    cache = K.PagedCache(num_pages=sum(-(-t // page) for t in total) + 2, page_size=page,
                         num_layers=layers, num_kv_heads=hkv, num_q_heads=hq, head_dim=dim,
                         max_requests=len(prompts) + 1, max_tokens=max(total), dtype=dtype)
    cache.k_pages.fill_(float("nan"))
    cache.v_pages.fill_(float("nan"))
    # a request that comes and goes before the others start
    cache.assign(ints([0] * len(prompts) + [2 * page]), 2 * page)
    cache.assign(ints([0] * len(prompts) + [-1]), 0)
    done, outs = [0] * len(prompts), [[[] for _ in prompts] for _ in range(layers)]
    while any(d < t for d, t in zip(done, total)):
        new = [min(chunk, n - d) if d < n else 1 if d < t else 0
               for d, n, t in zip(done, prompts, total)]
        rows = sum(new) + 2
        cache.assign(ints(new + [0]), rows, max_new=max(new))
        off = cache.offsets.tolist()
        assert off[:-1] == offsets_of(new)
        for layer in range(layers):
            q, k, v = (torch.zeros(rows, h, dim, dtype=dtype, device="cuda")
                       for h in (hq, hkv, hkv))
            for b, n in enumerate(new):
                for x, src in zip((q, k, v), qkv[layer][b]):
                    x[off[b]:off[b] + n] = src[done[b]:done[b] + n]
            cache.append(layer, k, v)
            out = cache.attend(layer, q)
            for b, n in enumerate(new):
                outs[layer][b].append(out[off[b]:off[b] + n])
        done = [d + n for d, n in zip(done, new)]
    assert cache.check_device_status() == 0
    for layer in range(layers):
        for b, t in enumerate(total):
            got = torch.cat(outs[layer][b])
            U.assert_close(got, *U.attend(*qkv[layer][b]), f"layer {layer} request {b}")
    # whole prompts without pages give the same
    packed = K.PackedAttention(num_kv_heads=hkv, num_q_heads=hq, head_dim=dim)
    q, k, v = (torch.cat([qkv[0][b][i] for b in range(len(total))]) for i in range(3))
    got = packed.attend(q, k, v, ints(offsets_of(total)))
    for b, (a, t) in enumerate(zip(offsets_of(total), total)):
        U.assert_close(got[a:a + t], *U.attend(*qkv[0][b]), f"packed {b}")
    assert packed.check_device_status() == 0
    assert cache.lengths.tolist() == total + [0]


@pytest.mark.parametrize("hkv,hq,dim,page,dtype", [(2, 8, 128, 16, BF16), (2, 2, 64, 64, FP16)])
def test_steps_of_a_server(kivi, hkv, hq, dim, page, dtype):
    run_steps(kivi, [150, 1, 333, 40], 64, 5, hkv, hq, dim, page, dtype)


def test_packed_equals_uniform_causal_attention(kivi):
    """The attention of uniform prompts that the library already has, within both bounds."""
    gen = gen_of(4)
    B, S, hkv, hq, dim = 3, 200, 2, 8, 128
    q, k, v = (randn(gen, B, h, S, dim) for h in (hq, hkv, hkv))
    want = kivi.kivi_causal_attention(q, k, v)
    rows = lambda x: x.transpose(1, 2).reshape(B * S, -1, dim).contiguous()  # noqa: E731
    got = kivi.kivi_packed_attention(rows(q), rows(k), rows(v), ints([0, S, 2 * S, 3 * S]),
                                     workspace(kivi, hkv, hq, dim))
    mean = torch.cat([U.attend(rows(q)[i * S:(i + 1) * S], rows(k)[i * S:(i + 1) * S],
                               rows(v)[i * S:(i + 1) * S])[1] for i in range(B)])
    err = (got.double() - rows(want).double()).abs()
    assert (err <= (5 * 2.0 ** -8 + 2.0 ** -10) * mean + 1e-6).all()


def graph_state(K, gen):
    cache = K.PagedCache(num_pages=40, page_size=16, num_layers=1, num_kv_heads=2, num_q_heads=8,
                         head_dim=128, max_requests=3, max_tokens=200)
    k, v = randn(gen, 3, 2, 128), randn(gen, 3, 2, 128)
    return cache, randn(gen, 3, 8, 128), k, v


def test_decode_steps_in_a_graph(kivi):
    """A captured decode step replayed 40 times, across page borders, against the plain form."""
    gen = gen_of(8)
    cache, q, k, v = graph_state(kivi, gen)
    first = [5, 14, 31]
    keys, values = [[] for _ in first], [[] for _ in first]

    def prompt():
        cache.assign(ints(first), sum(first))
        kk, vv = randn(gen, sum(first), 2, 128), randn(gen, sum(first), 2, 128)
        cache.append(0, kk, vv)
        at = 0
        for b, n in enumerate(first):
            keys[b].append(kk[at:at + n])
            values[b].append(vv[at:at + n])
            at += n

    prompt()
    one = ints([1, 1, 1])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    cache.slots = torch.empty(3, dtype=torch.int32, device="cuda")
    cache.positions = torch.empty_like(cache.slots)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        cache.assign(one, 3, max_new=1)
        cache.append(0, k, v)
        cache.attend(0, q, out=out)
    for _ in range(40):
        for x, n in ((q, 8), (k, 2), (v, 2)):
            x.copy_(randn(gen, 3, n, 128))
        graph.replay()
        for b in range(3):
            keys[b].append(k[b:b + 1].clone())
            values[b].append(v[b:b + 1].clone())
            U.assert_close(out[b:b + 1], *U.attend(q[b:b + 1], torch.cat(keys[b]),
                                                   torch.cat(values[b])), f"request {b}")
    assert cache.lengths.tolist() == [45, 54, 71] and cache.check_device_status() == 0


def test_other_stream_and_repeated_calls_agree(kivi):
    gen = gen_of(12)
    pool = Pool(gen, [3000, 700, 50], 2, 128, 32, BF16)
    q = randn(gen, 230, 8, 128)
    off, kv = ints([0, 200, 201, 230]), ints([3000, 700, 50])
    call = lambda ws, **kw: kivi.kivi_paged_attention(  # noqa: E731
        q, pool.k, pool.v, pool.table, kv, off, ws, **kw)
    want = call(workspace(kivi, 2, 8, 128))
    ws = workspace(kivi, 2, 8, 128)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = [call(ws, stream=stream) for _ in range(3)]
    stream.synchronize()
    for g in got:  # the split over keys and its join do not depend on the order of arrival
        assert torch.equal(g, want)


def test_binding_checks(kivi):
    gen = gen_of(13)
    q, k = randn(gen, 6, 4, 64), randn(gen, 6, 2, 64)
    ws, off = workspace(kivi, 2, 4, 64), ints([0, 6])
    for bad in (lambda: kivi.kivi_packed_attention(q, k, k.to(FP16), off, ws),
                lambda: kivi.kivi_packed_attention(q.float(), k.float(), k.float(), off, ws),
                lambda: kivi.kivi_packed_attention(q, k[:5], k, off, ws),
                lambda: kivi.kivi_packed_attention(q, k, k, off.long(), ws),
                lambda: kivi.kivi_packed_attention(q, k, k, off.cpu(), ws),
                lambda: kivi.kivi_packed_attention(q.transpose(0, 1), k, k, off, ws),
                lambda: kivi.kivi_paged_append(k, k, ints([1, 2]), k[None], k[None])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kivi.KiviError, match="BUFFER_TOO_SMALL"):
        kivi.kivi_packed_attention(q, k, k, off, ws[:128])
    pages = k[None, :2].contiguous()  # one page of 2 "tokens": refused by the library
    table, one = ints([[0]]), ints([6])
    for bad in (lambda: kivi.kivi_paged_attention(q, pages, pages, table.long(), one, off, ws),
                lambda: kivi.kivi_paged_attention(q, pages, pages, table[0], one, off, ws),
                lambda: kivi.kivi_paged_attention(q, pages, pages, table, ints([6, 6]), off, ws),
                lambda: kivi.kivi_paged_attention(q, pages, pages.float(), table, one, off, ws),
                lambda: kivi.kivi_paged_attention(q, pages, pages, table, one, off, ws, out=q[:3]),
                lambda: kivi.kivi_paged_attention(q, pages, pages, table, one, off, ws,
                                                  max_new=2 ** 31),
                lambda: kivi.kivi_packed_attention(q[0], k, k, off, ws),
                lambda: kivi.kivi_packed_attention(q, k, k, off, ws, out=q.transpose(0, 1)),
                lambda: kivi.kivi_packed_attention(q[..., ::2], k[..., ::2], k[..., ::2], off, ws)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: kivi.kivi_packed_attention(q, None, k, off, ws),
                lambda: kivi.kivi_packed_attention(q, k, k, off, ws, sm_scale="x"),
                lambda: kivi.kivi_paged_attention(q, pages, pages, table, one, off, ws, max_new=1.5)):
        with pytest.raises(TypeError):
            bad()


def test_mixed_steps_in_two_graphs(kivi):
    """Two captured steps with a workspace each, replayed in turn and with an eager step between,
    against the plain form: cut items, joined by the second kernel."""
    gen = gen_of(17)
    lengths, new = [2100, 333, 64, 900], [1, 120, 64, 30]
    off, total = offsets_of(new), sum(new)
    states = []
    for i in range(2):
        pool = Pool(gen, lengths, 2, 128, 32, BF16)
        q = randn(gen, total, 8, 128)
        out = torch.zeros_like(q)
        states.append((pool, q, out, workspace(kivi, 2, 8, 128), ints(lengths), ints(off)))

    def call(st, out):
        pool, q, _, ws, kv, offsets = st
        return kivi.kivi_paged_attention(q, pool.k, pool.v, pool.table, kv, offsets, ws,
                                         max_new=max(new), out=out)

    graphs = []
    for st in states:
        call(st, None)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(st, st[2])
        graphs.append(graph)
    for _ in range(3):
        for st, graph in zip(states, graphs):
            st[1].copy_(randn(gen, total, 8, 128))
            st[2].fill_(-1.0)
            graph.replay()
            eager = call(st, None)
            assert torch.equal(eager, st[2])
            for b, (a, e) in enumerate(zip(off, off[1:])):
                U.assert_close(st[2][a:e], *U.attend(st[1][a:e], st[0].keys[b], st[0].values[b]),
                               f"request {b}")
    assert all(kivi.kivi_attention_status(st[3]) == 0 for st in states)


def test_cache_steps_of_changing_size_keep_a_captured_step(kivi):
    """A captured decode step of a PagedCache stays valid when an eager step has another size."""
    gen = gen_of(19)
    cache, q, k, v = graph_state(kivi, gen)
    first, keys, values = [5, 14, 31], [], []
    kk, vv = randn(gen, sum(first), 2, 128), randn(gen, sum(first), 2, 128)
    cache.assign(ints(first), sum(first))
    cache.append(0, kk, vv)
    for a, e in zip(offsets_of(first), offsets_of(first)[1:]):
        keys.append(kk[a:e])
        values.append(vv[a:e])
    one, out = ints([1, 1, 1]), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.assign(one, 3, max_new=1)
        cache.append(0, k, v)
        cache.attend(0, q, out=out)

    def replay():
        for x, n in ((q, 8), (k, 2), (v, 2)):
            x.copy_(randn(gen, 3, n, 128))
        graph.replay()
        for b in range(3):
            keys[b] = torch.cat([keys[b], k[b:b + 1]])
            values[b] = torch.cat([values[b], v[b:b + 1]])
            U.assert_close(out[b:b + 1], *U.attend(q[b:b + 1], keys[b], values[b]), f"request {b}")

    replay()
    kk, vv = randn(gen, 70, 2, 128), randn(gen, 70, 2, 128)
    cache.assign(ints([0, 70, 0]), 70)
    cache.append(0, kk, vv)
    keys[1], values[1] = torch.cat([keys[1], kk]), torch.cat([values[1], vv])
    replay()
    assert cache.check_device_status() == 0
