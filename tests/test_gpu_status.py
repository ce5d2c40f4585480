"""The status queries on the GPU (needs a B200): what they read and clear runs on the caller's stream
and is complete on return.

The default stream is kept busy by a kernel that sleeps while the query runs on another stream: a
query that touches the default stream would come back only when that kernel has ended."""
import pytest
import torch

import paged_util as U
from gpu_util import load_kivi
from test_gpu_paged import Pool, gen_of, ints, randn, workspace

pytestmark = pytest.mark.gpu
BUSY_CYCLES = 1_000_000_000  # about half a second


@pytest.fixture(scope="module")
def kivi():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    return load_kivi()


def busy_default_stream():
    """An event behind about half a second of work on the default stream."""
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY_CYCLES)
    end = torch.cuda.Event()
    end.record()
    return end


@pytest.mark.parametrize("new", [[1, 1], [200, 30]])
def test_attention_status_clears_on_its_stream(kivi, new):
    """A call that reports a bad page, the query, and at once calls whose items are cut and joined."""
    gen = gen_of(41)
    lengths, off = [3000, 700], ints([0, new[0], sum(new)])
    pool = Pool(gen, lengths, 2, 128, 32, torch.bfloat16)
    bad = pool.table.clone()
    bad[0, 1] = -1
    q, ws, kv = randn(gen, sum(new), 8, 128), workspace(kivi, 2, 8, 128), ints(lengths)
    outs = [torch.empty_like(q) for _ in range(6)]
    stream = torch.cuda.Stream()

    def call(table, out):
        kivi.kivi_paged_attention(q, pool.k, pool.v, table, kv, off, ws, max_new=max(new), out=out,
                                  stream=stream)

    call(pool.table, outs[0])  # loads the kernels
    end = busy_default_stream()
    for out in outs:
        call(bad, out)
        assert kivi.kivi_attention_status(ws, stream) == 2
        call(pool.table, out)
    assert kivi.kivi_attention_status(ws, stream) == 0
    assert not end.query(), "the query waited for the default stream"
    torch.cuda.synchronize()
    assert ws[64:8192].count_nonzero() == 0
    for out in outs:
        for b, (a, e) in enumerate(zip([0, new[0]], [new[0], sum(new)])):
            U.assert_close(out[a:e], *U.attend(q[a:e], pool.keys[b], pool.values[b]), f"request {b}")


def small_cache(K):
    return K.KiviCache(batch=2, num_layers=1, num_kv_heads=2, num_q_heads=4, head_dim=64, bits=2,
                       max_tokens=300)


def query_of(K, which):
    """A status query, and the buffer whose first word it takes (None: not reachable from here)."""
    if which == "cache":
        cache = small_cache(K)
        return cache.check_device_status, cache.workspace
    if which == "bf16":
        attention = K.Bf16Attention(batch=2, num_kv_heads=2, num_q_heads=4, head_dim=64)
        return attention.check_device_status, attention.workspace
    return K.kivi_static_scratch_status, None


@pytest.mark.parametrize("which", ["cache", "bf16", "static"])
def test_older_queries_clear_on_their_stream(kivi, which):
    """The word and a ticket set as a failed call leaves them, the query, and a read at once."""
    query, words = query_of(kivi, which)
    stream = torch.cuda.Stream()
    if words is not None:
        words[:64].fill_(0)  # loads the fill's kernel: loading one waits for what runs
    assert query(stream) == 0
    end = busy_default_stream()
    with torch.cuda.stream(stream):
        for _ in range(4):
            if words is not None:
                words[:64].fill_(1)
            assert query(stream) == (0 if words is None else 0x01010101)
            if words is not None:
                left = words[:64].cpu()
                assert left.count_nonzero() == 0
        assert query(stream) == 0
    assert not end.query(), "the query waited for the default stream"
    torch.cuda.synchronize()


def test_a_new_handle_is_clear_on_return(kivi):
    """No clear of a new handle's workspace is pending behind the default stream's work."""
    cache = small_cache(kivi)
    cache.workspace[:4].fill_(1)
    cache.close()
    stream = torch.cuda.Stream()
    end = busy_default_stream()
    with torch.cuda.stream(stream):
        cache = small_cache(kivi)
        assert end.query()
        cache.workspace[:4].fill_(1)
        assert cache.check_device_status(stream) == 0x01010101
        assert cache.check_device_status(stream) == 0
    cache.close()


def test_a_new_cache_takes_a_block_with_work_pending(kivi):
    """The workspace's memory held another tensor, whose last write on the stream is still to come."""
    sample = small_cache(kivi)
    shapes = [t.numel() for t in (sample.records, sample.resid_k, sample.resid_v, sample.workspace)]
    sample.close()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        torch.cuda.synchronize()
        old = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in shapes]
        torch.cuda._sleep(BUSY_CYCLES // 4)
        for t in old:
            t.fill_(1)
        del old, t
        cache = small_cache(kivi)
        assert cache.check_device_status(stream) == 0
    cache.close()


@pytest.mark.parametrize("raw", [False, True])
def test_paged_cache_query_clears_on_its_stream(kivi, raw):
    """Steps that fail on a stream beside a busy default stream: each query has its own step's bits."""
    cache = kivi.PagedCache(num_pages=4, page_size=16, num_layers=1, num_kv_heads=1, num_q_heads=2,
                            head_dim=64, max_requests=2, max_tokens=64)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    fits, pages, long = ints([1, 0]), ints([50, 50]), ints([65, 0])
    cache.assign(fits, 1)
    cache.assign(pages, 100)
    cache.check_device_status()
    end = busy_default_stream()
    for _ in range(3):
        cache.assign(pages, 100, stream=stream)
        assert cache.check_device_status(stream) == 8
        cache.assign(long, 100, stream=stream)
        assert cache.check_device_status(stream) == 4
        cache.assign(fits, 1, stream=stream)
        assert cache.check_device_status(stream) == 0
    assert not end.query(), "the query waited for the default stream"
    torch.cuda.synchronize()
    assert cache.lengths.tolist() == [4, 0]
