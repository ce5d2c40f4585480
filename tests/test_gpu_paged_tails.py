"""Rows with a few strong keys and a long tail of weak ones (needs a B200): the tail's weights lie
around 2^-25 of the largest, where fp16 has lost its bits, and all of the output comes from them.

Tolerance: that of paged_util, with two of its terms for these inputs.
  - sum |q k| / sqrt(D) stays below 32 here, not 16, so the scores' part is 2 * 2^-11.
  - A weight is rounded to fp16 after a factor that brings the row's largest to 2^6 at least, so
    one in the subnormal range is off by at most half a step, 2^-25, which is 2^-31 of the largest;
    the L weights' errors are at most L 2^-31 max |v| of the output.
"""
import pytest
import torch

import paged_util as U
from gpu_util import load_kivi
from test_gpu_paged import BF16, FP16, Pool, gen_of, ints, offsets_of, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kivi():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    return load_kivi()


def tail_rows(gen, L, hkv, dim, strong, depth, dtype):
    """Keys and values of one request: the keys `strong` score 2^depth times the others and have
    values of zero, the others values around 16."""
    k = torch.randn(L, hkv, dim, generator=gen, device="cuda")
    k[..., 0] = 0.0
    k[strong, :, 0] = depth * 0.6931472 * dim ** 0.5 / 8.0  # q is 8 there
    v = 16.0 + torch.randn(L, hkv, dim, generator=gen, device="cuda")
    v[strong] = 0.0
    return k.to(dtype), v.to(dtype)


def tail_queries(gen, n, hq, dim, dtype):
    q = 0.05 * torch.randn(n, hq, dim, generator=gen, device="cuda")
    q[..., 0] = 8.0
    return q.to(dtype)


def check(got, q, k, v, what):
    u, L = torch.finfo(got.dtype).eps / 2, k.shape[0]
    assert (q.abs().amax(0).double().amax(0) * k.abs().double().amax((0, 1))).sum() \
        / q.shape[-1] ** 0.5 < 32
    out, mean = U.attend(q, k, v)
    err = (got.double() - out).abs()
    bound = (3 * u + 2 * 2.0 ** -11) * mean + 1e-6 + L * 2.0 ** -31 * v.abs().max().item()
    assert torch.isfinite(got).all() and (err <= bound).all(), \
        f"{what}: max err {err.max().item():.3e} of {mean.max().item():.3e}"


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("depth", [17.0, 25.5])
@pytest.mark.parametrize("requests,L,new,ratio,dim", [
    (160, 4096, 1, 2, 64),      # an item or so per SM
    (1, 131072, 1, 4, 64),      # cut into many pieces
    (2, 20000, 40, 4, 128),     # a chunk
    (1, 131072, 70, 2, 64)])
def test_tail_over_pages(kivi, requests, L, new, ratio, dim, depth, dtype):
    gen = gen_of(L + new)
    pool = Pool(gen, [L] * requests, 1, dim, 64, dtype)
    j = torch.arange(L, device="cuda")
    for b in range(requests):
        # one strong key for each 16 keys of the first tile
        pool.keys[b], pool.values[b] = tail_rows(gen, L, 1, dim, [3, 21, 40, 63], depth, dtype)
        ids = pool.table[b].long()[j // 64]
        pool.k[ids, :, j % 64] = pool.keys[b]
        pool.v[ids, :, j % 64] = pool.values[b]
    q = tail_queries(gen, requests * new, ratio, dim, dtype)
    ws = workspace(kivi, 1, ratio, dim)
    got = kivi.kivi_paged_attention(q, pool.k, pool.v, pool.table, ints([L] * requests),
                                    ints(offsets_of([new] * requests)), ws, max_new=new)
    for b in range(requests):
        at = slice(b * new, (b + 1) * new)
        check(got[at], q[at], pool.keys[b], pool.values[b], f"request {b}")
    assert kivi.kivi_attention_status(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("depth", [17.0, 25.5])
def test_tail_of_a_packed_prompt(kivi, depth, dtype):
    gen, n = gen_of(77), 9000
    k, v = tail_rows(gen, n, 2, 128, [0, 21, 40, 63], depth, dtype)
    q = tail_queries(gen, n, 4, 128, dtype)
    ws = workspace(kivi, 2, 4, 128)
    got = kivi.kivi_packed_attention(q, k, v, ints([0, n]), ws)
    for a in range(0, n, 3000):  # in parts: the rows a .. a + 2999 see the keys up to their own
        check(got[a:a + 3000], q[a:a + 3000], k[:a + 3000], v[:a + 3000], f"rows from {a}")
    assert kivi.kivi_attention_status(ws) == 0
