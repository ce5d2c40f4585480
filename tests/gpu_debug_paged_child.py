"""Run by test_gpu_debug_paged.py in a child process whose KIVI_LIBRARY points at the debug build:
waits of the attention over pages and packed rows that run out after about 1 ms (not a test module).

The kernels are told to expect more bytes than their copies bring; every copy still lands whole."""
import sys

import torch

import paged_util as U
from gpu_util import load_kivi
from test_gpu_paged import BF16, FP16, Pool, gen_of, ints, offsets_of, randn, workspace


def cases(K):
    """(what, workspace, call, check) of each kernel and each way of joining cut items."""
    for what, lengths, new, hkv, hq, dim, dtype in [
            ("decode", [3000, 700, 64, 1], [1, 1, 1, 1], 2, 8, 128, BF16),
            ("decode of many", [100 + b for b in range(70)], [1] * 70, 1, 2, 64, FP16),
            ("chunks", [2100, 333, 64, 900], [1, 120, 64, 30], 2, 8, 128, BF16),
            ("chunks of many", [90 + b for b in range(40)], [b % 5 for b in range(40)], 1, 8, 64, FP16)]:
        gen = gen_of(len(lengths))
        pool, off = Pool(gen, lengths, hkv, dim, 32, dtype), offsets_of(new)
        q, ws = randn(gen, off[-1], hq, dim, dtype=dtype), workspace(K, hkv, hq, dim)
        kv, offsets = ints(lengths), ints(off)

        def call(pool=pool, q=q, ws=ws, kv=kv, offsets=offsets, new=new):
            return K.kivi_paged_attention(q, pool.k, pool.v, pool.table, kv, offsets, ws,
                                          max_new=max(new))

        def check(out, pool=pool, q=q, off=off, what=what):
            for b, (a, e) in enumerate(zip(off, off[1:])):
                U.assert_close(out[a:e], *U.attend(q[a:e], pool.keys[b], pool.values[b]),
                               f"{what}: request {b}")

        yield what, ws, call, check
    # few rows: cut items are joined by the second kernel; many: by their last CTA
    for what, lengths in [("packed", [700, 5, 300]), ("packed, joined by the last", [9000, 1, 1500])]:
        gen, off = gen_of(len(what)), offsets_of(lengths)
        q, k, v = (randn(gen, off[-1], h, 64) for h in (16, 2, 2))
        ws, offsets = workspace(K, 2, 16, 64), ints(off)

        def call(q=q, k=k, v=v, ws=ws, offsets=offsets):
            return K.kivi_packed_attention(q, k, v, offsets, ws)

        def check(out, q=q, k=k, v=v, off=off, what=what):
            for a, e in zip(off, off[1:]):
                for x in range(a, e, 1500):  # in parts
                    y = min(x + 1500, e)
                    U.assert_close(out[x:y], *U.attend(q[x:y], k[a:y], v[a:y]), f"{what}: {x}")

        yield what, ws, call, check


def waits_run_out(K, overstate):
    for what, ws, call, check in cases(K):
        check(call())
        assert K.kivi_attention_status(ws) == 0, what
        assert overstate(16) == 0
        call()
        code = K.kivi_attention_status(ws)
        assert code & 1, f"{what}: the waits did not report running out (status word {code})"
        assert ws[:8192].count_nonzero() == 0, f"{what}: the header is not clear"
        assert overstate(0) == 0
        for _ in range(2):
            check(call())
        assert K.kivi_attention_status(ws) == 0, what
        print(f"{what}: ok", flush=True)


if __name__ == "__main__":
    kivi = load_kivi()
    from decode_attention_kivi_b200 import _native

    waits_run_out(kivi, _native.lib().kivi_debug_overstate_copies)
    print("waits: ok")
    sys.exit(0)
