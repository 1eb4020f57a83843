"""Scalar arguments at and past their limits through the host-side checks of
the 4-bit cache's entry points, with no CUDA device visible: a call that passes
its checks stops at its first CUDA call, so the pointers below, which nothing
may read, are never used.  Run by tests/test_q4_sanitizers.py against a build
whose host code has UndefinedBehaviorSanitizer; a report aborts this process."""
import ctypes
import itertools
import os
import sys

import torch

if torch.cuda.is_available():   # never with a device: the pointers below are not real
    sys.exit("a CUDA device is visible; refusing to run")

L = ctypes.CDLL(sys.argv[1], mode=os.RTLD_LAZY)
vp, i32, i64, u64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
L.pkv_reshape_and_cache_q4.argtypes = [vp, i64, vp, i64, i32, vp, vp, vp, i32, i32, i32, i32, i64, vp, vp]
L.pkv_gather_cache_q4.argtypes = [vp, i64, vp, i64, i32, vp, vp, i32, vp, i32, i32, i32, i32, i64, vp, vp]
L.pkv_paged_attention_decode_q4.argtypes = [vp, i32, vp, i64, i32, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, i32, f32,
                                            i32, vp, u64, vp, vp]
L.pkv_paged_attention_q4_workspace_bytes.argtypes = [i32] * 7
L.pkv_paged_attention_q4_workspace_bytes.restype = u64
P, BIG, HUGE = 16 * 1024, 2**31 - 1, 2**63 - 1
n = 0
for a in itertools.product([-1, 0, 1, 65535, BIG], [0, 1, 8, BIG], [0, 1, 8, BIG], [1, 128, BIG], [-1, 8, 31, 32, BIG], [-1, 0, 1, 4096, BIG],
                           [-1, 0, 32, 2**31 - 32, BIG]):
    L.pkv_paged_attention_q4_workspace_bytes(*a)
    n += 1
for T, Hk, D, bs, nb, st in itertools.product([0, 1, 2, BIG], [1, 3, 65535, BIG], [64, 128, BIG], [8, 32, BIG], [1, BIG, HUGE],
                                              [-HUGE - 1, -8, 0, 128, 65535 * 128, 2**40, HUGE - 7, HUGE]):
    L.pkv_reshape_and_cache_q4(P, st, P, st, 2, P, P, P, T, Hk, D, bs, nb, P, None)
    L.pkv_gather_cache_q4(P, st, P, st, 0, P, P, 1, P, T, Hk, D, bs, nb, P, None)
    n += 2
for mb, B, H, Hk, D, bs, mcl, part, st in itertools.product([1, 2**20, BIG], [0, 1, 2, 65535, BIG], [1, 8, BIG], [1, 8, 65536], [64, 128, BIG],
                                                            [8, 32, BIG], [0, 1, 2**20, BIG], [0, 32, 2**31 - 32], [0, 2**20, HUGE]):
    L.pkv_paged_attention_decode_q4(P, 0, P, st, 2, P, P, P, mb, P, B, H, Hk, D, bs, BIG, mcl, 1.0, part, P, 2**62, P, None)
    n += 1
print("calls", n)
