"""Scalar arguments at and past their limits through the host-side checks of
the 8-bit cache's and the block selection's entry points, with no CUDA device
visible: a call that passes its checks stops at its first CUDA call, so the
pointers below, which nothing may read, are never used.  Run by
tests/test_q8_sanitizers.py against a build whose host code has
UndefinedBehaviorSanitizer; a report aborts this process."""
import ctypes
import itertools
import os
import sys

import torch

if torch.cuda.is_available():   # never with a device: the pointers below are not real
    sys.exit("a CUDA device is visible; refusing to run")

L = ctypes.CDLL(sys.argv[1], mode=os.RTLD_LAZY)
vp, i32, i64, u64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
L.pkv_append_cache_q8.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i64, vp, vp]
L.pkv_summarize_blocks.argtypes = [vp, i32, vp, vp, i32, vp, i32, vp, vp, i32, i32, i32, i32, i32, i64, vp, vp]
L.pkv_select_blocks.argtypes = [vp, vp, i32, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32, i64, i32, i32, i32, i32, vp, u64, vp, vp]
L.pkv_select_blocks_workspace_bytes.argtypes = [i32] * 4
L.pkv_select_blocks_workspace_bytes.restype = u64
L.pkv_paged_attention_list_workspace_bytes.argtypes = [i32] * 7
L.pkv_paged_attention_list_workspace_bytes.restype = u64
L.pkv_paged_attention_decode_q8.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, i32, f32,
                                            i32, vp, u64, vp, vp]
L.pkv_paged_attention_decode_selected.argtypes = [vp, i32, vp, i32, vp, vp, i32, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32,
                                                  i32, i64, i32, f32, i32, vp, u64, vp, vp]
P, BIG = 16 * 1024, 2**31 - 1
EDGES = [-2**31, -1, 0, 1, 8, 32, 65535, 65536, BIG]
n = 0
for a in itertools.product(EDGES, repeat=4):
    L.pkv_select_blocks_workspace_bytes(*a)
    n += 1
for a in itertools.product([0, 1, 65535, BIG], [1, 8, BIG], [1, 8, BIG], [1, 128, BIG], [1, 8, 31, 32, BIG], [0, 1, 4096, BIG],
                           [-1, 0, 32, 2**31 - 32, BIG]):
    L.pkv_paged_attention_list_workspace_bytes(*a)
    n += 1
for B, T, Hk, D, bs, mb, nb in itertools.product([0, 1, 65536, BIG], [0, 1, BIG], [1, 3, 65535, BIG], [64, 128, BIG], [8, 32, BIG],
                                                 [1, 2**26, BIG], [1, BIG, 2**63 - 1]):
    for qs in (P, None):
        L.pkv_append_cache_q8(P, P, 2, P, P, P, P, P, mb, P, qs, B, T, Hk, D, bs, nb, P, None)
        L.pkv_summarize_blocks(P, 3, P, P, 2, P, mb, P, qs, B, T, Hk, D, bs, nb, P, None)
        n += 2
for mb, B, H, Hk, D, bs, mcl, K in itertools.product([1, 2**20, BIG], [0, 1, 65535, BIG], [1, 8, BIG], [1, 8, 65536], [64, 128, BIG],
                                                     [8, 32, BIG], [0, 1, 2**20, BIG], [1, 64, BIG]):
    for part in (0, 32, 2**31 - 32):
        L.pkv_paged_attention_decode_q8(P, 0, P, 2, P, P, P, P, P, mb, P, B, H, Hk, D, bs, BIG, mcl, 1.0, part, P, 2**62, P, None)
        L.pkv_paged_attention_decode_selected(P, 0, P, 2, P, P, 3, P, P, P, mb, P, P, K, B, H, Hk, D, bs, BIG, mcl, 1.0, part, P,
                                              2**62, P, None)
        n += 2
    for first, last in ((0, 0), (1, 0), (BIG, BIG)):
        L.pkv_select_blocks(P, P, 2, P, 2, P, mb, P, B, H, Hk, D, bs, BIG, mcl, K, first, last, P, 2**62, P, None)
        n += 1
print("calls", n)
