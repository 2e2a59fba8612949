"""What the contract of the operators around the layer promises on the host."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import quantized_routed_expert_sigmoid_amd as qre
from quantized_routed_expert_sigmoid_amd import block

P = 1 << 20  # a well aligned address that no call here may touch


@pytest.fixture(scope="module")
def L():
    return block._f()


@pytest.mark.parametrize("N,K,bits,group", [(10240, 6144, 4, 0), (4096, 4096, 4, 0), (4096, 4096, 8, 128), (130, 2080, 2, 0),
                                            (64, 512, 8, 0), (1, 32768, 4, 32), (32768, 2048, 4, 64), (2100, 224, 4, 0)])
@pytest.mark.parametrize("out_type", [32, 16])
def test_linear_workspace_grows_with_the_batch(L, N, K, bits, group, out_type):
    """A workspace for S tokens serves every smaller batch: its size never falls."""
    w = qre.QBankDesc(data=P, row_scale=P, n_mat=1, rows=N, K=K, qtype=bits, group=group)
    sizes = sorted({1, 2, 4, 5, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 300, 333, 511, 512, 513, 640, 1000,
                    1023, 1024, 1025, 2047, 2048, 2049, 4095, 4096, 8191, 8192, 16384, 65535, 65536})
    most = [L.colibri_linear_workspace_bytes(ctypes.byref(w), S, out_type) for S in sizes]
    assert all(a <= b for a, b in zip(most, most[1:])), list(zip(sizes, most))


@pytest.mark.parametrize("heads,kv_heads,D", [(64, 8, 128), (8, 1, 64), (4, 4, 256), (48, 3, 192), (16, 16, 128)])
@pytest.mark.parametrize("type_", [32, 16])
def test_attention_workspace_grows_with_the_batch(L, heads, kv_heads, D, type_):
    """A workspace for a batch serves one with fewer sequences, rows, rows of a sequence or cached tokens."""
    c = block.KVCacheDesc(P, P, P, P, 64, kv_heads, D)

    def size(n_seq, n_tokens, max_q, max_kv):
        b = block.KVBatchDesc(None, None, None, n_seq, 0, n_tokens, max_q)
        a = block.KVAttnDesc(None, None, None, 0, 0, type_, heads, 1, 0, max_kv, 1.0)
        return L.colibri_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a))

    seqs, runs, kvs = (1, 2, 3, 5, 8, 16, 31, 32, 64, 100, 300), (1, 2, 3, 4, 5, 8, 9, 33, 128, 700, 2048), (1, 64, 500, 9000, 131072)
    whole = {(n, q, kv): size(n, n * q, q, kv) for n in seqs for q in runs for kv in kvs}
    for (n, q, kv), most in whole.items():
        less = [whole[m, r, k] for m in seqs for r in runs for k in kvs if m <= n and r <= q and k <= kv]
        assert most >= max(less), (n, q, kv)
        for tokens in (1, q, (n * q + 1) // 2):
            assert size(n, tokens, q, kv) <= most, (n, q, kv, tokens)
        assert most <= 1 << 28  # a few rows in many ranges, or many rows in few


def test_package_imports_without_private_torch_symbols():
    """A torch without the handles that the binding takes as a short cut (a CPU build) imports the package."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import quantized_routed_expert_sigmoid_amd as qre
try:
    qre.add_rms_norm(torch.zeros(2, 64), torch.ones(64))
except ValueError as e:
    print("refused:", e)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused: device tensor" in r.stdout, r.stderr


def test_workspace_tensors_lie_in_one_piece():
    """A view with gaps or repeats is refused: its bytes are not the ones that its size counts."""
    whole = torch.empty(64, dtype=torch.uint8)
    assert block._room(whole) == (whole.data_ptr(), 64) and block._room(torch.empty(8))[1] == 32
    for t in (whole[::2], whole[:1].expand(64), whole.view(8, 8).t(), whole.view(8, 8)[:, :4]):
        with pytest.raises(ValueError, match="ws: contiguous"):
            block._room(t)


@pytest.mark.parametrize("given,want", [(0, 0), (7, 7), (-1, -1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                        (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63, 2 ** 31 - 1), (5 - 2 ** 32, -1), (-2 ** 31 - 1, -1)])
def test_lengths_do_not_wrap(given, want):
    """A length beyond 32 bits counts as the largest, one below zero stays negative (and is refused)."""
    assert block._length(given) == want


def test_sizes_beyond_32_bits(L):
    """Plans and workspace sizes are computed in 64 bits: activations of 4 GiB, partial sums of 139 GB (a longest run
    of rows far below the real one), and a window beside which the cache's length is nothing."""
    w = qre.QBankDesc(data=P, row_scale=P, n_mat=1, rows=1 << 20, K=1 << 15, qtype=4, group=0)
    assert L.colibri_linear_workspace_bytes(ctypes.byref(w), 65536, 16) == (1 << 32) + 65536 * 4
    c = block.KVCacheDesc(P, P, P, P, 64, 8, 128)

    def size(n_tokens, window):
        b = block.KVBatchDesc(None, None, None, 1, 0, n_tokens, 1)
        a = block.KVAttnDesc(None, None, None, 0, 0, 32, 64, 1, window, 131072, 1.0)
        return L.colibri_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a))

    assert size(65536, 0) == 64 * 65536 * 64 * (128 * 4 + 8)  # 64 ranges
    for window in (131072, 2 ** 31 - 2, 2 ** 31 - 1):
        assert size(65536, window) == size(65536, 0)


@pytest.mark.parametrize("T,n,least,want", [
    (0, 0, 1024, 0), (7, 0, 1024, 7), (0, 5, 1024, 0), (64, 64, 1024, 1), (128, 32, 1024, 4), (50, 32, 1024, 2), (160, 32, 1024, 5),
    (512, 32, 1024, 16), (963, 64, 1024, 963), (2063, 64, 1024, 1024), (8000, 200, 1024, 1024), (32768, 16, 1024, 4096),
    (2048, 1, 1024, 2048), (5, 1, 1024, 5), (7000, 16, 8192, 7000)])
def test_expected_run_of_rows(T, n, least, want):
    """What is taken as the longest run of rows of a sequence where the caller does not say."""
    assert block._longest(T, n, least) == want
