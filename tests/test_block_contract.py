"""What the contract of the operators around the layer promises on the host."""

import ctypes

import pytest

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
