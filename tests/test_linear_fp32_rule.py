"""Which fp32 products go to the tensor cores, told by the workspace they ask for, against times of both forms
measured on a B200 (us).  Runs without a GPU: the rule does not depend on the device."""
import pytest

import mhc_hyper_connections_b200 as mhc

torch = pytest.importorskip("torch")
F32 = torch.float32

# T, K, N: forward from bf16 parts, forward on CUDA cores, backward from parts, backward on CUDA cores
MEASURED = [(9, 4096, 4096, 93.8, 56.0, 134.2, 96.1), (16, 1024, 4096, 28.9, 16.5, 47.1, 40.2),
            (17, 2880, 1536, 28.5, 36.8, 49.7, 47.1), (24, 4096, 1024, 28.1, 41.8, 49.2, 41.3),
            (24, 1024, 4096, 27.8, 22.2, 49.6, 88.2), (48, 1024, 1024, 17.7, 13.5, 34.6, 26.7),
            (48, 1024, 4096, 27.9, 22.9, 50.2, 93.5), (64, 2880, 1536, 28.7, 38.6, 50.4, 55.8),
            (64, 4096, 4096, 93.7, 77.1, 137.0, 153.9), (65, 4096, 4096, 93.7, 148.9, 139.6, 234.0),
            (65, 1024, 4096, 28.4, 42.4, 51.7, 100.9), (65, 4096, 1024, 28.8, 62.0, 51.3, 68.5),
            (128, 512, 512, 17.5, 9.0, 33.6, 22.3), (192, 1001, 777, 19.9, 26.1, 42.1, 45.5),
            (192, 4096, 1024, 31.2, 75.3, 54.6, 127.8), (512, 512, 512, 17.2, 14.4, 38.3, 31.2),
            (1024, 256, 256, 15.1, 12.8, 35.5, 28.7), (1024, 512, 512, 19.1, 24.9, 40.3, 48.3),
            (2048, 256, 256, 15.7, 15.7, 37.5, 52.8), (2048, 4096, 1024, 103.2, 580.3, 206.5, 915.7)]


@pytest.mark.parametrize("T,K,N,fp,fc,bp,bc", MEASURED)
def test_the_faster_form_is_taken(T, K, N, fp, fc, bp, bc):
    parts = mhc.mhc_linear_workspace_bytes(T, K, N, F32) >= 6 * (T + N) * K     # three bf16 planes of x and W
    assert (fp if parts else fc) <= 1.1 * min(fp, fc)
    parts = mhc.mhc_linear_backward_workspace_bytes(T, K, N, F32) >= 6 * (T * K + N * K + T * N)
    assert (bp if parts else bc) <= 1.1 * min(bp, bc)
