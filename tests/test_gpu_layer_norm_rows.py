"""Layer norm on rows that 16-byte vectors do not divide, and on the widest: the checks and bounds of the small cases.

Short rows share vectors with many others, the last ones end inside the tensor's last vector, and the few lengths
below 16384 take one vector more than the others.
"""
import pytest
import torch

import test_gpu_layer_norm as M

pytestmark = pytest.mark.gpu
la = M.la
F32, BF16 = torch.float32, torch.bfloat16

CASES = [((5, 1), F32), ((9, 3), BF16), ((8, 3), F32), ((257, 5), BF16), ((2049, 33), F32), ((2047, 63), BF16),
         ((999, 121), BF16), ((100, 250), BF16), ((77, 1026), BF16), ((1000, 4099), BF16), ((33, 4102), F32),
         ((50, 8197), BF16), ((9, 16377), BF16), ((9, 16379), BF16), ((9, 16382), F32), ((700, 5120), BF16),
         ((400, 6144), F32), ((300, 8192), F32), ((300, 12000), BF16), ((200, 16384), BF16), ((170, 12288), F32),
         ((170, 16384), F32)]


@pytest.mark.parametrize("shape,dtype", CASES)
def test_fwd(la, shape, dtype):
    M.test_fwd(la, shape, dtype)


@pytest.mark.parametrize("shape,dtype", CASES)
def test_bwd(la, shape, dtype):
    M.test_bwd(la, shape, dtype)
