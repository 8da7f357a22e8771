"""The Python binding of the serving entry points reports wrong arguments as the library does."""
import pytest

import bit_matvec_lb_gb300 as lb


class Tensor:  # a tensor's face, without a GPU; never dereferenced
    is_cuda = True

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return 8


@pytest.mark.parametrize("stride", [0, -1, 3])
def test_mask_without_a_stride(stride):
    t = Tensor()
    with pytest.raises(lb.LBError) as e:
        lb.lb_logits_adjust(t, lb.OUT_F32, 100, t, 100, 2, 100, mask=t, mask_stride=stride, stream=0)
    assert e.value.status == -3
