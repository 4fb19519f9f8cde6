"""The branch norm's gradients on long rows of which a block takes more than one: the sums
that are kept from row to row, in shared memory or in the block's row of the workspace."""
import pytest

import test_gpu_add_rmsnorm as norm

pytestmark = pytest.mark.gpu


# more rows than SMs, on 16-byte boundaries and off them; rows of more than 65536 values,
# of more than fit in shared memory, and of some that fit
@pytest.mark.parametrize("shape,types", [((160, 65544), ("bf16", "f32")), ((160, 50008), ("f32", "f32")),
                                         ((330, 20001), ("bf16", "bf16"))])
def test_backward_of_many_long_rows(ro, shape, types):
    norm.test_backward(ro, shape, types)
