"""Block-scaled decode of more sequences than leave room for a long ring of stages in shared memory: short rings, with
items of every number of tiles one behind the other."""
import pytest

from tests import test_gpu_scaled as scaled

pytestmark = pytest.mark.gpu


@pytest.fixture
def pkv(pkv_lib, cuda_device):
    pkv_lib.device_error(reset=True)
    prev = pkv_lib.set_kernel_path(pkv_lib.PATH_TENSOR)
    yield pkv_lib
    pkv_lib.set_kernel_path(prev)
    assert pkv_lib.device_error(reset=True) == 0


CASES = [
    # act, Hq, Hkv, D, bs, partition, scales
    ("f16", 8, 1, 128, 16, 0, "narrow"),
    ("bf16", 8, 1, 128, 16, 0, "narrow"),
    ("f16", 8, 1, 128, 32, -1, "narrow"),
    ("bf16", 8, 1, 128, 16, 128, "wide"),
    ("f16", 8, 1, 64, 32, 0, "narrow"),
    ("bf16", 8, 1, 64, 16, -1, "wide"),
    ("bf16", 4, 1, 128, 16, 0, "narrow"),
    ("f16", 1, 1, 128, 16, 0, "narrow"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("rows", [700, 1030])
def test_many_sequences_with_items_of_every_length(pkv, case, rows):
    """Segments of four tiles followed by one to three more, so that an item begins at any stage of the ring."""
    lens = [(i * 131) % 385 + (514 if i % 3 else 0) for i in range(rows)]
    scaled._check_decode(pkv, case, lens)
