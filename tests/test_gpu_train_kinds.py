"""The shared expert's training calls in every kind of launch (test_train_kinds.LAYERS) against float64, with the bounds
of test_gpu_train_large.  Tiles and splits are what the library says for the size."""

import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B
from tests.test_gpu_train_large import test_every_tile_configuration as check_call
from tests.test_train_kinds import BF, LAYERS, LAYOUTS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.load()


@pytest.mark.parametrize("layout", LAYOUTS, ids=["kn", "nk"])
@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "x".join(map(str, c)))
def test_every_kind_of_launch(case, layout):
    tiles, *splits = B.moe_shared_train_tiles(BF, *case, layout)
    check_call(case, tiles, tuple(splits), layout)
