"""Batches of no rows and rows of no width: torch gives their tensors null
addresses, and there is nothing to do."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sl():
    from prng_seeded_decompress_b200 import build
    build.build()
    from prng_seeded_decompress_b200 import seedlm
    return seedlm


@pytest.mark.parametrize("M,cols", [(0, 64), (3, 0), (0, 0)])
def test_null_addresses_where_there_is_nothing(sl, M, cols):
    s = sl._NormStruct(cols, 0, 1, 1, 1, 1e-6, 0, 1, 1, None, None, None, None)
    assert sl.lib.seedlm_block_norm(ctypes.byref(s), M, None, cols, None, cols, None, cols, None, cols, 1, None, cols, 1,
                                    None) == 0
    assert sl.lib.seedlm_glu(M, cols, 0, None, 2 * cols, None, cols, 1, None) == 0
    # What can be told to be wrong without a row is refused all the same.
    s.kind = 2
    assert sl.lib.seedlm_block_norm(ctypes.byref(s), M, None, cols, None, cols, None, cols, None, cols, 1, None, cols, 1,
                                    None) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("M,cols", [(0, 64), (3, 0), (0, 0)])
def test_a_step_of_nothing(sl, M, cols):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    new = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    y, h, x = new(M, cols, t=torch.float32), new(M, cols), new(M, cols)
    nm = sl.BlockNorm(cols, w_post=new(cols), w_pre=new(cols))
    sl.block_norm(nm, y, h, h_out=h, x=x, gate=new(M, cols))
    sl.block_norm(nm, y, None, x=x)
    sl.block_norm(nm, None, h, h_out=h)
    sl.glu(new(M, 2 * cols, t=torch.float32), x)
    ad = sl.Adapters(new(2, 4, cols), new(2, cols, 4))
    plan = sl.adapter_plan(torch.zeros(M, dtype=torch.int32, device="cuda"), 2)
    sl.adapter_apply(ad, plan, x, y)
    torch.cuda.synchronize()
