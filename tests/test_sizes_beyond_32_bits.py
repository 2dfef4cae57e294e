"""Sizes that the library counts in 32 bits and that do not fit are refused by
the binding, never cut off (tensors of no memory stand for the large ones)."""
import pytest

torch = pytest.importorskip("torch")

BIG = 2 ** 32 + 64  # cut off to 32 bits: 64


@pytest.fixture(scope="module")
def sl():
    from prng_seeded_decompress_b200 import build
    build.build()
    from prng_seeded_decompress_b200 import seedlm
    return seedlm


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def refused(call, *args, **kw):
    with pytest.raises(ValueError, match="32 bits"):
        call(*args, **kw)


def test_plans_and_workspaces(sl):
    refused(sl.AdapterPlan, BIG, 3, device="cpu")
    refused(sl.AdapterPlan, 3, BIG, device="cpu")
    refused(sl.AdapterPlan, -BIG, 3, device="cpu")
    refused(sl.adapter_plan, meta(BIG, dtype=torch.int32), 3)
    ad = sl.Adapters(meta(3, 8, 64), meta(3, 32, 8))
    refused(sl.adapter_workspace_bytes, ad, BIG)


@pytest.mark.parametrize("n,rank,cols,rows", [(BIG, 8, 64, 32), (3, BIG, 64, 32), (3, 8, BIG, 32), (3, 8, 64, BIG)])
def test_adapters(sl, n, rank, cols, rows):
    refused(sl.Adapters, meta(n, rank, cols), meta(n, rows, rank))


def test_norms_and_glu(sl):
    refused(sl.BlockNorm, BIG)
    nm = sl.BlockNorm(64)
    refused(sl.block_norm, nm, meta(BIG, 64, dtype=torch.float32), None, x=meta(BIG, 64))
    refused(sl.glu, meta(BIG, 128, dtype=torch.float32), meta(BIG, 64))
    refused(sl.glu, meta(3, 2 * BIG, dtype=torch.float32), meta(3, BIG))
