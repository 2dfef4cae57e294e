"""What the second product gets to see of the sums between the two, S = x A^T:
sums of full 24-bit significands, from one row's largest down to 2^-24 of it.
bf16: three cut-off parts hold all 24 bits.  fp16: two rounded parts of the sum,
scaled by a power of two per row and 64 ranks, leave at most 2^-23 of it, or
2^-39 of the largest of those 64 where that is more."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHIFTS = 25


@pytest.fixture(scope="module")
def sl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from prng_seeded_decompress_b200 import build
    build.build()
    from prng_seeded_decompress_b200 import seedlm
    seedlm.init()
    return seedlm


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rank", [25, 90])
@pytest.mark.parametrize("M,outs", [(1, 96), (40, 96), (2048, 6000)])
def test_sums_of_24_bits_reach_the_outputs(sl, M, outs, rank, dtype):
    # S_r = (h + m / 2^8 + l / 2^16) 2^-k: three products of an 8-bit number and a
    # power of two, exact in either type; k = 0 .. 24, of which A takes what X's
    # fp16 range leaves.  Output j takes S_(j % rank) alone.
    g = torch.Generator().manual_seed(rank + M)
    h = torch.randint(128, 256, (M, rank), generator=g).double()
    m, l = (torch.randint(0, 256, (M, rank), generator=g).double() for _ in range(2))
    h[:, 0], m[:, 0], l[:, 0] = 128, 8, 1  # 1 + 2^-12 + 2^-23: two halves keep 1 + 2^-12
    l[:, 1::2] = l[:, 1::2] // 2 * 2 + 1   # odd: all 24 bits are needed
    k = torch.arange(rank) % SHIFTS
    k_x = k.clamp(max=16)
    X, A, B = torch.zeros(M, rank, 3).double(), torch.zeros(rank, rank, 3).double(), torch.zeros(outs, rank)
    for i, part in enumerate((h, m, l)):
        X[:, :, i] = part * 2.0 ** -k_x
        A[torch.arange(rank), torch.arange(rank), i] = 2.0 ** (-8 * i - (k - k_x)).double()
    B[torch.arange(outs), torch.arange(outs) % rank] = 1
    S = (h + m / 2 ** 8 + l / 2 ** 16) * 2.0 ** -k
    X, A = X.flatten(1), A.flatten(1)
    assert torch.equal(X.to(dtype).double(), X) and torch.equal(A.to(dtype).double(), A)
    ad = sl.Adapters(A.to(dtype).cuda()[None], B.to(dtype).cuda()[None])
    plan = sl.adapter_plan(torch.zeros(M, dtype=torch.int32, device="cuda"), 1)
    Y = torch.zeros(M, outs, device="cuda")
    sl.adapter_apply(ad, plan, X.to(dtype).cuda(), Y)
    got, want = Y.cpu().double(), S[:, torch.arange(outs) % rank]
    if dtype == torch.bfloat16:
        assert torch.equal(got, want)
    else:
        # The largest of the row's block of 64 ranks; the two parts are added up,
        # and added to Y, with at most half a step each, 2^-24 of the value.
        top = torch.cat([S[:, b:b + 64].max(1, keepdim=True)[0].expand(-1, min(64, rank - b)) for b in range(0, rank, 64)], 1)
        bound = torch.maximum(2.0 ** -23 * want, 2.0 ** -39 * top[:, torch.arange(outs) % rank]) + 2.0 ** -23 * want
        assert bool(((got - want).abs() <= bound).all())
