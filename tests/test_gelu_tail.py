"""The gated GELU's negative tail, where 1 + erf(g / sqrt 2) cancels: relative to
the value, against 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from prng_seeded_decompress_b200 import build
    build.build()
    from prng_seeded_decompress_b200 import seedlm
    seedlm.init()
    return seedlm


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,cols", [(1, 4096), (3, 1001), (40, 200), (2, 6000)])
def test_relative_error_of_the_negative_tail(sl, M, cols, dtype):
    # In units of 2^-23, relative, for g <= 0 (m = -g; Q(m) = e^(-m^2/2) t P(t),
    # t = 1 / (1 + 0.35 m)): P's fit 0.3; t 1.5 (half for the sum, one for the
    # reciprocal), which counts |d ln(t P) / d ln t| <= 2.3 times, at m = 0; the
    # last steps of P and its product with t 1.5; the exponential 2 + 1.2 m^2 / 2
    # (its table entry), its argument's rounding m^2 / 4; two more products 1.
    # Together less than g^2 + 9.  Above 0 the value is g - g Q, off by less.
    # Down to -12.5 e^(-m^2/2) is a normal fp32 number.
    gate = torch.linspace(-12.5, 1.0, M * cols).view(M, cols)[:, torch.randperm(cols, generator=torch.Generator().manual_seed(1))]
    # fp16 ends at 6e-8: the factor brings the tail into its range, up to 2^15.
    ref = 0.5 * gate.double() * torch.special.erfc(-gate.double() / 2 ** 0.5)
    up = 2.0 ** torch.floor(4 - torch.log2(ref.abs().clamp(min=1e-40)).clamp(min=-100)) if dtype == "f16" else torch.ones(M, cols, dtype=torch.float64)
    GU = torch.cat([gate, up.float()], 1)
    X = torch.empty(M, cols, dtype=DT[dtype], device="cuda")
    sl.glu(GU.cuda(), X, act="gelu")
    ref = ref * up.float().double()
    bound = (torch.finfo(DT[dtype]).eps / 2 + (gate.double() ** 2 + 9) * 2.0 ** -23) * ref.abs()
    assert bool(((X.cpu().double() - ref).abs() <= bound + 2.0 ** -25).all() if dtype == "f16"
                else ((X.cpu().double() - ref).abs() <= bound).all())
