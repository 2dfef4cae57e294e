"""Low-rank adapters of many requests beside a shared projection: the plan that
sorts a batch's rows by adapter, and Y = base + s_a (x A_a^T) B_a^T.

Two kinds of numbers are used.  Small whole numbers, with scales that are
powers of two: every product and every partial sum is a whole number below
2^24 times a power of two, exact in fp32 in any order of summation, so the
result has to equal the 64-bit one bit for bit (a sum between the two products
that were rounded to 16 bits would not).  And normal numbers, under a bound
from the arithmetic: the first product adds at most cols / 16 + 16 times to
one fp32 sum (16 products at a time), the second at most rank times, each
addition and each kept or scaled value is off by at most one unit in the last
place, 2^-23 of the sum of the absolute values."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sl():
    from prng_seeded_decompress_b200 import build
    build.build()
    from prng_seeded_decompress_b200 import seedlm
    return seedlm


@pytest.fixture(scope="module")
def gpu(sl):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sl.init()
    return sl


# ------------------------------------------------------- refusals (no GPU)

def _struct(sl, **kw):
    s = sl._AdaptersStruct(4, 16, 64, 1, 1)
    s.rows[0], s.A[0], s.B[0] = 32, 0x1000, 0x2000
    s.a_adapter[0], s.a_row[0], s.b_adapter[0], s.b_row[0] = 1024, 64, 512, 16
    for k, v in kw.items():
        if k in ("rows", "A", "B", "a_adapter", "a_row", "b_adapter", "b_row"):
            getattr(s, k)[0] = v
        else:
            setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), -1), (dict(rank=0), -1), (dict(cols=-1), -1), (dict(slices=0), -1), (dict(dtype=2), -1),
    (dict(n=1025), -2), (dict(rank=257), -2), (dict(slices=5), -2), (dict(rows=-1), -1),
    (dict(cols=(1 << 30) + 1), -2), (dict(rows=(1 << 30) + 1), -2),
    (dict(A=0), -1), (dict(B=0), -1), (dict(A=0x1001), -1), (dict(B=0x2001), -1), (dict(a_adapter=-1), -1),
    (dict(a_row=-1), -1), (dict(b_adapter=-1), -1), (dict(b_row=-1), -1), (dict(ranks=0x3002), -1),
    (dict(scales=0x3002), -1),
])
def test_bad_adapters_are_refused_before_cuda(sl, kw, code):
    s = _struct(sl, **kw)
    assert sl.lib.seedlm_adapters_apply(ctypes.byref(s), 0x4000, 3, 0x5000, 64, None, 0, 0x6000, 32, 0x7000,
                                        1 << 20, None) == code
    assert sl.lib.seedlm_adapters_workspace_bytes(ctypes.byref(s), 3) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(plan=None), -1), (dict(plan=0x4004), -1), (dict(M=-1), -1), (dict(M=(1 << 24) + 1), -2),
    (dict(X=None), -1), (dict(X=0x5001), -1), (dict(ldx=63), -1), (dict(Y=None), -1), (dict(Y=0x6002), -1),
    (dict(ldy=31), -1), (dict(base=0x8002, ldb=32), -1), (dict(base=0x8000, ldb=31), -1),
    (dict(base=0x6000, ldb=40), -1), (dict(wsb=-1), -1),
])
def test_bad_calls_are_refused_before_cuda(sl, kw, code):
    a = dict(plan=0x4000, M=3, X=0x5000, ldx=64, base=None, ldb=0, Y=0x6000, ldy=32, ws=0x7000, wsb=1 << 20)
    a.update(kw)
    s = _struct(sl)
    assert sl.lib.seedlm_adapters_apply(ctypes.byref(s), a["plan"], a["M"], a["X"], a["ldx"], a["base"], a["ldb"],
                                        a["Y"], a["ldy"], a["ws"], a["wsb"], None) == code


def test_plan_arguments_and_empty_work(sl):
    L = sl.lib
    assert L.seedlm_adapters_apply(None, 0x4000, 3, 0x5000, 64, None, 0, 0x6000, 32, 0x7000, 1 << 20, None) == -1
    for M, n, code in ((-1, 4, -1), (4, 0, -1), ((1 << 24) + 1, 4, -2), (4, 1025, -2)):
        assert L.seedlm_adapters_plan(M, n, 0x1000, 0x2000, None) == code
        assert L.seedlm_adapters_plan_words(M, n) == -1
    assert L.seedlm_adapters_plan(4, 4, None, 0x2000, None) == -1
    assert L.seedlm_adapters_plan(4, 4, 0x1002, 0x2000, None) == -1
    assert L.seedlm_adapters_plan(4, 4, 0x1000, None, None) == -1
    assert L.seedlm_adapters_plan(4, 4, 0x1000, 0x2004, None) == -1
    for M, n in ((0, 1), (1, 1), (64, 64), (1 << 24, 1024)):
        assert L.seedlm_adapters_plan_words(M, n) >= M + n + 1 + 4
    # No rows, or no outputs: nothing to do, nothing touched.
    s = _struct(sl)
    assert L.seedlm_adapters_apply(ctypes.byref(s), None, 0, None, 0, None, 0, None, 0, None, 0, None) == 0
    s = _struct(sl, rows=0, A=0, B=0)
    assert L.seedlm_adapters_apply(ctypes.byref(s), None, 5, None, 0, None, 0, None, 0, None, 0, None) == 0


def test_binding_refuses_what_it_cannot_pass(sl):
    A, B = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 32, 8, dtype=torch.bfloat16)
    ok = sl.Adapters(A, B)
    assert (ok.n, ok.rank, ok.cols, ok.rows, ok.total_rows) == (3, 8, 64, [32], 32)
    two = sl.Adapters([A, A], [B, B[:, :5]])
    assert two.rows == [32, 5] and two.struct.slices == 2
    with pytest.raises(ValueError):
        sl.Adapters([A] * 5, [B] * 5)
    with pytest.raises(ValueError):
        sl.Adapters([A, A], [B])
    with pytest.raises(ValueError):
        sl.Adapters(A, B[:2])
    with pytest.raises(ValueError):
        sl.Adapters(A, B[:, :, :4])
    with pytest.raises(ValueError):
        sl.Adapters(A[0], B[0])
    with pytest.raises(ValueError, match="unit stride"):
        sl.Adapters(A.transpose(1, 2).contiguous().transpose(1, 2), B)
    with pytest.raises(TypeError):
        sl.Adapters(A, B.half())
    with pytest.raises(TypeError):
        sl.Adapters(A.float(), B.float())
    with pytest.raises(TypeError):
        sl.Adapters(A, B, ranks=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        sl.Adapters(A, B, scales=torch.zeros(2))
    with pytest.raises(sl.SeedLMError):
        sl.AdapterPlan(4, 0, device="cpu")
    plan = sl.AdapterPlan(4, 3, device="cpu")
    assert plan.order.shape == (4,) and plan.offsets.shape == (4,)
    with pytest.raises(TypeError):
        sl.adapter_plan(torch.zeros(4, dtype=torch.int64), 3, plan=plan)
    with pytest.raises(ValueError, match="contiguous"):
        sl.adapter_plan(torch.zeros(8, dtype=torch.int32)[::2], 3, plan=plan)
    with pytest.raises(ValueError, match="the plan is for"):
        sl.adapter_plan(torch.zeros(5, dtype=torch.int32), 3, plan=plan)
    with pytest.raises(ValueError, match="CUDA"):
        sl.adapter_plan(torch.zeros(4, dtype=torch.int32), 3, plan=plan)
    X, Y, ws = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 32), torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(TypeError):
        sl.adapter_apply(ok, plan, X.half(), Y, workspace=ws)
    with pytest.raises(TypeError):
        sl.adapter_apply(ok, plan, X, Y.half(), workspace=ws)
    with pytest.raises(ValueError, match="4 x 64"):
        sl.adapter_apply(ok, plan, X[:3], Y, workspace=ws)
    with pytest.raises(ValueError, match="4 x 32"):
        sl.adapter_apply(ok, plan, X, Y[:, :31], workspace=ws)
    with pytest.raises(ValueError, match="unit column stride"):
        sl.adapter_apply(ok, plan, X, torch.zeros(32, 4).t(), workspace=ws)
    with pytest.raises(ValueError, match="4 x 32"):
        sl.adapter_apply(ok, plan, X, Y, base=Y[:2], workspace=ws)
    with pytest.raises(ValueError, match="adapters"):
        sl.adapter_apply(ok, sl.AdapterPlan(4, 2, device="cpu"), X, Y, workspace=ws)
    with pytest.raises(ValueError, match="CUDA"):
        sl.adapter_apply(ok, plan, X, Y, workspace=ws)


# ---------------------------------------------------------------- the plan

def check_plan(ids, n, plan):
    ids = np.asarray(ids)
    key = np.where((ids >= 0) & (ids < n), ids, n)
    assert np.array_equal(plan.order.cpu().numpy(), np.argsort(key, kind="stable"))
    assert np.array_equal(plan.offsets.cpu().numpy(), np.searchsorted(np.sort(key), np.arange(n + 1)))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [0, 1, 2, 31, 32, 33, 256, 257, 1000, 4097, 70000])
@pytest.mark.parametrize("n", [1, 2, 33, 1023, 1024])
def test_plan_sorts_rows_by_adapter(gpu, M, n):
    rng = np.random.default_rng(M * 1031 + n)
    kinds = [rng.integers(-1, n, M), np.full(M, n - 1), np.full(M, -1), np.sort(rng.integers(0, n, M))[::-1],
             np.where(rng.random(M) < 0.3, rng.choice([-2 ** 31, -7, n, n + 5, 2 ** 31 - 1], M), rng.integers(0, n, M))]
    plan = gpu.AdapterPlan(M, n)
    for ids in kinds:
        t = torch.from_numpy(np.ascontiguousarray(ids.astype(np.int32))).cuda()
        assert gpu.adapter_plan(t, n, plan=plan) is plan
        check_plan(ids, n, plan)


# ------------------------------------------------------------ the products

def make(M, cols, rows, n, rank, dtype, kind, seed, pad=0, off=0, ranks="mixed", none=0.15):
    """Inputs on the GPU.  pad widens every row stride, off moves every array
    that many elements from an aligned address; what lies in the padding and
    beyond an adapter's rank is NaN."""
    g = torch.Generator().manual_seed(seed)

    def values(shape, dt, lo=3 if cols * rank < 500000 else 1):
        if kind == "whole":
            return torch.randint(-lo, lo + 1, shape, generator=g).to(dt)
        return torch.randn(shape, generator=g).to(dt)

    def placed(t):
        *lead, last = t.shape
        buf = torch.full((off + int(np.prod(lead, dtype=np.int64)) * (last + pad),), float("nan"), dtype=t.dtype,
                         device="cuda")
        v = buf[off:].view(*lead, last + pad)[..., :last]
        v.copy_(t)
        return v

    dt = DT[dtype]
    r = torch.full((n,), rank, dtype=torch.int32)
    if ranks == "mixed":
        r = torch.randint(0, rank + 1, (n,), generator=g).to(torch.int32)
        r[torch.randint(0, n, (1,), generator=g)] = rank
    beyond = torch.arange(rank)[None, :] >= r[:, None]
    d = dict(X=values((M, cols), dt), base=values((M, sum(rows)), torch.float32, 1000), ranks=r)
    d["A"] = [values((n, rank, cols), dt).masked_fill(beyond[:, :, None], float("nan")) for _ in rows]
    d["B"] = [values((n, R, rank), dt).masked_fill(beyond[:, None, :], float("nan")) for R in rows]
    d["scales"] = 2.0 ** torch.randint(0, 3, (n,), generator=g).float() if kind == "whole" else \
        torch.rand(n, generator=g) + 0.5
    ids = torch.randint(0, n, (M,), generator=g)
    ids[torch.rand(M, generator=g) < none] = -1
    d["ids"] = ids.to(torch.int32)
    out = {k: placed(v) for k, v in d.items() if k in ("X", "base")}
    for k in ("A", "B"):
        out[k] = [placed(v) for v in d[k]]
    out |= {k: d[k].cuda() for k in ("ranks", "scales", "ids")}
    out["placed"] = placed
    return out


def reference(d, base=None):
    """(Y, sum of absolute values) in 64 bits."""
    ids, base = d["ids"].cpu(), (d["base"] if base is None else base).cpu().double()
    Y, mag = base.clone(), base.abs()
    X = d["X"].cpu().double()
    for a in range(d["ranks"].numel()):
        rows, r, j = (ids == a).nonzero().flatten(), int(d["ranks"][a]), 0
        s = float(d["scales"][a])
        for A, B in zip(d["A"], d["B"]):
            Aa, Ba = A[a, :r].cpu().double(), B[a, :, :r].cpu().double()
            R = B.shape[1]
            Y[rows, j:j + R] += s * (X[rows] @ Aa.T) @ Ba.T
            mag[rows, j:j + R] += abs(s) * (X[rows].abs() @ Aa.abs().T) @ Ba.abs().T
            j += R
    return Y, mag


def apply(sl, d, Y, base=None, workspace=None, plan=None, stream=None):
    ad = sl.Adapters(d["A"], d["B"], ranks=d["ranks"], scales=d["scales"])
    plan = plan or sl.adapter_plan(d["ids"], ad.n, stream=stream)
    sl.adapter_apply(ad, plan, d["X"], Y, base=base, workspace=workspace, stream=stream)
    return Y


#: M, cols, rows of the slices, adapters, rank: one token to many, sides that
#: divide nothing, one of everything, every slice count.
LOW = [
    (1, 64, [32], 1, 8), (1, 8192, [1024], 3, 16), (2, 1, [1], 2, 1), (3, 7, [5], 2, 3), (5, 4099, [1021], 4, 12),
    (8, 256, [128], 1, 16), (9, 256, [128], 1, 64), (64, 512, [96, 40], 64, 20), (37, 1024, [256, 64, 64], 20, 16),
    (100, 300, [33, 1, 70, 31], 6, 37), (255, 96, [64], 300, 8), (256, 130, [130], 5, 130), (257, 130, [130], 5, 130),
    (300, 1000, [500], 1, 256), (333, 513, [127], 7, 12), (700, 64, [1000, 24], 3, 16), (1025, 264, [72], 1024, 4),
    (17, 20000, [16], 2, 256), (600, 9001, [64], 2, 8), (64, 0, [40], 3, 8), (30, 2000, [300], 2, 256),
    (60, 9001, [64], 2, 8),
]
#: The same for batches that take tiles of 64 rows.
TALL = [
    (2000, 2000, [2000], 3, 16), (2100, 4099, [1021], 7, 12), (1500, 2048, [1024, 512, 520], 2, 64),
    (3000, 1000, [2001, 33], 5, 37), (1200, 3001, [4000], 1, 130), (1300, 2500, [3000], 2, 256),
    (2600, 64, [6000], 9, 4), (2500, 9000, [64], 2, 8), (4096, 1024, [2048], 40, 20), (3000, 0, [9000], 2, 8),
    (2049, 1, [7001], 1, 1), (1800, 5000, [258], 2, 97),
]
SHAPES = LOW + TALL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("M,cols,rows,n,rank", SHAPES)
def test_whole_numbers_are_exact(gpu, M, cols, rows, n, rank, pad, off, dtype):
    d = make(M, cols, rows, n, rank, dtype, "whole", M + cols + rank, pad, off)
    ref, mag = reference(d)
    assert float(mag.max()) < 2 ** 24  # so every partial sum is exact
    Y = d["placed"](torch.full((M, sum(rows)), float("nan")))
    around = Y.as_strided((M, Y.stride(0)), (Y.stride(0), 1)) if pad else None
    apply(gpu, d, Y, base=d["base"])
    assert torch.equal(Y.cpu().double(), ref)
    if pad:  # nothing beyond the outputs is written
        assert bool(around[:, sum(rows):].isnan().all())
    # In place, from another state of Y.
    Y2 = d["placed"](d["base"].cpu())
    apply(gpu, d, Y2)
    assert torch.equal(Y2.cpu(), Y.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,cols,rows,n,rank", SHAPES)
def test_normal_numbers_within_the_bound(gpu, M, cols, rows, n, rank, dtype):
    d = make(M, cols, rows, n, rank, dtype, "normal", 7 * M + cols + rank)
    ref, mag = reference(d)
    Y = torch.full((M, sum(rows)), float("nan"), device="cuda")
    apply(gpu, d, Y, base=d["base"])
    err = (Y.cpu().double() - ref).abs()
    assert bool((err <= (cols / 16 + 16 + rank + 4) * 2.0 ** -23 * mag).all())
    again = torch.empty_like(Y)
    apply(gpu, d, again, base=d["base"])
    assert torch.equal(again, Y)  # the same bits every time


@pytest.mark.gpu
@pytest.mark.parametrize("M,outs", [(1, 16), (40, 16), (2048, 6000)])
def test_sums_between_the_products_keep_24_bits_whatever_their_size(gpu, M, outs):
    # x A^T of very different sizes in one row (2^-15 to 1 of each other): the
    # outputs that take only the small one must see it whole.
    n, rank, cols = 1, 16, 32
    for dtype in ("bf16", "f16"):
        A = torch.zeros(n, rank, cols)
        B = torch.zeros(n, outs, rank)
        for r in range(rank):
            A[0, r, 2 * r], A[0, r, 2 * r + 1] = 1.0, 2.0 ** -8
            B[0, r::rank, r] = 1.0
        X = torch.zeros(M, cols)
        for r in range(rank):
            X[:, 2 * r] = 2.0 ** (r - 8) * 1.5
            X[:, 2 * r + 1] = 2.0 ** (r - 8) * 1.25
        dt = DT[dtype]
        ad = gpu.Adapters(A.to(dt).cuda(), B.to(dt).cuda())
        plan = gpu.adapter_plan(torch.zeros(M, dtype=torch.int32, device="cuda"), n)
        Y = torch.zeros(M, outs, device="cuda")
        gpu.adapter_apply(ad, plan, X.to(dt).cuda(), Y)
        want = torch.tensor([2.0 ** (r % rank - 8) * (1.5 + 1.25 * 2.0 ** -8) for r in range(outs)]).expand(M, outs)
        assert torch.equal(Y.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,outs", [(6, 90), (290, 90), (2048, 6000)])
def test_infinities_and_nan_stay_in_their_rows(gpu, M, outs, dtype):
    d = make(M, 200, [outs], 2, 9, dtype, "whole", 5, none=0.0, ranks="full")
    d["ids"].zero_()
    clean = apply(gpu, d, torch.empty(M, outs, device="cuda"), base=d["base"])
    d["X"][1, 3], d["X"][4, 0] = float("nan"), float("inf")
    d["A"][0][0, :, 0] = 1.0  # the infinity reaches every sum with one sign ...
    d["B"][0][0] = 2.0        # ... and every output
    ref, _ = reference(d)
    Y = apply(gpu, d, torch.empty(M, outs, device="cuda"), base=d["base"])
    assert bool(Y[1].isnan().all())
    assert bool((Y[4] == float("inf")).all())
    keep = [m for m in range(M) if m not in (1, 4)]
    assert torch.equal(Y[keep].cpu().double(), ref[keep])
    assert clean.isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,cols,rows", [(4, 128, [64, 10]), (300, 128, [64, 10]), (4000, 2000, [1900, 102])])
def test_rows_without_an_adapter_are_left_alone(gpu, M, cols, rows):
    d = make(M, cols, rows, 3, 8, "bf16", "whole", 9, none=0.5)
    d["ids"][0] = -1
    off = (d["ids"] < 0).nonzero().flatten()
    d["X"][off] = float("nan")
    Y = d["base"].clone()
    Y[off] = float("nan")
    want = apply(gpu, d, torch.empty_like(Y), base=d["base"])
    assert torch.equal(want[off], d["base"][off])
    apply(gpu, d, Y)
    assert bool(Y[off].isnan().all())
    on = (d["ids"] >= 0).nonzero().flatten()
    assert torch.equal(Y[on], want[on])


@pytest.mark.gpu
@pytest.mark.parametrize("M,cols,outs", [(20, 64, 32), (2048, 1024, 3000)])
def test_a_slice_without_outputs_is_not_looked_at(gpu, M, cols, outs):
    d = make(M, cols, [outs, 0, 17], 4, 8, "bf16", "whole", 12)
    ad = gpu.Adapters(d["A"], d["B"], ranks=d["ranks"], scales=d["scales"])
    ad.struct.A[1] = ad.struct.B[1] = None
    Y = torch.empty(M, outs + 17, device="cuda")
    gpu.adapter_apply(ad, gpu.adapter_plan(d["ids"], 4), d["X"], Y, base=d["base"])
    assert torch.equal(Y.cpu().double(), reference(d)[0])


@pytest.mark.gpu
def test_without_ranks_and_scales(gpu):
    d = make(20, 64, [32], 4, 8, "f16", "whole", 3, ranks="full")
    d["scales"] = torch.ones(4, device="cuda")
    ref, _ = reference(d)
    ad = gpu.Adapters(d["A"], d["B"])
    Y = torch.empty(20, 32, device="cuda")
    gpu.adapter_apply(ad, gpu.adapter_plan(d["ids"], 4), d["X"], Y, base=d["base"])
    assert torch.equal(Y.cpu().double(), ref)


@pytest.mark.gpu
def test_ranks_outside_their_range_are_clamped(gpu):
    d = make(20, 64, [32], 4, 8, "f16", "whole", 4, ranks="full")
    d["ranks"].copy_(torch.tensor([-3, 8, 1000, 2 ** 31 - 1]))
    ad = gpu.Adapters(d["A"], d["B"], ranks=d["ranks"], scales=d["scales"])
    Y = torch.empty(20, 32, device="cuda")
    gpu.adapter_apply(ad, gpu.adapter_plan(d["ids"], 4), d["X"], Y, base=d["base"])
    d["ranks"].clamp_(0, 8)
    assert torch.equal(Y.cpu().double(), reference(d)[0])


@pytest.mark.gpu
def test_shared_and_strided_adapters(gpu):
    # One A for all adapters (stride 0), B a view of a larger tensor.
    d = make(50, 96, [40], 5, 16, "bf16", "whole", 6, ranks="full")
    d["A"] = [d["A"][0][:1].expand(5, 16, 96)]
    big = torch.full((5, 60, 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, 20:, 8:] = d["B"][0]
    d["B"] = [big[:, 20:, 8:]]
    Y = apply(gpu, d, torch.empty(50, 40, device="cuda"), base=d["base"])
    assert torch.equal(Y.cpu().double(), reference(d)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("M,cols,outs", [(3, 264, 136), (2048, 1024, 2048)])
def test_offsets_beyond_32_bits(gpu, M, cols, outs):
    # Adapters 2^31 elements apart; for a few rows also outputs 2^30 floats apart.
    n, rank, far = 2, 16, 1 << 31
    d = make(M, cols, [outs], n, rank, "bf16", "whole", 77, ranks="full")
    for k, shape in (("A", (n, rank, cols)), ("B", (n, outs, rank))):
        big = torch.empty(far + shape[1] * shape[2], dtype=torch.bfloat16, device="cuda")
        v = big.as_strided(shape, (far, shape[2], 1))
        v.copy_(d[k][0])
        d[k] = [v]
    ref, _ = reference(d)
    Y = torch.empty(M, outs, device="cuda")
    if M == 3:
        ld = (1 << 30) + 4
        Y = torch.empty(2 * ld + outs, device="cuda").as_strided((M, outs), (ld, 1))
    apply(gpu, d, Y, base=d["base"])
    assert torch.equal(Y.cpu().double(), ref)


@pytest.mark.gpu
def test_a_plan_of_another_batch_changes_nothing_and_says_so(gpu):
    d = make(20, 64, [32], 4, 8, "f16", "whole", 3)
    plan = gpu.adapter_plan(d["ids"], 4)
    other = gpu.AdapterPlan(20, 4)  # never made: all zeros
    ad = gpu.Adapters(d["A"], d["B"], ranks=d["ranks"], scales=d["scales"])
    Y = torch.full((20, 32), 7.0, device="cuda")
    gpu.adapter_apply(ad, other, d["X"], Y, base=d["base"])
    torch.cuda.synchronize()
    assert gpu.device_error() == 4 and gpu.device_error() == 0
    assert bool((Y == 7.0).all())
    gpu.adapter_apply(ad, plan, d["X"], Y, base=d["base"])
    assert torch.equal(Y.cpu().double(), reference(d)[0])


@pytest.mark.gpu
def test_a_workspace_that_is_too_small_or_misaligned_is_refused(gpu):
    d = make(20, 64, [32], 4, 8, "f16", "whole", 3)
    ad = gpu.Adapters(d["A"], d["B"])
    plan = gpu.adapter_plan(d["ids"], 4)
    ws = gpu.adapter_workspace(ad, 20)
    need = gpu.adapter_workspace_bytes(ad, 20)
    Y = torch.full((20, 32), 7.0, device="cuda")
    for bad in (ws[:need - 1], torch.empty(need + 256, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(gpu.SeedLMError):
            gpu.adapter_apply(ad, plan, d["X"], Y, workspace=bad)
    with pytest.raises(ValueError, match="same CUDA device"):
        gpu.adapter_apply(ad, plan, d["X"], torch.empty(20, 32), workspace=ws)
    with pytest.raises(ValueError, match="same CUDA device"):
        gpu.adapter_apply(ad, plan, d["X"].cpu(), Y, workspace=ws)
    with pytest.raises(ValueError, match="same CUDA device"):
        gpu.adapter_plan(d["ids"].cpu(), 4, plan=plan)
    with pytest.raises(ValueError, match="same CUDA device"):
        gpu.Adapters(d["A"][0].cpu(), d["B"])
    torch.cuda.synchronize()
    assert bool((Y == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,cols,rows", [(12, 512, [200, 56]), (400, 512, [200, 56]), (2048, 1024, [1500, 548])])
def test_captured_graphs_that_share_a_workspace_and_follow_their_inputs(gpu, M, cols, rows):
    n = 6
    d = make(M, cols, rows, n, 16, "bf16", "whole", 21)
    e = make(M, cols, rows, n, 16, "bf16", "whole", 22)
    ads = [gpu.Adapters(v["A"], v["B"], ranks=v["ranks"], scales=v["scales"]) for v in (d, e)]
    ws = gpu.adapter_workspace(ads[0], M)
    ws.fill_(255)  # any content
    plans = [gpu.AdapterPlan(M, n) for _ in ads]
    Ys = [torch.empty(M, sum(rows), device="cuda") for _ in ads]
    graphs = []
    gpu.adapter_plan(d["ids"], n, plan=plans[0])
    gpu.adapter_apply(ads[0], plans[0], d["X"], Ys[0], base=d["base"], workspace=ws)
    torch.cuda.synchronize()
    for v, ad, plan, Y in zip((d, e), ads, plans, Ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gpu.adapter_plan(v["ids"], n, plan=plan)
            gpu.adapter_apply(ad, plan, v["X"], Y, base=v["base"], workspace=ws)
            gpu.adapter_apply(ad, plan, v["X"], Y, workspace=ws)  # and once more, in place
        graphs.append(g)
    for step in range(3):
        for v in (d, e):
            v["ids"].copy_(torch.randint(-1, n, (M,), dtype=torch.int32))
            v["X"].copy_(torch.randint(-2, 3, v["X"].shape))
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for v, Y in zip((d, e), Ys):
            once, _ = reference(v)
            assert torch.equal(Y.cpu().double(), reference(v, base=once)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("M,cols,outs", [(70, 1024, 300), (2048, 1024, 2048)])
def test_streams_of_their_own(gpu, M, cols, outs):
    ds = [make(M, cols, [outs], 5, 16, "f16", "whole", 31 + i) for i in range(3)]
    refs = [reference(d)[0] for d in ds]
    ads = [gpu.Adapters(d["A"], d["B"], ranks=d["ranks"], scales=d["scales"]) for d in ds]
    wss = [gpu.adapter_workspace(ad, M) for ad in ads]
    plans = [gpu.AdapterPlan(M, 5) for _ in ads]
    Ys = [torch.empty(M, outs, device="cuda") for _ in ads]
    streams = [torch.cuda.Stream() for _ in ads]
    torch.cuda.synchronize()
    for _ in range(10):
        for d, ad, ws, plan, Y, st in zip(ds, ads, wss, plans, Ys, streams):
            gpu.adapter_plan(d["ids"], 5, plan=plan, stream=st)
            gpu.adapter_apply(ad, plan, d["X"], Y, base=d["base"], workspace=ws, stream=st)
    torch.cuda.synchronize()
    for Y, ref in zip(Ys, refs):
        assert torch.equal(Y.cpu().double(), ref)
