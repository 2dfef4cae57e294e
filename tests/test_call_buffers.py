"""Buffers that a call makes for itself belong to the stream it runs on: what
fills them is ordered before the call, and memory that is handed back is not
given to work of another stream while the call still uses it.  On the CPU with
torch's streams replaced by names; on the GPU with the other stream kept busy,
so that a buffer of the wrong stream would be filled, or used by others, at the
wrong time."""
import contextlib
import types

import numpy as np
import pytest

from prng_seeded_decompress_b200 import inputs

torch = pytest.importorskip("torch")

BUSY = 40_000_000  # clock cycles: 20 ms


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


class FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


@pytest.fixture
def made_on(sl, monkeypatch):
    """The handles of the streams that buffers were made on, in order; the
    current stream's is 7."""
    seen, current = [], [7]

    @contextlib.contextmanager
    def stream(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def maker(kind):
        real = getattr(torch, kind)

        def make(*size, dtype=None, device=None):
            seen.append(current[-1])
            return real(*size, dtype=dtype)
        return make

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: FakeStream(current[-1]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda d=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(sl, "_place", lambda tensors: 0)
    monkeypatch.setattr(sl, "_run_on", lambda *a: None)
    monkeypatch.setattr(sl, "adapter_workspace_bytes", lambda ad, M: 1000)

    def then(make):
        monkeypatch.setattr(torch, "zeros", maker("zeros"))
        monkeypatch.setattr(torch, "empty", maker("empty"))
        make()
        return seen
    return then


@pytest.mark.parametrize("stream,handle", [(None, 7), (FakeStream(9), 9), (9, 9), (7, 7), (0, 0), (FakeStream(0), 0)])
def test_a_plan_and_a_workspace_are_made_on_the_calls_stream(sl, made_on, stream, handle):
    ids = torch.zeros(4, dtype=torch.int32)
    ad = sl.Adapters(torch.zeros(3, 8, 64).half(), torch.zeros(3, 32, 8).half())
    ad.device = 0
    plan, X, Y = sl.AdapterPlan(4, 3, device="cpu"), torch.zeros(4, 64).half(), torch.zeros(4, 32)

    def calls():
        sl.adapter_plan(ids, 3, stream=stream)
        sl.adapter_apply(ad, plan, X, Y, stream=stream)
    assert made_on(calls) == [handle, handle]


@pytest.mark.parametrize("stream,handle", [(None, 7), (FakeStream(9), 9), (9, 9), (7, 7), (0, 0)])
def test_a_products_workspace_is_made_on_the_calls_stream(sl, made_on, monkeypatch, stream, handle):
    fmt = inputs.make_layer(64, 128, 8, 3, seed=1)["fmt"]
    rec, X, Y = torch.zeros(64, 16, dtype=torch.int32), torch.zeros(20, 128).half(), torch.zeros(20, 64)
    monkeypatch.setattr(sl, "gemm_workspace_bytes", lambda f, M: 1000)
    monkeypatch.setattr(sl, "gemm_any_workspace_bytes", lambda f, M: 1000)
    monkeypatch.setattr(sl, "_check", lambda fn, rc: None)
    monkeypatch.setattr(sl, "lib", types.SimpleNamespace(seedlm_gemm=lambda *a: 0, seedlm_gemm_smallM=lambda *a: 0))

    def calls():
        sl.gemm(fmt, rec, None, X, Y, stream=stream)
        sl.gemm_smallM(fmt, rec, None, X, Y, stream=stream)
    assert made_on(calls) == [handle, handle]


@pytest.mark.parametrize("device,want", [(None, "cuda"), (0, 0), (1, 1), ("cuda:0", "cuda:0")])
def test_device_0_is_device_0(sl, monkeypatch, device, want):
    seen, real = [], torch.zeros

    def zeros(*size, dtype=None, device=None):
        seen.append(device)
        return real(*size, dtype=dtype)
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(sl, "gemm_workspace_bytes", lambda f, M: 1000)
    sl.AdapterPlan(4, 3, device=device)
    sl.gemm_workspace(None, 4, device=device)
    assert seen == [want, want]


def batch(M, seed):
    g = torch.Generator().manual_seed(seed)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g)  # noqa: E731
    A, B, X, base = whole(5, 8, 256), whole(5, 320, 8), whole(M, 256), whole(M, 320).float()
    ids = torch.randint(-1, 5, (M,), generator=g).to(torch.int32)
    ref = base.double()
    for a in range(5):
        on = ids == a
        ref[on] += (X[on].double() @ A[a].double().T) @ B[a].double().T
    return [t.cuda() for t in (A.bfloat16(), B.bfloat16(), X.bfloat16(), base, ids)], ref


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("M", [60, 2048])
def test_a_plan_made_by_a_call_outlives_the_current_streams_work(gpu, M, handle):
    (A, B, X, base, ids), ref = batch(M, M)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)  # the current stream: nothing put on it runs before the sort is done
    plan = gpu.adapter_plan(ids, 5, stream=side.cuda_stream if handle else side)
    side.synchronize()
    torch.cuda.synchronize()
    key = np.where(ids.cpu().numpy() < 0, 5, ids.cpu().numpy())
    assert np.array_equal(plan.order.cpu().numpy(), np.argsort(key, kind="stable"))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [60, 2048])
def test_a_workspace_made_by_a_call_is_not_the_current_streams(gpu, M):
    (A, B, X, base, ids), ref = batch(M, M + 1)
    ad, side = gpu.Adapters(A, B), torch.cuda.Stream()
    plan, Y = gpu.adapter_plan(ids, 5), torch.empty(M, 320, device="cuda")
    size = gpu.adapter_workspace_bytes(ad, M)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    gpu.adapter_apply(ad, plan, X, Y, base=base, stream=side)
    # The current stream's next buffer of that size, filled before the call above runs.
    mine = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert bool((mine == 255).all())
    assert torch.equal(Y.cpu().double(), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [16, 600])
def test_a_products_workspace_is_cleared_before_the_product(gpu, oracle_mod, M):
    L = inputs.make_layer(256, 512, 8, 3, seed=M)
    W = torch.from_numpy(oracle_mod.decompress(L["fmt"], L["rec"], None)).double()
    rec = torch.from_numpy(L["rec"].view(np.int32)).cuda()
    X = torch.randn(M, 512, generator=torch.Generator().manual_seed(M)).half()
    Xd, side = X.cuda(), torch.cuda.Stream()
    size = gpu.gemm_any_workspace_bytes(L["fmt"], M)
    for call in (gpu.gemm, gpu.gemm_smallM)[:2 if M <= 64 else 1]:
        Y = torch.full((M, 256), float("nan"), device="cuda")
        with torch.cuda.stream(side):  # memory that the workspace may come to lie in
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        call(L["fmt"], rec, None, Xd, Y, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        ref = X.double() @ W.T
        assert bool(((Y.cpu().double() - ref).abs() <= 1e-5 * (X.double().abs() @ W.abs().T)).all())
