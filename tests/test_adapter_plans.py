"""What adapter_apply() makes of plan memory that is not this batch's plan:
plans of other sizes, zeros and parts of other plans are found out and change
nothing; memory that was written over behind a good head leads to no access
outside the arrays (the kernels check every tile and row number that they
follow), and says so."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

#: M, cols, outputs, adapters, rank: tiles of 8 rows, tiles of 64.
FORMS = [(100, 64, 40, 50, 8), (2000, 2000, 2000, 3, 16), (1300, 2500, 3000, 2, 256)]


@pytest.fixture(scope="module")
def sl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from prng_seeded_decompress_b200 import build
    build.build()
    from prng_seeded_decompress_b200 import seedlm
    seedlm.init()
    return seedlm


class Batch:
    def __init__(self, sl, M, cols, outs, n, rank, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(M + n)
        whole = lambda *s: torch.randint(-1, 2, s, generator=g)  # noqa: E731
        A, B, X, self.base = whole(n, rank, cols), whole(n, outs, rank), whole(M, cols), whole(M, outs).float()
        self.ids = torch.randint(-1, n, (M,), generator=g).to(torch.int32)
        self.ref = self.base.double()
        for a in range(n):
            on = self.ids == a
            self.ref[on] += (X[on].double() @ A[a].double().T) @ B[a].double().T
        self.sl, self.M, self.n, self.outs = sl, M, n, outs
        self.ad = sl.Adapters(A.to(dtype).cuda(), B.to(dtype).cuda())
        self.X = X.to(dtype).cuda()
        self.plan = sl.adapter_plan(self.ids.cuda(), n)
        # Y between rows and columns that nothing may write.
        self.around = torch.full((M + 2, outs + 8), 7.0, device="cuda")
        self.Y = self.around[1:-1, 4:-4]
        self.ws = sl.adapter_workspace(self.ad, M)

    def apply(self, plan, in_place=False):
        """The flag, and whether Y is as it was."""
        self.Y.copy_(self.base)
        before = self.around.clone()
        base = None if in_place else self.base.cuda() + 1  # (so that a row that is written is seen)
        self.sl.adapter_apply(self.ad, plan, self.X, self.Y, base=base, workspace=self.ws)
        torch.cuda.synchronize()
        frame = self.around.clone()
        frame[1:-1, 4:-4] = before[1:-1, 4:-4]
        assert torch.equal(frame, before)
        return self.sl.device_error(), torch.equal(self.around, before)

    def still_right(self):
        flag, _ = self.apply(self.plan, in_place=True)
        assert flag == 0 and torch.equal(self.Y.cpu().double(), self.ref)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("form", FORMS)
def test_plans_of_other_sizes_change_nothing_and_say_so(sl, form, in_place):
    b = Batch(sl, *form)
    for M, n in ((b.M, b.n + 1), (b.M, max(1, b.n - 1)), (b.M - 1, b.n), (b.M + 1, b.n), (2 * b.M, b.n)):
        other = sl.AdapterPlan(b.M, b.n)
        words = sl.adapter_plan(torch.zeros(M, dtype=torch.int32, device="cuda"), n).buffer
        k = min(words.numel(), other.buffer.numel())
        other.buffer[:k] = words[:k]
        assert b.apply(other, in_place) == (4, True)
    assert b.apply(sl.AdapterPlan(b.M, b.n), in_place) == (4, True)  # zeros
    b.still_right()


def test_a_part_of_another_plan_is_not_taken_for_a_head(sl):
    # A plan of 200 rows whose order reads 100, 50, 2, 3 where the head of a plan
    # of 100 rows and 50 adapters lies, and goes on as its tiles might.
    b = Batch(sl, *FORMS[0])
    order = np.full(200, -1)
    order[152:156] = 100, 50, 2, 3
    order[160:172] = 0, 10, 4, 120, 1, 14, 5, 121, 6, 20, 7, 122
    order[order < 0] = np.setdiff1d(np.arange(200), order)
    ids = np.empty(200, np.int32)
    ids[order] = np.arange(200)
    words = sl.adapter_plan(torch.from_numpy(ids).cuda(), 200)
    assert np.array_equal(words.order.cpu().numpy(), order) and int(order[10:28].max()) < 100
    other = sl.AdapterPlan(b.M, b.n)
    other.buffer.copy_(words.buffer[:other.buffer.numel()])
    assert b.apply(other) == (4, True)
    b.still_right()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("form", FORMS)
def test_plans_that_were_written_over_are_followed_nowhere_outside(sl, form, dtype, in_place):
    b = Batch(sl, *form, dtype=dtype)
    rng = np.random.default_rng(b.M)
    good = b.plan.buffer.cpu().numpy()
    head = (b.M + b.n + 1 + 3) // 4 * 4
    first_tile, words = head + 8, good.size

    def follow(content):
        other = sl.AdapterPlan(b.M, b.n)
        other.buffer.copy_(torch.from_numpy(content.astype(np.int32)))
        flag, _ = b.apply(other, in_place)
        assert flag == 4
        return other

    wild = rng.choice([-2 ** 31, -1, -7, b.M, b.M + 1, 2 ** 30, 2 ** 31 - 1], words)
    rows = good.copy()
    rows[:b.M] = wild[:b.M]
    follow(rows)
    some = good.copy()  # one wrong row number in each tile of 64
    some[:b.M:50] = b.M
    follow(some)
    for field in range(4):  # adapter, first, count of every tile; all of them
        tiles = good.copy()
        if field < 3:
            tiles[first_tile + field::4] = wild[first_tile + field::4]
        else:
            tiles[first_tile:] = wild[first_tile:]
        if field == 0:  # (-1 is a tile without an adapter)
            tiles[first_tile::4] = np.where(tiles[first_tile::4] == -1, b.n, tiles[first_tile::4])
        follow(tiles)
    near = good.copy()  # tiles that just leave the batch, or have one row too many
    near[first_tile + 1::4] = b.M - near[first_tile + 2::4] + 1
    follow(near)
    for at in (2, 3, 6, 7):  # numbers of tiles
        heads = good.copy()
        heads[head + at] = 2 ** 31 - 1
        heads[head + (at ^ 4)] = 2 ** 31 - 1
        follow(heads)
    b.still_right()
