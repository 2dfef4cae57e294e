"""The products and what runs between them, together, as a server's step uses
them: norm, gate+up product, adapters, gated activation, down product,
adapters, residual sum and norm, enqueued on one stream without a wait between
them.  Every stage's output is compared with the 64-bit formula of that stage
on the inputs it was given, so each bound is the stage's own."""
import os
import subprocess
import sys

import numpy as np
import pytest

from prng_seeded_decompress_b200 import inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
N, RANK = 5, 12


@pytest.fixture(scope="module")
def sl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from prng_seeded_decompress_b200 import build
    build.build(check=os.environ.get("SEEDLM_CHECKED", "0") == "1")
    from prng_seeded_decompress_b200 import seedlm
    seedlm.init()
    return seedlm


class Step:
    """The MLP half of a decoder layer over M rows, D wide, F inside."""

    def __init__(self, sl, oracle_mod, M, dtype, C, P, D=264, F=200):
        self.sl, self.M, self.F = sl, M, F
        self.dt = dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        g = torch.Generator().manual_seed(M)
        rnd = lambda *s, std=1.0: torch.randn(s, generator=g) * std  # noqa: E731
        self.layers = [inputs.make_layer(2 * F, D, C, P, seed=M), inputs.make_layer(D, F, C, P, seed=M + 1)]
        self.W = [torch.from_numpy(oracle_mod.decompress(L["fmt"], L["rec"], L["eplane"])) for L in self.layers]
        self.planes = [(torch.from_numpy(L["rec"].view(np.int32)).cuda(),
                        torch.from_numpy(L["eplane"]).cuda() if P == 4 else None) for L in self.layers]
        self.ranks = torch.tensor([12, 3, 0, 8, 5], dtype=torch.int32).cuda()
        self.scales = torch.tensor([1.0, 0.5, 2.0, 1.5, 0.25]).cuda()

        def adapters(cols, rows):
            A = [rnd(N, RANK, cols, std=cols ** -0.5).to(dt).cuda() for _ in rows]
            B = [rnd(N, R, RANK, std=0.1).to(dt).cuda() for R in rows]
            return sl.Adapters(A, B, ranks=self.ranks, scales=self.scales)

        self.ad = [adapters(D, [F, F]), adapters(F, [D])]
        w = [(1 + rnd(D, std=0.2)).to(dt).cuda() for _ in range(3)]
        self.norms = [sl.BlockNorm(D, w_pre=w[0]), sl.BlockNorm(D, w_post=w[1], w_pre=w[2], y_scale=0.5)]
        self.w = w
        self.ids = torch.randint(-1, N, (M,), generator=g).to(torch.int32).cuda()
        self.h = rnd(M, D, std=2.0).to(dt).cuda()
        new = lambda n, t: torch.empty(M, n, dtype=t, device="cuda")  # noqa: E731
        self.x, self.x2, self.act = new(D, dt), new(D, dt), new(F, dt)
        self.h2, self.gu, self.y = new(D, dt), new(2 * F, torch.float32), new(D, torch.float32)
        self.gu0, self.y0 = new(2 * F, torch.float32), new(D, torch.float32)
        self.plan = sl.AdapterPlan(M, N)
        self.ws = [sl.adapter_workspace(a, M) for a in self.ad]
        need = max(sl.gemm_any_workspace_bytes(L["fmt"], M) for L in self.layers)
        self.gws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")

    def product(self, i, X, Y):
        rec, ep = self.planes[i]
        if self.M == 1:
            self.sl.gemv(self.layers[i]["fmt"], rec, ep, X[0], Y[0])
        else:
            self.sl.gemm(self.layers[i]["fmt"], rec, ep, X, Y, workspace=self.gws)

    def run(self):
        sl = self.sl
        sl.adapter_plan(self.ids, N, plan=self.plan)
        sl.block_norm(self.norms[0], None, self.h, x=self.x)
        self.product(0, self.x, self.gu0)
        sl.adapter_apply(self.ad[0], self.plan, self.x, self.gu, base=self.gu0, workspace=self.ws[0])
        sl.glu(self.gu, self.act)
        self.product(1, self.act, self.y0)
        sl.adapter_apply(self.ad[1], self.plan, self.act, self.y, base=self.y0, workspace=self.ws[1])
        sl.block_norm(self.norms[1], self.y, self.h, h_out=self.h2, x=self.x2)

    # Each stage in 64 bits from the inputs it had.

    def check(self):
        d = lambda t: t.cpu().double()  # noqa: E731
        step = torch.finfo(self.dt).eps / 2
        tiny = 2.0 ** -25 if self.dt == torch.float16 else 2.0 ** -134

        def rounded(got, ref, err):
            assert bool(((d(got) - ref).abs() <= step * ref.abs() + tiny + 1.01 * err).all())

        def rms(v, w):
            return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * d(w)

        def product(i, X, Y):
            ref, mag = d(X) @ self.W[i].T, d(X).abs() @ self.W[i].abs().T
            assert bool(((d(Y) - ref).abs() <= 1e-5 * mag).all())

        def adapted(i, X, base, Y):
            ref, mag = d(base), d(base).abs()
            ids, A, B = self.ids.cpu(), self.ad[i].tensors[:len(self.ad[i].rows)], self.ad[i].tensors[len(self.ad[i].rows):-2]
            for a in range(N):
                rows, r, s, j = (ids == a).nonzero().flatten(), int(self.ranks[a]), float(self.scales[a]), 0
                for At, Bt in zip(A, B):
                    p, q = d(At[a, :r]), d(Bt[a, :, :r])
                    ref[rows, j:j + q.shape[0]] += s * (d(X)[rows] @ p.T) @ q.T
                    mag[rows, j:j + q.shape[0]] += s * (d(X)[rows].abs() @ p.abs().T) @ q.abs().T
                    j += q.shape[0]
            assert bool(((d(Y) - ref).abs() <= (X.shape[1] / 16 + 20 + RANK) * 2.0 ** -23 * mag).all())

        u = 96 * 2.0 ** -24
        ref = rms(d(self.h), self.w[0])
        rounded(self.x, ref, u * ref.abs())
        product(0, self.x, self.gu0)
        adapted(0, self.x, self.gu0, self.gu)
        g, up = d(self.gu)[:, :self.F], d(self.gu)[:, self.F:]
        rounded(self.act, g * torch.sigmoid(g) * up, 2.0 ** -21 * (g * up).abs())
        product(1, self.act, self.y0)
        adapted(1, self.act, self.y0, self.y)
        v = 0.5 * rms(d(self.y), self.w[1])
        h2 = d(self.h) + v
        err = u * (d(self.h).abs() + v.abs())
        rounded(self.h2, h2, err)
        rstd = 1 / torch.sqrt((h2 * h2).mean(1, keepdim=True) + 1e-6)
        x2 = rms(h2, self.w[2])
        rounded(self.x2, x2, err * rstd * d(self.w[2]).abs() + (u + (err * err).mean(1, keepdim=True).sqrt() * rstd) * x2.abs())

    def outputs(self):
        return [t.clone() for t in (self.x, self.gu0, self.gu, self.act, self.y0, self.y, self.h2, self.x2)]


#: 2048 rows of this width take the adapters' tensor-memory kernels, between
#: products that take all of it.
WIDE = dict(D=1032, F=1100)


@pytest.mark.parametrize("M,dtype,C,P", [(2048, "bf16", 8, 3), (2048, "f16", 12, 4), (1, "bf16", 8, 3), (1, "f16", 12, 4), (3, "bf16", 12, 4), (17, "f16", 8, 3),
                                         (64, "bf16", 8, 3), (300, "bf16", 12, 4), (300, "f16", 8, 3)])
def test_a_layers_mlp_half_stage_by_stage(sl, oracle_mod, M, dtype, C, P):
    s = Step(sl, oracle_mod, M, dtype, C, P, **(WIDE if M == 2048 else {}))
    s.run()
    torch.cuda.synchronize()
    s.check()
    first = s.outputs()
    for t in (s.x, s.gu0, s.gu, s.act, s.y0, s.y, s.h2, s.x2):
        t.fill_(float("nan"))
    for _ in range(3):
        s.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, s.outputs()))


@pytest.mark.parametrize("M", [1, 20, 300, 2048])
def test_the_same_step_captured_into_a_graph(sl, oracle_mod, M):
    s = Step(sl, oracle_mod, M, "bf16", 8, 3, **(WIDE if M == 2048 else {}))
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for seed in range(3):  # the graph follows its inputs, the batch's adapters among them
        gen = torch.Generator().manual_seed(seed)
        s.h.copy_(torch.randn(s.h.shape, generator=gen))
        s.ids.copy_(torch.randint(-1, N, (M,), generator=gen).to(torch.int32))
        g.replay()
        torch.cuda.synchronize()
        s.check()
        replayed = s.outputs()
        s.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, s.outputs()))


def test_the_suites_pass_in_the_checked_build(sl):
    # Every global and shared index compared with its extent; the fixture in
    # conftest.py then finds the flag clear after each test.
    if sl.CHECKED:
        pytest.skip("already running against the checked build")
    from prng_seeded_decompress_b200 import build
    build.build(check=True)
    env = dict(os.environ, SEEDLM_CHECKED="1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                          "tests/test_adapters.py", "tests/test_block_norm.py", "tests/test_layer_chain.py"],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-2000:]
    assert " passed" in res.stdout and " failed" not in res.stdout
