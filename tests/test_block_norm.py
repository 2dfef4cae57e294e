"""The end of one block and the start of the next (norm, gate, residual sum,
norm) and the gated activation, against the formulas in 64 bits.

Bounds: an output rounded to a type t is off by half a step, eps_t / 2 of its
value (or half the smallest subnormal number), on top of the error of the fp32
value.  In fp32 every operation is off by at most 2^-24 of its result; a sum
over a row is at most cols / 256 + 48 additions deep (at least 256 threads that
add their part each, then trees), so a mean or a mean square is off by that many
times 2^-24 of the mean of the absolute terms.  16 more operations bound each
value's own chain."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


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

@pytest.mark.parametrize("nm,call,code", [
    (dict(cols=-1), {}, -1), (dict(cols=(1 << 20) + 1), {}, -2), (dict(kind=2), {}, -1), (dict(dtype=3), {}, -1),
    (dict(post=2), {}, -1), (dict(pre=-1), {}, -1), (dict(eps=-1e-6), {}, -1), (dict(eps=float("nan")), {}, -1),
    (dict(w_post=0x1001), {}, -1), (dict(b_post=0x1001), {}, -1), (dict(w_pre=0x1001), {}, -1),
    (dict(b_pre=0x1001), {}, -1), ({}, dict(M=-1), -1), ({}, dict(y=None, h=None), -1),
    ({}, dict(h_out=None, x=None), -1), ({}, dict(y=0x1002), -1), ({}, dict(ldy=63), -1), ({}, dict(gate=0x1001), -1),
    ({}, dict(gate=0x1000, ldg=63), -1), ({}, dict(gate=0x1000, ldg=-64), -1), ({}, dict(h=0x1001), -1),
    ({}, dict(ldh=63), -1), ({}, dict(h_out=0x1001), -1), ({}, dict(ldo=63), -1), ({}, dict(ht=3), -1),
    ({}, dict(ht=2, h=0x1002), -1), ({}, dict(xt=2), -1), ({}, dict(x=0x1001), -1), ({}, dict(ldx=63), -1),
    ({}, dict(h_out=0x3000, ldo=72), -1),
])
def test_bad_norm_calls_are_refused_before_cuda(sl, nm, call, code):
    f = dict(cols=64, kind=0, dtype=1, post=0, pre=1, eps=1e-6, weight_offset=0, h_scale=1, y_scale=1, w_post=None,
             b_post=None, w_pre=0x1000, b_pre=None)
    f.update(nm)
    s = sl._NormStruct(*f.values())
    a = dict(M=3, y=0x2000, ldy=64, gate=None, ldg=0, h=0x3000, ldh=64, h_out=0x4000, ldo=64, ht=1, x=0x5000, ldx=64,
             xt=1)
    a.update(call)
    assert sl.lib.seedlm_block_norm(ctypes.byref(s), *a.values(), None) == code


def test_empty_norm_and_null(sl):
    s = sl._NormStruct(64, 0, 1, 0, 1, 1e-6, 0, 1, 1, None, None, 0x1000, None)
    args = (0x2000, 64, None, 0, 0x3000, 64, 0x4000, 64, 1, 0x5000, 64, 1, None)
    assert sl.lib.seedlm_block_norm(None, 3, *args) == -1
    assert sl.lib.seedlm_block_norm(ctypes.byref(s), 0, *args) == 0
    s.cols = 0
    assert sl.lib.seedlm_block_norm(ctypes.byref(s), 3, *args) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -1), (dict(cols=-1), -1), (dict(act=3), -1), (dict(act=-1), -1), (dict(xt=2), -1), (dict(GU=None), -1),
    (dict(GU=0x1002), -1), (dict(ldgu=127), -1), (dict(X=None), -1), (dict(X=0x2001), -1), (dict(ldx=63), -1),
    (dict(M=0), 0), (dict(cols=0), 0), (dict(cols=(1 << 30) + 1), -2),
])
def test_bad_glu_calls_are_refused_before_cuda(sl, kw, code):
    a = dict(M=3, cols=64, act=0, GU=0x1000, ldgu=128, X=0x2000, ldx=64, xt=0)
    a.update(kw)
    assert sl.lib.seedlm_glu(*a.values(), None) == code


def test_binding_refuses_what_it_cannot_pass(sl):
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="kind"):
        sl.BlockNorm(64, kind="group")
    with pytest.raises(ValueError):
        sl.BlockNorm(64, w_pre=w[:63])
    with pytest.raises(TypeError):
        sl.BlockNorm(64, w_pre=w, w_post=w.float())
    with pytest.raises(TypeError):
        sl.BlockNorm(64, w_pre=w.double())
    nm = sl.BlockNorm(64, w_pre=w)
    assert nm.struct.post == 0 and nm.struct.pre == 1
    assert sl.BlockNorm(64, w_post=w, w_pre=w).struct.post == 1
    y, h, x = torch.zeros(3, 64), torch.zeros(3, 64, dtype=torch.float16), torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be given"):
        sl.block_norm(nm, None, None, x=x)
    with pytest.raises(ValueError, match="must be given"):
        sl.block_norm(nm, y, h)
    with pytest.raises(TypeError):
        sl.block_norm(nm, y.half(), h, x=x)
    with pytest.raises(TypeError):
        sl.block_norm(nm, y, h, h_out=torch.zeros(3, 64), x=x)
    with pytest.raises(TypeError):
        sl.block_norm(nm, y, h, x=torch.zeros(3, 64))
    with pytest.raises(ValueError, match="3 x 64"):
        sl.block_norm(nm, y, h[:2], x=x)
    with pytest.raises(ValueError, match="unit column stride"):
        sl.block_norm(nm, torch.zeros(64, 3).t(), h, x=x)
    with pytest.raises(TypeError):
        sl.block_norm(nm, y, h, x=x, gate=torch.zeros(64))
    with pytest.raises(ValueError, match="gate"):
        sl.block_norm(nm, y, h, x=x, gate=w[:32])
    with pytest.raises(ValueError, match="CUDA"):
        sl.block_norm(nm, y, h, x=x)
    with pytest.raises(ValueError, match="act"):
        sl.glu(torch.zeros(3, 128), x, act="relu")
    with pytest.raises(ValueError, match="3 x 128"):
        sl.glu(torch.zeros(3, 127), x)
    with pytest.raises(TypeError):
        sl.glu(torch.zeros(3, 128), torch.zeros(3, 64))
    with pytest.raises(ValueError, match="CUDA"):
        sl.glu(torch.zeros(3, 128), x)


# -------------------------------------------------------------------- norms

def placed(t, pad, off):
    M, cols = t.shape
    buf = torch.full((off + M * (cols + pad),), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[off:].view(M, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def unit(cols):
    return (cols / 256 + 64) * 2.0 ** -24


def normed(v, err, kind, eps, off, w, b):
    """(norm(v), bound of the fp32 error), v in 64 bits with error bound err."""
    U = unit(v.shape[1])
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    c = v - mean
    rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    size = v.abs() + v.abs().mean(1, keepdim=True)
    own = err + err.mean(1, keepdim=True) + U * size  # of v - mean
    rel = U + (own * own).mean(1, keepdim=True).sqrt() * rstd  # of rstd
    g = off + w if w is not None else torch.ones_like(v[:1])
    b = b if b is not None else torch.zeros_like(v[:1])
    out = c * rstd * g + b
    return out, (own * rstd + (rel + U) * (c * rstd).abs()) * g.abs() + U * b.abs()


def half_step(ref, t):
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[t]
    return torch.finfo(t).eps / 2 * ref.abs() + tiny


def norm_reference(c, t):
    """(h', bound, x, bound) in 64 bits."""
    d = {k: (v.cpu().double() if torch.is_tensor(v) else None) for k, v in t.items()}
    M, cols = c["M"], c["cols"]
    U = unit(cols)
    zero = torch.zeros(M, cols, dtype=torch.float64)
    v, err = (d["y"] if d["y"] is not None else zero), zero
    off = c.get("offset", 0.0)
    if d["y"] is not None and c["post"]:
        v, err = normed(v, err, c["kind"], c["eps"], off, d["w_post"], d["b_post"])
    g = (d["gate"] if d["gate"] is not None else torch.ones(1, cols, dtype=torch.float64)).view(-1, cols)
    hs, ys = c.get("h_scale", 1.0), c.get("y_scale", 1.0)
    a = hs * (d["h"] if d["h"] is not None else zero)
    h = a + ys * g * v
    err = (ys * g).abs() * err + U * (a.abs() + (ys * g * v).abs())
    x, xerr = normed(h, err, c["kind"], c["eps"], off, d["w_pre"], d["b_pre"]) if c.get("pre", True) else (h, err)
    return h, err, x, xerr


def norm_case(gpu, c, pad=0, off=0):
    g = torch.Generator().manual_seed(c["M"] * 7919 + c["cols"])
    M, cols, dt = c["M"], c["cols"], DT[c["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g) * std + mean

    def vector(std, mean=0.0):
        v = torch.full((off + cols,), float("nan"), dtype=dt, device="cuda")[off:]
        return v.copy_(normal(cols, std=std, mean=mean))

    w_mean = 0.0 if c.get("offset") else 1.0
    bias = c.get("bias", c["kind"] == "layer")
    t = dict(y=placed(normal(M, cols, mean=c.get("mean", 0.0)), pad, off) if c.get("y", True) else None,
             h=placed(normal(M, cols, std=3.0, mean=c.get("mean", 0.0)).to(DT[c["h"]]), pad, off) if c["h"] else None,
             w_post=vector(0.3, w_mean) if c["post"] and c.get("weights", True) else None,
             b_post=vector(0.3) if c["post"] and bias else None,
             w_pre=vector(0.3, w_mean) if c.get("pre", True) and c.get("weights", True) else None,
             b_pre=vector(0.3) if c.get("pre", True) and bias else None,
             gate={None: None, "cols": vector(0.5), "rows": placed(normal(M, cols, std=0.5).to(dt), pad, off)}[c["gate"]])
    nm = gpu.BlockNorm(cols, kind=c["kind"], eps=c["eps"], h_scale=c.get("h_scale", 1.0), y_scale=c.get("y_scale", 1.0),
                       weight_offset=c.get("offset", 0.0), w_post=t["w_post"], b_post=t["b_post"], w_pre=t["w_pre"],
                       b_pre=t["b_pre"], post=c["post"], pre=c.get("pre", True), dtype=dt)
    return t, nm


def check_norm(gpu, c, pad=0, off=0, in_place=False):
    t, nm = norm_case(gpu, c, pad, off)
    M, cols, ht, xt = c["M"], c["cols"], DT[c["h"] or "bf16"], DT[c.get("x", "bf16")]
    h, herr, x, xerr = norm_reference(c, t)
    h_out = t["h"] if in_place else placed(torch.full((M, cols), float("nan"), dtype=ht), pad, off)
    x_out = placed(torch.full((M, cols), float("nan"), dtype=xt), pad, off)
    gpu.block_norm(nm, t["y"], t["h"], h_out=h_out, x=x_out, gate=t["gate"])
    got_h, got_x = h_out.cpu().double(), x_out.cpu().double()
    assert bool(((got_h - h).abs() <= half_step(h, ht) + (1 + torch.finfo(ht).eps) * herr).all())
    assert bool(((got_x - x).abs() <= half_step(x, xt) + (1 + torch.finfo(xt).eps) * xerr).all())
    if pad:
        for o in (h_out, x_out):
            assert bool(o.as_strided((M, cols + pad), (cols + pad, 1))[:, cols:].isnan().all())
    return t, nm, h_out, x_out


NORMS = [
    dict(kind="rms", post=False, gate=None, eps=1e-5, dtype="bf16", h="bf16"),
    dict(kind="rms", post=True, gate="cols", eps=1e-6, dtype="f16", h="f16", x="f16", offset=1.0, h_scale=0.5, y_scale=0.22),
    dict(kind="layer", post=True, gate="rows", eps=1e-5, dtype="f32", h="f32", mean=5.0),
    dict(kind="layer", post=False, gate="rows", eps=1e-5, dtype="bf16", h="f32", x="f16", bias=False),
    dict(kind="rms", post=True, gate="rows", eps=1e-6, dtype="f16", h="bf16", bias=True, weights=False, y_scale=-1.5),
]
SIZES = [(1, 1), (1, 8192), (3, 7), (2, 64), (5, 129), (4, 1000), (7, 4096), (3, 5001), (2, 8191), (3, 16384), (2, 28672),
         (1, 32769), (2, 100003), (300, 512), (700, 1001), (2000, 24), (400, 8192), (310, 387), (320, 3333), (300, 8191)]


@pytest.mark.gpu
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("M,cols", SIZES)
@pytest.mark.parametrize("which", range(len(NORMS)))
def test_norms_within_the_bound(gpu, which, M, cols, pad, off):
    check_norm(gpu, dict(NORMS[which], M=M, cols=cols), pad, off)


@pytest.mark.gpu
@pytest.mark.parametrize("M,cols", [(1, 8192), (3, 5001), (2, 100003), (300, 512), (700, 1001), (400, 8191)])
def test_norm_parts_left_out(gpu, M, cols):
    base = dict(NORMS[0], M=M, cols=cols)
    check_norm(gpu, dict(base, y=False))                    # the first block's norm
    check_norm(gpu, dict(base, h=None, post=True))          # no residual stream yet
    check_norm(gpu, dict(base, pre=False))                  # x is the rounded sum
    check_norm(gpu, dict(base, h="f32"), in_place=True)
    t, nm, h_out, x_out = check_norm(gpu, base)
    h2, x2 = torch.empty_like(h_out), torch.empty_like(x_out)
    gpu.block_norm(nm, t["y"], t["h"], h_out=h2)            # either output alone, the same bits
    gpu.block_norm(nm, t["y"], t["h"], x=x2)
    assert torch.equal(h2, h_out) and torch.equal(x2, x_out)
    gpu.block_norm(nm, t["y"], t["h"], h_out=t["h"])        # in place
    assert torch.equal(t["h"], h_out)


@pytest.mark.gpu
def test_offsets_beyond_32_bits(gpu):
    ld, cols = (1 << 30) + 4, 600
    far = torch.empty(2 * ld + 2 * cols, device="cuda").as_strided((3, 2 * cols), (ld, 1))
    near = torch.randn(3, 2 * cols, device="cuda")
    far.copy_(near)
    nm = gpu.BlockNorm(cols, kind="layer")
    x, x_far = (torch.empty(3, cols, dtype=torch.float16, device="cuda") for _ in range(2))
    gpu.block_norm(nm, near[:, :cols], None, x=x)
    gpu.block_norm(nm, far[:, :cols], None, x=x_far)
    assert torch.equal(x, x_far)
    gpu.glu(near, x)
    gpu.glu(far, x_far)
    assert torch.equal(x, x_far)


@pytest.mark.gpu
def test_norm_of_constant_huge_and_special_rows(gpu):
    cols = 512
    nm = gpu.BlockNorm(cols, kind="layer", eps=1e-5)
    y = torch.zeros(6, cols, device="cuda")
    y[1] = 7.0                      # no variance: 0
    y[2], y[2, 5] = 1.0, float("nan")
    y[3], y[3, 5] = 1.0, float("inf")
    y[4] = torch.linspace(-1e18, 1e18, cols)
    x = torch.empty(6, cols, dtype=torch.bfloat16, device="cuda")
    gpu.block_norm(nm, y, None, x=x)
    assert bool((x[:2] == 0).all()) and bool(x[2:4].isnan().all())
    ref = torch.nn.functional.layer_norm(y[4].cpu().double(), (cols,), eps=1e-5)
    assert bool(((x[4].cpu().double() - ref).abs() <= half_step(ref, torch.bfloat16) + 2 * unit(cols) * (ref.abs() + 1)).all())
    assert bool((x[5] == 0).all())
    rms = gpu.BlockNorm(cols, eps=0.0)
    gpu.block_norm(rms, y, None, x=x)
    assert bool(x[0].isnan().all())  # 0 / 0, as the formula has it
    assert bool((x[1] == 1).all())


@pytest.mark.gpu
def test_one_gate_row_expanded_over_the_batch(gpu):
    c = dict(NORMS[1], M=9, cols=200)
    t, nm = norm_case(gpu, c)
    out = [torch.empty(9, 200, dtype=torch.float16, device="cuda") for _ in range(2)]
    gpu.block_norm(nm, t["y"], t["h"], h_out=out[0], gate=t["gate"])
    gpu.block_norm(nm, t["y"], t["h"], h_out=out[1], gate=t["gate"].expand(9, 200))
    assert torch.equal(*out)


# ---------------------------------------------------------------------- glu

def activation(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * torch.special.erfc(-g / 2 ** 0.5)
    return g * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("M,cols", [(1, 1), (1, 28672), (3, 7), (2, 64), (5, 1001), (130, 96), (1000, 257), (70000, 3)])
def test_glu_within_the_bound(gpu, M, cols, pad, off, dtype, act):
    # fp32: exp, erf and tanh are off by at most 2 steps (2^-23 of values up to
    # 1), their arguments by 2^-22 relative, which the functions' slopes
    # (x f'(x) < 1/2) halve; with the products less than 2^-21 |g u| in all.
    g = torch.Generator().manual_seed(M + cols)
    GU = torch.randn((M, 2 * cols), generator=g) * 4
    GU[0, 0] = -90.0
    src = placed(GU, pad, off)
    X = placed(torch.full((M, cols), float("nan"), dtype=DT[dtype]), pad, off)
    gpu.glu(src, X, act=act)
    gate, up = GU[:, :cols].double(), GU[:, cols:].double()
    ref = activation(gate, act) * up
    assert bool(((X.cpu().double() - ref).abs() <= half_step(ref, DT[dtype]) + 2.0 ** -21 * (gate * up).abs()).all())
    if pad:
        assert bool(X.as_strided((M, cols + pad), (cols + pad, 1))[:, cols:].isnan().all())


@pytest.mark.gpu
def test_glu_at_the_ends(gpu):
    inf, nan = float("inf"), float("nan")
    G = torch.tensor([[inf, 200.0, -200.0, nan, 0.0, -0.0, 1.0, 3e38]])
    Uv = torch.tensor([[1.0, 2.0, 2.0, 1.0, 5.0, 5.0, nan, 1e-38]])
    for act in ("silu", "gelu", "gelu_tanh"):
        X = torch.empty(1, 8, dtype=torch.bfloat16, device="cuda")
        gpu.glu(torch.cat([G, Uv], 1).cuda(), X, act=act)
        x = X.cpu().float()[0]
        assert x[0] == inf and x[1] == 400 and x[2] == 0 and x[3].isnan() and x[4] == 0 and x[5] == 0 and x[6].isnan()
        assert 2.9 < float(x[7]) < 3.1
