"""What runs around the compressed products of a decoder layer, as measured work:

* ``plan``     -- rows of a batch sorted by the adapter each of them uses;
* ``adapters`` -- the low-rank adapters of many requests added to a shared projection;
* ``norm``     -- the end of one block and the start of the next: norm of the block's output, gate,
                  residual sum, norm for the next projection;
* ``glu``      -- the gated activation between the gate+up and the down projection.

Each case is one call on one GPU.  `own` false computes the plain form with elementary torch operations;
`own` true calls the framework.  Projections of the framework take fp16 or bf16 activations and give fp32
sums, so that is what goes in and comes out here.
"""
import math

import torch

own = False

#: Of every norm case: epsilon and the scales of the residual stream and of the block's output.
EPS, H_SCALE, Y_SCALE = 1e-5, 1.0, 0.75

_F = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # Made once for every step of a server: 64 running requests, up to 64 adapters in memory.
        dict(name="plan 64 rows", op="plan", M=64, n=64, none=5),
        # The rows of a large prefill batch (many prompts in one step) over many resident adapters.
        dict(name="plan 16384 rows", op="plan", M=16384, n=500, none=1000),
        # One user, one token: the attention output projection (8192 x 8192) of the 70B layer.
        dict(name="adapters 1 token", op="adapters", M=1, cols=8192, outs="8192", n=16, rank=16, mixed=False,
             none=0, dtype="bf16"),
        # Decoding 64 requests, an adapter for each, of different ranks, on the fused gate+up projection
        # of the 70B layer (one adapter pair for gate and one for up).
        dict(name="adapters 64 tokens", op="adapters", M=64, cols=8192, outs="28672+28672", n=64, rank=64, mixed=True,
             none=0, dtype="bf16"),
        # A half-full batch on the fused QKV projection of the 8B layer, some requests without an adapter.
        dict(name="adapters 37 tokens qkv", op="adapters", M=37, cols=4096, outs="4096+1024+1024", n=20, rank=16,
             mixed=False, none=9, dtype="f16"),
        # Odd everything: prompts of unequal lengths over a matrix whose sides no tile divides.
        dict(name="adapters odd sizes", op="adapters", M=333, cols=4099, outs="1021", n=7, rank=12, mixed=True,
             none=40, dtype="bf16"),
        # Prefill: 4096 prompt tokens of eight tenants through the 70B layer's gate+up.
        dict(name="adapters 4096 tokens", op="adapters", M=4096, cols=8192, outs="28672+28672", n=8, rank=64,
             mixed=False, none=0, dtype="bf16"),
        # One token of the 70B layer: residual sum and the norm before the next projection.
        dict(name="norm 1 token", op="norm", M=1, cols=8192, kind="rms", post=False, gate="none", dtype="bf16", h="bf16"),
        # A prefill batch with norms on both sides of the block.
        dict(name="norm 4096 tokens", op="norm", M=4096, cols=8192, kind="rms", post=True, gate="none", dtype="bf16",
             h="bf16"),
        # Odd width, layer norms with biases, a gate for each row, the residual stream in fp32.
        dict(name="norm odd width", op="norm", M=1000, cols=5001, kind="layer", post=True, gate="rows", dtype="f16",
             h="f32"),
        # One token between the 70B layer's gate+up and down projections.
        dict(name="glu 1 token", op="glu", M=1, cols=28672, act="silu", dtype="bf16"),
        # A prefill batch of the 8B layer.
        dict(name="glu 2048 tokens", op="glu", M=2048, cols=14336, act="gelu_tanh", dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "adapters", "adapters", "adapters", "norm", "norm", "glu"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "plan":
        M = _log(rng, 1, 16384)
        return dict(op=op, M=M, n=_log(rng, 1, 500), none=rng.randint(0, M // 4))
    M = _log(rng, 1, 4096)
    if op == "adapters":
        cols, outs = rng.choice([(8192, "8192+1024+1024"), (8192, "8192"), (8192, "28672+28672"), (28672, "8192"),
                                 (4096, "4096+1024+1024"), (4096, "14336+14336"), (14336, "4096"), None, None]) or \
            (_log(rng, 64, 12000), str(_log(rng, 64, 12000)))
        rank = rng.choice([4, 8, 8, 16, 16, 16, 32, 32, 64, 20, 37])
        return dict(op=op, M=M, cols=cols, outs=outs, n=_log(rng, 1, 64 if M <= 256 else 8), rank=rank,
                    mixed=rng.random() < 0.5, none=rng.randint(0, M // 4), dtype=dtype)
    if op == "norm":
        return dict(op=op, M=M, cols=rng.choice([4096, 8192, _log(rng, 64, 8192)]), kind=rng.choice(["rms", "rms", "layer"]),
                    post=rng.random() < 0.5, gate=rng.choice(["none", "cols", "rows"]), dtype=dtype,
                    h=rng.choice(["f32", dtype]))
    return dict(op=op, M=M, cols=rng.choice([14336, 28672, _log(rng, 64, 28672)]),
                act=rng.choice(["silu", "gelu_tanh", "gelu"]), dtype=dtype)


def _outs(case):
    return [int(v) for v in case["outs"].split("+")]


def _ranks(case):
    r = case["rank"]
    return [max(1, r >> (a % 4)) if case["mixed"] else r for a in range(case["n"])]


def _rows_of(case):
    """How many rows use adapter a: the rows with one are dealt out in turn (the seed says which rows)."""
    left = case["M"] - case["none"]
    return [left // case["n"] + (a < left % case["n"]) for a in range(case["n"])]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t.normal_(mean, std, generator=g)

    op, M = case["op"], case["M"]
    s = {"case": case}
    if op in ("plan", "adapters"):
        n = case["n"]
        rows = torch.tensor(_rows_of(case), device="cuda")
        ids = torch.cat([torch.repeat_interleave(torch.arange(n, device="cuda"), rows),
                         torch.full((case["none"],), -1, device="cuda")])
        if op == "plan":  # requests come and go: which adapters are used changes from step to step
            ids = torch.where(ids < 0, ids, torch.randint(0, n, (M,), generator=g, device="cuda"))
        s["ids"] = ids[torch.randperm(M, generator=g, device="cuda")].to(torch.int32)
    if op == "adapters":
        dt, cols, rank = _F[case["dtype"]], case["cols"], case["rank"]
        s["X"] = normal(M, cols, dtype=dt)
        s["A"] = [normal(n, rank, cols, std=cols ** -0.5, dtype=dt) for _ in _outs(case)]
        s["B"] = [normal(n, R, rank, std=0.1, dtype=dt) for R in _outs(case)]
        s["ranks"] = torch.tensor(_ranks(case), dtype=torch.int32, device="cuda")
        s["scales"] = torch.empty(n, device="cuda").uniform_(0.5, 2.0, generator=g)
        s["base"] = normal(M, sum(_outs(case)))
        s["Y"] = torch.empty_like(s["base"])
    elif op == "norm":
        dt, D = _F[case["dtype"]], case["cols"]
        s["y"] = normal(M, D)
        s["h"] = normal(M, D, std=2.0, dtype=_F[case["h"]])
        layer = case["kind"] == "layer"
        for k in ("post", "pre"):
            on = k == "pre" or case["post"]
            s["w_" + k] = normal(D, mean=1.0, std=0.2, dtype=dt) if on else None
            s["b_" + k] = normal(D, std=0.2, dtype=dt) if on and layer else None
        s["gate"] = {"none": None, "cols": (D,), "rows": (M, D)}[case["gate"]]
        if s["gate"] is not None:
            s["gate"] = normal(*s["gate"], std=0.5, dtype=dt)
        s["h_out"] = torch.empty_like(s["h"])
        s["x"] = torch.empty(M, D, dtype=dt, device="cuda")
    elif op == "glu":
        s["GU"] = normal(M, 2 * case["cols"], std=1.5)
        s["X"] = torch.empty(M, case["cols"], dtype=_F[case["dtype"]], device="cuda")
    if own:  # what a program keeps: handles on its weights, the batch's plan, workspaces
        from prng_seeded_decompress_b200 import seedlm
        s["lib"] = seedlm
        if op == "plan":
            s["plan"] = seedlm.AdapterPlan(M, n, device="cuda")
        elif op == "adapters":  # one plan serves every projection of every layer of the step
            s["adapters"] = seedlm.Adapters(s["A"], s["B"], ranks=s["ranks"], scales=s["scales"])
            s["plan"] = seedlm.adapter_plan(s["ids"], n)
            s["workspace"] = seedlm.adapter_workspace(s["adapters"], M)
        elif op == "norm":
            s["norm"] = seedlm.BlockNorm(D, kind=case["kind"], eps=EPS, h_scale=H_SCALE, y_scale=Y_SCALE,
                                         w_post=s["w_post"], b_post=s["b_post"], w_pre=s["w_pre"], b_pre=s["b_pre"])
    return s



# ------------------------------------------------------------------- a pass

def run(s):
    return (_framework if own else _plain)[s["case"]["op"]](s)


def _own_plan(s):
    p = s["lib"].adapter_plan(s["ids"], s["case"]["n"], plan=s["plan"])
    return [p.order, p.offsets]


def _own_adapters(s):
    s["lib"].adapter_apply(s["adapters"], s["plan"], s["X"], s["Y"], base=s["base"], workspace=s["workspace"])
    return s["Y"]


def _own_norm(s):
    s["lib"].block_norm(s["norm"], s["y"], s["h"], h_out=s["h_out"], x=s["x"], gate=s["gate"])
    return [s["h_out"], s["x"]]


def _own_glu(s):
    s["lib"].glu(s["GU"], s["X"], act=s["case"]["act"])
    return s["X"]


_framework = {"plan": _own_plan, "adapters": _own_adapters, "norm": _own_norm, "glu": _own_glu}


def _plain_plan(s):
    """Rows in the order of their adapter, rows without one last, rows of one adapter in their own order."""
    n, ids = s["case"]["n"], s["ids"]
    key = torch.where((ids >= 0) & (ids < n), ids, n)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(n + 1, dtype=key.dtype, device=key.device))
    return [order.to(torch.int32), offsets.to(torch.int32)]


def _plain_adapters(s):
    """Y = base + scale_a (x A_a^T) B_a^T for each row's adapter a; `ranks` says how much of A and B is used."""
    ids, M, n, rank = s["ids"].long(), s["case"]["M"], s["case"]["n"], s["case"]["rank"]
    on = ids >= 0
    a = torch.where(on, ids, 0)
    used = on[:, None] & (torch.arange(rank, device=ids.device) < s["ranks"][a][:, None])  # M x rank
    X, scale = s["X"].float(), s["scales"][a][:, None]
    out = []
    # One pass for each fused part of the projection, as a module for each part would make it.
    for A, B in zip(s["A"], s["B"]):
        if M <= n:  # an adapter for about every row: take each row's own
            S = torch.where(used, torch.einsum("mk,mrk->mr", X, A[a].float()), 0) * scale
            out.append(torch.einsum("mr,mjr->mj", S, B[a].float()))
        else:  # few adapters: all of them at once, then each row's own
            S = (X @ A.float().flatten(0, 1).T).view(M, n, rank)
            mine = torch.arange(n, device=ids.device) == a[:, None]
            S = torch.where(mine[:, :, None] & used[:, None, :], S, 0) * scale[:, :, None]
            out.append(S.flatten(1) @ B.float().transpose(1, 2).flatten(0, 1))
    return s["base"] + torch.cat(out, 1)


def _normed(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * w.float()
    return v if b is None else v + b.float()


def _plain_norm(s):
    """h' = h_scale h + y_scale gate norm_post(y);  x = norm_pre(h')."""
    kind, v = s["case"]["kind"], s["y"]
    if s["w_post"] is not None:
        v = _normed(v, kind, s["w_post"], s["b_post"])
    if s["gate"] is not None:
        v = v * s["gate"].float()
    h = H_SCALE * s["h"].float() + Y_SCALE * v
    return [h.to(s["h"].dtype), _normed(h, kind, s["w_pre"], s["b_pre"]).to(s["x"].dtype)]


def _plain_glu(s):
    g, u = s["GU"].chunk(2, 1)
    act = s["case"]["act"]
    if act == "silu":
        v = g / (1 + torch.exp(-g))
    elif act == "gelu":
        v = 0.5 * g * (1 + torch.erf(g * 0.5 ** 0.5))
    else:
        v = 0.5 * g * (1 + torch.tanh((2 / math.pi) ** 0.5 * (g + 0.044715 * g * g * g)))
    return (v * u).to(s["X"].dtype)


_plain = {"plan": _plain_plan, "adapters": _plain_adapters, "norm": _plain_norm, "glu": _plain_glu}


# ------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, M = case["op"], case["M"]
    if op == "plan":
        ids = s["ids"].tolist()
        order, offsets = [], []
        lists = [[] for _ in range(case["n"] + 1)]
        for i, a in enumerate(ids):
            lists[a if 0 <= a < case["n"] else case["n"]].append(i)
        for rows in lists:
            offsets.append(len(order))
            order += rows
        return [torch.tensor(order, dtype=torch.int32), torch.tensor(offsets, dtype=torch.int32)]
    if op == "adapters":
        Y = s["base"].double()
        for a, r in enumerate(_ranks(case)):
            rows = (s["ids"] == a).nonzero().flatten()
            x, scale, j = s["X"][rows].double(), s["scales"][a].double(), 0
            for A, B in zip(s["A"], s["B"]):
                y = (x @ A[a, :r].double().mT) @ B[a, :, :r].double().mT
                Y[rows, j:j + B.shape[1]] += scale * y
                j += B.shape[1]
        return Y
    if op == "norm":
        D = case["cols"]

        def norm(v, k):
            if case["kind"] == "layer":
                out = (v - v.sum(-1, True) / D) / torch.sqrt(v.var(-1, correction=0, keepdim=True) + EPS)
            else:
                out = v / torch.sqrt((v * v).sum(-1, True) / D + EPS)
            out = out * s["w_" + k].double()
            return out + s["b_" + k].double() if s["b_" + k] is not None else out

        y = s["y"].double()
        y = norm(y, "post") if case["post"] else y
        y = y * s["gate"].double() if s["gate"] is not None else y
        h = H_SCALE * s["h"].double() + Y_SCALE * y
        return [h, norm(h, "pre")]
    F = case["cols"]
    g, u = s["GU"][:, :F].double(), s["GU"][:, F:].double()
    if case["act"] == "silu":
        return g * torch.sigmoid(g) * u
    if case["act"] == "gelu":
        return g * torch.special.ndtr(g) * u
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)) * u


# -------------------------------------------------------------------- work

def work(case):
    op, M = case["op"], case["M"]
    if op == "plan":
        return {"bytes": 4 * M + 4 * M + 4 * (case["n"] + 1), "flops": 0}
    if op == "adapters":
        outs, cols = _outs(case), case["cols"]
        used = sum(r for r, rows in zip(_ranks(case), _rows_of(case)) if rows)
        per_row = sum(r * rows for r, rows in zip(_ranks(case), _rows_of(case)))
        weights = 2 * used * (len(outs) * cols + sum(outs))
        return {"bytes": weights + 2 * M * cols + 8 * M * sum(outs) + 4 * M,
                "flops": 2 * per_row * (len(outs) * cols + sum(outs))}
    if op == "norm":
        D, hb = case["cols"], 4 if case["h"] == "f32" else 2
        return {"bytes": M * D * (4 + 2 * hb + 2 + (2 if case["gate"] == "rows" else 0)) + 4 * D,
                "flops": 12 * M * D}
    return {"bytes": M * case["cols"] * 10, "flops": 20 * M * case["cols"]}
