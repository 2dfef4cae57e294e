#!/usr/bin/env python
"""Benchmark of the SeedLM hot path on B200: fused reconstruction + GEMV.

    python bench.py [--gpus N] [--steps K] [--warmup W] [--impl seedlm|reference]

Default workload (one step): the four batch-1 GEMVs of one Llama-3-70B-shaped
decoder layer at 4 bits per weight (C=8, P=3, K=16) -- QKV 10240x8192,
O 8192x8192, gate+up 57344x8192, down 8192x28672 -- with 80 distinct layer
copies resident in HBM (34.2 GB compressed, i.e. every down-projection of the
model) and step k using layer k mod 80, so no step finds its weights in L2.
Inputs are synthetic (seeded PCG64; seed uniform on [1,65535], q on [-8,7],
e on [8,12], x ~ N(0,1) in fp16); the run time of the method does not depend
on the weight values.

Prints ONE JSON line (rank 0).  ``value`` is the FP16-equivalent weight
throughput (2 bytes per weight processed per second, all ranks); ``e2e`` the
same through the public API with the activations copied in from pinned host
memory and the results copied back every step; ``roofline`` the GEMV
kernel's achieved compressed-byte bandwidth against the measured HBM copy
bandwidth; ``cpu_baseline`` the fp64 CPU oracle timed on a bounded sample;
``extras`` the other workloads (square sweep, 3-bit 8B layer, small-M GEMM,
decompression, dense fp16 GEMV reference point) at one GPU.

``--impl reference`` times the oracle itself (the reference arm of this
build), on the host cores, on the same workload, one bounded sample per step.
"""
from __future__ import annotations

import argparse
import json
import math
import os
import statistics
import sys
import threading
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

METRIC = ("µs/GEMV and FP16-equiv weight GB/s; achieved % of HBM roofline on "
          "compressed bytes")
UNIT = "GB/s (FP16-equivalent weight bytes)"
FALLBACK_HBM_GBS = 6650.0

LAYER_70B = [("qkv", 10240, 8192), ("o", 8192, 8192), ("gate_up", 57344, 8192),
             ("down", 8192, 28672)]
LAYER_8B = [("qkv", 6144, 4096), ("o", 4096, 4096), ("gate_up", 28672, 4096),
            ("down", 4096, 14336)]
WORKLOAD = "llama3-70b decoder layer, 4-bit SeedLM GEMV x4 (QKV, O, gate+up, down)"


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def dist_env():
    return (int(os.environ.get("RANK", "0")), int(os.environ.get("WORLD_SIZE", "1")),
            int(os.environ.get("LOCAL_RANK", "0")))


def load_peaks():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        with open(p) as fh:
            d = json.load(fh)
        return float(d["hbm_gbs"]), "measured"
    return FALLBACK_HBM_GBS, "fallback"


def profile_traffic(kernel: str):
    """Per-launch DRAM bytes of `kernel` from the committed ncu summary, if the
    kernel's sources are unchanged since that capture (else None)."""
    import hashlib
    path = os.path.join(ROOT, "profiles", "traffic.json")
    if not os.path.exists(path):
        return None
    with open(path) as fh:
        d = json.load(fh).get(kernel)
    if not d:
        return None
    h = hashlib.sha256()
    for f in d["sources"]:
        with open(os.path.join(ROOT, f), "rb") as fh:
            h.update(fh.read())
    if h.hexdigest() != d["sources_sha256"]:
        return None
    return d


# ---------------------------------------------------------------- clocks

class ClockSampler:
    """Samples SM clock and throttle reasons with NVML while running."""

    REASONS = {0x1: "gpu_idle", 0x2: "applications_clocks_setting", 0x4: "sw_power_cap",
               0x8: "hw_slowdown", 0x10: "sync_boost", 0x20: "sw_thermal_slowdown",
               0x40: "hw_thermal_slowdown", 0x80: "hw_power_brake_slowdown",
               0x100: "display_clock_setting"}

    def __init__(self, torch_dev: int, period_s: float = 0.02):
        self.period = period_s
        self.samples = []
        self.reasons = 0
        self.error = None
        self._stop = threading.Event()
        self._thread = None
        try:
            import pynvml
            pynvml.nvmlInit()
            import torch
            self.h = None
            try:
                uuid = str(torch.cuda.get_device_properties(torch_dev).uuid)
                self.h = pynvml.nvmlDeviceGetHandleByUUID("GPU-" + uuid)
            except Exception:
                pass
            if self.h is None:
                vis = os.environ.get("CUDA_VISIBLE_DEVICES", "")
                idx = int(vis.split(",")[torch_dev]) if vis and vis.split(",")[0].isdigit() \
                    else torch_dev
                self.h = pynvml.nvmlDeviceGetHandleByIndex(idx)
            self.nv = pynvml
            self.max_mhz = pynvml.nvmlDeviceGetMaxClockInfo(self.h, pynvml.NVML_CLOCK_SM)
        except Exception as e:  # no NVML: report the failure, do not guess
            self.error = f"nvml unavailable: {e}"
            self.nv = None
            self.max_mhz = None

    def _run(self):
        while not self._stop.is_set():
            try:
                self.samples.append(self.nv.nvmlDeviceGetClockInfo(self.h, self.nv.NVML_CLOCK_SM))
                self.reasons |= int(self.nv.nvmlDeviceGetCurrentClocksEventReasons(self.h))
            except Exception as e:
                self.error = str(e)
                return
            time.sleep(self.period)

    def __enter__(self):
        if self.nv is not None:
            self._thread = threading.Thread(target=self._run, daemon=True)
            self._thread.start()
        return self

    def __exit__(self, *exc):
        self._stop.set()
        if self._thread:
            self._thread.join()

    def result(self):
        out = {"sm_mhz": statistics.median(self.samples) if self.samples else None,
               "sm_max_mhz": self.max_mhz, "samples": len(self.samples),
               "reasons": [n for b, n in self.REASONS.items() if self.reasons & b]}
        if self.error:
            out["error"] = self.error
        return out


# ------------------------------------------------------------ CPU oracle

def oracle_sample(shapes, fmt_cp, rows_per_shape, threads, seed=5):
    """Time the fp64 oracle on the first rows of each shape; (weights, seconds)."""
    import numpy as np

    import oracle
    from prng_seeded_decompress_b200 import inputs
    oracle.build()
    weights, secs = 0, 0.0
    for i, (_, R, N) in enumerate(shapes):
        r = min(R, rows_per_shape)
        L = inputs.make_layer(r, N, *fmt_cp, seed=seed + i)
        _, xv = inputs.make_activations((N,), "f16", 77 + i)
        t0 = time.perf_counter()
        oracle.gemv(L["fmt"], L["rec"], L["eplane"], xv, threads=threads)
        secs += time.perf_counter() - t0
        weights += r * N
        del L
    return weights, secs


def cpu_model() -> str:
    try:
        with open("/proc/cpuinfo") as fh:
            for line in fh:
                if line.startswith("model name"):
                    return line.split(":", 1)[1].strip()
    except OSError:
        pass
    import platform
    return platform.processor() or "unknown"


def cpu_single_thread(shapes, fmt_cp, target_s=3.0):
    """The oracle on one host thread: GB/s FP16-equivalent on the first rows
    of each layer shape, about `target_s` of work."""
    w0, s0 = oracle_sample(shapes, fmt_cp, 8, 1)
    rows = max(8, int(8 * target_s / max(s0, 1e-3)))
    w, s = oracle_sample(shapes, fmt_cp, rows, 1)
    return {"value": round(2 * w / s / 1e9, 6), "unit": UNIT, "cores": 1,
            "sample": f"first {rows} rows of each of the 4 layer shapes: "
                      f"{w / 1e6:.1f} M weights in {s:.1f} s, fp64, 1 host thread"}


def cpu_baseline(shapes, fmt_cp, target_s=12.0):
    """The oracle on the host cores: the first rows of each layer shape (all
    rows if that is quick), repeated until about `target_s` of CPU work."""
    threads = os.cpu_count() or 1
    w0, s0 = oracle_sample(shapes, fmt_cp, threads, threads)
    rows = max(threads, int(threads * target_s / max(s0, 1e-3)))
    w = s = 0
    passes = 0
    while s < target_s and passes < 64:
        dw, ds = oracle_sample(shapes, fmt_cp, rows, threads)
        w += dw
        s += ds
        passes += 1
    return {"value": round(2 * w / s / 1e9, 6), "unit": UNIT, "cores": threads,
            "kind": "oracle",
            "sample": f"first {rows} rows of each of the 4 layer shapes, {passes} pass(es): "
                      f"{w / 1e6:.1f} M weights in {s:.1f} s, fp64, {threads} host threads",
            "cpu_model": cpu_model(),
            "single_thread": cpu_single_thread(shapes, fmt_cp),
            "encode": cpu_encode_baseline()}


def cpu_encode_baseline(blocks: int = 24):
    """The oracle's seed search (NumPy, vectorised over seeds) on Gaussian
    4-bit blocks, for comparison with the GPU encoder in `extras`."""
    import numpy as np

    from oracle.search import _tables, seed_search
    t0 = time.perf_counter()
    _tables(8, 3)                                   # pinv of all 65,535 seeds, once
    setup = time.perf_counter() - t0
    rng = np.random.default_rng(11)
    W = rng.standard_normal((blocks, 8)) * 0.02
    t0 = time.perf_counter()
    for b in range(blocks):
        seed_search(W[b], 8, 3)
    s = time.perf_counter() - t0
    return {"blocks_per_s": round(blocks / s, 2), "sample": f"{blocks} Gaussian 4-bit blocks "
            f"in {s:.1f} s after {setup:.1f} s of pseudo-inverse tables (NumPy, fp64)"}


# --------------------------------------------------------------- GPU arm

def make_layer_on_device(torch, shapes, cp, seed):
    import numpy as np

    from prng_seeded_decompress_b200 import inputs
    out = []
    for i, (name, R, N) in enumerate(shapes):
        L = inputs.make_layer(R, N, *cp, seed=seed + i)
        rec = torch.from_numpy(L["rec"].view(np.int32)).cuda()
        ep = torch.from_numpy(L["eplane"]).cuda() if cp[1] == 4 else None
        out.append(dict(name=name, fmt=L["fmt"], rec=rec, ep=ep, R=R, N=N))
        del L
    return out


def replicate(torch, layer, copies):
    res = [layer]
    for _ in range(copies - 1):
        res.append([dict(m, rec=m["rec"].clone(), ep=None if m["ep"] is None else m["ep"].clone())
                    for m in layer])
    return res


def time_median(torch, fn, reps, regions=5):
    """Median over `regions` timed regions of `reps` calls each: ms per call."""
    return statistics.median(time_region(torch, fn, reps) / reps for _ in range(regions))


def time_region(torch, fn, reps):
    """Device time of `reps` calls of fn() on the current stream, in ms."""
    s = torch.cuda.current_stream()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    e0.record(s)
    for i in range(reps):
        fn(i)
    e1.record(s)
    e1.synchronize()
    return e0.elapsed_time(e1)


def layer_bytes(shapes, cp):
    """(weights, compressed stored bytes, algorithmic bytes) of one layer pass."""
    C, P = cp
    w = comp = alg = 0
    for _, R, N in shapes:
        nb = (N + C - 1) // C
        w += R * N
        rec_pitch = (nb + 3) // 4 * 4
        e_pitch = ((nb + 1) // 2 + 15) // 16 * 16 if P == 4 else 0
        comp += R * (4 * rec_pitch + e_pitch)
        ideal = (16 + 4 * P + 4) * nb / 8
        alg += R * ideal + 2 * N + 4 * R
    return w, comp, alg


def extras(torch, sl, args):
    """The other workloads, one GPU: square sweep, 3-bit 8B layer, small-M
    GEMM, decompression, the encoder, dense fp16 GEMV reference point."""
    import numpy as np

    from prng_seeded_decompress_b200 import inputs
    l2 = torch.cuda.get_device_properties(0).L2_cache_size
    out = {}

    # Square sweep (512..2048): 1000 back-to-back calls, a CUDA-graph replay
    # of 1000 calls, and a cold-L2 rotation over >= 4x L2 of distinct copies.
    sweep = {}
    for n in (512, 1024, 2048):
        layer = make_layer_on_device(torch, [("sq", n, n)], (8, 3), 500 + n)[0]
        xb, _ = inputs.make_activations((n,), "f16", 600 + n)
        x = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.float16)
        y = torch.empty(n, device="cuda")
        f = sl.Format.from_dict(layer["fmt"])
        call = lambda i: sl.gemv(f, layer["rec"], None, x, y)  # noqa: E731
        for i in range(20):
            call(i)
        warm = time_median(torch, call, 1000) * 1e3
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call(0)
            with torch.cuda.graph(g, stream=s):
                for i in range(1000):
                    sl.gemv(f, layer["rec"], None, x, y, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        g.replay()
        graph = time_median(torch, lambda i: g.replay(), 1) / 1000 * 1e3
        del g
        copies = max(2, math.ceil(4 * l2 / layer["rec"].numel() / 4))
        recs = [layer["rec"].clone() for _ in range(copies)]
        cold = time_median(torch, lambda i: sl.gemv(f, recs[i % copies], None, x, y),
                           max(1000, copies)) * 1e3
        del recs
        comp = n * layer["fmt"]["rec_pitch"] * 4
        sweep[f"{n}x{n}"] = {"us_per_call": round(warm, 3), "us_per_call_graph": round(graph, 3),
                             "us_per_call_cold_l2": round(cold, 3), "cold_copies": copies,
                             "fp16_equiv_gbs_cold": round(2 * n * n / cold / 1e3, 1),
                             "compressed_gbs_cold": round(comp / cold / 1e3, 1)}
    out["square_sweep_4bit"] = sweep

    # The 70B layer's four GEMVs as one CUDA graph vs launched one by one
    # (4 resident copies rotating, 428 MB of records each, so L2 stays cold):
    # how much a fused layer launch could save.
    layer = make_layer_on_device(torch, LAYER_70B, (8, 3), 1300)
    copies = replicate(torch, layer, 4)
    fm = [sl.Format.from_dict(m["fmt"]) for m in layer]
    xl = {}
    for _, _, N in LAYER_70B:
        if N not in xl:
            xb, _ = inputs.make_activations((N,), "f16", 1400 + N)
            xl[N] = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.float16)
    yl = [torch.empty(R, device="cuda") for _, R, _ in LAYER_70B]

    def run70(lay, stream=None):
        for m, f, y in zip(lay, fm, yl):
            sl.gemv(f, m["rec"], None, xl[m["N"]], y, stream=stream)
    for i in range(8):
        run70(copies[i % 4])
    eager = time_median(torch, lambda i: run70(copies[i % 4]), 80) * 1e3
    graphs = []
    gs = torch.cuda.Stream()
    gs.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(gs):
        for c in copies:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=gs):
                run70(c, stream=gs)
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(gs)
    for i in range(8):
        graphs[i % 4].replay()
    graph = time_median(torch, lambda i: graphs[i % 4].replay(), 80) * 1e3
    out["llama3_70b_layer_graph_vs_eager"] = {"us_per_layer_eager": round(eager, 2),
                                             "us_per_layer_graph": round(graph, 2)}
    # The same four GEMVs as one batched launch (seedlm_gemv_batch).
    batched = time_median(torch, lambda i: sl.gemv_batch(
        [(f, m["rec"], None, xl[m["N"]], y) for m, f, y in zip(copies[i % 4], fm, yl)]), 80) * 1e3
    out["llama3_70b_layer_batched"] = {"us_per_layer": round(batched, 2),
                                      "us_per_layer_separate_calls": round(eager, 2)}
    del graphs, copies, layer

    # 3-bit Llama-3-8B layer: as specified (one layer) and 32 copies (cold).
    layer = make_layer_on_device(torch, LAYER_8B, (12, 4), 700)
    xs = {}
    for _, _, N in LAYER_8B:
        if N not in xs:
            xb, _ = inputs.make_activations((N,), "f16", 800 + N)
            xs[N] = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.float16)
    ys = [torch.empty(R, device="cuda") for _, R, _ in LAYER_8B]
    fmts = [sl.Format.from_dict(m["fmt"]) for m in layer]

    def run_layer(lay):
        for m, f, y in zip(lay, fmts, ys):
            sl.gemv(f, m["rec"], m["ep"], xs[m["N"]], y)
    for i in range(5):
        run_layer(layer)
    one = time_median(torch, lambda i: run_layer(layer), 100) * 1e3
    copies = replicate(torch, layer, 32)
    cold = time_median(torch, lambda i: run_layer(copies[i % 32]), 64) * 1e3
    del copies
    w, comp, _ = layer_bytes(LAYER_8B, (12, 4))
    out["llama3_8b_layer_3bit"] = {
        "us_per_layer_single_copy": round(one, 2), "us_per_layer_32_copies": round(cold, 2),
        "us_per_gemv_32_copies": round(cold / 4, 2),
        "fp16_equiv_gbs": round(2 * w / cold / 1e3, 1),
        "compressed_gbs": round(comp / cold / 1e3, 1)}
    del layer

    # Small-M GEMM on the 70B MLP shapes, 4-bit and 3-bit, M in {1,8,16,64},
    # rotating over distinct record copies totalling >= 4x L2.
    gemm = {}
    for cp, tag in (((8, 3), "4bit"), ((12, 4), "3bit")):
        for name, R, N in (("up_28672x8192", 28672, 8192), ("down_8192x28672", 8192, 28672)):
            base = make_layer_on_device(torch, [(name, R, N)], cp, 900 + R)[0]
            nbytes = base["rec"].numel() * 4 + (0 if base["ep"] is None else base["ep"].numel())
            ncp = max(2, math.ceil(4 * l2 / nbytes))
            mats = [base] + [dict(base, rec=base["rec"].clone(),
                                  ep=None if base["ep"] is None else base["ep"].clone())
                             for _ in range(ncp - 1)]
            f = sl.Format.from_dict(base["fmt"])
            # bf16 activations at every M (M = 2 and 4 run on the CUDA cores;
            # from M = 5 on the tensor cores take them as fp16 with a
            # power-of-two scale per row), fp16 at M = 16 and 64.
            for M, dt in ((1, "bf16"), (2, "bf16"), (4, "bf16"), (8, "bf16"), (16, "bf16"),
                          (64, "bf16"), (16, "f16"), (64, "f16")):
                Xb, _ = inputs.make_activations((M, N), dt, 950 + M)
                X = torch.from_numpy(Xb.view(np.int16)).cuda().view(
                    torch.bfloat16 if dt == "bf16" else torch.float16)
                Y = torch.empty((M, R), device="cuda")
                ws = sl.gemm_workspace(f, M)
                fn = lambda i: sl.gemm_smallM(f, mats[i % ncp]["rec"], mats[i % ncp]["ep"], X, Y,  # noqa
                                              workspace=ws)
                fn(0)
                us = time_median(torch, fn, 4 * ncp) * 1e3
                key = f"{tag}/{name}/M={M}" + ("" if dt == "bf16" else "/f16")
                gemm[key] = {
                    "us_per_call": round(us, 2), "weights_per_s_e9": round(R * N / us / 1e3, 2),
                    "tflops_useful": round(2 * M * R * N / us / 1e6, 2), "copies": ncp}
            xb, _ = inputs.make_activations((N,), "bf16", 990)
            x = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.bfloat16)
            y = torch.empty(R, device="cuda")
            fn = lambda i: sl.gemv(f, mats[i % ncp]["rec"], mats[i % ncp]["ep"], x, y)  # noqa
            fn(0)
            gemm[f"{tag}/{name}/gemv_bf16"] = {"us_per_call": round(time_median(torch, fn, 4 * ncp)
                                                                    * 1e3, 2)}
            # Larger batches (prefill) through seedlm_gemm: passes of at most
            # 256 rows of X, 4-bit gate/up shape only.
            if tag == "4bit" and name.startswith("up"):
                for M in (128, 256, 1024):
                    Xb, _ = inputs.make_activations((M, N), "bf16", 960 + M)
                    X = torch.from_numpy(Xb.view(np.int16)).cuda().view(torch.bfloat16)
                    Y = torch.empty((M, R), device="cuda")
                    ws = torch.zeros(max(sl.gemm_any_workspace_bytes(f, M), 256),
                                     dtype=torch.uint8, device="cuda")
                    fn = lambda i: sl.gemm(f, mats[i % ncp]["rec"], mats[i % ncp]["ep"], X, Y,  # noqa
                                           workspace=ws)
                    fn(0)
                    us = time_median(torch, fn, 2 * ncp) * 1e3
                    gemm[f"{tag}/{name}/M={M}"] = {
                        "us_per_call": round(us, 2), "weights_per_s_e9": round(R * N / us / 1e3, 2),
                        "tflops_useful": round(2 * M * R * N / us / 1e6, 2), "copies": ncp,
                        "entry": "seedlm_gemm"}
                    del ws
            del mats, base
    out["gemm_smallM"] = gemm

    # Dense fp16 reference for the crossover on the same shapes: the weights
    # as fp16 (2 bytes each), Y = X W^T through cuBLAS (torch.matmul, fp32
    # accumulation) at M >= 2 and the in-house dense GEMV at M = 1,
    # rotating over copies totalling >= 4x L2.
    dense_mm = {}
    for name, R, N in (("up_28672x8192", 28672, 8192), ("down_8192x28672", 8192, 28672)):
        Wd = torch.randn((R, N), device="cuda", dtype=torch.float16) * 0.02
        ncp = max(2, math.ceil(4 * l2 / (Wd.numel() * 2)))
        Ws = [Wd] + [Wd.clone() for _ in range(ncp - 1)]
        for M in ((1, 2, 4, 8, 16, 64, 128, 256, 1024) if name.startswith("up") else (1, 2, 4, 8, 16, 64)):
            X = torch.randn((M, N), device="cuda", dtype=torch.float16)
            if M == 1:
                y = torch.empty(R, device="cuda")
                fn = lambda i: sl.dense_gemv_f16(Ws[i % ncp], X[0], y)  # noqa
            else:
                fn = lambda i: torch.matmul(X, Ws[i % ncp].t())  # noqa
            fn(0)
            us = time_median(torch, fn, 4 * ncp) * 1e3
            dense_mm[f"{name}/M={M}"] = {"us_per_call": round(us, 2),
                                         "hbm_gbs": round(2 * R * N / us / 1e3, 1),
                                         "impl": "in-house GEMV" if M == 1 else "cuBLAS"}
        del Ws, Wd
    out["dense_fp16_smallM"] = dense_mm

    # Decompression of the 70B down projection (fp32 output).
    m = make_layer_on_device(torch, [("down", 8192, 28672)], (8, 3), 1100)[0]
    f = sl.Format.from_dict(m["fmt"])
    W = torch.empty((8192, 28672), device="cuda")
    sl.decompress(f, m["rec"], None, W)
    us = time_median(torch, lambda i: sl.decompress(f, m["rec"], None, W), 10) * 1e3
    moved = W.numel() * 4 + m["rec"].numel() * 4
    out["decompress_4bit_8192x28672"] = {"us_per_call": round(us, 1),
                                        "hbm_gbs_read_plus_write": round(moved / us / 1e3, 1)}
    del W, m

    # Encoder (offline): full seed / coefficient / exponent search of a
    # Gaussian 4096 x 4096 matrix at 4 and 3 bits (2.1 M / 1.4 M blocks x
    # 65,535 seeds x 16 exponents), one call after a warm-up call.
    rng = np.random.default_rng(11)
    We = torch.from_numpy((rng.standard_normal((4096, 4096)) * 0.02).astype(np.float32)).cuda()
    for bits, (C, P) in ((4, (8, 3)), (3, (12, 4))):
        fe = inputs.make_format(4096, 4096, C, P)
        rec_e = torch.empty((4096, fe["rec_pitch"]), dtype=torch.int32, device="cuda")
        ep_e = (torch.empty((4096, fe["e_pitch"]), dtype=torch.uint8, device="cuda")
                if P == 4 else None)
        err_e = torch.empty((4096, fe["nb"]), dtype=torch.float64, device="cuda")
        sl.encode(fe, We, rec_e, ep_e, err_e)
        ms = time_region(torch, lambda i: sl.encode(fe, We, rec_e, ep_e), 1)
        blocks = 4096 * fe["nb"]
        # Relative reconstruction error of the fit (Gaussian weights, as in
        # the pages' design-space exploration): ||W - W_hat|| / ||W||.
        rel = math.sqrt(float(err_e.sum()) / float((We.double() ** 2).sum()))
        out[f"encode_{bits}bit_4096x4096"] = {
            "ms_per_call": round(ms, 1), "blocks_per_s": round(blocks / (ms / 1e3)),
            "seeds_per_s_e9": round(blocks * 65535 / (ms / 1e3) / 1e9, 1),
            "relative_reconstruction_error": round(rel, 4)}
        del rec_e, ep_e, err_e
    del We

    # Design-space sweep: exhaustive search (all 2^K - 1 seeds, 16 exponents)
    # on Gaussian blocks for other block sizes C, latent dimensions P and
    # seed widths K; relative reconstruction error against bits per weight
    # ((K + 4P + 4) / C).
    sweep_ds = {}
    for C, P, K, nblk in ((8, 3, 16, 4096), (8, 4, 16, 4096), (8, 2, 16, 4096),
                          (12, 3, 16, 4096), (12, 4, 16, 4096), (16, 4, 16, 4096),
                          (16, 3, 16, 4096), (8, 3, 12, 4096), (8, 3, 14, 4096),
                          (8, 3, 18, 1024), (8, 3, 20, 256)):
        rng = np.random.default_rng(1000 + C * 100 + P * 10 + K)
        Wb = torch.from_numpy((rng.standard_normal((nblk, C)) * 0.02).astype(np.float32)).cuda()
        sd = torch.empty(nblk, dtype=torch.int32, device="cuda")
        qd = torch.empty((nblk, P), dtype=torch.int8, device="cuda")
        ed = torch.empty(nblk, dtype=torch.uint8, device="cuda")
        er = torch.empty(nblk, dtype=torch.float64, device="cuda")
        sl.search_blocks(C, P, K, Wb, sd, qd, ed, er)
        ms = time_region(torch, lambda i: sl.search_blocks(C, P, K, Wb, sd, qd, ed, er), 1)
        rel = math.sqrt(float(er.sum()) / float((Wb.double() ** 2).sum()))
        sweep_ds[f"C={C},P={P},K={K}"] = {
            "bits_per_weight": round((K + 4 * P + 4) / C, 3), "relative_error": round(rel, 4),
            "blocks": nblk, "ms": round(ms, 1)}
        del Wb, sd, qd, ed, er
    out["design_space_sweep"] = sweep_ds

    # Dense fp16 GEMV (in-house) on the 70B layer shapes, 4 rotating copies.
    rng = np.random.default_rng(3)
    dense = []
    for name, R, N in LAYER_70B:
        Wh = torch.from_numpy((rng.standard_normal((R, N), dtype=np.float32) * 0.02)
                              .astype(np.float16).view(np.int16)).cuda().view(torch.float16)
        dense.append((Wh, [Wh] + [Wh.clone() for _ in range(3)]))
    xsd = {N: torch.randn(N, device="cuda").half() for N in (8192, 28672)}
    ysd = [torch.empty(R, device="cuda") for _, R, _ in LAYER_70B]

    def dense_layer(i):
        for (Wh, cps), (_, R, N), y in zip(dense, LAYER_70B, ysd):
            sl.dense_gemv_f16(cps[i % 4], xsd[N], y)
    for i in range(4):
        dense_layer(i)
    us = time_median(torch, dense_layer, 20) * 1e3
    w, _, _ = layer_bytes(LAYER_70B, (8, 3))
    out["dense_fp16_gemv_70b_layer"] = {"us_per_layer": round(us, 2),
                                       "hbm_gbs": round(2 * w / us / 1e3, 1)}
    del dense

    # The same reference on the Llama-3-8B layer shapes (the 3-bit workload).
    dense8 = []
    for name, R, N in LAYER_8B:
        Wh = (torch.randn((R, N), device="cuda") * 0.02).half()
        dense8.append([Wh] + [Wh.clone() for _ in range(7)])
    xs8 = {N: torch.randn(N, device="cuda").half() for N in (4096, 14336)}
    ys8 = [torch.empty(R, device="cuda") for _, R, _ in LAYER_8B]

    def dense_layer8(i):
        for cps, (_, R, N), y in zip(dense8, LAYER_8B, ys8):
            sl.dense_gemv_f16(cps[i % 8], xs8[N], y)
    for i in range(8):
        dense_layer8(i)
    us = time_median(torch, dense_layer8, 40) * 1e3
    w8, _, _ = layer_bytes(LAYER_8B, (12, 4))
    out["dense_fp16_gemv_8b_layer"] = {"us_per_layer": round(us, 2),
                                      "hbm_gbs": round(2 * w8 / us / 1e3, 1)}
    del dense8
    return out


def summarize(result, hbm_peak):
    """The figures a reader looks for first, compact, at the end of the line."""
    ex = result["extras"]
    out = {"llama3_70b_4bit_us_per_layer": round(result["ms_per_step"] * 1e3, 2),
           "llama3_70b_4bit_roofline_frac": result["roofline"]["frac"]}
    d70 = ex.get("dense_fp16_gemv_70b_layer", {}).get("us_per_layer")
    if d70:
        out["llama3_70b_speedup_vs_dense_fp16"] = round(d70 / (result["ms_per_step"] * 1e3), 3)
    l8 = ex.get("llama3_8b_layer_3bit")
    if l8:
        _, comp8, alg8 = layer_bytes(LAYER_8B, (12, 4))
        us8 = l8["us_per_layer_32_copies"]
        out["llama3_8b_3bit_us_per_layer"] = us8
        out["llama3_8b_3bit_roofline_frac"] = round(alg8 / us8 / 1e3 / hbm_peak, 4)
        d8 = ex.get("dense_fp16_gemv_8b_layer", {}).get("us_per_layer")
        if d8:
            out["llama3_8b_speedup_vs_dense_fp16"] = round(d8 / us8, 3)
    g = ex.get("gemm_smallM", {})
    dm = ex.get("dense_fp16_smallM", {})
    for M in (2, 4, 8, 16, 64, 128, 256, 1024):
        k = f"4bit/up_28672x8192/M={M}"
        if k in g:
            out[f"gemm_4bit_28672x8192_M{M}_us"] = g[k]["us_per_call"]
        kd = f"up_28672x8192/M={M}"
        if kd in dm:
            out[f"dense_fp16_28672x8192_M{M}_us"] = dm[kd]["us_per_call"]
    bt = ex.get("llama3_70b_layer_batched")
    if bt:
        out["llama3_70b_4bit_us_per_layer_one_batched_launch"] = bt["us_per_layer"]
    sq = ex.get("square_sweep_4bit", {})
    for n, v in sq.items():
        out[f"square_{n}_us_graph"] = v["us_per_call_graph"]
    return out


def seedlm_arm(args):
    import numpy as np
    import torch

    rank, world, local_rank = dist_env()
    torch.cuda.set_device(local_rank)
    if world > 1:
        import datetime

        import torch.distributed as dist
        dist.init_process_group("nccl", timeout=datetime.timedelta(seconds=120),
                                device_id=torch.device("cuda", local_rank))
    from prng_seeded_decompress_b200 import build
    if rank == 0 or world == 1:
        build.build()
    if world > 1:
        torch.distributed.barrier()
    from prng_seeded_decompress_b200 import dist_util, inputs, seedlm as sl
    sl.init()
    hbm_peak, peak_kind = load_peaks()

    shapes, cp = LAYER_70B, (8, 3)
    t0 = time.time()
    base = make_layer_on_device(torch, shapes, cp, seed=1000 + rank)
    layers = replicate(torch, base, args.layers)
    torch.cuda.synchronize()
    log(f"[rank {rank}] {args.layers} layer copies resident "
        f"({sum(m['rec'].numel() * 4 for lay in layers for m in lay) / 1e9:.1f} GB) "
        f"in {time.time() - t0:.1f} s")
    xs = {}
    for _, _, N in shapes:
        if N not in xs:
            xb, _ = inputs.make_activations((N,), "f16", 2000 + N)
            xs[N] = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.float16)
    ys = [torch.empty(R, device="cuda") for _, R, _ in shapes]
    fmts = [sl.Format.from_dict(m["fmt"]) for m in base]

    def step(k):
        lay = layers[k % args.layers]
        for m, f, y in zip(lay, fmts, ys):
            sl.gemv(f, m["rec"], m["ep"], xs[m["N"]], y)

    for k in range(args.warmup):
        step(k)
    torch.cuda.synchronize()
    if world > 1:
        torch.distributed.barrier()
    n0 = sl.launch_count()
    with ClockSampler(local_rank) as clk:
        ms = time_region(torch, step, args.steps)
    launches = sl.launch_count() - n0
    ms = dist_util.max_over_ranks(ms, device="cuda")
    w, comp, alg = layer_bytes(shapes, cp)
    secs = ms / 1e3
    value = 2 * w * args.steps * world / secs / 1e9
    achieved = alg * args.steps / secs / 1e9          # per launch avg bytes / avg duration
    comp_gbs = comp * args.steps / secs / 1e9

    # End to end through the public API: every step, the four GEMVs'
    # activation vectors come in from pinned host memory (one packed copy)
    # and their four results go back to pinned host memory (one packed
    # copy), as a serving loop would run it: inputs on an H2D stream, results
    # on a D2H stream, double-buffered on the device, so step k's copies
    # overlap the compute of steps k-1 / k+1.  The timed region ends when the
    # last step's results are on the host.
    xoff = [0]
    for _, _, N in shapes:
        xoff.append(xoff[-1] + N)
    yoff = [0]
    for _, R, _ in shapes:
        yoff.append(yoff[-1] + R)
    hx = torch.cat([xs[N].cpu() for _, _, N in shapes]).pin_memory()
    hy = [torch.empty(yoff[-1], dtype=torch.float32).pin_memory() for _ in range(2)]
    dx = [torch.empty_like(hx, device="cuda") for _ in range(2)]
    dy = [torch.empty(yoff[-1], device="cuda") for _ in range(2)]
    dxs = [[d[xoff[i]:xoff[i + 1]] for i in range(len(shapes))] for d in dx]
    dys = [[d[yoff[i]:yoff[i + 1]] for i in range(len(shapes))] for d in dy]
    h2d = hx.numel() * 2    # one input vector per GEMV
    d2h = yoff[-1] * 4      # one output vector per GEMV
    cs = torch.cuda.current_stream()
    s_in, s_out = torch.cuda.Stream(), torch.cuda.Stream()
    ev_in = [torch.cuda.Event() for _ in range(2)]
    ev_done = [torch.cuda.Event() for _ in range(2)]
    ev_out = [torch.cuda.Event() for _ in range(2)]
    for b in range(2):
        ev_done[b].record(cs)
        ev_out[b].record(cs)

    def e2e_step(k):
        b = k % 2
        lay = layers[k % args.layers]
        with torch.cuda.stream(s_in):
            s_in.wait_event(ev_done[b])          # step k-2 finished reading dx[b]
            dx[b].copy_(hx, non_blocking=True)
            ev_in[b].record(s_in)
        cs.wait_event(ev_in[b])
        cs.wait_event(ev_out[b])                 # step k-2's results left dy[b]
        for m, f, xv, yv in zip(lay, fmts, dxs[b], dys[b]):
            sl.gemv(f, m["rec"], m["ep"], xv, yv)
        ev_done[b].record(cs)
        with torch.cuda.stream(s_out):
            s_out.wait_event(ev_done[b])
            hy[b].copy_(dy[b], non_blocking=True)
            ev_out[b].record(s_out)

    def e2e_region(reps):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        e0.record(cs)
        for k in range(reps):
            e2e_step(k)
        for b in range(2):
            cs.wait_event(ev_out[b])             # every result is on the host
        e1.record(cs)
        e1.synchronize()
        return e0.elapsed_time(e1)

    for k in range(args.warmup):
        e2e_step(k)
    torch.cuda.synchronize()
    if world > 1:
        torch.distributed.barrier()
    e2e_ms = e2e_region(args.steps)
    e2e_ms = dist_util.max_over_ranks(e2e_ms, device="cuda")
    e2e_value = 2 * w * args.steps * world / (e2e_ms / 1e3) / 1e9

    # Per-shape times (same rotation over the resident copies).
    per_shape = {}
    for i, (name, R, N) in enumerate(shapes):
        f, y = fmts[i], ys[i]
        fn = lambda k, i=i, f=f, y=y: sl.gemv(f, layers[k % args.layers][i]["rec"], None,  # noqa
                                             xs[layers[0][i]["N"]], y)
        reps = min(args.steps, 400)
        us = time_region(torch, fn, reps) / reps * 1e3
        C, P = cp
        nb = (N + C - 1) // C
        per_shape[name] = {"us": round(us, 2),
                           "compressed_gbs": round(R * nb * 4 / us / 1e3, 1),
                           "fp16_equiv_gbs": round(2 * R * N / us / 1e3, 1)}

    traffic = profile_traffic("gemv_kernel<8>")
    result = {
        "metric": METRIC, "value": round(value, 1), "unit": UNIT, "n_gpus": world,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": round(ms / args.steps, 5),
        # Arithmetic: weights rebuilt exactly in int32, products and sums in fp32.
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f32",
        "data": "synthetic (seeded PCG64 records and N(0,1) fp16 activations; runtime does not "
                "depend on weight values)",
        "config": {"workload": WORKLOAD, "format": "C=8, P=3, K=16 (32 bits per 8 weights)",
                   "shapes": {n: [R, N] for n, R, N in shapes}, "batch": 1,
                   "layer_copies_resident": args.layers,
                   "resident_compressed_gb": round(comp * args.layers / 1e9, 2),
                   "l2": "inputs larger than L2: each step reads one layer copy "
                         f"({comp / 1e6:.0f} MB) of {args.layers} resident",
                   "parallelism": f"replicas x{world} (independent layer stacks per GPU)"},
        "us_per_gemv": round(ms * 1e3 / (args.steps * len(shapes)), 3),
        "per_shape": per_shape,
        "compressed_gbs": round(comp_gbs, 1),
        "hbm_roofline_pct": round(100 * comp_gbs / hbm_peak, 2),
        "hbm_roofline_pct_of_8tbs_spec": round(100 * comp_gbs / 8000, 2),
        "roofline": {"bound": "hbm", "achieved": round(achieved, 1), "peak": hbm_peak,
                     "peak_kind": peak_kind, "unit": "GB/s", "frac": round(achieved / hbm_peak, 4),
                     "kernel": "gemv_kernel<8>",
                     "traffic": None if traffic is None else traffic["bytes_per_launch"],
                     "algorithmic_bytes_per_launch": round(alg / len(shapes))},
        "clocks": clk.result(),
        "e2e": {"value": round(e2e_value, 1), "unit": UNIT, "h2d_bytes_per_step": h2d,
                "d2h_bytes_per_step": d2h, "ms_per_step": round(e2e_ms / args.steps, 5)},
        "gpu_launches": int(launches),
    }
    # The same kernel against its instruction-issue bound: blocks per second if
    # every warp scheduler issued one instruction per cycle at the measured SM
    # clock, with the kernel's own instruction count per block (ncu, same
    # source hash as the traffic figure).
    sm_mhz = result["clocks"].get("sm_mhz")
    if traffic is not None and traffic.get("thread_instructions_per_block") and sm_mhz:
        ipb = traffic["thread_instructions_per_block"]
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        peak_bps = sms * 4 * 32 * sm_mhz * 1e6 / ipb
        got_bps = achieved * 1e9 / 4  # 4 record bytes per 8-weight block
        result["roofline_issue"] = {
            "bound": "alu", "achieved": round(got_bps / 1e9, 2), "peak": round(peak_bps / 1e9, 2),
            "unit": "Gblock/s", "frac": round(got_bps / peak_bps, 4),
            "thread_instructions_per_block": ipb, "sm_mhz": sm_mhz, "sms": sms,
            "kernel": "gemv_kernel<8>"}
    del layers, base
    torch.cuda.empty_cache()
    if world == 1 and not args.no_extras:
        result["extras"] = extras(torch, sl, args)
    if rank == 0 and world == 1 and not args.no_cpu_baseline:
        result["cpu_baseline"] = cpu_baseline(shapes, cp, target_s=args.cpu_seconds)
    if "extras" in result:
        result["summary"] = summarize(result, hbm_peak)
    if world > 1:
        torch.distributed.barrier()
        torch.distributed.destroy_process_group()
    if rank == 0:
        print(json.dumps(result), flush=True)


def reference_arm(args):
    rank, world, _ = dist_env()
    if rank != 0:
        return
    shapes, cp = LAYER_70B, (8, 3)
    threads = os.cpu_count() or 1
    # One step = the oracle on the first `rows` rows of each of the 4 shapes,
    # sized so that one step takes about `--ref-step-seconds`.
    w0, s0 = oracle_sample(shapes, cp, threads, threads)
    rows = max(threads, int(threads * args.ref_step_seconds / max(s0, 1e-3)))
    for _ in range(args.warmup):
        oracle_sample(shapes, cp, rows, threads)
    tot_w, tot_s = 0, 0.0
    for _ in range(args.steps):
        w, s = oracle_sample(shapes, cp, rows, threads)
        tot_w += w
        tot_s += s
    value = 2 * tot_w / tot_s / 1e9
    sample = (f"first {rows} rows of each of the 4 layer shapes per step "
              f"({tot_w / args.steps / 1e6:.1f} M weights), fp64, {threads} host threads")
    print(json.dumps({
        "impl": "reference", "metric": METRIC, "value": round(value, 6), "unit": UNIT,
        "n_gpus": world, "steps": args.steps, "warmup": args.warmup,
        "ms_per_step": round(1e3 * tot_s / args.steps, 3), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "f64",
        "data": "synthetic (seeded PCG64 records and N(0,1) fp16 activations)",
        "config": {"workload": WORKLOAD, "format": "C=8, P=3, K=16 (32 bits per 8 weights)",
                   "shapes": {n: [R, N] for n, R, N in shapes}, "batch": 1,
                   "parallelism": "host threads (rows split)"},
        "cpu_baseline": {"value": round(value, 6), "unit": UNIT, "cores": threads,
                         "kind": "oracle", "sample": sample},
        "e2e": {"value": round(value, 6), "unit": UNIT, "h2d_bytes_per_step": 0,
                "d2h_bytes_per_step": 0},
    }), flush=True)


def flush_l2(torch):
    """Leave L2 holding clean lines only: the uploads of the inputs are
    written back now rather than during the captured kernel."""
    junk = torch.empty(int(4 * torch.cuda.get_device_properties(0).L2_cache_size) // 4,
                       dtype=torch.float32, device="cuda")
    junk.zero_()
    float(junk.sum())  # a read pass over 4x L2 evicts every dirty line
    del junk
    torch.cuda.synchronize()


def profile_case(name: str):
    """One small single-kernel workload for an ncu capture (inputs > L2)."""
    import numpy as np
    import torch

    from prng_seeded_decompress_b200 import build, inputs
    build.build()
    from prng_seeded_decompress_b200 import seedlm as sl
    sl.init()
    if name == "decompress":
        L = inputs.make_layer(8192, 28672, 8, 3, seed=1)
        rec = torch.from_numpy(L["rec"].view(np.int32)).cuda()
        W = torch.empty((8192, 28672), device="cuda")
        for _ in range(3):
            sl.decompress(L["fmt"], rec, None, W)
    elif name in ("gemm64", "gemm16"):
        M = 64 if name == "gemm64" else 16
        L = inputs.make_layer(28672, 8192, 8, 3, seed=2)
        rec = torch.from_numpy(L["rec"].view(np.int32)).cuda()
        Xb, _ = inputs.make_activations((M, 8192), "bf16", 3)
        X = torch.from_numpy(Xb.view(np.int16)).cuda().view(torch.bfloat16)
        Y = torch.empty((M, 28672), device="cuda")
        ws = sl.gemm_workspace(L["fmt"], M)
        for _ in range(3):
            sl.gemm_smallM(L["fmt"], rec, None, X, Y, workspace=ws)
    elif name == "gemm3x2":
        # 2 rows of X at 3 bits (the CUDA-core kernel), 28672 x 8192, three
        # calls (capture with -s 1 -c 1).
        L = inputs.make_layer(28672, 8192, 12, 4, seed=4)
        rec = torch.from_numpy(L["rec"].view(np.int32)).cuda()
        ep = torch.from_numpy(L["eplane"]).cuda()
        Xb, _ = inputs.make_activations((2, 8192), "bf16", 5)
        X = torch.from_numpy(Xb.view(np.int16)).cuda().view(torch.bfloat16)
        Y = torch.empty((2, 28672), device="cuda")
        for _ in range(3):
            sl.gemm_smallM(L["fmt"], rec, ep, X, Y)
    elif name in ("gemv", "gemv-cycle"):
        # The four GEMVs of one 4-bit Llama-3-70B layer, twice (the first
        # round warms up; capture with -s 4 -c 4).  "gemv-cycle" stores each
        # seed's position in the register's cycle instead of the seed, the
        # record form of a library built with SEEDLM_GEMV_LFSR=2 (the
        # full-cycle window table; for the LFSR variant comparison only).
        pos = None
        if name == "gemv-cycle":
            pos = np.zeros(65536, np.uint32)
            st = 1
            for p in range(65535):
                pos[st] = p
                st = (st >> 1) | (((st ^ (st >> 2) ^ (st >> 3) ^ (st >> 5)) & 1) << 15)
        lay = []
        for i, (_, R, N) in enumerate(LAYER_70B):
            L = inputs.make_layer(R, N, 8, 3, seed=10 + i)
            rec = L["rec"]
            if pos is not None:
                rec = ((pos[rec >> 16] << 16) | (rec & 0xffff)).astype(np.uint32)
            xb, _ = inputs.make_activations((N,), "f16", 20 + i)
            lay.append((L["fmt"], torch.from_numpy(rec.view(np.int32)).cuda(),
                        torch.from_numpy(xb.view(np.int16)).cuda().view(torch.float16),
                        torch.empty(R, device="cuda")))
        flush_l2(torch)
        for _ in range(2):
            for f, rec, x, y in lay:
                sl.gemv(f, rec, None, x, y)
    elif name == "gemv3":
        # The four GEMVs of one 3-bit Llama-3-8B layer, twice (capture with
        # -s 4 -c 4; the third launch is gate+up, 28672 x 4096).
        lay = []
        for i, (_, R, N) in enumerate(LAYER_8B):
            L = inputs.make_layer(R, N, 12, 4, seed=30 + i)
            xb, _ = inputs.make_activations((N,), "f16", 40 + i)
            lay.append((L["fmt"], torch.from_numpy(L["rec"].view(np.int32)).cuda(),
                        torch.from_numpy(L["eplane"]).cuda(),
                        torch.from_numpy(xb.view(np.int16)).cuda().view(torch.float16),
                        torch.empty(R, device="cuda")))
        flush_l2(torch)
        for _ in range(2):
            for f, rec, ep, x, y in lay:
                sl.gemv(f, rec, ep, x, y)
    elif name == "encode":
        # Full seed / coefficient / exponent search of a Gaussian 2048 x 2048
        # matrix at 4 bits (524,288 blocks), twice.
        rng = np.random.default_rng(11)
        We = torch.from_numpy((rng.standard_normal((2048, 2048)) * 0.02).astype(np.float32)).cuda()
        fe = inputs.make_format(2048, 2048, 8, 3)
        rec_e = torch.empty((2048, fe["rec_pitch"]), dtype=torch.int32, device="cuda")
        for _ in range(2):
            sl.encode(fe, We, rec_e)
    elif name in ("adapters", "adapters-prefill"):
        # Low-rank adapters on the 70B layer's fused gate+up: 64 rows with an
        # adapter each, or 1024 rows of eight adapters, rank 64, three calls.
        M, n = (64, 64) if name == "adapters" else (1024, 8)
        A = [torch.randn((n, 64, 8192), device="cuda").bfloat16() * 8192 ** -0.5 for _ in range(2)]
        B = [torch.randn((n, 28672, 64), device="cuda").bfloat16() * 0.1 for _ in range(2)]
        ad = sl.Adapters(A, B)
        ids = torch.arange(M, dtype=torch.int32, device="cuda") % n
        plan = sl.adapter_plan(ids, n)
        X = torch.randn((M, 8192), device="cuda").bfloat16()
        Y = torch.zeros((M, 57344), device="cuda")
        ws = sl.adapter_workspace(ad, M)
        for _ in range(3):
            sl.adapter_apply(ad, plan, X, Y, workspace=ws)
    elif name == "norm":
        # Residual sum and both norms of 4096 rows of 8192, three calls.
        w = torch.ones(8192, dtype=torch.bfloat16, device="cuda")
        nm = sl.BlockNorm(8192, w_post=w, w_pre=w)
        y = torch.randn((4096, 8192), device="cuda")
        h = torch.randn((4096, 8192), device="cuda").bfloat16()
        x, h_out = torch.empty_like(h), torch.empty_like(h)
        for _ in range(3):
            sl.block_norm(nm, y, h, h_out=h_out, x=x)
    elif name == "glu":
        GU = torch.randn((2048, 2 * 14336), device="cuda")
        X = torch.empty((2048, 14336), dtype=torch.bfloat16, device="cuda")
        for _ in range(3):
            sl.glu(GU, X)
    elif name == "dense":
        W = torch.randn((57344, 8192), device="cuda").half()
        x = torch.randn(8192, device="cuda").half()
        y = torch.empty(57344, device="cuda")
        for _ in range(3):
            sl.dense_gemv_f16(W, x, y)
    torch.cuda.synchronize()
    if sl.device_error():
        raise SystemExit("device error flag raised")
    print(f"case {name} ok", flush=True)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=2000)
    ap.add_argument("--warmup", type=int, default=20)
    ap.add_argument("--impl", choices=("seedlm", "reference"), default="seedlm")
    ap.add_argument("--layers", type=int, default=80, help="distinct layer copies resident")
    ap.add_argument("--no-extras", action="store_true")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--cpu-seconds", type=float, default=12.0)
    ap.add_argument("--ref-step-seconds", type=float, default=1.0)
    ap.add_argument("--case", choices=("gemv", "gemv3", "gemv-cycle", "decompress", "gemm64", "gemm3x2",
                                       "gemm16", "dense", "encode", "adapters", "adapters-prefill",
                                       "norm", "glu"),
                    help="run one small single-kernel workload (for ncu) and exit")
    args = ap.parse_args()
    if args.case:
        profile_case(args.case)
        return
    if args.warmup < 3:
        ap.error("--warmup must be at least 3")
    if args.impl == "reference":
        reference_arm(args)
    else:
        seedlm_arm(args)


if __name__ == "__main__":
    main()
