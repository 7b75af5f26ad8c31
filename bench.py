#!/usr/bin/env python
"""Benchmark of the groupwise int4/int5 small-batch projection on GB300.

Metric: µs/call and achieved HBM GB/s (fraction of the measured HBM roofline) for Q4/Q5
skinny GEMM at T=1..8. Algorithmic bytes per call = packed codes + fp16 scales + X + Y,
each read or written once.

Default workload (the headline line): decode GEMV Q4, T=1, K=5120, N=17408 (a 27B-class FFN
up-projection). One step = one projection call on one of R packed weight copies; the copies
rotate so that R * bytes > 3 x L2 and every step streams its weights from HBM. The K timed
steps are replayed as one CUDA graph of K back-to-back launches (how a decode engine issues
them), bracketed by CUDA events on the launching stream.

  python bench.py [--gpus N] [--steps K] [--warmup W] [--impl ours|reference]
                  [--workload decode_q4|verify_q5|swiglu_block|swiglu_block_q5|swiglu_block_fp4|layer_stack] [--T T]
                  [--no-sweep] [--no-cpu-baseline]

--impl reference times the CPU oracle (the deliberately slow fp64 definition) on the host
cores instead, on the same workload, metric and unit.
"""
from __future__ import annotations

import argparse
import hashlib
import json
import os
import statistics
import subprocess
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

L2_BYTES = 129 * 1000 * 1000
FALLBACK_HBM_GBS = 6800.0
METRIC = "µs/call and achieved HBM GB/s (% of roofline) for Q4/Q5 skinny GEMM, T=1..8"
MAX_T = 64
# What decides a projection's DRAM traffic: its kernels, their work split, the tensor maps and the choice of
# kernel, grid and cluster on the host. All sources but those of the serving step's own kernels.
STEP_SOURCES = {"nq_attn.cu", "nq_attn.cuh", "nq_pages.cu", "nq_sample.cu", "nq_step.h"}
KERNEL_SOURCES = sorted(f for f in os.listdir(os.path.join(ROOT, "weight_only_groupwise_gb300", "csrc"))
                        if f.endswith((".cu", ".cuh", ".h")) and f not in STEP_SOURCES)


# ---------------------------------------------------------------- ranks

def max_over_ranks(x: float, device=None) -> float:
    """The largest x over all ranks of the default process group (the slowest rank's time);
    x itself when no group is running or it has one rank."""
    import torch
    import torch.distributed as dist
    if not (dist.is_available() and dist.is_initialized()) or dist.get_world_size() == 1:
        return x
    t = torch.tensor([x], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def job_rate_gbs(bytes_per_step_per_rank: int, ms_per_step: float, world: int) -> float:
    """Whole-job GB/s: the bytes all ranks processed per step over the slowest rank's step."""
    return bytes_per_step_per_rank * world / (ms_per_step * 1e-3) / 1e9


# ---------------------------------------------------------------- workloads

FP4 = 14  # format tag of NVFP4 weights in the library's calls


def weight_bytes(bits: int, K: int, N: int) -> int:
    """Packed codes + packed scales of one K x N matrix: Q4 / Q5 codes with an fp16 scale per
    64 along K; NVFP4 e2m1 codes (K*N/2) with an e4m3 scale per 16 (N*K/16)."""
    if bits == FP4:
        return K * N // 2 + N * K // 16
    return K * N * bits // 8 + N * (K // 64) * 2


def proj_bytes(bits: int, T: int, K: int, N: int) -> int:
    return weight_bytes(bits, K, N) + T * K * 2 + T * N * 2


def fp4_bytes(T: int, K: int, N: int) -> int:
    """NVFP4: e2m1 codes (K*N/2) + e4m3 block scales (N*K/16) + X + Y."""
    return proj_bytes(FP4, T, K, N)


def swiglu_bytes(T: int, K: int, N: int, bits: int = 4) -> int:
    return 2 * weight_bytes(bits, K, N) + T * K * 2 + T * N * 2


WORKLOADS = {
    "decode_q4": dict(kind="proj", bits=4, T=1, K=5120, N=17408,
                      desc="decode GEMV Q4, T=1, K=5120, N=17408 (27B-class FFN up-projection)"),
    "verify_q5": dict(kind="proj", bits=5, T=8, K=5120, N=6144,
                      desc="spec-verify Q5, T=8, K=5120, N=6144 (attention gate/value projection)"),
    "decode_fp4": dict(kind="proj", bits=FP4, T=1, K=5120, N=17408,
                       desc="decode GEMV NVFP4, T=1, K=5120, N=17408 (e2m1 codes, an e4m3 scale per 16, "
                            "an fp32 tensor scale)"),
    "swiglu_block": dict(kind="swiglu", bits=4, T=8, K=5120, N=17408, Kd=17408, Nd=5120,
                         desc="SwiGLU block Q4, T=8: fused gate+up K=5120 N=17408, then down K=17408 N=5120"),
    "swiglu_block_q5": dict(kind="swiglu", bits=5, T=8, K=5120, N=17408, Kd=17408, Nd=5120,
                            desc="SwiGLU block Q5, T=8: fused gate+up K=5120 N=17408, then down K=17408 N=5120"),
    "swiglu_block_fp4": dict(kind="swiglu", bits=FP4, T=8, K=5120, N=17408, Kd=17408, Nd=5120,
                             desc="SwiGLU block NVFP4, T=8: fused gate+up K=5120 N=17408, then down K=17408 N=5120"),
    "layer_stack": dict(kind="stack", T=8, layers=64,
                        desc="64 independent 27B-class layers: fused gate+up and down (Q4), "
                             "q-gate 5120x6144, kv 5120x1024, out 6144x5120 (Q5)"),
}


# The pages' own single-op numbers for this path ("NInfer-4090" release post, section "实测数据"):
# another GPU (an RTX 4090 fork) and shapes the pages do not state, so context for the line,
# not a baseline (vs_baseline stays null).
PAGES_CONTEXT = {
    "source": "\"NInfer-4090\" release post, section 实测数据",
    "hardware": "RTX 4090 (sm_89 fork)",
    "t8_attention_q5_gate_value_us": {"before": 57.344, "after": 39.936},
    "t8_gdn_qk_q4_us": {"before": 35.840, "after": 31.744},
    "note": "shapes not stated on the pages; this GPU's calls are judged against its HBM roofline",
}


def workload_bytes(w: dict) -> int:
    if w["kind"] == "proj":
        return proj_bytes(w["bits"], w["T"], w["K"], w["N"])
    if w["kind"] == "swiglu":
        return (swiglu_bytes(w["T"], w["K"], w["N"], w["bits"])
                + proj_bytes(w["bits"], w["T"], w["Kd"], w["Nd"]))
    T = w["T"]
    per_layer = (swiglu_bytes(T, 5120, 17408, 4) + proj_bytes(4, T, 17408, 5120) + proj_bytes(5, T, 5120, 6144)
                 + proj_bytes(5, T, 5120, 1024) + proj_bytes(5, T, 6144, 5120))
    return per_layer * w["layers"]


def launches_per_step(w: dict) -> int:
    """Kernel launches per step. T <= 8: one per call (the stack's q-gate and kv share one).
    8 < T <= 64: one per projection on the tensor-core kernel, two for a fused SwiGLU call
    (gate, then up) and two for the stack's grouped q-gate/kv call (one per matrix)."""
    T = w.get("T", 1)
    big = T > 8
    swiglu = 2 if big else 1
    grouped = 2 if big else 1
    if w["kind"] == "proj":
        return 1
    if w["kind"] == "swiglu":
        return swiglu + 1
    return (swiglu + 1 + grouped + 1) * w.get("layers", 1)


# ---------------------------------------------------------------- environment helpers

def measured_peak():
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        with open(p) as f:
            d = json.load(f)
        return float(d["hbm_gbs"]), "measured"
    except Exception:
        return FALLBACK_HBM_GBS, "fallback"


def kernel_hash() -> str:
    """Hash of the kernel sources with comments and blank space removed, so that an edit of
    comments alone keeps the committed ncu traffic record valid."""
    import re
    h = hashlib.sha256()
    for f in KERNEL_SOURCES:
        with open(os.path.join(ROOT, "weight_only_groupwise_gb300", "csrc", f), encoding="utf-8") as fh:
            src = fh.read()
        src = re.sub(r"/\*.*?\*/", " ", src, flags=re.S)
        src = re.sub(r"//[^\n]*", " ", src)
        h.update(" ".join(src.split()).encode())
    return h.hexdigest()[:16]


def ncu_traffic(workload: str, T: int):
    """DRAM bytes per launch of the dominant kernel of `workload` at T tokens (key
    "<workload>@T<T>") from the committed ncu summary, or None when the summary is absent or
    was taken on different kernel sources."""
    p = os.path.join(ROOT, "profiles", "traffic.json")
    try:
        with open(p) as f:
            d = json.load(f)
        e = d[f"{workload}@T{T}"]
        if e.get("kernel_hash") != kernel_hash():
            return None
        return int(e["dram_bytes_per_launch"])
    except Exception:
        return None


class ClockSampler:
    """nvidia-smi sampling of SM clock, power and throttle reasons while the GPU works."""
    FIELDS = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, gpu_index: int):
        self.gpu = gpu_index
        self.proc = None
        self.out = None

    def __enter__(self):
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", "-i", str(self.gpu), f"--query-gpu={self.FIELDS}",
                 "--format=csv,noheader,nounits", "-lms", "100"],
                stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
        except Exception:
            self.proc = None
        return self

    def __exit__(self, *a):
        if self.proc is not None:
            self.proc.terminate()
            try:
                self.out, _ = self.proc.communicate(timeout=5)
            except Exception:
                self.proc.kill()
                self.out = ""

    def summary(self) -> dict:
        if not self.out:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["clock sampling unavailable"]}
        sm, mx, reasons = [], [], set()
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for line in self.out.strip().splitlines():
            f = [x.strip() for x in line.split(",")]
            if len(f) < 9:
                continue
            try:
                sm.append(float(f[1]))
                mx.append(float(f[2]))
            except ValueError:
                continue
            for n, v in zip(names, f[5:9]):
                if v.lower().startswith("active"):
                    reasons.add(n)
        if not sm:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["no samples"]}
        return {"sm_mhz": statistics.median(sm), "sm_max_mhz": max(mx), "samples": len(sm),
                "reasons": sorted(reasons)}


# ---------------------------------------------------------------- device setup

def make_proj_copies(nq, bits, K, N, copies, seed, dev):
    import torch
    import seeded_inputs as si
    gen = torch.Generator(device=dev)
    out = []
    for r in range(copies):
        gen.manual_seed(seed * 1000 + r)
        wn = si.device_code_words(N, K // 8, gen, dev)
        if bits == 5:
            wh = si.device_code_words(N, K // 32, gen, dev)
        s = si.device_scales(N, K, gen, dev)
        if bits == 4:
            out.append(nq.pack_q4(wn, s, K, N))
        else:
            out.append(nq.pack_q5(wn, wh, s, K, N))
        del wn, s
    torch.cuda.synchronize()
    return out


def make_fp4_copies(nq, K, N, copies, seed, dev):
    import torch
    import seeded_inputs as si
    gen = torch.Generator(device=dev)
    out = []
    for r in range(copies):
        gen.manual_seed(seed * 1000 + r)
        codes = si.device_code_words(N, K // 8, gen, dev)
        sf = si.device_fp4_scales(N, K, gen, dev)
        out.append(nq.pack_fp4(codes, sf, K, N))
        del codes, sf
    torch.cuda.synchronize()
    return out


def proj_copies_and_call(nq, bits: int, K: int, N: int, R: int, dev, seed=None):
    """R packed weight copies of one K x N matrix and the library call fn(x, w, s, N, out=y)
    that projects through one of them (NVFP4: with the seeded inputs' tensor scale)."""
    import seeded_inputs as si
    if bits == FP4:
        copies = make_fp4_copies(nq, K, N, R, 9 if seed is None else seed, dev)

        def fn(x, wq, s, n, out, stream=None):
            nq.gemm_fp4(x, wq, s, si.FP4_GLOBAL_SCALE, n, out=out, stream=stream)
        return copies, fn
    copies = make_proj_copies(nq, bits, K, N, R, (1 if bits == 4 else 2) if seed is None else seed, dev)
    return copies, (nq.gemm_q4 if bits == 4 else nq.gemm_q5)


def build_step(nq, w: dict, dev, T_override=None):
    """Returns (step(i) -> None launching one step, bytes_per_step, copies, note)."""
    import torch
    import seeded_inputs as si
    gen = torch.Generator(device=dev)
    gen.manual_seed(12345)
    if w["kind"] == "proj":
        bits, T, K, N = w["bits"], T_override or w["T"], w["K"], w["N"]
        b = proj_bytes(bits, T, K, N)
        R = max(2, -(-3 * L2_BYTES // b))
        copies, fn = proj_copies_and_call(nq, bits, K, N, R, dev)
        x = si.device_activations(T, K, gen, dev)
        y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)

        def step(i):
            fn(x, *copies[i % R], N, out=y)
        return step, b, R, f"rotate {R} packed weight copies ({R * b / 1e6:.0f} MB > 3x L2)", (x, y)
    if w["kind"] == "swiglu":
        bits, T, K, N, Kd, Nd = w["bits"], T_override or w["T"], w["K"], w["N"], w["Kd"], w["Nd"]
        b = swiglu_bytes(T, K, N, bits) + proj_bytes(bits, T, Kd, Nd)
        R = max(2, -(-3 * L2_BYTES // b))
        if bits == FP4:
            gate = make_fp4_copies(nq, K, N, R, 33, dev)
            up = make_fp4_copies(nq, K, N, R, 34, dev)
            down = make_fp4_copies(nq, Kd, Nd, R, 35, dev)
            gsc = si.FP4_GLOBAL_SCALE

            def fused(x, wg, sg, wu, su, n, out):
                nq.swiglu_fp4(x, wg, sg, gsc, wu, su, gsc, n, out=out)

            def fn(x, wd, sd, n, out):
                nq.gemm_fp4(x, wd, sd, gsc, n, out=out)
        else:
            gate = make_proj_copies(nq, bits, K, N, R, 3 + 10 * (bits - 4), dev)
            up = make_proj_copies(nq, bits, K, N, R, 4 + 10 * (bits - 4), dev)
            down = make_proj_copies(nq, bits, Kd, Nd, R, 5 + 10 * (bits - 4), dev)
            fused = nq.swiglu_q4 if bits == 4 else nq.swiglu_q5
            fn = nq.gemm_q4 if bits == 4 else nq.gemm_q5
        x = si.device_activations(T, K, gen, dev)
        h = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        y = torch.empty((T, Nd), dtype=torch.bfloat16, device=dev)

        def step(i):
            j = i % R
            fused(x, *gate[j], *up[j], N, out=h)
            fn(h, *down[j], Nd, out=y)
        return step, b, R, f"rotate {R} weight sets ({R * b / 1e6:.0f} MB > 3x L2)", (x, y)
    # layer stack: 64 independent layers, ~12 GB of packed weights (no reuse within a pass)
    T = T_override or w["T"]
    layers = build_layers(nq, w["layers"], dev)
    step, keep = stack_step(nq, layers, T, dev, grouped=True)
    w2 = dict(w, T=T)
    return step, workload_bytes(w2), 1, "64 distinct layers (~12 GB) per pass, no reuse", (keep, layers)


def build_layers(nq, L: int, dev):
    import seeded_inputs as si
    layers = []
    for l in range(L):
        layers.append(dict(
            gate=make_proj_copies(nq, 4, 5120, 17408, 1, si.layer_seed(l, 0), dev)[0],
            up=make_proj_copies(nq, 4, 5120, 17408, 1, si.layer_seed(l, 1), dev)[0],
            down=make_proj_copies(nq, 4, 17408, 5120, 1, si.layer_seed(l, 2), dev)[0],
            qg=make_proj_copies(nq, 5, 5120, 6144, 1, si.layer_seed(l, 3), dev)[0],
            kv=make_proj_copies(nq, 5, 5120, 1024, 1, si.layer_seed(l, 4), dev)[0],
            out=make_proj_copies(nq, 5, 6144, 5120, 1, si.layer_seed(l, 5), dev)[0]))
    return layers


def stack_step(nq, layers, T: int, dev, grouped: bool):
    """One pass over the layers: fused gate/up + down (Q4); q-gate and kv (Q5, the same X) as
    one grouped launch or two calls; out (Q5)."""
    import torch
    import seeded_inputs as si
    gen = torch.Generator(device=dev)
    gen.manual_seed(12345)
    x = si.device_activations(T, 5120, gen, dev)
    x6 = si.device_activations(T, 6144, gen, dev)
    h = torch.empty((T, 17408), dtype=torch.bfloat16, device=dev)
    yd = torch.empty((T, 5120), dtype=torch.bfloat16, device=dev)
    yq = torch.empty((T, 6144), dtype=torch.bfloat16, device=dev)
    ykv = torch.empty((T, 1024), dtype=torch.bfloat16, device=dev)
    yo = torch.empty((T, 5120), dtype=torch.bfloat16, device=dev)

    def step(i):
        for ly in layers:
            nq.swiglu_q4(x, *ly["gate"], *ly["up"], 17408, out=h)
            nq.gemm_q4(h, *ly["down"], 5120, out=yd)
            if grouped:
                nq.gemm_q5_grouped(x, [(*ly["qg"], 6144), (*ly["kv"], 1024)], outs=[yq, ykv])
            else:
                nq.gemm_q5(x, *ly["qg"], 6144, out=yq)
                nq.gemm_q5(x, *ly["kv"], 1024, out=ykv)
            nq.gemm_q5(x6, *ly["out"], 5120, out=yo)
    return step, (x, x6, h, yd, yq, ykv, yo)


def stack_program(nq, layers, T: int, dev):
    """The calls of stack_step (grouped) recorded once into a library program (nq_program_*),
    replayed by one graph launch per pass."""
    import torch
    import seeded_inputs as si
    gen = torch.Generator(device=dev)
    gen.manual_seed(12345)
    x = si.device_activations(T, 5120, gen, dev)
    x6 = si.device_activations(T, 6144, gen, dev)
    h = torch.empty((T, 17408), dtype=torch.bfloat16, device=dev)
    yd = torch.empty((T, 5120), dtype=torch.bfloat16, device=dev)
    yq = torch.empty((T, 6144), dtype=torch.bfloat16, device=dev)
    ykv = torch.empty((T, 1024), dtype=torch.bfloat16, device=dev)
    yo = torch.empty((T, 5120), dtype=torch.bfloat16, device=dev)
    prog = nq.Program()
    for ly in layers:
        prog.swiglu_q4(x, *ly["gate"], *ly["up"], 17408, out=h)
        prog.gemm_q4(h, *ly["down"], 5120, out=yd)
        prog.grouped_q5(x, [(*ly["qg"], 6144), (*ly["kv"], 1024)], outs=[yq, ykv])
        prog.gemm_q5(x6, *ly["out"], 5120, out=yo)
    prog.build()
    return prog


def time_launches(launch, steps: int, warmup: int, stream, reps: int = 5):
    """`warmup` untimed calls of launch(), then `reps` timed runs of `steps` calls, each
    bracketed by CUDA events on `stream`. Returns the run times in milliseconds."""
    import torch
    with torch.cuda.stream(stream):
        for _ in range(warmup):
            launch()
    torch.cuda.synchronize()
    out = []
    for _ in range(reps):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        with torch.cuda.stream(stream):
            e0.record(stream)
            for _ in range(steps):
                launch()
            e1.record(stream)
        torch.cuda.synchronize()
        out.append(e0.elapsed_time(e1))
    return out


def time_graph(step, steps: int, warmup: int, stream, soak_s: float = 0.0, reps: int = 5):
    """Eager warm-up, capture `steps` steps into one CUDA graph, replay it untimed (and for
    `soak_s` seconds), then time `reps` replays, each bracketed by CUDA events on the
    launching stream. Returns the list of replay times in milliseconds."""
    import torch
    with torch.cuda.stream(stream):
        for i in range(warmup):
            step(i)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        for i in range(steps):
            step(i)
    g.replay()
    torch.cuda.synchronize()
    t_end = time.time() + soak_s
    while time.time() < t_end:
        g.replay()
        torch.cuda.synchronize()
    out = []
    for _ in range(reps):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        with torch.cuda.stream(stream):
            start.record(stream)
            g.replay()
            end.record(stream)
        torch.cuda.synchronize()
        out.append(start.elapsed_time(end))
    del g
    return out


def time_e2e(nq, w: dict, steps: int, warmup: int, stream, dev):
    """End to end through the public call: every step copies its X from pinned host memory,
    runs the projection and reads its Y back to pinned host memory. The copies go on two copy
    streams (host->device, device->host) and overlap the kernels, as a serving loop would
    pipeline them: X is copied up to eight steps ahead into a ring of twelve device buffers,
    and each step's Y is read back while the next steps' kernels run. A kernel that waits on
    another stream loses its early (programmatic) start behind the preceding kernel, so the
    waits are batched: the kernel of every fourth step waits once, for the X copies of its
    four steps and for the reads of the Y buffers they reuse. The K steps are captured in one
    CUDA graph (copies included) like the device-timed value; each timed replay starts before
    the first step's copy and ends when the last step's Y has reached the host. Median of 5
    replays."""
    import torch
    import seeded_inputs as si
    bits, T, K, N = w["bits"], w["T"], w["K"], w["N"]
    b = proj_bytes(bits, T, K, N)
    R = max(2, -(-3 * L2_BYTES // b))
    copies, fn = proj_copies_and_call(nq, bits, K, N, R, dev, seed=7)
    gen = torch.Generator(device="cpu")
    gen.manual_seed(99)
    B, NR = 4, 12                                     # steps per wait, device ring buffers
    xs = [torch.randn((T, K), generator=gen).to(torch.bfloat16).pin_memory() for _ in range(4)]
    ys = [torch.empty((T, N), dtype=torch.bfloat16).pin_memory() for _ in range(4)]
    xd = [torch.empty((T, K), dtype=torch.bfloat16, device=dev) for _ in range(NR)]
    yd = [torch.empty((T, N), dtype=torch.bfloat16, device=dev) for _ in range(NR)]
    h2d, d2h = torch.cuda.Stream(device=dev), torch.cuda.Stream(device=dev)

    def steps_on_streams(n):
        """n steps; events order every reuse of the ring buffers."""
        fork = torch.cuda.Event()
        fork.record(stream)
        h2d.wait_event(fork)
        d2h.wait_event(fork)
        ev_k, ev_x, ev_y = {}, {}, {}

        def copy_x(i):
            if i >= NR:
                h2d.wait_event(ev_k[i - NR])           # kernel i-NR has read xd[i % NR]
            with torch.cuda.stream(h2d):
                xd[i % NR].copy_(xs[i % 4], non_blocking=True)
                ev_x[i] = torch.cuda.Event()
                ev_x[i].record(h2d)

        for i in range(min(B, n)):
            copy_x(i)
        for i in range(n):
            if i % B == 0:
                stream.wait_event(ev_x[min(i + B, n) - 1])   # X of steps i .. i+B-1 landed
                if i + B - 1 >= NR:
                    stream.wait_event(ev_y[i + B - 1 - NR])  # their Y buffers were read back
                for j in range(i + B, min(i + 2 * B, n)):
                    copy_x(j)
            fn(xd[i % NR], *copies[i % R], N, out=yd[i % NR], stream=stream)
            ev_k[i] = torch.cuda.Event()
            ev_k[i].record(stream)
            d2h.wait_event(ev_k[i])
            with torch.cuda.stream(d2h):
                ys[i % 4].copy_(yd[i % NR], non_blocking=True)
                ev_y[i] = torch.cuda.Event()
                ev_y[i].record(d2h)
        stream.wait_stream(h2d)
        stream.wait_stream(d2h)

    with torch.cuda.stream(stream):
        steps_on_streams(warmup)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        steps_on_streams(steps)
    g.replay()
    torch.cuda.synchronize()
    times = []
    for _ in range(5):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        with torch.cuda.stream(stream):
            start.record(stream)
            g.replay()
            end.record(stream)
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end))
    ms = statistics.median(times)
    return ms, b, T * K * 2, T * N * 2


# ---------------------------------------------------------------- CPU oracle timing

def oracle_sample(w: dict, budget_s: float):
    """Time the CPU oracle on a bounded sample of the workload. Returns
    (GB/s over the sample's algorithmic bytes, µs per full-workload call, threads, description)."""
    import numpy as np
    import oracle
    import seeded_inputs as si
    if w["kind"] != "proj":
        w = dict(kind="proj", bits=w.get("bits", 4), T=w.get("T", 8), K=5120, N=17408)
    bits, T, K, N = w["bits"], w["T"], w["K"], w["N"]
    if bits == FP4:
        p = si.fp4_problem(T, K, N, 3)

        def run(rows):
            oracle.gemm_fp4_rows(p["x"], p["codes"], p["sf"], p["g"], T, K, rows)
    elif bits == 4:
        p = si.q4_problem(T, K, N, 1)

        def run(rows):
            oracle.gemm_q4_rows(p["x"], p["wq"], p["s"], T, K, rows)
    else:
        p = si.q5_problem(T, K, N, 2)

        def run(rows):
            oracle.gemm_q5_rows(p["x"], p["wn"], p["wh"], p["s"], T, K, rows)
    rows_all = np.arange(N, dtype=np.int32)
    # first: one pass over a 1/16 row sample to size the run
    n0 = max(16, N // 16)
    t0 = time.perf_counter()
    run(rows_all[:n0])
    t_row = (time.perf_counter() - t0) / n0
    rows = int(min(N, max(n0, budget_s / max(t_row, 1e-12))))
    # the whole problem fits the budget: repeat full passes until the budget is used
    reps = max(1, int(budget_s / max(t_row * N, 1e-9))) if rows == N else 1
    t0 = time.perf_counter()
    for _ in range(reps):
        run(rows_all[:rows])
    dt = (time.perf_counter() - t0) / reps
    frac = rows / N
    sample_bytes = proj_bytes(bits, T, K, N) * frac
    gbs = sample_bytes / dt / 1e9
    us_full = dt / frac * 1e6
    fmt = "NVFP4" if bits == FP4 else f"{bits}-bit"
    desc = (f"CPU fp64 oracle on {rows}/{N} output rows of the {fmt} T={T} K={K} N={N} "
            f"projection, {reps} pass(es) of {dt:.2f} s, bytes scaled by the row fraction")
    return gbs, us_full, oracle.num_threads(), desc, (rows, dt)


# ---------------------------------------------------------------- main

def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--warmup", type=int, default=10)
    ap.add_argument("--impl", default="ours", choices=["ours", "reference"])
    ap.add_argument("--workload", default="decode_q4", choices=list(WORKLOADS))
    ap.add_argument("--T", type=int, default=0, help="override the workload's T")
    ap.add_argument("--no-sweep", action="store_true")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-e2e", action="store_true")
    ap.add_argument("--cpu-budget", type=float, default=10.0, help="seconds of CPU oracle work")
    ap.add_argument("--soak", type=float, default=1.0,
                    help="seconds of untimed graph replays before the timed ones (clock sampling)")
    ap.add_argument("--reps", type=int, default=5, help="timed replays of the K-step graph (median reported)")
    args = ap.parse_args()
    warmup = max(3, args.warmup)

    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    local_rank = int(os.environ.get("LOCAL_RANK", "0"))
    w = dict(WORKLOADS[args.workload])
    if args.T:
        w["T"] = args.T

    if args.impl == "reference":
        if rank != 0:
            return
        # the deliberately slow fp64 definition on the host cores; one step = one bounded sample
        per_step = max(0.5, min(5.0, 120.0 / max(1, args.steps + warmup)))
        for _ in range(warmup):
            oracle_sample(w, per_step)
        vals, times = [], []
        for _ in range(args.steps):
            gbs, us_full, cores, desc, (rows, dt) = oracle_sample(w, per_step)
            vals.append(gbs)
            times.append(dt)
        v = statistics.mean(vals)
        print(json.dumps({
            "impl": "reference", "metric": METRIC, "value": round(v, 4), "unit": "GB/s", "n_gpus": 1,
            "steps": args.steps, "warmup": warmup, "ms_per_step": round(1e3 * statistics.mean(times), 3),
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64",
            "data": "synthetic",
            "config": {"workload": w["desc"], "bits": w.get("bits", 4), "T": w["T"]},
            "cpu_baseline": {"value": round(v, 4), "unit": "GB/s", "cores": cores, "kind": "oracle",
                             "sample": desc},
            "e2e": {"value": round(v, 4), "unit": "GB/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
        }))
        return

    import torch
    if world > 1:
        import torch.distributed as dist
        dist.init_process_group("nccl")
    torch.cuda.set_device(local_rank)
    dev = torch.device("cuda", local_rank)
    from weight_only_groupwise_gb300 import build as nqbuild
    nqbuild.build()
    from weight_only_groupwise_gb300 import nq
    nq.reserve(8, 17408, 17408)
    stream = torch.cuda.Stream(device=dev)
    peak, peak_kind = measured_peak()

    step, bytes_step, R, l2_note, _keep = build_step(nq, w, dev)
    if world > 1:
        torch.distributed.barrier()
    torch.cuda.synchronize()
    with ClockSampler(local_rank) as clk:
        reps = time_graph(step, args.steps, warmup, stream, soak_s=args.soak, reps=args.reps)
    ms = max_over_ranks(statistics.median(reps), dev)
    nq.device_error()
    ms_step = ms / args.steps
    value = job_rate_gbs(bytes_step, ms_step, world)
    launches = launches_per_step(w)
    # dominant kernel: the step's projection launches, one rank's bytes over its launch time
    achieved = job_rate_gbs(bytes_step, ms_step, 1)
    result = {
        "metric": METRIC, "value": round(value, 2), "unit": "GB/s", "n_gpus": world,
        "steps": args.steps, "warmup": warmup, "ms_per_step": round(ms_step, 6),
        "us_per_call": round(1e3 * ms_step / launches, 3),
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
        "data": "synthetic (seeded; codes uniform, scales fp16(0.01*exp(N(0,0.25))), X ~ N(0,1))",
        "config": {"workload": w["desc"], "bits": w.get("bits"), "T": w["T"], "K": w.get("K"),
                   "N": w.get("N"), "l2": l2_note, "launch": "CUDA graph of K back-to-back calls",
                   "parallelism": f"replicas x{world}" if world > 1 else "single GPU"},
        "roofline": {"bound": "hbm", "achieved": round(achieved, 1), "peak": peak, "unit": "GB/s",
                     "frac": round(achieved / peak, 4), "peak_kind": peak_kind,
                     "traffic": ncu_traffic(args.workload, w["T"])},
        "gpu_launches": launches * args.steps * args.reps,
        "spread": {"replays": args.reps, "statistic": "median",
                   "us_per_step_min": round(1e3 * min(reps) / args.steps, 3),
                   "us_per_step_median": round(1e3 * statistics.median(reps) / args.steps, 3),
                   "us_per_step_max": round(1e3 * max(reps) / args.steps, 3)},
        "clocks": clk.summary(),
        "pages_context": PAGES_CONTEXT,
    }
    if not args.no_e2e and w["kind"] == "proj":
        e_ms, b, h2d, d2h = time_e2e(nq, w, args.steps, warmup, stream, dev)
        e_ms = max_over_ranks(e_ms, dev)
        result["e2e"] = {"value": round(job_rate_gbs(b, e_ms / args.steps, world), 2), "unit": "GB/s",
                         "us_per_call": round(1e3 * e_ms / args.steps, 3),
                         "h2d_bytes_per_step": h2d, "d2h_bytes_per_step": d2h,
                         "pipeline": "CUDA graph of K steps; each step's pinned host->device copy of X "
                                     "(up to 8 steps ahead) and device->host copy of Y on two copy "
                                     "streams, overlapping the kernels; one cross-stream wait per 4 "
                                     "kernels"}
    if not args.no_sweep and rank == 0:
        result["sweep"] = sweep(nq, dev, stream, peak)
    if rank == 0 and not args.no_cpu_baseline:
        gbs_c, us_c, cores, desc, _ = oracle_sample(w, args.cpu_budget)
        result["cpu_baseline"] = {"value": round(gbs_c, 4), "unit": "GB/s", "cores": cores, "kind": "oracle",
                                  "sample": desc, "us_per_call_full": round(us_c, 1)}
    if rank == 0:
        print(json.dumps(result))
    if world > 1:
        torch.distributed.destroy_process_group()


def sweep(nq, dev, stream, peak):
    """µs/call and GB/s of the other shapes (context, not the headline): the decode Q4 and
    verify Q5 projections at every T = 1..8 and at T = 16, 32, 64 (larger verify batches, on
    the tensor-core kernel) with one weight set per shape, reused across T; NVFP4 on the
    decode shape; the Q4 and Q5 SwiGLU blocks at T=8 and the Q4 block at T = 16 and 64; the
    64-layer stack at T = 1 and 8, grouped, ungrouped and as one recorded library program.
    Each entry is the median of 5 timed runs (graph replays, or program launches)."""
    import torch
    out = []

    def record(name, T, reps, steps, b, launches):
        us = 1e3 * statistics.median(reps) / steps
        gbs = b / (us * 1e-6) / 1e9
        out.append({"workload": name, "T": T, "us_per_step": round(us, 3),
                    "us_min": round(1e3 * min(reps) / steps, 3), "us_max": round(1e3 * max(reps) / steps, 3),
                    "calls_per_step": launches, "GB_s": round(gbs, 1), "frac": round(gbs / peak, 4)})

    import seeded_inputs as si
    gen = torch.Generator(device=dev)
    gen.manual_seed(777)
    for name in ("decode_q4", "verify_q5"):
        w = WORKLOADS[name]
        bits, K, N = w["bits"], w["K"], w["N"]
        R = max(2, -(-3 * L2_BYTES // proj_bytes(bits, 8, K, N)))
        copies = make_proj_copies(nq, bits, K, N, R, 1 if bits == 4 else 2, dev)
        fn = nq.gemm_q4 if bits == 4 else nq.gemm_q5
        for T in list(range(1, 9)) + [16, 32, 64]:
            x = si.device_activations(T, K, gen, dev)
            y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)

            def step(i, x=x, y=y):
                fn(x, *copies[i % R], N, out=y)
            steps = 100
            record(name, T, time_graph(step, steps, 5, stream), steps, proj_bytes(bits, T, K, N), 1)
        del copies
        torch.cuda.empty_cache()
    # NVFP4 weights on the decode shape (the pages' NVFP4 MLP-projection A16 kernel)
    K, N = 5120, 17408
    R = max(2, -(-3 * L2_BYTES // fp4_bytes(8, K, N)))
    copies = make_fp4_copies(nq, K, N, R, 9, dev)
    for T in (1, 2, 4, 8, 16, 64):
        x = si.device_activations(T, K, gen, dev)
        y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)

        def step(i, x=x, y=y):
            nq.gemm_fp4(x, *copies[i % R], si.FP4_GLOBAL_SCALE, N, out=y)
        record("decode_fp4", T, time_graph(step, 100, 5, stream), 100, fp4_bytes(T, K, N), 1)
    del copies
    torch.cuda.empty_cache()
    for name, T in (("swiglu_block", 8), ("swiglu_block_q5", 8), ("swiglu_block", 16), ("swiglu_block", 64),
                    ("swiglu_block_fp4", 8), ("swiglu_block_fp4", 16)):
        w = dict(WORKLOADS[name], T=T)
        step, b, R, note, keep = build_step(nq, w, dev)
        steps = 100
        record(name, T, time_graph(step, steps, 5, stream), steps, b, launches_per_step(w))
        del step, keep
        torch.cuda.empty_cache()
    layers = build_layers(nq, WORKLOADS["layer_stack"]["layers"], dev)
    for T in (1, 8):
        w = dict(WORKLOADS["layer_stack"], T=T)
        for grouped in (True, False):
            step, keep = stack_step(nq, layers, T, dev, grouped)
            record("layer_stack" if grouped else "layer_stack_ungrouped", T, time_graph(step, 2, 1, stream), 2,
                   workload_bytes(w), launches_per_step(w) + (0 if grouped else w["layers"]))
            del step, keep
        # the same pass recorded once as a library program (one graph launch per pass)
        prog = stack_program(nq, layers, T, dev)
        kernels = prog.info()["kernels"]
        record("layer_stack_program", T, time_launches(lambda: prog.launch(stream), 2, 1, stream), 2,
               workload_bytes(w), kernels)
        prog.close()
        del prog
    del layers
    torch.cuda.empty_cache()
    return out


if __name__ == "__main__":
    main()
