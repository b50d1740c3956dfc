"""Benchmark: certified decode-attention tokens/s/layer at 128K context on one GB300.

One step = one certified decode step of every layer of the workload (each layer:
INT8 scoring + top-K* selection, mixed-precision pass with certificate and ladder plan,
second pass for rungs 1-2, dense rungs 3-4, certificate write-out), with the caches
already resident (tier 1 in HBM, tier 2 in pinned host memory).

  python bench.py [--gpus N] [--steps K] [--warmup W] [--impl ours|reference]

Prints one JSON line.  Under torchrun (N > 1) every rank runs an independent replica
(the path has no data exchange between sequences or heads) and rank 0 reports the
aggregate.  `--impl reference` times the CPU oracle on a bounded sample of the same
workload.
"""

from __future__ import annotations

import argparse
import json
import os
import statistics
import subprocess
import sys
import tempfile
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402

WORKLOAD = dict(name="c3_llama8b_ctx128k_32l", batch=1, ctx=131072, layers=32, q_heads=32,
                kv_heads=8, head_dim=128, tau_cov=0.995, eps=0.25, seed=2)
ROPE = dict(base=500000.0, scaling="parts", factor=8.0, original_ctx=8192, low=1.0, high=4.0)   # Llama-3.1-8B's
METRIC = "certified decode-attn tokens/s/layer at 128K ctx; HBM GB/s vs peak"
UNIT = "tokens/s/layer"
TIER1_BYTES_PER_TOKEN_HEAD = 212        # 128 K codes + 4 K scales + 64 V codes + 16 V scale/offset
SCORE_BYTES_PER_TOKEN_HEAD = 132        # K codes + K scales (scoring pass)
MIX_BYTES_PER_TOKEN_HEAD = 80           # V codes + V scale/offset (mixed pass, tail blocks)
F16_BLOCK = 16384
F16_BYTES_PER_TOKEN_HEAD = 512          # FP16 key + value of one token (tier-2 mirror)
APPEND_HBM_BYTES_PER_TOKEN_HEAD = 512 + 212   # FP16 K/V read + tier 1 written (quantiser)


def _peaks():
    try:
        with open(os.path.join(ROOT, "MEASURED_PEAKS.json")) as f:
            p = json.load(f)
        return float(p["hbm_gbs"]), "measured"
    except Exception:
        return 6800.0, "fallback"


class ClockSampler:
    """nvidia-smi clocks and throttle reasons sampled every 200 ms."""

    FIELDS = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, gpu_index: int):
        self.gpu = gpu_index
        self.proc = None
        self.path = None

    def __enter__(self):
        fd, self.path = tempfile.mkstemp(suffix=".csv")
        os.close(fd)
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", "-i", str(self.gpu), f"--query-gpu={self.FIELDS}", "--format=csv,noheader,nounits",
                 "-lms", "200"], stdout=open(self.path, "w"), stderr=subprocess.DEVNULL)
        except Exception:
            self.proc = None
        time.sleep(0.3)
        return self

    def __exit__(self, *a):
        if self.proc is not None:
            self.proc.terminate()
            try:
                self.proc.wait(timeout=5)
            except Exception:
                self.proc.kill()

    def summary(self):
        sm, mx, reasons = [], [], set()
        try:
            for line in open(self.path):
                f = [x.strip() for x in line.split(",")]
                if len(f) < 9:
                    continue
                try:
                    sm.append(float(f[1])); mx.append(float(f[2]))
                except ValueError:
                    continue
                for name, val in zip(("hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown",
                                      "sw_power_cap"), f[5:9]):
                    if val.lower() == "active":
                        reasons.add(name)
        finally:
            os.unlink(self.path)
        if not sm:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["unsampled"]}
        return {"sm_mhz": statistics.median(sm), "sm_max_mhz": max(mx), "reasons": sorted(reasons),
                "samples": len(sm)}


# ---------------------------------------------------------------------------------
# reference arm / CPU baseline: the oracle on a bounded sample
# ---------------------------------------------------------------------------------

def oracle_sample(wl: dict, groups: int = 1) -> dict:
    """Time the oracle on `groups` (sequence, KV head) groups of one layer of the workload.

    Runs single-threaded (BLAS threads pinned to 1 by the caller's environment).
    Returns the per-layer time scaled from the sample.
    """
    import oracle as O
    import workloads as W
    q, K, V = W.c3_layer(0, device="cpu", seed=wl["seed"], batch=wl["batch"], ctx=wl["ctx"],
                         Hq=wl["q_heads"], Hkv=wl["kv_heads"])
    n_rep = wl["q_heads"] // wl["kv_heads"]
    total = 0.0
    for g in range(groups):
        qs = q[:, g * n_rep:(g + 1) * n_rep].numpy()
        Ks, Vs = K[:, g:g + 1].numpy(), V[:, g:g + 1].numpy()
        t0 = time.perf_counter()
        t1 = O.quantize_layer(Ks, Vs)          # the oracle derives tier 1 itself; not timed below
        total_q = time.perf_counter() - t0
        t0 = time.perf_counter()
        O.decode_layer(qs, Ks, Vs, t1, wl["tau_cov"], wl["eps"], O.OracleConfig(n_rep=n_rep))
        total += time.perf_counter() - t0
        del total_q
    per_group = total / groups
    t_layer = per_group * wl["batch"] * wl["kv_heads"]
    return {"t_layer_s": t_layer, "sample_s": total, "groups": groups}


# ---------------------------------------------------------------------------------
# the oracle on every host core: one process per (sequence, KV head) group
# ---------------------------------------------------------------------------------

def _oracle_group_worker(idx, q, K, V, tau, eps, n_rep, barrier, out_q, rounds):
    """Spawned worker: derive tier 1 of its group once (untimed), then decode it once per
    round, every round starting on a barrier shared by all workers."""
    for var in ("OMP_NUM_THREADS", "OPENBLAS_NUM_THREADS", "MKL_NUM_THREADS"):
        os.environ[var] = "1"
    sys.path.insert(0, ROOT)
    import oracle as O
    t1 = O.quantize_layer(K, V)
    cfg = O.OracleConfig(n_rep=n_rep)
    for _ in range(rounds):
        barrier.wait(timeout=900)
        t0 = time.time()
        O.decode_layer(q, K, V, t1, tau, eps, cfg)
        out_q.put((idx, t0, time.time()))


def oracle_parallel(groups: list, tau: float, eps: float, n_rep: int, rounds: int) -> list:
    """Decode the given (q, K, V) groups concurrently, one spawned process per group
    (each single-threaded), `rounds` times.  Returns the makespan of every round in
    seconds (first start to last finish)."""
    import multiprocessing as mp
    ctx = mp.get_context("spawn")   # never fork a process that has touched the GPU
    barrier = ctx.Barrier(len(groups))
    out_q = ctx.Queue()
    saved = {v: os.environ.get(v) for v in ("OMP_NUM_THREADS", "OPENBLAS_NUM_THREADS", "MKL_NUM_THREADS",
                                            "CUDA_VISIBLE_DEVICES")}
    for v in saved:
        os.environ[v] = "" if v == "CUDA_VISIBLE_DEVICES" else "1"
    try:
        procs = [ctx.Process(target=_oracle_group_worker,
                             args=(i, q, K, V, tau, eps, n_rep, barrier, out_q, rounds), daemon=True)
                 for i, (q, K, V) in enumerate(groups)]
        for pr in procs:
            pr.start()
    finally:
        for v, val in saved.items():
            if val is None:
                os.environ.pop(v, None)
            else:
                os.environ[v] = val
    spans = []
    try:
        for _ in range(rounds):
            got = [out_q.get(timeout=1200) for _ in groups]
            spans.append(max(e for _, _, e in got) - min(s for _, s, _ in got))
    finally:
        for pr in procs:
            pr.join(timeout=60)
            if pr.is_alive():
                pr.terminate()
    return spans


def _split_groups(q, K, V, limit):
    """(q, K, V) numpy slices of the first `limit` (sequence, KV head) groups."""
    B, Hq = q.shape[0], q.shape[1]
    Hkv = K.shape[1]
    n_rep = Hq // Hkv
    out = []
    for b in range(B):
        for g in range(Hkv):
            if len(out) == limit:
                return out
            out.append((q[b:b + 1, g * n_rep:(g + 1) * n_rep].numpy().copy(),
                        K[b:b + 1, g:g + 1].numpy().copy(), V[b:b + 1, g:g + 1].numpy().copy()))
    return out


def oracle_config_baselines(rounds: int = 1) -> dict:
    """The oracle on the four workloads' shapes, on all host cores (one process per group,
    up to the core count) and on one core (one group), in tokens/s/layer.  Each figure is
    a bounded sample: the groups run, scaled to the layer (B sequences x Hkv groups)."""
    import workloads as W
    ncores = os.cpu_count() or 1
    shapes = {
        "c1_ctx4k": lambda: W.c1(),
        "c2_lowrank_ctx32k_b4": lambda: W.c2(),
        "c3_llama8b_ctx128k_32l": lambda: W.c3_layer(0, seed=WORKLOAD["seed"]),
        "c4_planted_ctx64k_b8": lambda: W.c4()[:3],
    }
    res = {}
    for name, make in shapes.items():
        cfg = W.WORKLOADS[name]
        q, K, V = make()
        B, Hkv = q.shape[0], K.shape[1]
        n_groups = B * Hkv
        n_rep = q.shape[1] // Hkv
        par = _split_groups(q, K, V, min(ncores, n_groups))
        span = min(oracle_parallel(par, cfg.tau_cov, cfg.eps, n_rep, rounds))
        one = oracle_parallel(par[:1], cfg.tau_cov, cfg.eps, n_rep, 1)[0]
        del q, K, V
        res[name] = {
            "all_cores": {"value": (len(par) / n_groups) * B / span, "unit": UNIT, "cores": len(par),
                          "sample": f"{len(par)} of {n_groups} groups concurrently, {span:.2f} s"},
            "one_core": {"value": B / (one * n_groups), "unit": UNIT, "cores": 1,
                         "sample": f"1 of {n_groups} groups, {one:.2f} s, scaled to the layer"},
        }
    res["nproc"] = ncores
    return res


def run_oracle_subprocess(wl: dict, groups: int = 1) -> dict:
    env = dict(os.environ, OMP_NUM_THREADS="1", OPENBLAS_NUM_THREADS="1", MKL_NUM_THREADS="1",
               CUDA_VISIBLE_DEVICES="")
    code = ("import json,sys; sys.path.insert(0, %r); import bench; "
            "print(json.dumps(bench.oracle_sample(json.loads(sys.argv[1]), %d)))" % (ROOT, groups))
    r = subprocess.run([sys.executable, "-c", code, json.dumps(wl)], capture_output=True, text=True,
                       env=env, timeout=1200)
    if r.returncode != 0:
        raise RuntimeError(r.stderr[-2000:])
    return json.loads(r.stdout.strip().splitlines()[-1])


def _c3_groups(wl: dict, limit: int) -> list:
    """(q, K, V) of up to `limit` (sequence, KV head) groups of the headline workload,
    layer after layer, drawn on the CPU."""
    import workloads as W
    out = []
    layer = 0
    while len(out) < limit and layer < wl["layers"]:
        q, K, V = W.c3_layer(layer, device="cpu", seed=wl["seed"], batch=wl["batch"], ctx=wl["ctx"],
                             Hq=wl["q_heads"], Hkv=wl["kv_heads"])
        out += _split_groups(q, K, V, limit - len(out))
        layer += 1
    return out


def reference_arm(args, wl):
    """The oracle, as it stands, on the host's cores: one single-threaded process per
    (sequence, KV head) group of the headline workload, as many groups as there are
    cores (drawn from consecutive layers), all decoding at once.  A step is one such
    round; its time is scaled to one layer of the workload."""
    rank = int(os.environ.get("RANK", "0"))
    if rank != 0:
        return
    ncores = os.cpu_count() or 1
    n_groups = wl["batch"] * wl["kv_heads"]
    n_rep = wl["q_heads"] // wl["kv_heads"]
    groups = _c3_groups(wl, ncores)
    spans = oracle_parallel(groups, wl["tau_cov"], wl["eps"], n_rep, args.warmup + args.steps)[args.warmup:]
    t_layer = float(np.mean(spans)) * n_groups / len(groups)
    value = wl["batch"] / t_layer
    sample = (f"oracle decode of {len(groups)} (sequence, KV head) groups of {wl['ctx']}-token layers "
              f"({len(groups) / n_groups:g} layers) per step, one single-threaded process per group "
              f"on {len(groups)} of {ncores} host cores, scaled to one layer")
    line = {"impl": "reference", "metric": METRIC, "value": value, "unit": UNIT, "n_gpus": args.gpus,
            "steps": args.steps, "warmup": args.warmup, "ms_per_step": t_layer * wl["layers"] * 1e3,
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64",
            "data": "synthetic", "config": _config(wl),
            "cpu_baseline": {"value": value, "unit": UNIT, "cores": len(groups), "kind": "oracle",
                             "sample": sample, "nproc": ncores},
            "e2e": {"value": value, "unit": UNIT, "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0}}
    print(json.dumps(line), flush=True)


def _source_hash() -> str:
    """Of the kernels that the summary covers (the paged cache and rotary positions are none of them)."""
    import hashlib
    d = os.path.join(ROOT, "certified_quantized_kv_gb300", "csrc")
    h = hashlib.sha256()
    for f in sorted(os.listdir(d)):
        if f.startswith(("kvq_paged", "kvq_rope")):
            continue
        with open(os.path.join(d, f), "rb") as fh:
            h.update(f.encode() + fh.read())
    return h.hexdigest()[:16]


def _ncu_traffic() -> dict:
    """Per-launch DRAM / host-link bytes per kernel from the committed ncu summary, if it
    was taken on the current kernel sources (else empty: traffic is reported as null)."""
    path = os.path.join(ROOT, "profiles", "ncu_traffic.txt")
    out = {}
    try:
        for line in open(path):
            f = dict(kv.split("=", 1) for kv in line.split() if "=" in kv)
            if f.get("src") != _source_hash() or "kernel" not in f:
                continue
            out[f["kernel"]] = {k: float(v) for k, v in f.items() if k.endswith("_bytes")}
    except OSError:
        pass
    return out


def _config(wl):
    return {"workload": wl["name"], "batch": wl["batch"], "ctx": wl["ctx"], "layers": wl["layers"],
            "q_heads": wl["q_heads"], "kv_heads": wl["kv_heads"], "head_dim": wl["head_dim"],
            "tau_cov": wl["tau_cov"], "eps": wl["eps"],
            "l2": "inputs larger than L2: tier 1 and tier 2 of all layers are streamed every step"}


# ---------------------------------------------------------------------------------
# our arm
# ---------------------------------------------------------------------------------

def aggregate_ranks(ms_local: float, units_local: int, device=None):
    """Whole-job timing over ranks: the slowest rank's time and the units of all ranks.

    Every rank runs an independent replica (no data exchange on the path), so the job's
    throughput is the total units over the max time.  Single-process runs pass through.
    """
    import torch
    import torch.distributed as dist
    if not (dist.is_available() and dist.is_initialized()) or dist.get_world_size() == 1:
        return ms_local, units_local
    t = torch.tensor([ms_local], dtype=torch.float64, device=device)
    u = torch.tensor([units_local], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    dist.all_reduce(u, op=dist.ReduceOp.SUM)
    dist.barrier()
    return float(t.item()), int(u.item())


REJECT_REASONS = ("hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown")


def clocks_rejected(clocks: dict) -> bool:
    """A timed region is not kept when the GPU slowed itself down (hardware or thermal
    slowdown) or ran with SM clocks well below their maximum and no reason reported (a
    clock lock left behind by another user).  Power capping alone is kept."""
    reasons = set(clocks.get("reasons") or [])
    if reasons & set(REJECT_REASONS):
        return True
    sm, mx = clocks.get("sm_mhz"), clocks.get("sm_max_mhz")
    return bool(sm and mx and sm < 0.85 * mx and not (reasons - {"unsampled"}))


def any_rank(flag: bool, device=None) -> bool:
    """True on every rank if it is true on any (single-process runs pass through)."""
    import torch
    import torch.distributed as dist
    if not (dist.is_available() and dist.is_initialized()) or dist.get_world_size() == 1:
        return flag
    t = torch.tensor([1.0 if flag else 0.0], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return bool(t.item() > 0)


def measure_h2d(torch):
    n = 256 << 20
    h = torch.empty(n, dtype=torch.uint8).pin_memory()
    d = torch.empty(n, dtype=torch.uint8, device="cuda")
    best = 1e9
    for _ in range(10):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(); d.copy_(h, non_blocking=True); e1.record(); e1.synchronize()
        best = min(best, e0.elapsed_time(e1))
    return n / best / 1e6   # GB/s


def measure_d2h(torch):
    n = 256 << 20
    h = torch.empty(n, dtype=torch.uint8).pin_memory()
    d = torch.empty(n, dtype=torch.uint8, device="cuda")
    best = 1e9
    for _ in range(10):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(); h.copy_(d, non_blocking=True); e1.record(); e1.synchronize()
        best = min(best, e0.elapsed_time(e1))
    return n / best / 1e6   # GB/s


def measure_append(torch, kvq, W, wl, hbm_peak, reps=2):
    """Bulk prefill of one layer (the workload's batch and context) through kvq_append:
    quantisation to tier 1 on the device plus the FP16 mirror to tier 2 over the host
    link, both inside the timed call.  Best of `reps` fresh caches."""
    B, N, Hq, Hkv = wl["batch"], wl["ctx"], wl["q_heads"], wl["kv_heads"]
    _, K, V = W.c3_layer(0, device="cuda", seed=wl["seed"], batch=B, ctx=N, Hq=Hq, Hkv=Hkv)
    K, V = K.contiguous(), V.contiguous()
    best_ms, kern_us = 1e9, None
    for _ in range(reps):
        c = kvq.Cache(1, B, Hq, Hkv, max_ctx=N)
        c.set_debug(kvq.DEBUG_PROFILE)
        c.profile_read(reset=True)
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(); c.append(0, K, V); e1.record(); torch.cuda.synchronize()
        ms = e0.elapsed_time(e1)
        prof = c.profile_read(reset=True)
        c.close()
        if ms < best_ms:
            best_ms = ms
            n, tot = prof.get("quantize_append", (1, float("nan")))
            kern_us = 1e3 * tot / max(1, n)
    units = B * Hkv * N
    d2h = measure_d2h(torch)
    hbm_bytes = units * APPEND_HBM_BYTES_PER_TOKEN_HEAD
    return {"tokens": B * N, "ms": best_ms, "tokens_per_s": B * N / (best_ms / 1e3),
            "mirror_bytes": units * F16_BYTES_PER_TOKEN_HEAD, "d2h_gbs_measured": d2h,
            "mirror_frac_of_d2h": units * F16_BYTES_PER_TOKEN_HEAD / (best_ms / 1e3) / 1e9 / d2h,
            "quantize_kernel_us": kern_us,
            "quantize_kernel_hbm": {"bytes": hbm_bytes, "achieved_gbs": hbm_bytes / (kern_us * 1e-6) / 1e9,
                                    "peak": hbm_peak, "frac": hbm_bytes / (kern_us * 1e-6) / 1e9 / hbm_peak,
                                    "traffic": _ncu_traffic().get("quantize_append", {}).get("dram_bytes"),
                                    "timing": "CUDA events around the kernel inside the append call, while the "
                                              "tier-2 mirror copy runs beside it"}}


def measure_fp16_values(args, wl):
    """The FP16-values configuration (value_bits 16) on the same synthetic caches: FP16
    values resident in VRAM, keys-only tier 2.  Same timing protocol as the headline."""
    import torch
    import certified_quantized_kv_gb300 as kvq
    import workloads as W
    B, L, N = wl["batch"], wl["layers"], wl["ctx"]
    Hq, Hkv, D = wl["q_heads"], wl["kv_heads"], wl["head_dim"]
    tau, eps = wl["tau_cov"], wl["eps"]
    cache = kvq.Cache(L, B, Hq, Hkv, max_ctx=N, value_bits=16)
    qs = []
    for layer in range(L):
        q, K, V = W.c3_layer(layer, device="cuda", seed=wl["seed"], batch=B, ctx=N, Hq=Hq, Hkv=Hkv)
        cache.append(layer, K.contiguous(), V.contiguous())
        qs.append(q.contiguous())
        del K, V
    out = torch.empty(B, Hq, D, dtype=torch.float16, device="cuda")
    certs = [torch.empty(B * Hq * 32, dtype=torch.uint8, device="cuda") for _ in range(L)]

    def step():
        for layer in range(L):
            cache.decode(layer, qs[layer], tau, eps, out, certs[layer])

    for _ in range(args.warmup):
        step()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(args.steps):
        step()
    e1.record()
    torch.cuda.synchronize()
    ms = e0.elapsed_time(e1) / args.steps
    hist, prom = [0] * 5, 0
    for layer in range(L):
        c = kvq.certificates(certs[layer]).reshape(B, Hq)
        for lv in c["level"].ravel():
            hist[int(lv)] += 1
        prom += int(c["promoted_bytes"][:, :: Hq // Hkv].sum())
    cache.close()
    return {"value": B * L / (ms / 1e3), "unit": UNIT, "ms_per_step": ms, "ladder_histogram": hist,
            "promoted_bytes_per_step": prom, "vram_bytes_per_token_head": 128 + 4 + 256,
            "what": "value_bits 16: INT8 keys, FP16 values in VRAM, keys-only tier 2"}


def measure_residency(args, wl, frac=0.25, layers=4):
    """Cross-step residency of paged-in FP16 blocks (kvq_config.resident_blocks: an option
    of this library, not of the paper), same timing protocol as the headline.
    (1) The headline caches, `layers` layers, each allowed to keep `frac` of its FP16
    tier-2 blocks (keys and values) in HBM.  (2) The concentrated 32K x 4 workload, with
    and without room for its whole working set.  Warm-up calls fill the slots; the timed
    calls report tokens/s/layer and the FP16 bytes read over the host link and from HBM."""
    import torch
    import certified_quantized_kv_gb300 as kvq
    import workloads as W
    B, N = wl["batch"], wl["ctx"]
    Hq, Hkv, D = wl["q_heads"], wl["kv_heads"], wl["head_dim"]
    tau, eps = wl["tau_cov"], wl["eps"]

    def run(cache, qs, n_layers, batch):
        out = torch.empty(batch, Hq, D, dtype=torch.float16, device="cuda")

        def step():
            for layer in range(n_layers):
                cache.decode(layer, qs[layer], tau, eps, out)

        for _ in range(args.warmup):
            step()
        torch.cuda.synchronize()
        for layer in range(n_layers):
            cache.residency_stats(layer, reset=True)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(args.steps):
            step()
        e1.record()
        torch.cuda.synchronize()
        ms = e0.elapsed_time(e1) / args.steps
        st = [cache.residency_stats(layer) for layer in range(n_layers)]
        per = args.steps * n_layers
        return {"value": batch * n_layers / (ms / 1e3), "unit": UNIT, "us_per_layer": 1e3 * ms / n_layers,
                "host_bytes_per_layer": sum(x["host_bytes"] for x in st) / per,
                "resident_bytes_per_layer": sum(x["resident_bytes"] for x in st) / per,
                "slots_in_use_per_layer": sum(x["slots_in_use"] for x in st) / n_layers}

    res = {}
    nblk = B * Hkv * (N // 64) * 2
    slots = int(frac * nblk)
    cache = kvq.Cache(layers, B, Hq, Hkv, max_ctx=N, resident_blocks=slots)
    qs = []
    for layer in range(layers):
        q, K, V = W.c3_layer(layer, device="cuda", seed=wl["seed"], batch=B, ctx=N, Hq=Hq, Hkv=Hkv)
        cache.append(layer, K.contiguous(), V.contiguous())
        qs.append(q.contiguous())
        del K, V
    r = run(cache, qs, layers, B)
    cache.close()
    r.update({"workload": f"{wl['name']} (first {layers} layers)", "resident_blocks": slots,
              "resident_fraction_of_tier2": frac, "extra_vram_bytes_per_layer": slots * F16_BLOCK})
    res["headline_shape"] = r
    q, K, V = W.c2(device="cuda", batch=4, ctx=32768)
    q = q.contiguous()
    for slots in (0, 4 * Hkv * 512 * 2):
        cache = kvq.Cache(1, 4, Hq, Hkv, max_ctx=32768, resident_blocks=slots)
        cache.append(0, K.contiguous(), V.contiguous())
        r = run(cache, [q], 1, 4)
        cache.close()
        r.update({"resident_blocks": slots, "extra_vram_bytes_per_layer": slots * F16_BLOCK})
        res[f"c2_ctx32k_b4_slots{slots}"] = r
    del K, V
    res["what"] = ("FP16 blocks paged in by one call kept in HBM for the next (not part of the paper); "
                   "outputs and certificates are bit-identical to the cache without residency")
    return res



def time_back_to_back(torch, call, reps=20, batches=5, warmup=3):
    """Device time per call (ms): `reps` calls enqueued back to back between two CUDA
    events, so the host's enqueue time hides behind the GPU; median over `batches`."""
    for _ in range(warmup):
        call()
    torch.cuda.synchronize()
    res = []
    for _ in range(batches):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(reps):
            call()
        e1.record()
        torch.cuda.synchronize()
        res.append(e0.elapsed_time(e1) / reps)
    return statistics.median(res)


def time_dense_hbm(torch, kvq, q, K, V):
    """Device time (ms) of one kvq_dense_attention call (dense FP16 attention over K/V in
    HBM) on these device tensors; K and V are read once per call."""
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    ws = kvq.dense_attention(q, K, V, out)
    return time_back_to_back(torch, lambda: kvq.dense_attention(q, K, V, out, ws))


def measure_dense_hbm(args, wl, t_cert_layer_us, t_unc_layer_us):
    """Dense FP16 decode attention with the whole FP16 cache in HBM (kvq_dense_attention)
    on one layer of the headline caches: the dense baseline the pages quote the certified
    step against (Results, performance overhead: 2.7-4.8x slower than dense attention,
    hardware unstated).  K and V (512 B per token and KV head) exceed L2 many times over,
    so every call streams them from HBM."""
    import torch
    import certified_quantized_kv_gb300 as kvq
    import workloads as W
    B, N, Hq, Hkv = wl["batch"], wl["ctx"], wl["q_heads"], wl["kv_heads"]
    q, K, V = W.c3_layer(0, device="cuda", seed=wl["seed"], batch=B, ctx=N, Hq=Hq, Hkv=Hkv)
    q, K, V = q.contiguous(), K.contiguous(), V.contiguous()
    ms = time_dense_hbm(torch, kvq, q, K, V)
    del K, V
    torch.cuda.empty_cache()
    hbm_peak, peak_kind = _peaks()
    b = B * Hkv * N * F16_BYTES_PER_TOKEN_HEAD
    us = 1e3 * ms
    return {"value": B / (ms / 1e3), "unit": UNIT, "us_per_layer": us,
            "roofline": {"bound": "hbm", "kernel": "dense_hbm (split pass + combine)", "achieved": b / (us * 1e-6) / 1e9,
                         "peak": hbm_peak, "peak_kind": peak_kind, "unit": "GB/s",
                         "frac": b / (us * 1e-6) / 1e9 / hbm_peak, "algorithmic_bytes_per_launch": b,
                         "traffic": _ncu_traffic().get("dense_hbm", {}).get("dram_bytes")},
            "certified_over_dense": t_cert_layer_us / us,
            "uncertified_over_dense": t_unc_layer_us / us,
            "pages_certified_over_dense": "2.7-4.8x (Results, performance overhead; hardware unstated)",
            "vram_bytes_per_token_head": {"dense_fp16": 512, "certified_tier1": TIER1_BYTES_PER_TOKEN_HEAD},
            "what": "kvq_dense_attention: exact FP16 attention, K/V resident in HBM, one 128K layer of the headline "
                    "caches; device time per call from batches of back-to-back calls between CUDA events"}


def measure_configs(args, with_oracle: bool) -> dict:
    """The other workloads' shapes (4K x 1, concentrated 32K x 4, planted-needle 64K x 8):
    device time per certified decode call (batches of 20 back-to-back calls after 5
    warm-up calls, median over the batches) and per dense FP16 call over the same K/V in
    HBM, next to the oracle on all host cores and on one core (bounded samples, scaled
    to the layer)."""
    import torch
    import certified_quantized_kv_gb300 as kvq
    import workloads as W
    res = {}
    for name, make in (("c1_ctx4k", lambda: W.c1(device="cuda")),
                       ("c2_lowrank_ctx32k_b4", lambda: W.c2(device="cuda")),
                       ("c4_planted_ctx64k_b8", lambda: W.c4(device="cuda")[:3])):
        cfg = W.WORKLOADS[name]
        q, K, V = make()
        B, Hq, Hkv, N = q.shape[0], q.shape[1], K.shape[1], K.shape[2]
        cache = kvq.Cache(1, B, Hq, Hkv, max_ctx=N)
        cache.append(0, K.contiguous(), V.contiguous())
        q = q.contiguous()
        dense_ms = time_dense_hbm(torch, kvq, q, K.contiguous(), V.contiguous())
        del K, V
        out = torch.empty(B, Hq, 128, dtype=torch.float16, device="cuda")
        cert = torch.empty(B * Hq * 32, dtype=torch.uint8, device="cuda")
        ms = time_back_to_back(torch, lambda: cache.decode(0, q, cfg.tau_cov, cfg.eps, out, cert), warmup=5)
        c = kvq.certificates(cert).reshape(B, Hq)
        res[name] = {"gpu": {"value": B / (ms / 1e3), "unit": UNIT, "us_per_call": 1e3 * ms,
                             "ladder_histogram": [int(x) for x in np.bincount(c["level"].ravel(), minlength=5)],
                             "promoted_bytes": int(c["promoted_bytes"][:, :: Hq // Hkv].sum())},
                     "dense_fp16_hbm": {"us_per_call": 1e3 * dense_ms, "value": B / (dense_ms / 1e3), "unit": UNIT,
                                        "certified_over_dense": ms / dense_ms}}
        cache.close()
        torch.cuda.empty_cache()
    if with_oracle:
        orc = oracle_config_baselines()
        for name in res:
            res[name]["oracle"] = orc[name]
        res["oracle_nproc"] = orc["nproc"]
    return res


def our_arm(args, wl):
    import torch
    import torch.distributed as dist
    import certified_quantized_kv_gb300 as kvq
    import workloads as W

    world = int(os.environ.get("WORLD_SIZE", "1"))
    rank = int(os.environ.get("RANK", "0"))
    local = int(os.environ.get("LOCAL_RANK", "0"))
    torch.cuda.set_device(local)
    if world > 1:
        dist.init_process_group("nccl")
    B, L, N = wl["batch"], wl["layers"], wl["ctx"]
    Hq, Hkv, D = wl["q_heads"], wl["kv_heads"], wl["head_dim"]
    tau, eps = wl["tau_cov"], wl["eps"]

    cache = kvq.Cache(L, B, Hq, Hkv, max_ctx=N)
    qs, qs_host = [], []
    t_fill = time.time()
    for layer in range(L):
        q, K, V = W.c3_layer(layer, device="cuda", seed=wl["seed"] + 1000 * rank, batch=B, ctx=N, Hq=Hq, Hkv=Hkv)
        cache.append(layer, K.contiguous(), V.contiguous())
        qs.append(q.contiguous())
        qs_host.append(q.cpu().pin_memory())
        del K, V
    torch.cuda.synchronize()
    t_fill = time.time() - t_fill
    outs = [torch.empty(B, Hq, D, dtype=torch.float16, device="cuda") for _ in range(L)]
    certs = [torch.empty(B * Hq * 32, dtype=torch.uint8, device="cuda") for _ in range(L)]
    lvls = [torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(L)]

    def step():
        for layer in range(L):
            cache.decode(layer, qs[layer], tau, eps, outs[layer], certs[layer], lvls[layer])

    for _ in range(args.warmup):
        step()
    torch.cuda.synchronize()
    if world > 1:
        dist.barrier()
    st = torch.cuda.current_stream()

    def timed_region():
        # one event per step boundary on the launching stream: the K steps are timed as a
        # whole, and the per-step times give the median
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(args.steps + 1)]
        with ClockSampler(local) as clk:
            torch.cuda.synchronize()
            ev[0].record(st)
            for i in range(args.steps):
                step()
                ev[i + 1].record(st)
            torch.cuda.synchronize()
        per = [ev[i].elapsed_time(ev[i + 1]) for i in range(args.steps)]
        return ev[0].elapsed_time(ev[-1]), per, clk.summary()

    ms, per_step, clocks = timed_region()
    if any_rank(clocks_rejected(clocks), "cuda" if world > 1 else None):
        # slowed down or clock-locked: measured once more, and the second run is reported
        if world > 1:
            dist.barrier()
        ms, per_step, clocks = timed_region()
        clocks["remeasured"] = True
    ms, units = aggregate_ranks(ms, B * L * args.steps, "cuda" if world > 1 else None)
    ms_per_step = ms / args.steps
    ms_median = statistics.median(per_step)
    value = units / (ms / 1e3)

    # the uncertified INT8/INT4 baseline on the same caches: the speed ceiling of tier 1
    def step_unc():
        for layer in range(L):
            cache.decode_uncertified(layer, qs[layer], outs[layer])

    for _ in range(args.warmup):
        step_unc()
    torch.cuda.synchronize()
    u0, u1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    u0.record(st)
    for _ in range(args.steps):
        step_unc()
    u1.record(st)
    torch.cuda.synchronize()
    unc_ms = u0.elapsed_time(u1) / args.steps
    uncertified = {"value": world * B * L / (unc_ms / 1e3), "unit": UNIT, "ms_per_step": unc_ms,
                   "what": "INT8 scores and INT4 values on every block: no page-in, no ladder"}

    # the tier-1 kernels alone: uncertified calls on one layer in a loop, CUDA events
    # around every kernel (the scoring pass and the INT4 value pass)
    cache.set_debug(kvq.DEBUG_PROFILE)
    for _ in range(3):
        cache.decode_uncertified(0, qs[0], outs[0])
    torch.cuda.synchronize()
    cache.profile_read(reset=True)
    for _ in range(20):
        cache.decode_uncertified(0, qs[0], outs[0])
    torch.cuda.synchronize()
    prof_alone = cache.profile_read(reset=True)
    cache.set_debug(0)

    # certificates of the last step: ladder histogram, promoted bytes
    hist = [0] * 5
    prom = 0
    n_rep = Hq // Hkv
    for layer in range(L):
        c = kvq.certificates(certs[layer]).reshape(B, Hq)
        for lv in c["level"].ravel():
            hist[int(lv)] += 1
        prom += int(c["promoted_bytes"][:, ::n_rep].sum())

    # per-kernel durations: a second pass with CUDA events around every kernel
    cache.set_debug(kvq.DEBUG_PROFILE)
    cache.profile_read(reset=True)
    for _ in range(args.steps):
        step()
    torch.cuda.synchronize()
    prof = cache.profile_read(reset=True)
    cache.set_debug(0)
    # FP16 blocks paged in per pass, from the selection state of every layer
    nb = N // 64
    u0 = u1_new = v1 = dense_blocks = 0
    for layer in range(L):
        cache.decode(layer, qs[layer], tau, eps, outs[layer], certs[layer], lvls[layer])
        st = cache.export_decode_state(nb)
        k0, k1, vv = st["kprom0"].sum().item(), st["kprom1"].sum().item(), st["vprom1"].sum().item()
        u0 += k0; u1_new += k1 - k0; v1 += vv
        c = kvq.certificates(certs[layer]).reshape(B, Hq)
        dense = (c["level"].reshape(B, Hkv, Hq // Hkv) >= 3).any(axis=2)
        # a dense group pages in every value block and the key blocks not paged in before
        kp1 = st["kprom1"].sum(dim=2).cpu().numpy()
        dense_blocks += int(((2 * nb - kp1) * dense).sum())
    torch.cuda.synchronize()
    host_bytes = {"mixed_round0": u0 * F16_BLOCK / L, "mixed_round1": (u1_new + v1) * F16_BLOCK / L,
                  "dense_fallback": dense_blocks * F16_BLOCK / L}

    # end to end through the C ABI with host buffers (q in, out + certificate back)
    outs_h = [torch.empty(B, Hq, D, dtype=torch.float16).pin_memory() for _ in range(L)]
    certs_h = [torch.empty(B * Hq * 32, dtype=torch.uint8).pin_memory() for _ in range(L)]
    lvls_h = [torch.empty(B, dtype=torch.int32).pin_memory() for _ in range(L)]

    def step_host():
        for layer in range(L):
            cache.decode(layer, qs_host[layer], tau, eps, outs_h[layer], certs_h[layer], lvls_h[layer])

    step_host()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(args.steps):
        step_host()
    torch.cuda.synchronize()
    e2e_s = (time.perf_counter() - t0) / args.steps
    e2e_value = world * B * L / e2e_s
    h2d = L * B * Hq * D * 2
    d2h = L * (B * Hq * D * 2 + B * Hq * 32 + B * 4)

    h2d_gbs = measure_h2d(torch)
    hbm_peak, peak_kind = _peaks()
    append = measure_append(torch, kvq, W, wl, hbm_peak) if rank == 0 else None
    if rank != 0:
        cache.close()
        if world > 1:
            dist.destroy_process_group()
        return

    kern = {}
    for name, (n, tot) in prof.items():
        kern[name] = {"launches": n, "avg_us": 1e3 * tot / max(1, n), "total_ms": tot}
    tot_all = sum(v["total_ms"] for v in kern.values()) or 1.0
    for v in kern.values():
        v["share"] = v["total_ms"] / tot_all
    units = B * Hkv * N      # token x KV-head units per layer
    traffic = _ncu_traffic()
    t_layer_us = 1e3 * ms_per_step / L
    # HBM-bound tier-1 kernels: algorithmic bytes per launch (tier-1 bytes they must read)
    hbm_algo = {"score": SCORE_BYTES_PER_TOKEN_HEAD * units}

    def host_roofline(k):
        b = host_bytes.get(k, 0.0)
        achieved = b / (kern[k]["avg_us"] * 1e-6) / 1e9
        t = traffic.get(k, {}).get("sysmem_bytes")
        return {"bound": "host_link", "kernel": k, "achieved": achieved, "peak": h2d_gbs,
                "peak_kind": "measured in this run (pinned H2D copy, 256 MiB)", "unit": "GB/s",
                "frac": achieved / h2d_gbs, "traffic": t, "algorithmic_bytes_per_launch": b,
                "timing": "CUDA events around this kernel in a separate pass that brackets every kernel "
                          "(that pass runs about 10% slower than the timed region)"}

    def hbm_roofline(k):
        achieved = hbm_algo[k] / (kern[k]["avg_us"] * 1e-6) / 1e9
        t = traffic.get(k, {}).get("dram_bytes")
        return {"bound": "hbm", "kernel": k, "achieved": achieved, "peak": hbm_peak, "peak_kind": peak_kind,
                "unit": "GB/s", "frac": achieved / hbm_peak, "traffic": t,
                "algorithmic_bytes_per_launch": hbm_algo[k]}

    # the decode step is bound by the FP16 blocks it pages in over the host link: the
    # roofline is that link, from the timed region (every tier-2 read of the step: the
    # first and second mixed passes and the dense rung, per layer call)
    prom_layer = prom / L
    link_traffic = [traffic.get(k, {}).get("sysmem_bytes") for k in ("mixed_round0", "mixed_round1", "dense_fallback")]
    roofline = {"bound": "host_link",
                "kernel": "decode call (tier-2 reads of mixed_round0, mixed_round1 and dense_fallback)",
                "achieved": prom_layer / (t_layer_us * 1e-6) / 1e9, "peak": h2d_gbs,
                "peak_kind": "measured in this run (pinned H2D copy, 256 MiB)", "unit": "GB/s",
                "frac": prom_layer / (t_layer_us * 1e-6) / 1e9 / h2d_gbs,
                "traffic": (sum(link_traffic) if all(x is not None for x in link_traffic) else None),
                "algorithmic_bytes_per_launch": prom_layer,
                "timing": "the timed region: ms_per_step / layers per decode call"}
    tier1_layer = TIER1_BYTES_PER_TOKEN_HEAD * units
    floor_us = 1e6 * (tier1_layer / (hbm_peak * 1e9) + prom_layer / (h2d_gbs * 1e9))
    two_link = {"tier1_bytes_per_layer": tier1_layer, "promoted_bytes_per_layer": prom_layer,
                "floor_us_per_layer": floor_us, "t_layer_us": t_layer_us, "frac": floor_us / t_layer_us,
                "what": "(tier-1 bytes / measured HBM + promoted bytes / measured H2D) / time per layer"}
    roofline_hbm = hbm_roofline("score") if "score" in kern else None
    # the same kernels timed alone (one layer, uncertified calls back to back)
    tier1_alone = {}
    for k, per_unit in (("score", SCORE_BYTES_PER_TOKEN_HEAD), ("int4_tail", MIX_BYTES_PER_TOKEN_HEAD + 4 * (Hq // Hkv))):
        if k in prof_alone:
            n, tot = prof_alone[k]
            us = 1e3 * tot / max(1, n)
            b = per_unit * units
            t = traffic.get(k, {}).get("dram_bytes")
            tier1_alone[k] = {"bound": "hbm", "kernel": k, "avg_us": us, "achieved": b / (us * 1e-6) / 1e9,
                              "peak": hbm_peak, "peak_kind": peak_kind, "unit": "GB/s",
                              "frac": b / (us * 1e-6) / 1e9 / hbm_peak, "traffic": t,
                              "algorithmic_bytes_per_launch": b}
    if "score" in tier1_alone and "int4_tail" in tier1_alone:
        b = tier1_alone["score"]["algorithmic_bytes_per_launch"] + tier1_alone["int4_tail"]["algorithmic_bytes_per_launch"]
        us = tier1_alone["score"]["avg_us"] + tier1_alone["int4_tail"]["avg_us"]
        tier1_alone["pair"] = {"bound": "hbm", "kernel": "score + int4_tail", "avg_us": us,
                               "achieved": b / (us * 1e-6) / 1e9, "peak": hbm_peak, "peak_kind": peak_kind,
                               "unit": "GB/s", "frac": b / (us * 1e-6) / 1e9 / hbm_peak,
                               "algorithmic_bytes_per_launch": b}
    line = {
        "metric": METRIC, "value": value, "unit": UNIT, "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": ms_per_step, "ms_per_step_median": ms_median,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
        "dtype": "f32 accumulate (int8/int4/f16 MMA operands)",
        "data": "synthetic (seeded Gaussian caches shaped like Llama-3.1-8B attention)",
        "config": _config(wl),
        "clocks": clocks,
        "e2e": {"value": e2e_value, "unit": UNIT, "h2d_bytes_per_step": h2d, "d2h_bytes_per_step": d2h},
        "gpu_launches": int(sum(v["launches"] for v in kern.values())) // max(1, args.steps) * args.steps,
        "roofline": roofline,
        "roofline_two_link": two_link,
        "roofline_hbm": roofline_hbm,
        "roofline_tier1_alone": tier1_alone,
    }
    if args.cpu_baseline:
        try:
            ncores = os.cpu_count() or 1
            n_groups = B * Hkv
            groups = _c3_groups(wl, ncores)
            span = min(oracle_parallel(groups, tau, eps, Hq // Hkv, 2))
            t_all = span * n_groups / len(groups)
            one = oracle_parallel(groups[:1], tau, eps, Hq // Hkv, 1)[0]
            line["cpu_baseline"] = {
                "value": B / t_all, "unit": UNIT, "cores": len(groups), "kind": "oracle", "nproc": ncores,
                "sample": (f"oracle decode of {len(groups)} (sequence, KV head) groups of {N}-token layers at "
                           f"once, one single-threaded process per group ({span:.2f} s), scaled to one layer"),
                "one_core": {"value": B / (one * n_groups), "unit": UNIT, "cores": 1,
                             "sample": f"1 of {n_groups} groups of one layer ({one:.2f} s), scaled to the layer"}}
        except Exception as e:  # pragma: no cover
            line["cpu_baseline"] = {"value": None, "unit": UNIT, "cores": 1, "kind": "oracle",
                                    "sample": f"failed: {e}"[:200]}
    line.update({
        "roofline_kernel_mixed_round0": host_roofline("mixed_round0") if "mixed_round0" in kern else None,
        "ladder_histogram": hist,
        "promoted_bytes_per_step": prom,
        "host_link": {"h2d_gbs_measured": h2d_gbs, "bytes_per_layer": host_bytes,
                      "floor_us_per_layer": prom / L / (h2d_gbs * 1e3) if h2d_gbs else None},
        "uncertified_baseline": uncertified,
        "kernels": kern,
        "fill_s": t_fill,
        "append": append,
    })
    cache.close()
    line["dense_fp16_hbm"] = measure_dense_hbm(args, wl, t_layer_us, 1e3 * unc_ms / L)
    line["fp16_values"] = measure_fp16_values(args, wl)
    line["residency"] = measure_residency(args, wl)
    line["configs"] = measure_configs(args, args.cpu_baseline)
    print(json.dumps(line), flush=True)
    if world > 1:
        dist.destroy_process_group()


C5_CTX = (4096, 8192, 16384, 32768, 65536, 131072)
C5_BATCH = (1, 8, 32)
C5_TAU = (0.99, 0.995, 0.999)


def sweep_c5(args):
    """Ladder sweep: one layer per (context, batch) point, keys with four x20 channels and
    values with four x8 channels per KV head, at three coverage targets.  One JSON line per
    (context, batch, tau_cov): time per decode call, the ladder histogram over the query
    heads, the promoted host-link bytes and the mean K*.  Inputs are drawn on the device
    (this sweep has no oracle leg)."""
    import torch
    import certified_quantized_kv_gb300 as kvq
    import workloads as W

    torch.cuda.set_device(int(os.environ.get("LOCAL_RANK", "0")))
    Hq, Hkv, D, eps = WORKLOAD["q_heads"], WORKLOAD["kv_heads"], WORKLOAD["head_dim"], WORKLOAD["eps"]
    ctxs = [args.ctx] if args.ctx else C5_CTX
    batches = [args.batch] if args.batch else C5_BATCH
    point = 0
    for N in ctxs:
        for B in batches:
            q, K, V = W.c5_point(N, B, device="cuda", seed=4 + point)
            point += 1
            cache = kvq.Cache(1, B, Hq, Hkv, max_ctx=N)
            cache.append(0, K, V)
            del K, V
            out = torch.empty(B, Hq, D, dtype=torch.float16, device="cuda")
            cert = torch.empty(B * Hq * 32, dtype=torch.uint8, device="cuda")
            lvl = torch.empty(B, dtype=torch.int32, device="cuda")
            for tau in C5_TAU:
                for _ in range(max(1, args.warmup)):
                    cache.decode(0, q, tau, eps, out, cert, lvl)
                times = []
                for _ in range(max(1, args.steps)):
                    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                    e0.record()
                    cache.decode(0, q, tau, eps, out, cert, lvl)
                    e1.record()
                    torch.cuda.synchronize()
                    times.append(e0.elapsed_time(e1))
                ms = sorted(times)[len(times) // 2]
                c = kvq.certificates(cert).reshape(B, Hq)
                hist = [int(x) for x in np.bincount(c["level"].ravel(), minlength=5)]
                prom = int(c["promoted_bytes"][:, :: Hq // Hkv].sum())
                print(json.dumps({
                    "sweep": "c5", "ctx": N, "batch": B, "tau_cov": tau, "eps": eps,
                    "ms_per_call": ms, "tokens_per_s_per_layer": B / (ms / 1e3),
                    "ladder_histogram": hist, "promoted_bytes": prom,
                    "promoted_fraction_of_tier2": prom / (B * Hkv * N * 2 * D * 2),
                    "host_gbs": prom / (ms / 1e3) / 1e9, "k_star_mean": float(c["k_star"].mean()),
                    "blocks": N // 64}), flush=True)
            cache.close()
            del q
            torch.cuda.empty_cache()


def decode_loop(args):
    """Token-by-token decode on the headline cache shape: every step appends one new
    token's K/V to each layer (quantiser + tier-2 mirror) and then decodes that layer's
    new query, as a serving loop does.  The cache is prefilled to ctx - warmup - steps
    tokens and ends at ctx.  Prints one JSON line."""
    import torch
    import certified_quantized_kv_gb300 as kvq
    import workloads as W

    torch.cuda.set_device(int(os.environ.get("LOCAL_RANK", "0")))
    wl = dict(WORKLOAD)
    B, L, N = args.batch or wl["batch"], args.layers or wl["layers"], args.ctx or wl["ctx"]
    Hq, Hkv, D, tau, eps = wl["q_heads"], wl["kv_heads"], wl["head_dim"], wl["tau_cov"], wl["eps"]
    T, Wm = args.steps, args.warmup
    n0 = N - T - Wm
    slots = int(args.resident * B * Hkv * (N // 64) * 2)   # a fraction of each layer's FP16 blocks
    cache = kvq.Cache(L, B, Hq, Hkv, max_ctx=N, resident_blocks=slots)
    for layer in range(L):
        _, K, V = W.c3_layer(layer, device="cuda", seed=wl["seed"], batch=B, ctx=n0, Hq=Hq, Hkv=Hkv)
        cache.append(layer, K.contiguous(), V.contiguous())
        del K, V
    gen = torch.Generator(device="cuda")
    gen.manual_seed(wl["seed"] + 77)
    steps = T + Wm
    knew = torch.randn(steps, L, B, Hkv, 1, D, generator=gen, device="cuda").half()
    vnew = torch.randn(steps, L, B, Hkv, 1, D, generator=gen, device="cuda").half()
    qnew = torch.randn(steps, L, B, Hq, D, generator=gen, device="cuda").half()
    out = torch.empty(B, Hq, D, dtype=torch.float16, device="cuda")
    cert = torch.empty(B * Hq * 32, dtype=torch.uint8, device="cuda")

    plan = kvq.RopePlan(D, **ROPE) if args.rope else None
    if plan:
        pos = torch.arange(n0, n0 + steps, dtype=torch.int32, device="cuda").repeat_interleave(B).reshape(steps, B)

    def step(t):
        for layer in range(L):
            q = qnew[t, layer]
            if plan:   # new tokens of a model's projections: rotated in place
                kvq.rope(q, pos[t], plan, out=q)
                k = knew[t, layer].squeeze(2)
                kvq.rope(k, pos[t], plan, out=k)
            cache.append(layer, knew[t, layer], vnew[t, layer])
            cache.decode(layer, q, tau, eps, out, cert)

    for t in range(Wm):
        step(t)
    torch.cuda.synchronize()
    for layer in range(L):
        cache.residency_stats(layer, reset=True)
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for t in range(Wm, steps):
        step(t)
    e1.record()
    torch.cuda.synchronize()
    ms = e0.elapsed_time(e1) / T
    rs = [cache.residency_stats(layer) for layer in range(L)]
    print(json.dumps({"mode": "decode_loop", "metric": "tokens/s/layer (append + certified decode per token)",
                      "value": B / (ms / L / 1e3), "ms_per_step": ms, "steps": T, "warmup": Wm,
                      "layers": L, "batch": B, "ctx_end": N, "tau_cov": tau, "eps": eps, "rope": bool(args.rope),
                      "resident_fraction": args.resident, "resident_blocks_per_layer": slots,
                      "host_bytes_per_step": sum(x["host_bytes"] for x in rs) / T if slots else None,
                      "resident_bytes_per_step": sum(x["resident_bytes"] for x in rs) / T if slots else None}),
          flush=True)
    cache.close()


def paged_loop(args):
    """The same loop on the paged 4-bit cache: every step turns a layer's new query and key by
    their position, appends the key and the value to its pages (one call) and attends over
    them (a second one).  The pool of pages lies in device memory, in shuffled order.  Prints
    one JSON line."""
    import torch
    import certified_quantized_kv_gb300 as kvq
    import workloads as W

    torch.cuda.set_device(int(os.environ.get("LOCAL_RANK", "0")))
    wl = dict(WORKLOAD)
    B, L, N = args.batch or wl["batch"], args.layers or wl["layers"], args.ctx or wl["ctx"]
    Hq, Hkv, D = wl["q_heads"], wl["kv_heads"], wl["head_dim"]
    T, Wm = args.steps, args.warmup
    steps = T + Wm
    n0, per = N - steps, -(-N // 64)
    plan = kvq.RopePlan(D, **ROPE)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(wl["seed"] + 77)
    table = torch.randperm(B * per, generator=gen, device="cuda").to(torch.int32).reshape(B, per)
    pools = [torch.empty(B * per, Hkv, kvq.paged_page_bytes(D), dtype=torch.uint8, device="cuda") for _ in range(L)]
    ws = torch.zeros(kvq.paged_attention_workspace(B, 1, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    at = torch.arange(N, device="cuda")
    slots = (table.long()[:, at // 64] * 64 + at % 64).to(torch.int32)           # [B, N]
    at = at.to(torch.int32)
    for layer in range(L):
        _, K, V = W.c3_layer(layer, device="cuda", seed=wl["seed"], batch=B, ctx=n0, Hq=Hq, Hkv=Hkv)
        for b in range(B):
            kvq.paged_append(pools[layer], K[b].transpose(0, 1), V[b].transpose(0, 1), slots[b, :n0].contiguous(),
                             positions=at[:n0], plan=plan)
        del K, V
    new = torch.randn(steps, L, B, Hq + 2 * Hkv, D, generator=gen, device="cuda").half()
    slot = [slots[:, n0 + t].contiguous() for t in range(steps)]
    pos = [torch.full((B,), n0 + t, dtype=torch.int32, device="cuda") for t in range(steps)]
    lens = [torch.full((B,), n0 + t + 1, dtype=torch.int32, device="cuda") for t in range(steps)]
    out = torch.empty(B, Hq, D, dtype=torch.float16, device="cuda")

    def step(t):
        for layer in range(L):
            x = new[t, layer]
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
            kvq.paged_append(pools[layer], k, v, slot[t], positions=pos[t], plan=plan, q=q, q_out=q)
            kvq.paged_attention(q, pools[layer], table, lens[t], out, workspace=ws)

    for t in range(Wm):
        step(t)
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for t in range(Wm, steps):
        step(t)
    e1.record()
    torch.cuda.synchronize()
    ms = e0.elapsed_time(e1) / T
    read = B * N * Hkv * (D + 8 * (D // 32))
    print(json.dumps({"mode": "paged_loop", "metric": "tokens/s/layer (append + attention over 4-bit pages per token)",
                      "value": B / (ms / L / 1e3), "ms_per_step": ms, "steps": T, "warmup": Wm, "layers": L, "batch": B,
                      "ctx_end": N, "page_bytes_read_per_layer": read, "page_gbs": read / (ms / L * 1e6)}), flush=True)


VTOL_SWEEP = (0.0, 0.2, 0.1, 0.05, 0.02)


def sweep_vtol(args):
    """Value-tolerance sweep on one layer of the headline workload: for each v_tol (0 = no
    budget beyond eps) the time per decode call, the ladder histogram, the paged-in bytes
    and the largest certified E_val."""
    import torch
    import certified_quantized_kv_gb300 as kvq
    import workloads as W

    torch.cuda.set_device(int(os.environ.get("LOCAL_RANK", "0")))
    wl = WORKLOAD
    B, N = args.batch or wl["batch"], args.ctx or wl["ctx"]
    Hq, Hkv, D, tau, eps = wl["q_heads"], wl["kv_heads"], wl["head_dim"], wl["tau_cov"], wl["eps"]
    q, K, V = W.c3_layer(0, device="cuda", seed=wl["seed"], batch=B, ctx=N, Hq=Hq, Hkv=Hkv)
    for v_tol in VTOL_SWEEP:
        cache = kvq.Cache(1, B, Hq, Hkv, max_ctx=N, v_tol=v_tol)
        cache.append(0, K, V)
        out = torch.empty(B, Hq, D, dtype=torch.float16, device="cuda")
        cert = torch.empty(B * Hq * 32, dtype=torch.uint8, device="cuda")
        for _ in range(max(1, args.warmup)):
            cache.decode(0, q, tau, eps, out, cert)
        times = []
        for _ in range(max(1, args.steps)):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            cache.decode(0, q, tau, eps, out, cert)
            e1.record()
            torch.cuda.synchronize()
            times.append(e0.elapsed_time(e1))
        ms = sorted(times)[len(times) // 2]
        c = kvq.certificates(cert).reshape(B, Hq)
        ok = c["level"] < 3
        print(json.dumps({
            "sweep": "vtol", "v_tol": v_tol, "ctx": N, "batch": B, "tau_cov": tau, "eps": eps,
            "ms_per_call": ms, "tokens_per_s_per_layer": B / (ms / 1e3),
            "ladder_histogram": [int(x) for x in np.bincount(c["level"].ravel(), minlength=5)],
            "promoted_bytes": int(c["promoted_bytes"][:, :: Hq // Hkv].sum()),
            "max_certified_e_val": float(c["e_val"][ok].max()) if ok.any() else None,
            "mean_certified_e_val": float(c["e_val"][ok].mean()) if ok.any() else None}), flush=True)
        cache.close()


def profile_layer(args):
    """A small fixed launch sequence for ncu captures (not a bench line): one 128K-token
    layer of the headline caches, quantised twice (two caches), then three certified,
    three uncertified and three dense-FP16-in-HBM decode calls on it.  Launch order:
    append_kernel x2; (score, select, mixed_kernel_r0, combine, mixed_kernel, combine,
    dense_kernel, finalize) x3; (score, select, tail_kernel, combine, finalize) x3;
    (dense_hbm_kernel, dense_hbm_combine_kernel) x3."""
    import torch
    import certified_quantized_kv_gb300 as kvq
    import workloads as W
    wl = WORKLOAD
    B, N, Hq, Hkv, D = wl["batch"], wl["ctx"], wl["q_heads"], wl["kv_heads"], wl["head_dim"]
    torch.cuda.set_device(0)
    q, K, V = W.c3_layer(0, device="cuda", seed=wl["seed"], batch=B, ctx=N, Hq=Hq, Hkv=Hkv)
    q, K, V = q.contiguous(), K.contiguous(), V.contiguous()
    first = kvq.Cache(1, B, Hq, Hkv, max_ctx=N)
    first.append(0, K, V)
    torch.cuda.synchronize()
    first.close()
    cache = kvq.Cache(1, B, Hq, Hkv, max_ctx=N)
    cache.append(0, K, V)
    out = torch.empty(B, Hq, D, dtype=torch.float16, device="cuda")
    for _ in range(3):
        cache.decode(0, q, wl["tau_cov"], wl["eps"], out)
    for _ in range(3):
        cache.decode_uncertified(0, q, out)
    ws = None
    for _ in range(3):
        ws = kvq.dense_attention(q, K, V, out, ws)
    torch.cuda.synchronize()
    cache.close()
    print(json.dumps({"profile_layer": "done", "workload": wl["name"] + " (layer 0)"}))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--warmup", type=int, default=10)
    ap.add_argument("--impl", default="ours", choices=["ours", "reference"])
    ap.add_argument("--layers", type=int, default=None, help="override the layer count (not the headline)")
    ap.add_argument("--ctx", type=int, default=None, help="override the context (not the headline)")
    ap.add_argument("--batch", type=int, default=None, help="override the batch (not the headline)")
    ap.add_argument("--no-cpu-baseline", dest="cpu_baseline", action="store_false")
    ap.add_argument("--resident", type=float, default=0.0,
                    help="with --loop: fraction of each layer's FP16 blocks kept resident in HBM")
    ap.add_argument("--loop", action="store_true",
                    help="token-by-token decode loop (append + decode per layer and step)")
    ap.add_argument("--cache", choices=["certified", "paged"], default="certified",
                    help="with --loop: the certified tiered cache, or the paged 4-bit cache in device memory")
    ap.add_argument("--rope", action="store_true",
                    help="with --loop on the certified cache: rotate each step's queries and keys first")
    ap.add_argument("--profile-layer", dest="profile_layer", action="store_true",
                    help="run the fixed launch sequence of profile_layer (for ncu captures) and exit")
    ap.add_argument("--sweep", choices=["c5", "vtol"], default=None,
                    help="run a sweep instead of the headline (one JSON line per point)")
    args = ap.parse_args()
    if args.sweep == "c5":
        sweep_c5(args)
        return
    if args.sweep == "vtol":
        sweep_vtol(args)
        return
    if args.loop:
        (paged_loop if args.cache == "paged" else decode_loop)(args)
        return
    if args.profile_layer:
        profile_layer(args)
        return
    wl = dict(WORKLOAD)
    for k in ("layers", "ctx", "batch"):
        v = getattr(args, k)
        if v is not None:
            wl[k] = v
            wl["name"] = f"c3_shape_custom_b{wl['batch']}_ctx{wl['ctx']}_{wl['layers']}l"
    if args.impl == "reference":
        reference_arm(args, wl)
    else:
        our_arm(args, wl)


if __name__ == "__main__":
    main()
