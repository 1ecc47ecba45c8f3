#!/usr/bin/env python
"""Benchmark of the packed-code weight-only GEMV/GEMM on B200 (one JSON line on rank 0).

Headline workload: decode of one token (M = 1) through the 36-layer Qwen3-4B-shaped body,
252 packed GEMVs back to back (v/up/down at 3 bits, the rest at 2 bits, fp16 block-256
scales), each module with its own seeded weights and a fresh seeded bf16 input. One step is
one pass over the body, captured in a CUDA graph. The packed body is 1.18 GB, larger than L2
(126 MB), so every step streams the weights from HBM.

Extra keys report the other rows of the path on the same synthetic recipe: the M = 8 body,
single-linear and per-module GEMVs, the prefill GEMM sweep (TFLOP/s), the ternary body and
the bf16 materializer. `--impl reference` times the fp64 CPU oracle on the host cores on a
bounded sample of the same workload instead.

Multi-GPU (torchrun): the path needs no exchange; each rank runs its own replica of the
body, the step time is the max over ranks and `value` is the aggregate over all ranks.
"""
from __future__ import annotations

import argparse
import json
import os
import statistics
import subprocess
import sys
import threading
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

METRIC = "decode GEMV HBM GB/s (% of 8 TB/s) & tokens/s; prefill GEMM TFLOP/s (% peak)"
E2E_QUARTERS = 4   # batched calls the end-to-end step splits the body into, to overlap host copies
HBM_FALLBACK_GBS, BF16_FALLBACK_TFLOPS = 6650.0, 1590.0


def parse_args():
    p = argparse.ArgumentParser()
    p.add_argument("--gpus", type=int, default=1)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--warmup", type=int, default=5)
    p.add_argument("--impl", choices=["wr", "reference"], default="wr")
    p.add_argument("--layers", type=int, default=36)
    p.add_argument("--tokens", type=int, default=1, help="decode tokens M of the headline body (1..8)")
    p.add_argument("--no-extras", action="store_true", help="headline body only")
    p.add_argument("--cpu-seconds", type=float, default=12.0, help="oracle sample budget (0: no CPU baseline)")
    p.add_argument("--case", default=None,
                   help="time one case alone and exit (for profiling): gemm:BITS:M:N:K, tgemm:M:N:K, or the ternary batched body tbody:M:LAYERS")
    return p.parse_args()


def peaks():
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        d = json.load(open(path))
        return float(d["hbm_gbs"]), float(d["bf16_tflops"]), float(d.get("bf16_tflops_sustained", d["bf16_tflops"])), "measured"
    except Exception:
        return HBM_FALLBACK_GBS, BF16_FALLBACK_TFLOPS, 1400.0, "fallback"


# ------------------------------------------------------------------------------ clocks

class ClockSampler:
    """nvidia-smi samples of SM clock and throttle reasons while the timed region runs."""
    FIELDS = ("clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, uuid: str | None):
        self.uuid, self.rows, self.proc = uuid, [], None

    def __enter__(self):
        cmd = ["nvidia-smi", f"--query-gpu={self.FIELDS}", "--format=csv,noheader,nounits", "-lms", "100"]
        if self.uuid:
            cmd += ["-i", self.uuid]
        try:
            self.proc = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
            self.thread = threading.Thread(target=self._read, daemon=True)
            self.thread.start()
            time.sleep(0.3)
        except Exception:
            self.proc = None
        return self

    def _read(self):
        for line in self.proc.stdout:
            self.rows.append([c.strip() for c in line.split(",")])

    def __exit__(self, *exc):
        if self.proc:
            time.sleep(0.2)
            self.proc.terminate()
            try:
                self.proc.wait(timeout=5)
            except Exception:
                self.proc.kill()

    def summary(self):
        sm, mx, reasons = [], [], set()
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for r in self.rows:
            try:
                sm.append(float(r[0]))
                mx.append(float(r[1]))
                for i, nm in enumerate(names):
                    if r[4 + i].lower().startswith("active"):
                        reasons.add(nm)
            except Exception:
                continue
        if not sm:
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["unsampled"], "samples": 0}
        return {"sm_mhz": statistics.median(sm), "sm_max_mhz": max(mx), "reasons": sorted(reasons),
                "samples": len(sm)}


# ------------------------------------------------------------------------------ workloads

def body_modules(layers: int):
    import wr_synth
    for layer in range(layers):
        for idx, (name, K, N, bits) in enumerate(wr_synth.QWEN3_4B_LAYER):
            yield layer, idx, name, K, N, bits


def build_q_module(wr, torch, seed, N, K, bits):
    import numpy as np
    import wr_synth
    W = wr_synth.weights_fp32(seed, N, K)
    codes, scales = wr.wr_quantize(bits, W)
    packed = wr.wr_pack(bits, codes)
    return (torch.from_numpy(packed).cuda(), torch.from_numpy(scales.view(np.int16)).cuda())


def module_bytes(wr, M, N, K, bits):
    fmt = bits
    return wr.wr_packed_bytes(fmt, N, K) + N * (K // 256) * 2 + M * K * 2 + M * N * 4


# DRAM traffic of the decode GEMV launch, (dram__bytes_read + dram__bytes_write) / algorithmic
# bytes, from one ncu capture of the current kernel at that token count (summary and command in
# profiles/). None: no capture of this kernel version, so no traffic figure is claimed.
# current kernel (weights copied with an L2 evict-first policy, activation tiles evict-last):
# M = 1 reads 1,181,419,520 and writes 3,914,240 bytes for 1,178,984,448 algorithmic; M = 8 reads
# 1,206,598,656 and writes 14,751,232 for 1,223,368,704 (part of y is still in L2 at the end)
_TRAFFIC_RATIO = {1: (1_181_419_520 + 3_914_240) / 1_178_984_448, 8: (1_206_598_656 + 14_751_232) / 1_223_368_704}


def split_ranges(n: int, parts: int):
    """Consecutive index ranges [(i0, i1), ...] that cover range(n) in at most `parts` pieces of
    ceil(n / parts) (the end-to-end step's batched calls)."""
    per = (n + parts - 1) // parts
    return [(i0, min(n, i0 + per)) for i0 in range(0, n, per)] if n > 0 else []


def traffic_per_launch(M: int, layers: int, algo_bytes: int):
    r = _TRAFFIC_RATIO.get(M)
    return None if r is None else int(r * algo_bytes)


def graph_time_ms(torch, fn, steps, warmup, stream, dist=None):
    """Capture fn() once in a CUDA graph; replay `warmup` times, then time `steps` replays with
    CUDA events recorded on the stream the replays are launched on, with a barrier and a
    device synchronize on both sides."""
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        fn()                                   # one eager pass (lazy init outside capture)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=stream):
            fn()
        for _ in range(warmup):
            g.replay()
        torch.cuda.synchronize()
        if dist:
            dist.barrier()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        assert torch.cuda.current_stream() == stream
        start.record(stream)
        for _ in range(steps):
            g.replay()
        end.record(stream)
        torch.cuda.synchronize()
    if dist:
        dist.barrier()
    ms = start.elapsed_time(end)
    del g
    return ms


def max_over_ranks(torch, dist, v, device="cuda"):
    """The slowest rank's time: every replica's device time, reduced with MAX."""
    if not dist:
        return v
    t = torch.tensor([v], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


# ------------------------------------------------------------------------------ reference arm

def cpu_model():
    try:
        for line in open("/proc/cpuinfo"):
            if line.startswith("model name"):
                return line.split(":", 1)[1].strip()
    except OSError:
        pass
    return "unknown"


def _oracle_run(budget_s: float, M: int):
    """One timed pass of the fp64 oracle over consecutive body modules until the budget is used:
    (GB/s over the algorithmic bytes, modules done, seconds)."""
    import wr_synth
    from oracle import wr_oracle as o
    done_bytes, t_total, mods = 0, 0.0, []
    for layer, idx, name, K, N, bits in body_modules(36):
        W = wr_synth.weights_fp32(wr_synth.module_seed(layer, idx), N, K)
        codes, scales = o.quantize_odd_grid(W, bits)
        x = wr_synth.activations_bf16(10_000 + 10 * layer + idx, M, K)
        t0 = time.perf_counter()
        o.gemm_codes(x, codes, scales, bits)
        t_total += time.perf_counter() - t0
        done_bytes += (o.packed_bytes(bits, N, K) + N * (K // 256) * 2 + M * K * 2 + M * N * 4)
        mods.append(f"L{layer}.{name}")
        if t_total >= budget_s:
            break
    return done_bytes / t_total / 1e9, mods, t_total


def cpu_oracle_sample(budget_s: float, M: int = 1):
    """The oracle as it stands, timed on this host's cores: three runs with numpy's thread pool
    limited to one thread and three with all cores, each over consecutive body modules for about
    budget_s / 6 seconds of CPU time; the medians are reported (GB/s over the same algorithmic
    bytes as the GPU step)."""
    import numpy  # noqa: F401  (loads the BLAS whose thread pool is reported)
    from threadpoolctl import threadpool_info, threadpool_limits
    cores = max([d.get("num_threads", 1) for d in threadpool_info()] + [1])
    per = max(0.3, budget_s / 6.0)
    single, allc, mods_all, secs = [], [], [], 0.0
    with threadpool_limits(limits=1):
        for _ in range(3):
            v, _, t = _oracle_run(per, M)
            single.append(v)
            secs += t
    for _ in range(3):
        v, mods, t = _oracle_run(per, M)
        allc.append(v)
        mods_all = mods
        secs += t
    return {"value": statistics.median(allc), "unit": "GB/s", "cores": cores, "kind": "oracle",
            "single_thread": {"value": statistics.median(single), "unit": "GB/s", "cores": 1},
            "cpu_model": cpu_model(), "nproc": os.cpu_count(),
            "sample": f"median of 3 runs per thread count; each run times the fp64 oracle (dequant + "
                      f"matmul) over consecutive body modules at M={M} for ~{per:.1f} s "
                      f"(all-core run: {len(mods_all)} modules, {mods_all[0]}..{mods_all[-1]}); "
                      f"{secs:.1f} s of CPU time in all"}


def run_reference(args, rank, world):
    if rank != 0:
        return
    per_step = []
    for _ in range(args.warmup):
        _oracle_run(0.3, 1)
    for _ in range(args.steps):
        per_step.append(_oracle_run(max(0.5, args.cpu_seconds / max(args.steps, 1)), 1)[0])
    gbs = statistics.median(per_step)
    tokps = gbs * 1e9 / 1_178_984_448
    cb = cpu_oracle_sample(args.cpu_seconds)
    cb["value"] = gbs
    cb["sample"] = (f"each step: the fp64 oracle over consecutive body modules at M=1 for "
                    f"~{max(0.5, args.cpu_seconds / max(args.steps, 1)):.1f} s (median of the steps, all cores); "
                    "single_thread: " + cb["sample"])
    line = {"impl": "reference", "metric": METRIC, "value": gbs, "unit": "GB/s", "n_gpus": args.gpus,
            "steps": args.steps, "warmup": args.warmup, "ms_per_step": 1e3 / tokps,
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64",
            "data": "synthetic", "tokens_per_s": tokps,
            "config": {"workload": "qwen3-4b body, 36 layers x 7 packed GEMVs, M=1 (oracle sample)",
                       "model": "Qwen3-4B-shaped linears", "global_batch": 1, "seq_len": 1,
                       "parallelism": "replicas"},
            "cpu_baseline": cb,
            "e2e": {"value": gbs, "unit": "GB/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0}}
    print(json.dumps(line), flush=True)


# ------------------------------------------------------------------------------ main arm

def main():
    args = parse_args()
    rank, world = int(os.environ.get("RANK", 0)), int(os.environ.get("WORLD_SIZE", 1))
    local_rank = int(os.environ.get("LOCAL_RANK", 0))
    if world > 1:
        os.environ["CUDA_VISIBLE_DEVICES"] = str(local_rank)
    if args.impl == "reference":
        run_reference(args, rank, world)
        return
    import numpy as np
    import torch
    import bit_weight_only_wr_b200 as wr
    import wr_synth

    torch.cuda.set_device(0)
    dist = None
    if world > 1:
        import datetime
        import torch.distributed as tdist
        tdist.init_process_group("nccl", timeout=datetime.timedelta(seconds=120),
                                 device_id=torch.device("cuda", 0))
        dist = tdist
    hbm_peak, bf16_peak, bf16_sust, peak_kind = peaks()
    stream = torch.cuda.Stream()
    uuid = None
    try:
        uuid = str(torch.cuda.get_device_properties(0).uuid)
        uuid = uuid if uuid.startswith("GPU-") else "GPU-" + uuid
    except Exception:
        pass

    if args.case:
        run_case(args, wr, torch, np, stream, bf16_peak)
        return

    # ---- the body: weights resident in HBM, fresh x per module
    t_setup = time.time()
    mods = []
    for layer, idx, name, K, N, bits in body_modules(args.layers):
        packed, scales = build_q_module(wr, torch, wr_synth.module_seed(layer, idx), N, K, bits)
        mods.append(dict(layer=layer, name=name, K=K, N=N, bits=bits, packed=packed, scales=scales))
    setup_s = time.time() - t_setup

    def body_run(M, steps, warmup, with_e2e, batched=True):
        xs_host = [wr_synth.activations_bf16(10_000 + 10 * m["layer"] + i % 7, M, m["K"])
                   for i, m in enumerate(mods)]
        x_all = torch.from_numpy(np.concatenate([x.ravel() for x in xs_host]).view(np.int16)).cuda()
        offs, o_ = [], 0
        for x in xs_host:
            offs.append(o_)
            o_ += x.size
        y_all = torch.empty(sum(M * m["N"] for m in mods), dtype=torch.float32, device="cuda")
        yoffs, o_ = [], 0
        for m in mods:
            yoffs.append(o_)
            o_ += M * m["N"]
        xp, yp = x_all.data_ptr(), y_all.data_ptr()
        if batched:
            # the whole body: one launch of the batched decode GEMV per token
            arr = wr._problems([(xp + 2 * offs[i], m["packed"], m["scales"], yp + 4 * yoffs[i], m["N"], m["K"],
                                 m["bits"]) for i, m in enumerate(mods)])
            nb = wr.wr_gemv_batched_workspace_bytes(M, arr)
            ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
            launches = 2 * ((len(mods) + 255) // 256)   # preparation pass + decode GEMV per batch

            def step():
                wr.wr_gemv_batched(M, arr, ws, nb)
        else:
            nb = max(wr.wr_gemv_workspace_bytes(M, m["N"], m["K"], m["bits"]) for m in mods)
            ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
            launches = 2 * len(mods)

            def step():
                for i, m in enumerate(mods):
                    wr.wr_gemv(M, m["N"], m["K"], xp + 2 * offs[i], m["packed"], m["scales"], m["bits"],
                               yp + 4 * yoffs[i], ws, nb)
        ms = graph_time_ms(torch, step, steps, warmup, stream, dist) / steps
        ms = max_over_ranks(torch, dist, ms)
        nbytes = sum(module_bytes(wr, M, m["N"], m["K"], m["bits"]) for m in mods)
        out = {"ms": ms, "bytes": nbytes, "gbs": nbytes / ms / 1e6, "launches": launches}
        if with_e2e:
            # end to end from pinned host memory: the body in layer quarters, each one batched
            # call; a quarter's x is copied in and its y copied out on side streams, so that the
            # host transfers overlap the decode of the other quarters (every step moves all of x
            # in and all of y out)
            xh = x_all.cpu().pin_memory()
            yh = torch.empty(y_all.numel(), dtype=torch.float32).pin_memory()
            quarters = []
            for i0, i1 in split_ranges(len(mods), E2E_QUARTERS):
                xo0, xo1 = offs[i0], (offs[i1] if i1 < len(mods) else x_all.numel())
                yo0, yo1 = yoffs[i0], (yoffs[i1] if i1 < len(mods) else y_all.numel())
                arr_q = wr._problems([(xp + 2 * offs[i], mods[i]["packed"], mods[i]["scales"], yp + 4 * yoffs[i],
                                       mods[i]["N"], mods[i]["K"], mods[i]["bits"]) for i in range(i0, i1)])
                quarters.append((xo0, xo1, yo0, yo1, arr_q, wr.wr_gemv_batched_workspace_bytes(M, arr_q)))
            nbq = max(q[5] for q in quarters)
            wsq = torch.zeros(nbq, dtype=torch.uint8, device="cuda")   # the quarters run in turn on one stream
            s_in, s_out = torch.cuda.Stream(), torch.cuda.Stream()
            ev_in = [torch.cuda.Event() for _ in quarters]
            ev_done = [torch.cuda.Event() for _ in quarters]

            def e2e_step():
                main = torch.cuda.current_stream()
                s_in.wait_stream(main)
                s_out.wait_stream(main)
                with torch.cuda.stream(s_in):
                    for (xo0, xo1, *_r), ev in zip(quarters, ev_in):
                        x_all[xo0:xo1].copy_(xh[xo0:xo1], non_blocking=True)
                        ev.record(s_in)
                for (_, _, yo0, yo1, arr_q, _), ei, ed in zip(quarters, ev_in, ev_done):
                    main.wait_event(ei)
                    wr.wr_gemv_batched(M, arr_q, wsq, nbq)
                    ed.record(main)
                    with torch.cuda.stream(s_out):
                        s_out.wait_event(ed)
                        yh[yo0:yo1].copy_(y_all[yo0:yo1], non_blocking=True)
                main.wait_stream(s_in)
                main.wait_stream(s_out)
            ms_e = graph_time_ms(torch, e2e_step, steps, warmup, stream, dist) / steps
            ms_e = max_over_ranks(torch, dist, ms_e)
            out["e2e"] = {"ms": ms_e, "gbs": nbytes / ms_e / 1e6, "h2d": x_all.numel() * 2,
                          "d2h": y_all.numel() * 4, "calls": len(quarters)}
        return out

    def dependent_body_run(M, steps, warmup):
        """The body as a decoder whose layers depend on each other issues it: per layer four
        calls in order, each a wr_gemv_grouped over the linears that read one input (q/k/v on the
        attention input, o, gate/up on the MLP input, down), with fresh seeded inputs standing in
        for the outputs of attention and the MLP activation; no launch spans two layers."""
        groups = [("qkv", (0, 1, 2)), ("o", (3,)), ("gate_up", (4, 5)), ("down", (6,))]
        calls, keep, nbytes, nb = [], [], 0, 0
        for layer in range(args.layers):
            lm = mods[7 * layer:7 * layer + 7]
            for gi, (gname, idxs) in enumerate(groups):
                K = lm[idxs[0]]["K"]
                x = torch.from_numpy(wr_synth.activations_bf16(20_000 + 10 * layer + gi, M, K).view(np.int16)).cuda()
                ys = [torch.empty(M, lm[i]["N"], dtype=torch.float32, device="cuda") for i in idxs]
                arr = wr._gitems([(lm[i]["packed"], lm[i]["scales"], y, lm[i]["N"], lm[i]["bits"])
                                  for i, y in zip(idxs, ys)])
                nb = max(nb, wr.wr_gemv_grouped_workspace_bytes(M, K, arr))
                calls.append((K, x, arr))
                keep += ys
                nbytes += 2 * M * K + sum(wr.wr_packed_bytes(lm[i]["bits"], lm[i]["N"], K) + lm[i]["N"] * (K // 256) * 2
                                          + 4 * M * lm[i]["N"] for i in idxs)
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")

        def step():
            for K, x, arr in calls:
                wr.wr_gemv_grouped(M, K, x, arr, ws, nb)
        ms = graph_time_ms(torch, step, steps, warmup, stream, dist) / steps
        ms = max_over_ranks(torch, dist, ms)
        return {"ms": ms, "bytes": nbytes, "gbs": nbytes / ms / 1e6, "frac_of_hbm": nbytes / ms / 1e6 / hbm_peak,
                "tokens_per_s": M * 1e3 / ms, "calls": len(calls), "launches": 2 * len(calls)}

    with ClockSampler(uuid) as clk:
        head = body_run(args.tokens, args.steps, args.warmup, True)
    clocks = clk.summary()
    total_gbs = head["gbs"] * world
    tokens_per_s = world * args.tokens * 1e3 / head["ms"]

    extras = {}
    if not args.no_extras:
        try:
            extras["body_m8"] = {k: v for k, v in body_run(8, max(5, args.steps // 2), 3, False).items()}
            extras["body_m8"]["tokens_per_s"] = 8e3 / extras["body_m8"]["ms"]
        except Exception as e:  # noqa: BLE001
            extras["body_m8"] = {"error": repr(e)}
        for M in (16, 32):
            # a 16- or 32-token chunk through the body, one batched call: the decode kernel's
            # 64- and 128-column forms
            try:
                extras[f"body_m{M}"] = body_run(M, max(5, args.steps // 2), 3, False)
                extras[f"body_m{M}"]["tokens_per_s"] = M * 1e3 / extras[f"body_m{M}"]["ms"]
                extras[f"body_m{M}"]["frac_of_hbm"] = extras[f"body_m{M}"]["gbs"] / hbm_peak
            except Exception as e:  # noqa: BLE001
                extras[f"body_m{M}"] = {"error": repr(e)}
        try:
            extras["body_m1_one_call_per_linear"] = body_run(1, max(5, args.steps // 2), 3, False, batched=False)
        except Exception as e:  # noqa: BLE001
            extras["body_m1_one_call_per_linear"] = {"error": repr(e)}
        for M in (1, 8):
            try:
                extras[f"body_dependent_grouped_m{M}"] = dependent_body_run(M, max(5, args.steps // 2), 3)
            except Exception as e:  # noqa: BLE001
                extras[f"body_dependent_grouped_m{M}"] = {"error": repr(e)}
        extras.update(run_extras(args, wr, torch, np, stream, dist, hbm_peak, bf16_peak))

    # the step is one wr_gemv_batched call: the preparation pass, then one launch of the decode
    # GEMV kernel over all 252 problems (about 96% of the two kernels' time in the ncu launch
    # list); achieved = algorithmic bytes of the launch / event-timed duration of the whole call
    achieved = head["gbs"]
    roof = {"bound": "hbm", "achieved": achieved, "peak": hbm_peak, "unit": "GB/s",
            "frac": achieved / hbm_peak, "traffic": traffic_per_launch(args.tokens, args.layers, head["bytes"]),
            "peak_kind": peak_kind,
            "kernel": "gemv_q_kernel (batched 2/3-bit decode GEMV on tcgen05 kind::i8), after prep_x_kernel",
            "note": "algorithmic bytes per launch (packed codes + fp16 scales + bf16 x + fp32 y) / CUDA-event "
                    "duration of the call (preparation pass + GEMV launch), inside the timed region"}
    cb = None
    if rank == 0 and world == 1 and args.cpu_seconds > 0:
        try:
            cb = cpu_oracle_sample(args.cpu_seconds)
        except Exception as e:  # noqa: BLE001
            cb = {"error": repr(e)}
    line = {
        "metric": METRIC, "value": total_gbs, "unit": "GB/s", "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": head["ms"], "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "i8", "data": "synthetic",
        "dtype_note": "int8 tensor-core products of the codes and four int8 limbs of each bf16 activation, "
                      "int32 accumulators, fp32 epilogue; y is fp32",
        "tokens_per_s": tokens_per_s, "pct_of_8TBps": 100.0 * head["gbs"] / 8000.0,
        "config": {"workload": f"qwen3-4b body, {args.layers} layers x 7 packed GEMVs (v/up/down 3-bit, "
                               "others 2-bit, fp16 block-256 scales), M=%d decode" % args.tokens,
                   "model": "Qwen3-4B-shaped linears (synthetic, W~N(0,0.02), x~N(0,1) bf16)",
                   "global_batch": world * args.tokens, "seq_len": 1, "parallelism": f"replicas x{world}",
                   "l2": "inputs larger than L2 (1.18 GB of packed weights per step)",
                   "bytes_per_step": head["bytes"], "setup_s": round(setup_s, 1)},
        "roofline": roof, "cpu_baseline": cb, "clocks": clocks,
        "e2e": {"value": head["e2e"]["gbs"] * world, "unit": "GB/s",
                "h2d_bytes_per_step": head["e2e"]["h2d"], "d2h_bytes_per_step": head["e2e"]["d2h"],
                "ms_per_step": head["e2e"]["ms"], "calls_per_step": head["e2e"]["calls"]},
        "gpu_launches": head["launches"] * args.steps,
        "step": f"{7 * args.layers} linears ({args.layers} layers x 7) in one wr_gemv_batched call "
                "(preparation pass + decode GEMV launch), CUDA graph replay",
        "extras": extras,
    }
    if rank == 0:
        print(json.dumps(line), flush=True)
    if dist:
        dist.barrier()
        dist.destroy_process_group()


def run_case(args, wr, torch, np, stream, bf16_peak):
    """One prefill GEMM shape alone, `--warmup` + `--steps` calls in a graph: a small, single-kernel
    command for profilers."""
    import wr_synth
    kind, *dims = args.case.split(":")
    if kind == "gemm":
        bits, M, N, K = (int(v) for v in dims)
        p, s = build_q_module(wr, torch, 5000 + K, N, K, bits)
        nb = wr.wr_gemm_workspace_bytes(M, N, K, bits)
        call = lambda x, y, ws: wr.wr_gemm(M, N, K, x, p, s, bits, y, ws, nb)  # noqa: E731
    elif kind == "tgemm":
        M, N, K = (int(v) for v in dims)
        signs = wr_synth.sign_bits(900, K)
        codes, alpha = wr.wr_quantize_ternary(wr_synth.weights_fp32(800, N, K), signs)
        p = torch.from_numpy(wr.wr_pack(1, codes)).cuda()
        a = torch.from_numpy(alpha.view(np.int16)).cuda()
        sg = torch.from_numpy(signs.view(np.int32)).cuda()
        nb = wr.wr_gemm_ternary_workspace_bytes(M, N, K)
        call = lambda x, y, ws: wr.wr_gemm_ternary(M, N, K, x, p, a, sg, y, ws, nb)  # noqa: E731
    elif kind == "tbody":
        # the ternary body: `layers` copies of one quantized layer's 7 linears, one batched call
        M, layers = (int(v) for v in dims)
        mods = []
        for idx, (_, K, N, _) in enumerate(wr_synth.QWEN3_4B_LAYER):
            signs = wr_synth.sign_bits(900 + idx, K)
            codes, alpha = wr.wr_quantize_ternary(wr_synth.weights_fp32(800 + idx, N, K), signs)
            mods.append((K, N, torch.from_numpy(wr.wr_pack(1, codes)).cuda(),
                         torch.from_numpy(alpha.view(np.int16)).cuda(), torch.from_numpy(signs.view(np.int32)).cuda()))
        body = [(K, N, p.roll(c * 4096), a, sg) for c in range(layers) for (K, N, p, a, sg) in mods]
        xs = [torch.from_numpy(wr_synth.activations_bf16(3000 + j, M, K).view(np.int16)).cuda()
              for j, (K, _, _, _, _) in enumerate(body)]
        ys = [torch.empty(M, N, dtype=torch.float32, device="cuda") for (_, N, _, _, _) in body]
        arr = wr._tproblems([(xs[j], p, a, sg, ys[j], N, K) for j, (K, N, p, a, sg) in enumerate(body)])
        nb = wr.wr_gemv_ternary_batched_workspace_bytes(M, arr)
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        ms = graph_time_ms(torch, lambda: wr.wr_gemv_ternary_batched(M, arr, ws, nb), args.steps, args.warmup,
                           stream) / args.steps
        b = sum(p.numel() + 2 * N + 4 * ((K + 31) // 32) + 2 * M * K + 4 * M * N for (K, N, p, _, _) in body)
        print(json.dumps({"case": args.case, "us": ms * 1e3, "gbs": b / ms / 1e6, "bytes": b}))
        return
    else:
        raise SystemExit(f"unknown --case {args.case!r}")
    x = torch.from_numpy(wr_synth.activations_bf16(M, M, K).view(np.int16)).cuda()
    y = torch.empty(M, N, dtype=torch.float32, device="cuda")
    ws = torch.zeros(max(nb, 256), dtype=torch.uint8, device="cuda")
    ms = graph_time_ms(torch, lambda: call(x, y, ws), args.steps, args.warmup, stream) / args.steps
    tf = 2.0 * M * N * K / ms / 1e9
    print(json.dumps({"case": args.case, "us": ms * 1e3, "tflops": tf, "pct_bf16_peak": 100 * tf / bf16_peak}))


def run_extras(args, wr, torch, np, stream, dist, hbm_peak, bf16_peak):
    """Other rows of the path: per-module GEMVs over rotating copies, single linear, unpack,
    prefill GEMM sweep and the ternary body."""
    import wr_synth
    out = {}
    l2 = torch.cuda.get_device_properties(0).L2_cache_size

    # config 0: single 2560x2560 2-bit linear, M=1, rotating over >= 3x L2 of distinct copies
    try:
        N = K = 2560
        per = wr.wr_packed_bytes(2, N, K) + N * (K // 256) * 2
        copies = max(3, int(3 * l2 // per) + 1)
        base_p, base_s = build_q_module(wr, torch, 0, N, K, 2)
        ps = [base_p.roll(i * 1024) for i in range(copies)]      # distinct buffers, same statistics
        x = torch.from_numpy(wr_synth.activations_bf16(1, 1, K).view(np.int16)).cuda()
        y = torch.empty(1, N, dtype=torch.float32, device="cuda")
        nb = wr.wr_gemv_workspace_bytes(1, N, K, 2)
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")

        def step():
            for p in ps:
                wr.wr_gemv(1, N, K, x, p, base_s, 2, y, ws, nb)
        ms = graph_time_ms(torch, step, 10, 3, stream) / 10 / copies
        b = module_bytes(wr, 1, N, K, 2)
        out["single_linear_2560"] = {"us": ms * 1e3, "gbs": b / ms / 1e6, "bytes": b, "copies": copies}
    except Exception as e:  # noqa: BLE001
        out["single_linear_2560"] = {"error": repr(e)}

    # unpack (materializer) on the gate shape, rotating copies
    try:
        N, K = 9728, 2560
        p, s = build_q_module(wr, torch, 7, N, K, 2)
        w = torch.empty(N, K, dtype=torch.int16, device="cuda")

        def step():
            wr.wr_unpack_bf16(2, N, K, p, s, w)
        ms = graph_time_ms(torch, step, 20, 3, stream) / 20
        b = wr.wr_packed_bytes(2, N, K) + N * (K // 256) * 2 + N * K * 2
        out["unpack_bf16_gate"] = {"us": ms * 1e3, "gbs": b / ms / 1e6}
    except Exception as e:  # noqa: BLE001
        out["unpack_bf16_gate"] = {"error": repr(e)}

    # the 2-bit trellis-coded format: one layer's 7 linears encoded once (Viterbi, host), the
    # 36-layer body made of 36 distinct byte copies, one batched decode GEMV call per token
    try:
        res = {}
        tmods = []
        for idx, (name, K, N, _) in enumerate(wr_synth.QWEN3_4B_LAYER):
            sym, sc = wr.wr_quantize_trellis(wr_synth.weights_fp32(600 + idx, N, K))
            tmods.append((K, N, torch.from_numpy(wr.wr_pack(wr.WR_FMT_T2, sym)).cuda(),
                          torch.from_numpy(sc.view(np.int16)).cuda()))
        body = [(K, N, p.roll(c * 4096), sc) for c in range(36) for (K, N, p, sc) in tmods]
        for M in (1, 8):
            xs = [torch.from_numpy(wr_synth.activations_bf16(5000 + j, M, K).view(np.int16)).cuda()
                  for j, (K, _, _, _) in enumerate(body)]
            ys = [torch.empty(M, N, dtype=torch.float32, device="cuda") for (_, N, _, _) in body]
            arr = wr._problems([(xs[j], p, sc, ys[j], N, K, wr.WR_FMT_T2) for j, (K, N, p, sc) in enumerate(body)])
            nb = wr.wr_gemv_batched_workspace_bytes(M, arr)
            ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")

            def tstep():
                wr.wr_gemv_batched(M, arr, ws, nb)
            ms = graph_time_ms(torch, tstep, 10, 3, stream) / 10
            b = sum(p.numel() + 2 * N * (K // 256) + 2 * M * K + 4 * M * N for (K, N, p, _) in body)
            res[f"body_M{M}"] = {"ms": ms, "bytes": b, "gbs": b / ms / 1e6, "tokens_per_s": M * 1e3 / ms}
        out["trellis2"] = res
    except Exception as e:  # noqa: BLE001
        out["trellis2"] = {"error": repr(e)}

    # the 8-state trellis over 4-weight symbols: one layer's 7 linears encoded once (Viterbi,
    # host), the 36-layer body made of 36 distinct byte copies, one batched decode GEMV call
    try:
        res = {}
        tmods = []
        for idx, (name, K, N, _) in enumerate(wr_synth.QWEN3_4B_LAYER):
            c8, sc = wr.wr_quantize_trellis8(wr_synth.weights_fp32(650 + idx, N, K))
            tmods.append((K, N, torch.from_numpy(wr.wr_pack(wr.WR_FMT_T8, c8)).cuda(),
                          torch.from_numpy(sc.view(np.int16)).cuda()))
        body = [(K, N, p.roll(c * 4096), sc) for c in range(36) for (K, N, p, sc) in tmods]
        for M in (1, 8):
            xs = [torch.from_numpy(wr_synth.activations_bf16(5500 + j, M, K).view(np.int16)).cuda()
                  for j, (K, _, _, _) in enumerate(body)]
            ys = [torch.empty(M, N, dtype=torch.float32, device="cuda") for (_, N, _, _) in body]
            arr = wr._problems([(xs[j], p, sc, ys[j], N, K, wr.WR_FMT_T8) for j, (K, N, p, sc) in enumerate(body)])
            nb = wr.wr_gemv_batched_workspace_bytes(M, arr)
            ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")

            def t8step():
                wr.wr_gemv_batched(M, arr, ws, nb)
            ms = graph_time_ms(torch, t8step, 10, 3, stream) / 10
            b = sum(p.numel() + 2 * N * (K // 256) + 2 * M * K + 4 * M * N for (K, N, p, _) in body)
            res[f"body_M{M}"] = {"ms": ms, "bytes": b, "gbs": b / ms / 1e6, "tokens_per_s": M * 1e3 / ms}
        out["trellis8"] = res
    except Exception as e:  # noqa: BLE001
        out["trellis8"] = {"error": repr(e)}

    # int8 block scales (fp16 row scale times an int8 multiplier per 256-block): one layer's 7
    # linears quantized once by the device quantizer, the 36-layer body made of 36 distinct byte
    # copies, one batched decode GEMV call per token
    try:
        res = {}
        smods = []
        for idx, (name, K, N, bits) in enumerate(wr_synth.QWEN3_4B_LAYER):
            fmt = bits | wr.WR_SCALES_I8
            W = torch.from_numpy(wr_synth.weights_fp32(700 + idx, N, K)).cuda()
            pk = torch.empty(wr.wr_packed_bytes(bits, N, K), dtype=torch.uint8, device="cuda")
            rec = torch.zeros(wr.wr_scales_bytes(fmt, N, K), dtype=torch.uint8, device="cuda")
            wr.wr_quantize_pack(fmt, N, K, W, pk, rec)
            torch.cuda.synchronize()
            del W
            smods.append((K, N, fmt, pk, rec))
        body = [(K, N, fmt, p.roll(c * 4096), r.clone()) for c in range(36) for (K, N, fmt, p, r) in smods]
        for M in (1, 8):
            xs = [torch.from_numpy(wr_synth.activations_bf16(6000 + j, M, K).view(np.int16)).cuda()
                  for j, (K, _, _, _, _) in enumerate(body)]
            ys = [torch.empty(M, N, dtype=torch.float32, device="cuda") for (_, N, _, _, _) in body]
            arr = wr._problems([(xs[j], p, r, ys[j], N, K, fmt) for j, (K, N, fmt, p, r) in enumerate(body)])
            nb = wr.wr_gemv_batched_workspace_bytes(M, arr)
            ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")

            def sstep():
                wr.wr_gemv_batched(M, arr, ws, nb)
            ms = graph_time_ms(torch, sstep, 10, 3, stream) / 10
            b = sum(p.numel() + 2 * N + N * (K // 256) + 2 * M * K + 4 * M * N for (K, N, _, p, _) in body)
            res[f"body_M{M}"] = {"ms": ms, "bytes": b, "gbs": b / ms / 1e6, "tokens_per_s": M * 1e3 / ms}
        out["scales_i8"] = res
    except Exception as e:  # noqa: BLE001
        out["scales_i8"] = {"error": repr(e)}

    # device quantizer + packer (fp32 W -> packed codes + fp16 scales) on the gate and up shapes
    try:
        res = {}
        for name, bits in (("gate", 2), ("up", 3)):
            N, K = 9728, 2560
            W = torch.from_numpy(wr_synth.weights_fp32(7 + bits, N, K)).cuda()
            pk = torch.empty(wr.wr_packed_bytes(bits, N, K), dtype=torch.uint8, device="cuda")
            sc = torch.empty(N * (K // 256), dtype=torch.int16, device="cuda")

            def step():
                wr.wr_quantize_pack(bits, N, K, W, pk, sc)
            ms = graph_time_ms(torch, step, 20, 3, stream) / 20
            b = 4 * N * K + wr.wr_packed_bytes(bits, N, K) + 2 * N * (K // 256)
            res[name] = {"us": ms * 1e3, "gbs": b / ms / 1e6, "bytes": b}
            # int8 block scales: a row pass over W, then the pack pass (W is read twice)
            fmt = bits | wr.WR_SCALES_I8
            rec = torch.zeros(wr.wr_scales_bytes(fmt, N, K), dtype=torch.uint8, device="cuda")

            def step8():
                wr.wr_quantize_pack(fmt, N, K, W, pk, rec)
            ms = graph_time_ms(torch, step8, 20, 3, stream) / 20
            b = 4 * N * K + wr.wr_packed_bytes(bits, N, K) + 2 * N + N * (K // 256)
            res[name + "_i8"] = {"us": ms * 1e3, "gbs": b / ms / 1e6, "bytes": b, "w_reads": 2}
        out["quantize_pack"] = res
    except Exception as e:  # noqa: BLE001
        out["quantize_pack"] = {"error": repr(e)}

    # prefill sweep: R calls back to back inside one CUDA graph (so that a replay's launch cost is
    # not charged to one short kernel), cycling over R distinct copies of the packed weights
    # whose total exceeds 3x L2
    try:
        res = {}
        shapes = [("gate", 2560, 9728, 2), ("up", 2560, 9728, 3), ("down", 9728, 2560, 3)]
        for name, K, N, bits in shapes:
            p, s = build_q_module(wr, torch, 5000 + K, N, K, bits)
            R = max(8, int(3 * l2 // p.numel()) + 1)
            ps = [p.roll(i * 1024) for i in range(R)]          # distinct buffers, same format
            for M in (16, 32, 128, 512, 2048, 4096):
                x = torch.from_numpy(wr_synth.activations_bf16(M, M, K).view(np.int16)).cuda()
                y = torch.empty(M, N, dtype=torch.float32, device="cuda")
                nb = wr.wr_gemm_workspace_bytes(M, N, K, bits)
                ws = torch.zeros(max(nb, 256), dtype=torch.uint8, device="cuda")

                def step():
                    for pc in ps:
                        wr.wr_gemm(M, N, K, x, pc, s, bits, y, ws, nb)
                reps = 2 if M >= 2048 else 5
                ms = graph_time_ms(torch, step, reps, 3, stream) / reps / R
                tf = 2.0 * M * N * K / ms / 1e9
                b = module_bytes(wr, M, N, K, bits)
                res[f"{name}_M{M}"] = {"us": ms * 1e3, "tflops": tf, "pct_bf16_peak": 100 * tf / bf16_peak,
                                       "gbs": b / ms / 1e6, "calls_per_graph": R}
            del ps
        out["prefill"] = res
    except Exception as e:  # noqa: BLE001
        out["prefill"] = {"error": repr(e)}

    # ternary: one layer's 7 shapes at M=1 (rotating over 6 copies of the layer > L2)
    try:
        mods = []
        for idx, (name, K, N, _) in enumerate(wr_synth.QWEN3_4B_LAYER):
            signs = wr_synth.sign_bits(900 + idx, K)
            W = wr_synth.weights_fp32(800 + idx, N, K)
            codes, alpha = wr.wr_quantize_ternary(W, signs)
            packed = wr.wr_pack(1, codes)
            mods.append(dict(K=K, N=N, p=torch.from_numpy(packed).cuda(),
                             a=torch.from_numpy(alpha.view(np.int16)).cuda(),
                             s=torch.from_numpy(signs.view(np.int32)).cuda()))
        per_layer = sum(m["p"].numel() for m in mods)
        copies = max(1, int(3 * l2 // per_layer) + 1)
        res = {}
        for M in (1, 512):
            xs = [torch.from_numpy(wr_synth.activations_bf16(M + i, M, m["K"]).view(np.int16)).cuda()
                  for i, m in enumerate(mods)]
            ys = [torch.empty(M, m["N"], dtype=torch.float32, device="cuda") for m in mods]
            nb = max(wr.wr_gemm_ternary_workspace_bytes(M, m["N"], m["K"]) for m in mods)
            ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
            rolled = [[m["p"].roll(c * 1024) for m in mods] for c in range(copies if M == 1 else 1)]

            def step():
                for c in range(len(rolled)):
                    for i, m in enumerate(mods):
                        wr.wr_gemm_ternary(M, m["N"], m["K"], xs[i], rolled[c][i], m["a"], m["s"], ys[i], ws, nb)
            reps = 10 if M == 1 else 3
            ms = graph_time_ms(torch, step, reps, 2, stream) / reps / len(rolled)
            b = sum(m["p"].numel() + 2 * m["N"] + 4 * ((m["K"] + 31) // 32) + 2 * M * m["K"] + 4 * M * m["N"]
                    for m in mods)
            fl = sum(2.0 * M * m["N"] * m["K"] for m in mods)
            res[f"layer_M{M}"] = {"us": ms * 1e3, "gbs": b / ms / 1e6, "tflops": fl / ms / 1e9,
                                  "tokens_per_s_layer": M * 1e3 / ms}
        # the 36-layer ternary body in one wr_gemv_ternary_batched call per token (36 distinct
        # copies of the quantized layer, 731 MB, far above L2)
        body = [(mods[i], m["p"].roll(c * 4096)) for c in range(36) for i, m in enumerate(mods)]
        for M in (1, 8):
            xs = [torch.from_numpy(wr_synth.activations_bf16(3000 + j, M, m["K"]).view(np.int16)).cuda()
                  for j, (m, _) in enumerate(body)]
            ys = [torch.empty(M, m["N"], dtype=torch.float32, device="cuda") for m, _ in body]
            arr = wr._tproblems([(xs[j], pk, m["a"], m["s"], ys[j], m["N"], m["K"]) for j, (m, pk) in enumerate(body)])
            nb = wr.wr_gemv_ternary_batched_workspace_bytes(M, arr)
            ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")

            def tstep():
                wr.wr_gemv_ternary_batched(M, arr, ws, nb)
            ms = graph_time_ms(torch, tstep, 10, 3, stream) / 10
            b = sum(pk.numel() + 2 * m["N"] + 4 * ((m["K"] + 31) // 32) + 2 * M * m["K"] + 4 * M * m["N"]
                    for m, pk in body)
            res[f"body_M{M}"] = {"ms": ms, "bytes": b, "gbs": b / ms / 1e6, "tokens_per_s": M * 1e3 / ms,
                                 "launches": 2}
        out["ternary"] = res
    except Exception as e:  # noqa: BLE001
        out["ternary"] = {"error": repr(e)}

    # the same body at 8 bits (random int8 weights of its shapes), layer by layer with its norms and the
    # codes of each linear's input; the attention output is a stand-in
    try:
        out["eight_bit"] = eight_bit_body(args, wr, torch, stream, hbm_peak, bf16_peak)
    except Exception as e:  # noqa: BLE001
        out["eight_bit"] = {"error": repr(e)}
    return out


def eight_bit_body(args, wr, torch, stream, hbm_peak, bf16_peak):
    """A decoder body whose linears are all at 8 bits, as dependent calls in one graph. Per layer: norm to
    codes, stacked q/k/v; codes of the attention output, o; residual and norm to codes, stacked gate/up; codes
    of silu(gate) up, down; the next layer's first norm takes down's output."""
    H, QKV, A, F = 2560, 6144, 4096, 9728
    g = torch.Generator(device="cuda").manual_seed(11)
    layers = []
    for _ in range(args.layers):
        layers.append([(torch.randint(-127, 128, (n, k), device="cuda", generator=g, dtype=torch.int8),
                        torch.full((n,), 1e-3 / k ** 0.5, device="cuda"), n, k)
                       for n, k in ((QKV, H), (H, A), (2 * F, H), (H, F))])
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    out = {}
    for M in (1, 8, 512):
        h, att = torch.randn(M, H, device="cuda", generator=g).bfloat16(), torch.randn(M, A, device="cuda", generator=g).bfloat16()
        q = {k: torch.empty(M, k, dtype=torch.int8, device="cuda") for k in (H, A, F)}
        s = {k: torch.empty(M, device="cuda") for k in (H, A, F)}
        y = {n: torch.empty(M, n, dtype=torch.bfloat16, device="cuda") for n in (QKV, 2 * F)}
        d = torch.empty(M, H, device="cuda")

        def linear(item, x, xs, yt, yo):
            wq, ws, n, k = item
            wr.wr_gemm_i8(M, n, k, x, k, xs, wq, k, ws, yt, yo, n, None, 0)

        def norm(block):
            wr.wr_residual_norm(M, H, block=block, ld_block=H, residual=h, ld_residual=H, residual_out=h, ld_residual_out=H,
                                residual_type=wr.WR_BF16, norm_weight=w, weight_type=wr.WR_BF16, y=q[H], ld_y=H,
                                y_type=wr.WR_I8, y_scale=s[H])

        def step():
            for i, (qkv, o, gate_up, down) in enumerate(layers):
                norm(d if i else None)
                linear(qkv, q[H], s[H], wr.WR_BF16, y[QKV])
                wr.wr_quantize_rows(wr.WR_BF16, M, A, att, A, q[A], A, s[A])
                linear(o, q[A], s[A], wr.WR_F32, d)
                norm(d)
                linear(gate_up, q[H], s[H], wr.WR_BF16, y[2 * F])
                gu = y[2 * F]
                wr.wr_quantize_rows(wr.WR_BF16, M, F, gu[:, F:], 2 * F, q[F], F, s[F], gate=gu, ldg=2 * F)
                linear(down, q[F], s[F], wr.WR_F32, d)
        ms = graph_time_ms(torch, step, 5, 3, stream) / 5
        weights = sum(n * k for it in layers for _, _, n, k in it)
        out[f"body_dependent_M{M}"] = {"ms": ms, "weight_bytes": weights, "gbs": weights / ms / 1e6,
                                       "frac_of_hbm": weights / ms / 1e6 / hbm_peak, "tops": 2 * M * weights / ms / 1e9,
                                       "frac_of_2x_bf16": 2 * M * weights / ms / 1e9 / (2 * bf16_peak), "tokens_per_s": M * 1e3 / ms,
                                       "launches": 8 * len(layers)}
    return out


if __name__ == "__main__":
    main()
