"""Decode-attention benchmark: tokens/s and KV-read HBM GB/s of one paged decode step.

Default workload (the one the headline metric is quoted on): the Llama-3-8B-shaped decode
layer -- batch 32, 32 query / 8 kv heads (GQA 4), head_dim 128, block 16, context lengths
U[3500, 4500] + 1, physical blocks shuffled over a shared pool.  One step = kv_append of the
new token of every sequence + paged_decode_attention over all cached tokens.  Inputs are
resident in HBM and rotate over 4 independent pool copies (2.3 GB in total, far above the
129 MB L2) so no step reads K/V that a previous step left in L2.  The step runs as one call of
paged_decode_attention_append (the append fused into the decode kernel; tests check it
against kv_append followed by paged decode).

  python bench.py [--gpus N] [--steps K] [--warmup W] [--impl ours|reference] [--no-secondary]

With torchrun (N > 1) every rank runs an independent replica of the workload (the path
shards by sequence with no exchange: weak scaling); rank 0 prints the JSON line with the
max time over ranks.  `--impl reference` times the fp64 CPU oracle on host cores instead.
"""
from __future__ import annotations

import argparse
import json
import math
import os
import statistics
import subprocess
import sys
import time

import numpy as np
import torch

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

METRIC = "decode-attn tokens/s and KV-read HBM GB/s (% of GB300 peak), 1 GPU"
WORKLOAD = "llama8b"
ROTATE = 4  # pool copies the timed steps rotate over (overridden by --rotate)


def _peaks():
    path = os.path.join(ROOT, "MEASURED_PEAKS.json")
    try:
        with open(path) as f:
            p = json.load(f)
        return float(p["hbm_gbs"]), "measured"
    except Exception:
        return 6800.0, "fallback"


def _tensor_peak():
    """Measured dense bf16 TFLOP/s (burst), for kernels timed alone."""
    try:
        with open(os.path.join(ROOT, "MEASURED_PEAKS.json")) as f:
            return float(json.load(f)["bf16_tflops"]), "measured"
    except Exception:
        return 1900.0, "fallback"


def _dist():
    ws = int(os.environ.get("WORLD_SIZE", "1"))
    if ws > 1:
        import torch.distributed as dist
        if not dist.is_initialized():
            backend = os.environ.get("PKV_DIST_BACKEND") or ("nccl" if torch.cuda.is_available() else "gloo")
            dist.init_process_group(backend=backend)
        return dist, dist.get_rank(), ws
    return None, 0, 1


def _barrier(dist):
    if dist is not None:
        dist.barrier()


def _max_over_ranks(dist, value: float, device) -> float:
    if dist is None:
        return value
    t = torch.tensor([value], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


class ClockSampler:
    """nvidia-smi sampling of SM clocks and throttle reasons while the timed region runs."""

    FIELDS = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
              "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
              "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")

    def __init__(self, device_index: int):
        self.idx = device_index
        self.proc = None

    def __enter__(self):
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", f"--id={self.idx}", f"--query-gpu={self.FIELDS}",
                 "--format=csv,noheader,nounits", "-lms", "200"],
                stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
        except Exception:
            self.proc = None
        return self

    def __exit__(self, *exc):
        self.samples = []
        if self.proc is None:
            return False
        self.proc.terminate()
        try:
            out, _ = self.proc.communicate(timeout=5)
        except Exception:
            self.proc.kill()
            out, _ = self.proc.communicate()
        for line in out.strip().splitlines():
            parts = [p.strip() for p in line.split(",")]
            if len(parts) >= 9:
                self.samples.append(parts)
        return False

    def summary(self):
        if not getattr(self, "samples", None):
            return {"sm_mhz": None, "sm_max_mhz": None, "reasons": ["no nvidia-smi samples"]}
        sm = [float(s[1]) for s in self.samples if s[1].replace(".", "").isdigit()]
        mx = [float(s[2]) for s in self.samples if s[2].replace(".", "").isdigit()]
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        reasons = sorted({names[i] for s in self.samples for i in range(4) if s[5 + i].lower() == "active"})
        return {"sm_mhz": statistics.median(sm) if sm else None, "sm_max_mhz": max(mx) if mx else None,
                "reasons": reasons, "samples": len(self.samples)}


KERNEL_SOURCES = ("paged_kv_cache_mapped_gb300/csrc/decode.cu", "paged_kv_cache_mapped_gb300/csrc/kernels.h",
                  "paged_kv_cache_mapped_gb300/csrc/ptx.cuh")


def kernel_source_hash() -> str:
    import hashlib
    h = hashlib.sha256()
    for rel in KERNEL_SOURCES:
        with open(os.path.join(ROOT, rel), "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


def profiled_traffic(name: str):
    """DRAM bytes per launch from the committed ncu summary, or None if it is missing or the
    decode kernel's sources changed since it was taken."""
    path = os.path.join(ROOT, "profiles", f"{name}_counters.txt")  # JSON text
    try:
        with open(path) as f:
            p = json.load(f)
    except Exception:
        return None
    if p.get("kernel_source_hash") != kernel_source_hash():
        return None
    return p.get("dram_bytes_per_launch")


def kv_bytes(lens: torch.Tensor, hkv: int, d: int, window: int = 0) -> int:
    """Algorithmic bytes of K and V one decode reads: attended tokens x Hkv x d x 2 x 2 B."""
    L = lens.to(torch.int64)
    att = torch.minimum(L, torch.full_like(L, window)) if window > 0 else L
    return int(att.sum()) * hkv * d * 2 * 2


def decode_bytes(lens, B, hq, hkv, d, window=0) -> int:
    """KV + q + out + the block-table entries and lengths the step needs."""
    blocks = int(((lens.to(torch.int64) + 15) // 16).sum())
    return kv_bytes(lens, hkv, d, window) + 2 * B * hq * d * 2 + blocks * 4 + B * 4


# ------------------------------------------------------------------------------- our arm

def arm_config(wl, lens, nb, world):
    """The workload's config record, the same for both arms."""
    return {
        "workload": "llama8b decode layer: B=32, Hq=32, Hkv=8, d=128, block 16, "
                    "L=U[3500,4500]+1, append of the new token + paged decode",
        "batch": wl.batch, "context_tokens": int(lens.sum()), "num_q_heads": wl.num_q_heads,
        "num_kv_heads": wl.num_kv_heads, "head_dim": wl.head_dim, "block_size": 16,
        "l2": f"inputs larger than L2: {ROTATE} rotating pool copies "
              f"({ROTATE * 2 * nb * wl.num_kv_heads * 16 * wl.head_dim * 2 / 1e9:.2f} GB)",
        "parallelism": f"replicas x{world}" if world > 1 else "single GPU",
        "inputs_ready": "the calls declare pools, tables and lengths final before the previous "
                        "call ends (PKV_DECODE_INPUTS_READY); figures without it are reported beside",
    }


def run_ours(args):
    import paged_kv_cache_mapped_gb300 as pkv
    from paged_kv_cache_mapped_gb300 import inputs as W

    dist, rank, world = _dist()
    local = int(os.environ.get("LOCAL_RANK", "0"))
    dev = torch.device(f"cuda:{local}")
    torch.cuda.set_device(dev)
    wl = W.WORKLOADS[WORKLOAD]
    lens = W.context_lengths(wl)
    B, hq, hkv, d = wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim

    # pool copy 0 from the CPU generator (also feeds the CPU baseline), 1..3 drawn on device
    global ROTATE
    ROTATE = args.rotate
    host0 = W.make_layer(wl, layer=0, device="cpu")
    copies = [{k: (v.to(dev) if torch.is_tensor(v) else v) for k, v in host0.items()}]
    for r in range(1, ROTATE):
        copies.append(W.make_layer(wl, layer=r, device=dev, device_rng=True))
    nb, mb = copies[0]["num_blocks"], copies[0]["max_blocks_per_seq"]
    for c in copies:
        assert c["num_blocks"] == nb and c["max_blocks_per_seq"] == mb
    ws_bytes = pkv.decode_workspace_bytes(B, hq, hkv, d, nb, mb)
    ws = torch.zeros(ws_bytes, dtype=torch.uint8, device=dev)
    out = torch.empty((B, hq, d), dtype=torch.bfloat16, device=dev)
    err = pkv.new_error_word(dev)
    stream = torch.cuda.current_stream(dev)

    # Consecutive steps rotate over independent pools, so a step's pools, tables and lengths are
    # final before the previous step ends: the calls declare it (inputs_ready), which lets each
    # call's partition and first tile copies overlap the previous call's last warps -- the case of
    # consecutive decode layers.  q and the new rows are still read after the previous call ends.
    def step(c, ready=True, st=None):
        pkv.paged_decode_attention_append(c["q"], c["k_cache"], c["v_cache"], c["k_new"], c["v_new"],
                                          c["block_tables"], c["context_lens"], c["scale"], out=out,
                                          workspace=ws, error_word=err, stream=stream if st is None else st,
                                          inputs_ready=ready)

    # The timed K steps are launched as one CUDA graph (captured beforehand, as a serving loop
    # would): launched one call at a time from Python (~60 us of host work per call) the GPU
    # idles until the first call arrives, which a 20-step region counts as ~3 us per step.  The
    # same steps launched call by call are reported beside ("eager").
    def capture(ready):
        g = torch.cuda.CUDAGraph()
        cs = torch.cuda.Stream(dev)
        cs.wait_stream(stream)
        with torch.cuda.stream(cs):
            step(copies[0], ready, cs)  # the library's per-device setup runs outside the capture
            torch.cuda.synchronize(dev)
            with torch.cuda.graph(g, stream=cs):
                for i in range(args.steps):
                    step(copies[i % ROTATE], ready, cs)
        torch.cuda.synchronize(dev)
        return g

    for i in range(args.warmup):
        step(copies[i % ROTATE])
    torch.cuda.synchronize(dev)
    if pkv.read_error(err) != 0:
        raise RuntimeError("device error during warm-up")
    graph_ready = capture(True)
    graph_plain = capture(False)
    graph_ready.replay()  # untimed: the graph's first launch uploads it
    graph_plain.replay()
    torch.cuda.synchronize(dev)

    # Steps run back to back between two events on the launching stream: an event recorded
    # between two calls would end the programmatic (PDL) overlap of one call's launch with the
    # previous call's tail, which back-to-back decode layers get.
    ev0 = torch.cuda.Event(enable_timing=True)
    ev1 = torch.cuda.Event(enable_timing=True)
    with ClockSampler(local) as clk:
        # same load for ~0.8 s before the timed region, so nvidia-smi (200 ms period) has
        # started sampling when the timed steps run
        t_end = time.perf_counter() + args.preload_s
        i = 0
        while time.perf_counter() < t_end:
            step(copies[i % ROTATE])
            i += 1
            if i % 256 == 0:
                torch.cuda.synchronize(dev)
        _barrier(dist)
        torch.cuda.synchronize(dev)
        ev0.record(stream)
        graph_ready.replay()
        ev1.record(stream)
        torch.cuda.synchronize(dev)
    _barrier(dist)
    ms = ev0.elapsed_time(ev1) / args.steps
    ms = _max_over_ranks(dist, ms, dev)
    dec_ms = ev0.elapsed_time(ev1) / args.steps  # this rank's own average step (one decode call)
    if pkv.read_error(err) != 0:
        raise RuntimeError("device error during the timed region")
    # the same K steps launched call by call from Python
    torch.cuda.synchronize(dev)
    host_t0 = time.perf_counter()
    ev4 = torch.cuda.Event(enable_timing=True)
    ev5 = torch.cuda.Event(enable_timing=True)
    ev4.record(stream)
    for i in range(args.steps):
        step(copies[i % ROTATE])
    ev5.record(stream)
    host_ms = (time.perf_counter() - host_t0) * 1e3 / args.steps
    torch.cuda.synchronize(dev)
    eager_ms = ev4.elapsed_time(ev5) / args.steps
    # the same K steps without the declaration (each call's start-up waits for the previous call)
    ev2 = torch.cuda.Event(enable_timing=True)
    ev3 = torch.cuda.Event(enable_timing=True)
    ev2.record(stream)
    graph_plain.replay()
    ev3.record(stream)
    torch.cuda.synchronize(dev)
    plain_ms = ev2.elapsed_time(ev3) / args.steps
    del graph_ready, graph_plain

    # the same step timed alone with L2 flushed before each: a buffer of twice the L2 size is
    # written between steps, outside the events; median of 50 single steps (one call each, so
    # no programmatic overlap with a previous call)
    l2 = int(getattr(torch.cuda.get_device_properties(dev), "L2_cache_size", 0) or 129 * 2 ** 20)
    flush = torch.empty(2 * l2, dtype=torch.uint8, device=dev)
    pairs = []
    for i in range(50):
        flush.fill_(i & 0xff)
        e0 = torch.cuda.Event(enable_timing=True)
        e1 = torch.cuda.Event(enable_timing=True)
        e0.record(stream)
        step(copies[0], False)
        e1.record(stream)
        pairs.append((e0, e1))
    torch.cuda.synchronize(dev)
    flushed_ms = float(np.median([a.elapsed_time(b) for a, b in pairs]))
    del flush
    if pkv.read_error(err) != 0:
        raise RuntimeError("device error during the L2-flushed steps")

    # end to end through the public API: pinned host inputs -> device, step, result -> host
    e2e = run_e2e(pkv, copies, host0, dev, stream, ws, args) if args.e2e else None

    hbm, peak_kind = _peaks()
    # KV read + q/out + table entries + the append (new K/V rows read and written)
    bytes_dec = decode_bytes(lens, B, hq, hkv, d) + 2 * (B * hkv * d * 2 * 2)
    achieved = bytes_dec / (dec_ms * 1e-3) / 1e9
    tokens_per_s = world * B / (ms * 1e-3)
    line = {
        "metric": METRIC,
        "value": round(tokens_per_s, 1),
        "unit": "tokens/s",
        "n_gpus": world,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "bf16",
        "data": "synthetic (seeded N(0,1) bf16 K/V/q; shuffled block tables)",
        "config": arm_config(wl, lens, nb, world),
        "kv_read_gbs": round(kv_bytes(lens, hkv, d) / (dec_ms * 1e-3) / 1e9, 1),
        "roofline": {
            "bound": "hbm",
            "kernel": "paged_decode_attention_append: split kernel (fused append) + merge kernel, "
                      "timed together as the step; the split kernel alone is faster",
            "achieved": round(achieved, 1),
            "peak": hbm,
            "peak_kind": peak_kind,
            "unit": "GB/s",
            "frac": round(achieved / hbm, 4),
            "frac_of_nominal_8000": round(achieved / 8000.0, 4),  # the part's nominal HBM3e figure
            "traffic": profiled_traffic("decode_split_llama8b"),
            "traffic_note": "ncu dram__bytes_read.sum + dram__bytes_write.sum of decode_split_kernel"
                            "<128,false,false,false> per launch on this workload, from the committed "
                            "counters while the kernel sources are unchanged; the merge kernel adds the "
                            "partials",
            "algorithmic_bytes_per_launch": bytes_dec,
            "launch_ms": round(dec_ms, 5),
        },
        "without_inputs_ready": {
            "ms_per_step": round(plain_ms, 5), "tokens_per_s": round(B / (plain_ms * 1e-3), 1),
            "frac": round(bytes_dec / (plain_ms * 1e-3) / 1e9 / hbm, 4),
            "what": "the same K steps, the calls not declaring their inputs final (each call's "
                    "start-up waits for the previous call to end)"},
        "launch": "the K timed steps as one CUDA graph replay (captured before the timed region)",
        "eager": {"ms_per_step": round(eager_ms, 5), "tokens_per_s": round(B / (eager_ms * 1e-3), 1),
                  "frac": round(bytes_dec / (eager_ms * 1e-3) / 1e9 / hbm, 4),
                  "what": "the same K steps launched call by call from Python"},
        "gpu_launches": 2 * args.steps,
        "host_launch_ms_per_step": round(host_ms, 5),
        "clocks": dict(clk.summary(), window=f"last {args.preload_s} s of identical warm-up load + the timed region"),
        "e2e": e2e,
        "l2_flushed": {"ms_median": round(flushed_ms, 5), "tokens_per_s": round(B / (flushed_ms * 1e-3), 1),
                       "frac": round(bytes_dec / (flushed_ms * 1e-3) / 1e9 / hbm, 4),
                       "what": f"median of 50 single steps, {2 * l2 / 1e6:.0f} MB written between steps"},
    }
    if rank == 0 and world == 1 and args.baseline:
        line["cpu_baseline"] = cpu_baseline(host0, wl, lens)
    if rank == 0 and args.secondary and world == 1:
        line["secondary"] = run_secondary(pkv, W, dev, stream, args)
    if rank == 0:
        print(json.dumps(line), flush=True)
    if dist is not None:
        dist.destroy_process_group()


def run_e2e(pkv, copies, host0, dev, stream, ws, args):
    """Same step through the public API with the step's inputs taken from pinned host memory
    and the result returned to pinned host memory, inside the timed region, the steps in order.
    The step's inputs (q, the new K/V rows, block tables, lengths) sit in one pinned host buffer
    at 256-byte aligned offsets.  The figure: the call reads them there and writes out into a
    pinned host buffer, its kernels crossing the host link (NVLink-C2C) in place, so no copy
    separates one step's kernels from the next.  Beside it (`copies`): one host-to-device copy of
    the packed inputs, the call on views into the device copy, one device-to-host copy of out."""
    names = ("q", "k_new", "v_new", "block_tables", "context_lens")
    offs, at = {}, 0
    for n in names:
        offs[n] = at
        at += (host0[n].numel() * host0[n].element_size() + 255) // 256 * 256
    total = at

    def packed(src):
        buf = torch.empty(total, dtype=torch.uint8).pin_memory()
        for n in names:
            t = src[n].detach().cpu().contiguous()
            nb = t.numel() * t.element_size()
            buf[offs[n]:offs[n] + nb].copy_(t.view(-1).view(torch.uint8))
        return buf

    def views(buf):
        v = {}
        for n in names:
            t = host0[n]
            nb = t.numel() * t.element_size()
            v[n] = buf[offs[n]:offs[n] + nb].view(t.dtype).view(t.shape)
        return v
    hosts = [packed(host0)] + [packed(c) for c in copies[1:]]
    dev_buf = [torch.empty(total, dtype=torch.uint8, device=dev) for _ in range(2)]
    dev_in = [views(b) for b in dev_buf]
    out_h = torch.empty((copies[0]["q"].shape), dtype=torch.bfloat16).pin_memory()
    out = torch.empty_like(copies[0]["q"])
    h2d = sum(host0[n].numel() * host0[n].element_size() for n in names)
    d2h = out.numel() * out.element_size()

    def one_copies(i):
        c, di = copies[i % ROTATE], dev_in[i % 2]
        dev_buf[i % 2].copy_(hosts[i % ROTATE], non_blocking=True)
        pkv.paged_decode_attention_append(di["q"], c["k_cache"], c["v_cache"], di["k_new"], di["v_new"],
                                          di["block_tables"], di["context_lens"], c["scale"], out=out,
                                          workspace=ws, stream=stream)
        out_h.copy_(out, non_blocking=True)

    # in place: the call reads the pinned input buffer and writes a pinned output buffer (two,
    # alternating); its inputs are final before the previous step (that step appended into
    # another pool copy), so it declares them ready like the device-timed steps
    host_in = [views(h) for h in hosts]
    outs_h = [torch.empty((copies[0]["q"].shape), dtype=torch.bfloat16).pin_memory() for _ in range(2)]

    def one_in_place(i):
        c, hv = copies[i % ROTATE], host_in[i % ROTATE]
        pkv.paged_decode_attention_append(hv["q"], c["k_cache"], c["v_cache"], hv["k_new"], hv["v_new"],
                                          hv["block_tables"], hv["context_lens"], c["scale"], out=outs_h[i % 2],
                                          workspace=ws, stream=stream, inputs_ready=True)

    def timed(one):
        for i in range(args.warmup):
            one(i)
        torch.cuda.synchronize(dev)
        # the K steps in 5 consecutive blocks, each between two events; the median block is the
        # figure (one stall of the shared host inside a block moves only that block)
        nblk = 5 if args.steps >= 10 else 1
        per = [args.steps // nblk + (1 if b < args.steps % nblk else 0) for b in range(nblk)]
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(nblk + 1)]
        ev[0].record(stream)
        i = 0
        for b in range(nblk):
            for _ in range(per[b]):
                one(i)
                i += 1
            ev[b + 1].record(stream)
        torch.cuda.synchronize(dev)
        blocks = [ev[b].elapsed_time(ev[b + 1]) / per[b] for b in range(nblk)]
        return (statistics.median(blocks), ev[0].elapsed_time(ev[nblk]) / args.steps, blocks,
                f"median of {nblk} consecutive blocks of the {args.steps} steps")

    ms_c, mean_c, blocks_c, how = timed(one_copies)
    ms, mean, blocks, how = timed(one_in_place)
    # the in-place step's result equals the copy path's for the same inputs (the append rewrites
    # the same rows, so repeating a step leaves the pools as they were)
    one_copies(0)
    one_in_place(0)
    torch.cuda.synchronize(dev)
    if not torch.equal(outs_h[0], out_h):
        raise RuntimeError("the in-place end-to-end step differs from the copy path")
    B = copies[0]["q"].shape[0]
    return {"value": round(B / (ms * 1e-3), 1), "unit": "tokens/s", "ms_per_step": round(ms, 5),
            "h2d_bytes_per_step": h2d, "d2h_bytes_per_step": d2h,
            "ms_per_step_mean": round(mean, 5), "blocks_ms": [round(x, 5) for x in blocks], "timing": how,
            "transfers_per_step": "the kernels read the step's inputs from the pinned host buffer and write out "
                                  "into a pinned host buffer over the host link (NVLink-C2C), in place",
            "copies": {"value": round(B / (ms_c * 1e-3), 1), "ms_per_step": round(ms_c, 5),
                       "ms_per_step_mean": round(mean_c, 5), "blocks_ms": [round(x, 5) for x in blocks_c],
                       "transfers_per_step": "one host-to-device copy of the packed inputs, one device-to-host "
                                             "copy of out, the call between them on the device copy"}}


def cpu_model() -> str:
    """The host CPU's model name (lscpu, else /proc/cpuinfo), with the machine type."""
    import platform
    name = ""
    try:
        out = subprocess.run(["lscpu"], capture_output=True, text=True, timeout=10).stdout
        fields = dict(line.split(":", 1) for line in out.splitlines() if ":" in line)
        fields = {k.strip(): v.strip() for k, v in fields.items()}
        name = fields.get("Model name", "")
        if fields.get("Vendor ID") and fields["Vendor ID"] not in name:
            name = f"{fields['Vendor ID']} {name}".strip()
    except Exception:
        pass
    if not name:
        try:
            with open("/proc/cpuinfo") as f:
                for line in f:
                    if line.lower().startswith(("model name", "cpu model", "hardware")):
                        name = line.split(":", 1)[1].strip()
                        break
        except Exception:
            pass
    return f"{name or 'unknown'} ({platform.machine()})"


def cpu_baseline(host0, wl, lens, budget_s: float = 10.0):
    """The fp64 oracle, as it stands, on the host cores: whole decode steps of the same
    workload (every row of the batch) until ~budget_s of CPU time."""
    import oracle
    q = host0["q"].view(torch.int16).numpy().view(np.uint16)
    kc = host0["k_cache"].view(torch.int16).numpy().view(np.uint16)
    vc = host0["v_cache"].view(torch.int16).numpy().view(np.uint16)
    bt = host0["block_tables"].numpy()
    ln = host0["context_lens"].numpy()
    steps = 0
    t0 = time.perf_counter()
    while True:
        oracle.paged_decode(q, kc, vc, bt, ln, wl.scale)
        steps += 1
        if time.perf_counter() - t0 >= budget_s:
            break
    dt = time.perf_counter() - t0
    cores = oracle.num_threads()
    # the same steps on one thread, for a per-core figure (a quarter of the budget)
    oracle.set_num_threads(1)
    steps1 = 0
    t1 = time.perf_counter()
    try:
        while True:
            oracle.paged_decode(q, kc, vc, bt, ln, wl.scale)
            steps1 += 1
            if time.perf_counter() - t1 >= budget_s / 4:
                break
    finally:
        oracle.set_num_threads(cores)
    dt1 = time.perf_counter() - t1
    return {"value": round(steps * wl.batch / dt, 2), "unit": "tokens/s", "cores": cores,
            "cpu": cpu_model(), "os_cpu_count": os.cpu_count(),
            "kind": "oracle", "value_1_thread": round(steps1 * wl.batch / dt1, 2),
            "sample": f"{steps} full decode steps of the llama8b workload (all {wl.batch}x{wl.num_q_heads} "
                      f"rows, {int(lens.sum())} context tokens each step; the append's pool copy excluded); "
                      f"{steps1} more on one thread for value_1_thread"}


def run_secondary(pkv, W, dev, stream, args):
    """Short device-timed measurements of the other workloads' paths (not the headline)."""
    res = {}
    hbm, _ = _peaks()
    # long-context split-K decode: B=4 x 131072 tokens
    wl = W.WORKLOADS["long128k"]
    c = W.make_layer(wl, device=dev, device_rng=True)
    ws = torch.zeros(pkv.decode_workspace_bytes(wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim,
                                                c["num_blocks"], c["max_blocks_per_seq"]),
                     dtype=torch.uint8, device=dev)
    out = torch.empty_like(c["q"])

    def f():
        pkv.paged_decode_attention(c["q"], c["k_cache"], c["v_cache"], c["block_tables"],
                                   c["context_lens"], c["scale"], out=out, workspace=ws, stream=stream)
    ms = _time(f, args.warmup, max(5, args.steps // 4), dev, stream)
    nbytes = decode_bytes(c["context_lens"].cpu(), wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim)
    res["long128k_decode"] = {"ms": round(ms, 4), "tokens_per_s": round(wl.batch / (ms * 1e-3), 1),
                              "gbs": round(nbytes / (ms * 1e-3) / 1e9, 1),
                              "frac": round(nbytes / (ms * 1e-3) / 1e9 / hbm, 4),
                              "l2": "2.1 GB of K/V per launch (> L2)"}
    del c, ws, out
    torch.cuda.empty_cache()
    res["llama8b_kv_append"] = _append_row(pkv, W, dev, stream, args)
    torch.cuda.empty_cache()
    res["llama8b_decode_with_scores"] = _scores_row(pkv, W, dev, stream, args, hbm)
    torch.cuda.empty_cache()
    res["llama8b_decode_int8"] = _q8_row(pkv, W, dev, stream, args, hbm)
    torch.cuda.empty_cache()
    res["sparse_layer_prefill_scores"] = _prefill_row(pkv, W, dev, stream, args)
    torch.cuda.empty_cache()
    res["qwen1p5b_step"] = _qwen_step(pkv, W, dev, stream, args, hbm)
    torch.cuda.empty_cache()
    res.update(_sparse_step(pkv, W, dev, stream, args, hbm))
    torch.cuda.empty_cache()
    return res


def _scores_row(pkv, W, dev, stream, args, hbm):
    """llama8b decode layer with the sparsification score emitted (logits kept, then turned
    into probabilities added to the scores), against the same decode without it."""
    wl = W.WORKLOADS["llama8b"]
    c = W.make_layer(wl, device=dev, device_rng=True)
    stride = c["max_blocks_per_seq"] * 16
    ws = torch.zeros(pkv.decode_workspace_bytes(wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim,
                                                c["num_blocks"], c["max_blocks_per_seq"]),
                     dtype=torch.uint8, device=dev)
    out = torch.empty_like(c["q"])
    acc = torch.zeros((wl.batch, wl.num_kv_heads, stride), dtype=torch.float32, device=dev)
    lse = torch.empty((wl.batch, wl.num_q_heads), dtype=torch.float32, device=dev)
    logits = torch.empty((wl.batch, wl.num_q_heads, stride), dtype=torch.float32, device=dev)

    def plain():
        pkv.paged_decode_attention(c["q"], c["k_cache"], c["v_cache"], c["block_tables"], c["context_lens"],
                                   c["scale"], out=out, workspace=ws, stream=stream)

    def scored():
        pkv.paged_decode_attention_scores(c["q"], c["k_cache"], c["v_cache"], c["block_tables"],
                                          c["context_lens"], c["scale"], acc, out=out, lse=lse, logits=logits,
                                          workspace=ws, stream=stream)
    steps = max(5, args.steps // 4)
    ms_plain = _time(plain, args.warmup, steps, dev, stream)
    ms_scored = _time(scored, args.warmup, steps, dev, stream)
    lens = c["context_lens"].cpu()
    kv = decode_bytes(lens, wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim)
    keys = int(lens.to(torch.int64).sum()) * wl.num_kv_heads
    extra = keys * (wl.group * 4 * 2 + 4 * 2)  # logits written and read back, scores read and written
    del c, ws, out, acc, logits
    return {"ms": round(ms_scored, 4), "ms_without_scores": round(ms_plain, 4),
            "overhead": round(ms_scored / ms_plain - 1.0, 4),
            "gbs": round((kv + extra) / (ms_scored * 1e-3) / 1e9, 1),
            "frac": round((kv + extra) / (ms_scored * 1e-3) / 1e9 / hbm, 4),
            "score_bytes": extra, "l2": "one 0.58 GB pool (> L2)"}


def _append_row(pkv, W, dev, stream, args):
    """The KV append on its own (llama8b layer: one new K and V row per sequence and kv head),
    bf16 and INT8, and the bf16 append followed by the decode against the fused call."""
    wl = W.WORKLOADS["llama8b"]
    c = W.make_layer(wl, device=dev, device_rng=True)
    nb, hkv, _, d = c["k_cache"].shape
    g = torch.Generator(device=dev).manual_seed(43)
    kq = torch.randint(1, 256, (nb, hkv, 16, d), generator=g, device=dev, dtype=torch.uint8)
    vq = torch.randint(1, 256, (nb, hkv, 16, d), generator=g, device=dev, dtype=torch.uint8)
    ks = torch.empty((nb, hkv, 16), device=dev).exponential_(generator=g) * 0.02
    vs = torch.empty((nb, hkv, 16), device=dev).exponential_(generator=g) * 0.02
    ws = torch.zeros(pkv.decode_workspace_bytes(wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim,
                                                c["num_blocks"], c["max_blocks_per_seq"]),
                     dtype=torch.uint8, device=dev)
    out = torch.empty_like(c["q"])

    def append(st=None):
        pkv.kv_append(c["k_cache"], c["v_cache"], c["k_new"], c["v_new"], c["slot_mapping"],
                      stream=st or torch.cuda.current_stream(dev))

    def append_q8():
        pkv.kv_append_q8(kq, vq, ks, vs, c["k_new"], c["v_new"], c["slot_mapping"],
                         stream=torch.cuda.current_stream(dev))

    def two_calls():
        append(stream)
        pkv.paged_decode_attention(c["q"], c["k_cache"], c["v_cache"], c["block_tables"], c["context_lens"],
                                   c["scale"], out=out, workspace=ws, stream=stream)

    def fused():
        pkv.paged_decode_attention_append(c["q"], c["k_cache"], c["v_cache"], c["k_new"], c["v_new"],
                                          c["block_tables"], c["context_lens"], c["scale"], out=out,
                                          workspace=ws, stream=stream)
    # the appends as 20 calls in one CUDA graph (host launch cost would otherwise bound them)
    n = 20
    gstream = torch.cuda.Stream(dev)
    with torch.cuda.stream(gstream):
        ms = _graph_time([append] * n, args.warmup, max(5, args.steps // 20), dev, gstream) / n
        ms_q8 = _graph_time([append_q8] * n, args.warmup, max(5, args.steps // 20), dev, gstream) / n
    ms_two = _time(two_calls, args.warmup, max(5, args.steps // 4), dev, stream)
    ms_fused = _time(fused, args.warmup, max(5, args.steps // 4), dev, stream)
    rows = wl.batch * hkv
    nbytes = rows * d * 2 * 2 * 2 + wl.batch * 8  # K and V rows read and written, slots
    nbytes_q8 = rows * d * 2 * 2 + rows * 2 * (d + 4) + wl.batch * 8  # bf16 in, codes + scales out
    del c, kq, vq, ks, vs, ws, out
    return {"ms": round(ms, 4), "bytes": nbytes, "gbs": round(nbytes / (ms * 1e-3) / 1e9, 1),
            "ms_int8": round(ms_q8, 4), "bytes_int8": nbytes_q8,
            "ms_append_then_decode": round(ms_two, 4), "ms_fused_append_decode": round(ms_fused, 4),
            "what": f"{rows} K and {rows} V rows of {d} bf16 per call, {n} calls in one CUDA graph; latency-bound"}


def _q8_row(pkv, W, dev, stream, args, hbm):
    """llama8b decode layer over INT8 pools (random codes, per-row scales ~ Exp, the same
    context lengths), against the bf16 decode of the same shape."""
    wl = W.WORKLOADS["llama8b"]
    c = W.make_layer(wl, device=dev, device_rng=True)
    nb, hkv, _, d = c["k_cache"].shape
    g = torch.Generator(device=dev).manual_seed(41)
    kq = torch.randint(1, 256, (nb, hkv, 16, d), generator=g, device=dev, dtype=torch.uint8)
    vq = torch.randint(1, 256, (nb, hkv, 16, d), generator=g, device=dev, dtype=torch.uint8)
    ks = torch.empty((nb, hkv, 16), device=dev).exponential_(generator=g) * 0.02
    vs = torch.empty((nb, hkv, 16), device=dev).exponential_(generator=g) * 0.02
    ws = torch.zeros(pkv.decode_workspace_bytes(wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim,
                                                c["num_blocks"], c["max_blocks_per_seq"]),
                     dtype=torch.uint8, device=dev)
    out = torch.empty_like(c["q"])

    def plain():
        pkv.paged_decode_attention(c["q"], c["k_cache"], c["v_cache"], c["block_tables"], c["context_lens"],
                                   c["scale"], out=out, workspace=ws, stream=stream)

    def q8(ready=False):
        pkv.paged_decode_attention_q8(c["q"], kq, vq, ks, vs, c["block_tables"], c["context_lens"], c["scale"],
                                      out=out, workspace=ws, inputs_ready=ready, stream=stream)

    def q8_ready():  # consecutive calls declaring their inputs final (as the headline's steps do)
        q8(True)
    stride = c["max_blocks_per_seq"] * 16
    acc = torch.zeros((wl.batch, wl.num_kv_heads, stride), dtype=torch.float32, device=dev)
    lse = torch.empty((wl.batch, wl.num_q_heads), dtype=torch.float32, device=dev)
    logits = torch.empty((wl.batch, wl.num_q_heads, stride), dtype=torch.float32, device=dev)

    def q8_scored():
        pkv.paged_decode_attention_scores_q8(c["q"], kq, vq, ks, vs, c["block_tables"], c["context_lens"],
                                             c["scale"], acc, out=out, lse=lse, logits=logits, workspace=ws,
                                             stream=stream)
    def q8_fused():  # this step's rows quantized into the pools inside the decode
        pkv.paged_decode_attention_append_q8(c["q"], kq, vq, ks, vs, c["k_new"], c["v_new"], c["block_tables"],
                                             c["context_lens"], c["scale"], out=out, workspace=ws, stream=stream)

    def q8_two_calls():
        pkv.kv_append_q8(kq, vq, ks, vs, c["k_new"], c["v_new"], c["slot_mapping"], stream=stream)
        q8()
    steps = max(5, args.steps // 4)
    ms_plain = _time(plain, args.warmup, steps, dev, stream)
    ms_q8_plain = _time(q8, args.warmup, steps, dev, stream)
    ms_q8 = _time(q8_ready, args.warmup, steps, dev, stream)
    ms_q8_scored = _time(q8_scored, args.warmup, steps, dev, stream)
    ms_q8_fused = _time(q8_fused, args.warmup, steps, dev, stream)
    ms_q8_two = _time(q8_two_calls, args.warmup, steps, dev, stream)
    lens = c["context_lens"].cpu()
    tokens = int(lens.to(torch.int64).sum())
    blocks = int(((lens.to(torch.int64) + 15) // 16).sum())
    nbytes = (tokens * wl.num_kv_heads * (wl.head_dim + 4) * 2 + 2 * wl.batch * wl.num_q_heads * wl.head_dim * 2
              + blocks * 4 + wl.batch * 4)  # codes + row scales of K and V, q, out, tables, lengths
    del c, kq, vq, ks, vs, ws, out, acc, logits
    return {"ms": round(ms_q8, 4), "ms_without_inputs_ready": round(ms_q8_plain, 4),
            "ms_bf16": round(ms_plain, 4), "speedup": round(ms_plain / ms_q8_plain, 3),
            "ms_with_scores": round(ms_q8_scored, 4), "scores_overhead": round(ms_q8_scored / ms_q8_plain - 1.0, 4),
            "ms_append_fused": round(ms_q8_fused, 4), "ms_append_then_decode": round(ms_q8_two, 4),
            "tokens_per_s": round(wl.batch / (ms_q8 * 1e-3), 1), "bytes": nbytes,
            "gbs": round(nbytes / (ms_q8 * 1e-3) / 1e9, 1), "frac": round(nbytes / (ms_q8 * 1e-3) / 1e9 / hbm, 4),
            "frac_without_inputs_ready": round(nbytes / (ms_q8_plain * 1e-3) / 1e9 / hbm, 4),
            "launch": "back-to-back calls declaring their inputs ready (ms_without_inputs_ready: the same calls "
                      "without; ms_bf16, ms_with_scores and the append rows are undeclared calls)",
            "l2": "0.29 GB of INT8 K/V + scales per call (> L2)"}


def _prefill_row(pkv, W, dev, stream, args, alpha=256):
    """One sparse layer's prefill-window score: 16 prompts of 16384 tokens, 32/8 heads, d = 128,
    a 256-token instruction window; with the forward pass's lse given (the score pass alone) and
    with the lse computed first (two passes over the keys)."""
    wl = W.WORKLOADS["sparse"]
    c = W.make_layer(wl, device=dev, device_rng=True)
    B, hq, hkv, d = wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim
    g = torch.Generator(device=dev).manual_seed(51)
    q_win = torch.randn((B, alpha, hq, d), generator=g, device=dev).to(torch.bfloat16)
    acc = torch.zeros((B, hkv, c["max_blocks_per_seq"] * 16), dtype=torch.float32, device=dev)
    lse = torch.empty((B, hq, alpha), dtype=torch.float32, device=dev)
    pkv.prefill_window_scores(q_win, c["k_cache"], c["block_tables"], c["context_lens"], wl.scale, acc, lse=lse,
                              stream=stream)

    def given():
        pkv.prefill_window_scores(q_win, c["k_cache"], c["block_tables"], c["context_lens"], wl.scale, acc, lse=lse,
                                  lse_given=True, stream=stream)

    def computed():
        pkv.prefill_window_scores(q_win, c["k_cache"], c["block_tables"], c["context_lens"], wl.scale, acc, lse=lse,
                                  stream=stream)
    ms_given = _time(given, args.warmup, 10, dev, stream)
    ms_both = _time(computed, args.warmup, 10, dev, stream)
    lens = c["context_lens"].cpu().to(torch.int64)
    # attended (row, key) pairs: window row j sees keys [0, j]
    pairs = sum(int(sum(int(L) - alpha + r + 1 for r in range(alpha) if int(L) - alpha + r >= 0)) for L in lens)
    flop = 2 * d * pairs * hq  # q.k per attended (row, head, key); the score pass alone
    peak, kind = _tensor_peak()
    tf = flop / (ms_given * 1e-3) / 1e12
    del c, q_win, acc, lse
    # the exponential unit's bound: one ex2 per probability on the MUFU, 16 per clock per SM
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    ex2_peak = sms * 16 * 2.07e9
    exps = pairs * hq / (ms_given * 1e-3)
    return {"ms_lse_given": round(ms_given, 4), "ms_lse_computed": round(ms_both, 4), "tflops": round(tf, 1),
            "frac": round(tf / peak, 4), "peak": peak, "peak_kind": kind, "bound": "tensor",
            "exps_per_s": round(exps, 1),
            "ex2_roofline": {"peak_per_s": ex2_peak, "frac": round(exps / ex2_peak, 4),
                             "what": f"MUFU ex2: {sms} SMs x 16 per clock x 2.07 GHz (maximum SM clock)"},
            "what": "16 prompts x 16384 tokens, 32/8 heads, d 128, window 256 (tcgen05 UMMA bf16 into TMEM + ex2)"}


def _graph_time(calls, warmup, steps, dev, stream):
    """Capture `calls` (a list of no-arg launchers) into one CUDA graph; time its replays."""
    for f in calls:
        f()
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        for f in calls:
            f()
    return _time(g.replay, warmup, steps, dev, stream)


def _qwen_step(pkv, W, dev, stream, args, hbm):
    """Qwen2.5-1.5B-shaped decode step: 28 layers, each with its own pool, append + decode per
    layer, the 28 calls replayed as one CUDA graph."""
    wl = W.WORKLOADS["qwen1p5b"]
    lens = W.context_lengths(wl)
    layers = [W.make_layer(wl, layer=l, device=dev, device_rng=True) for l in range(wl.layers)]
    need = max(pkv.decode_workspace_bytes(wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim,
                                          c["num_blocks"], c["max_blocks_per_seq"]) for c in layers)
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    out = torch.empty_like(layers[0]["q"])
    gstream = torch.cuda.Stream(dev)

    # each layer has its own pools, so every call declares its inputs final (inputs_ready): a
    # layer's start-up overlaps the previous layer's last warps
    def call(c, ready=True):
        return lambda: pkv.paged_decode_attention_append(
            c["q"], c["k_cache"], c["v_cache"], c["k_new"], c["v_new"], c["block_tables"],
            c["context_lens"], c["scale"], out=out, workspace=ws, stream=torch.cuda.current_stream(dev),
            inputs_ready=ready)
    with torch.cuda.stream(gstream):
        ms = _graph_time([call(c) for c in layers], args.warmup, max(5, args.steps // 20), dev, gstream)
        ms_plain = _graph_time([call(c, False) for c in layers], args.warmup, max(5, args.steps // 20), dev,
                               gstream)
    nbytes = wl.layers * (decode_bytes(lens, wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim)
                          + 2 * wl.batch * wl.num_kv_heads * wl.head_dim * 2 * 2)
    # the same step over INT8 pools (random codes, row scales ~ Exp): the fused INT8 append
    g8 = torch.Generator(device=dev).manual_seed(53)
    hkv, d = wl.num_kv_heads, wl.head_dim
    pools8 = []
    for c in layers:
        nb = c["num_blocks"]
        codes = lambda: torch.randint(1, 256, (nb, hkv, 16, d), generator=g8, device=dev, dtype=torch.uint8)
        rs = lambda: torch.empty((nb, hkv, 16), device=dev).exponential_(generator=g8) * 0.02
        pools8.append((codes(), codes(), rs(), rs()))

    def call8(c, p):
        return lambda: pkv.paged_decode_attention_append_q8(
            c["q"], p[0], p[1], p[2], p[3], c["k_new"], c["v_new"], c["block_tables"], c["context_lens"],
            c["scale"], out=out, workspace=ws, stream=torch.cuda.current_stream(dev), inputs_ready=True)
    with torch.cuda.stream(gstream):
        ms8 = _graph_time([call8(c, p) for c, p in zip(layers, pools8)], args.warmup, max(5, args.steps // 20),
                          dev, gstream)
    tokens = int(lens.to(torch.int64).sum())
    bytes8 = wl.layers * (tokens * hkv * (d + 4) * 2 + 2 * wl.batch * wl.num_q_heads * d * 2
                          + 2 * wl.batch * hkv * d * 2 + 2 * wl.batch * hkv * (d + 4))
    del layers, pools8
    return {"ms": round(ms, 4), "tokens_per_s": round(wl.batch / (ms * 1e-3), 1),
            "gbs": round(nbytes / (ms * 1e-3) / 1e9, 1), "frac": round(nbytes / (ms * 1e-3) / 1e9 / hbm, 4),
            "layers": wl.layers, "launch": "28 fused append+decode calls in one CUDA graph, inputs_ready",
            "without_inputs_ready": {"ms": round(ms_plain, 4),
                                     "frac": round(nbytes / (ms_plain * 1e-3) / 1e9 / hbm, 4)},
            "l2": f"{wl.layers} separate pools, {nbytes / 1e9:.2f} GB per step (> L2)",
            "int8": {"ms": round(ms8, 4), "tokens_per_s": round(wl.batch / (ms8 * 1e-3), 1), "bytes": bytes8,
                     "gbs": round(bytes8 / (ms8 * 1e-3) / 1e9, 1),
                     "frac": round(bytes8 / (ms8 * 1e-3) / 1e9 / hbm, 4),
                     "launch": "28 fused INT8 append+decode calls in one CUDA graph, inputs_ready"}}


def _sparse_step(pkv, W, dev, stream, args, hbm):
    """Layer-wise sparse decode step (B16 x 16384, 32 layers): layers 0-3 paged decode over the
    full cache, layers 4-31 paged decode over compacted pools of 1540 kept tokens, replayed as
    one CUDA graph; plus one sparse layer's selection, compaction and gather-decode."""
    wl = W.WORKLOADS["sparse"]
    lens = W.context_lengths(wl)
    B, hq, hkv, d, K = wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim, wl.keep_max
    full = [W.make_layer(wl, layer=l, device=dev, device_rng=True) for l in range(wl.full_layers)]
    dbt_cpu, dnb = W.compact_tables(K, B, seed=5)
    dbt = dbt_cpu.to(dev)
    klens = torch.full((B,), K, dtype=torch.int32, device=dev)
    comp = []
    for l in range(wl.full_layers, wl.layers):
        g = torch.Generator(device=dev).manual_seed(W.layer_seed(wl, l))
        pool = lambda: torch.randn((dnb, hkv, 16, d), generator=g, device=dev).to(torch.bfloat16)
        comp.append({"q": torch.randn((B, hq, d), generator=g, device=dev).to(torch.bfloat16),
                     "k_cache": pool(), "v_cache": pool()})
    need = max(pkv.decode_workspace_bytes(B, hq, hkv, d, c["num_blocks"], c["max_blocks_per_seq"]) for c in full)
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    out = torch.empty((B, hq, d), dtype=torch.bfloat16, device=dev)
    gstream = torch.cuda.Stream(dev)

    # every layer reads its own pools: the calls declare their inputs final (inputs_ready)
    def full_call(c):
        return lambda: pkv.paged_decode_attention(c["q"], c["k_cache"], c["v_cache"], c["block_tables"],
                                                  c["context_lens"], c["scale"], out=out, workspace=ws,
                                                  stream=torch.cuda.current_stream(dev), inputs_ready=True)

    def comp_call(c):
        return lambda: pkv.paged_decode_attention(c["q"], c["k_cache"], c["v_cache"], dbt, klens, wl.scale,
                                                  out=out, workspace=ws, stream=torch.cuda.current_stream(dev),
                                                  inputs_ready=True)
    with torch.cuda.stream(gstream):
        ms = _graph_time([full_call(c) for c in full] + [comp_call(c) for c in comp], args.warmup,
                         max(5, args.steps // 20), dev, gstream)
    full_bytes = decode_bytes(lens, B, hq, hkv, d)
    sparse_bytes = decode_bytes(torch.full((B,), K, dtype=torch.int32), B, hq, hkv, d)
    nbytes = wl.full_layers * full_bytes + (wl.layers - wl.full_layers) * sparse_bytes
    res = {"sparse_step": {"ms": round(ms, 4), "tokens_per_s": round(B / (ms * 1e-3), 1),
                           "gbs": round(nbytes / (ms * 1e-3) / 1e9, 1),
                           "frac": round(nbytes / (ms * 1e-3) / 1e9 / hbm, 4),
                           "launch": "32 decode calls in one CUDA graph (4 full, 28 over compacted pools), "
                                     "inputs_ready",
                           "dense_equivalent_gb": round(wl.layers * full_bytes / 1e9, 2)}}
    # the same step over INT8 pools (random codes, row scales ~ Exp, the same tables and q)
    gq8 = torch.Generator(device=dev).manual_seed(47)

    def q8_pools(nblocks):
        codes = lambda: torch.randint(1, 256, (nblocks, hkv, 16, d), generator=gq8, device=dev, dtype=torch.uint8)
        rs = lambda: torch.empty((nblocks, hkv, 16), device=dev).exponential_(generator=gq8) * 0.02
        return codes(), codes(), rs(), rs()
    full8 = [q8_pools(c["num_blocks"]) for c in full]
    comp8 = [q8_pools(dnb) for _ in comp]

    def q8_call(c, p, tables, clens, scale):
        return lambda: pkv.paged_decode_attention_q8(c["q"], p[0], p[1], p[2], p[3], tables, clens, scale, out=out,
                                                     workspace=ws, stream=torch.cuda.current_stream(dev),
                                                     inputs_ready=True)
    calls8 = ([q8_call(c, p, c["block_tables"], c["context_lens"], c["scale"]) for c, p in zip(full, full8)]
              + [q8_call(c, p, dbt, klens, wl.scale) for c, p in zip(comp, comp8)])
    with torch.cuda.stream(gstream):
        ms8 = _graph_time(calls8, args.warmup, max(5, args.steps // 20), dev, gstream)
    qo = 2 * B * hq * d * 2
    bytes8 = (wl.full_layers * (int(lens.to(torch.int64).sum()) * hkv * (d + 4) * 2 + qo)
              + (wl.layers - wl.full_layers) * (B * K * hkv * (d + 4) * 2 + qo))
    res["sparse_step_int8"] = {"ms": round(ms8, 4), "tokens_per_s": round(B / (ms8 * 1e-3), 1), "bytes": bytes8,
                               "gbs": round(bytes8 / (ms8 * 1e-3) / 1e9, 1),
                               "frac": round(bytes8 / (ms8 * 1e-3) / 1e9 / hbm, 4), "ms_bf16": round(ms, 4),
                               "launch": "32 INT8 decode calls in one CUDA graph (4 full, 28 over compacted "
                                         "pools), inputs_ready"}
    del full8, comp8, calls8
    torch.cuda.empty_cache()
    # one sparse layer: select -> compact, and gather decode over the full pool
    src = full[0]
    scores = W.make_scores(wl, wl.full_layers, lens, device=dev, device_rng=True)
    kept = torch.empty((B, hkv, K), dtype=torch.int32, device=dev)
    kl = torch.empty((B,), dtype=torch.int32, device=dev)
    cur = lambda: torch.cuda.current_stream(dev)  # the capturing stream inside _graph_time
    sel = lambda: pkv.kv_select_topk(scores, src["context_lens"], wl.n_sink, wl.n_recent, wl.k_top,
                                     kept_out=kept, kept_lens_out=kl, stream=cur())
    # the selections of 16 layers one after another, each from its own scores (134 MB > L2): the
    # scores are final, so the calls declare it and each loads and counts its scores while the
    # previous one finishes; the same calls without the declaration beside
    layer_scores = [W.make_scores(wl, 100 + l, lens, device=dev, device_rng=True) for l in range(16)]
    sel_layer = [lambda sc=sc, r=r: pkv.kv_select_topk(sc, src["context_lens"], wl.n_sink, wl.n_recent, wl.k_top,
                                                       kept_out=kept, kept_lens_out=kl, inputs_ready=r,
                                                       stream=cur())
                 for r in (True, False) for sc in layer_scores]
    # the compactions of the 4 full layers one after another, each from its own pool (1.07 GB) into
    # its own compact pool through final kept lists: the calls declare it (inputs_ready) and each
    # reads its kept rows while the previous one stores; the same calls without the declaration beside
    cmp_layer = [lambda s_=s_, c_=c_, r=r: pkv.kv_compact(c_["k_cache"], c_["v_cache"], dbt, s_["k_cache"],
                                                          s_["v_cache"], s_["block_tables"], s_["context_lens"],
                                                          kept, kl, inputs_ready=r, stream=cur())
                 for r in (True, False) for s_, c_ in zip(full, comp)]
    n_cmp = len(full)
    ws_s = torch.zeros(pkv.sparse_decode_workspace_bytes(B, hq, hkv, d, src["num_blocks"],
                                                         src["max_blocks_per_seq"], K),
                       dtype=torch.uint8, device=dev)
    # consecutive gather calls over unchanged pools and lists: the calls declare their inputs final
    gat = lambda ready=True: pkv.sparse_decode_attention(src["q"], src["k_cache"], src["v_cache"],
                                                         src["block_tables"], src["context_lens"], kept, kl,
                                                         wl.scale, out=out, workspace=ws_s, stream=cur(),
                                                         inputs_ready=ready)
    # each per-layer call is microseconds of device work: time it as 10 calls in one CUDA graph
    # (as a decode step runs), not as Python launches that the host would bound
    with torch.cuda.stream(gstream):
        ms_sel = _graph_time(sel_layer[:16], args.warmup, 5, dev, gstream) / 16
        ms_sel_plain = _graph_time(sel_layer[16:], args.warmup, 5, dev, gstream) / 16
        ms_sel_same = _graph_time([sel] * 10, args.warmup, 5, dev, gstream) / 10
        ms_cmp = _graph_time(cmp_layer[:n_cmp] * 3, args.warmup, 5, dev, gstream) / (3 * n_cmp)
        ms_cmp_plain = _graph_time(cmp_layer[n_cmp:] * 3, args.warmup, 5, dev, gstream) / (3 * n_cmp)
        ms_gat = _graph_time([gat] * 10, args.warmup, 5, dev, gstream) / 10
        ms_gat_plain = _graph_time([lambda: gat(False)] * 10, args.warmup, 5, dev, gstream) / 10
    sel_bytes = int(scores.numel()) * 4 + B * hkv * K * 4
    cmp_bytes = B * hkv * K * d * 2 * 2 * 2
    res["sparse_layer_select_topk"] = {"ms": round(ms_sel, 4), "gbs": round(sel_bytes / (ms_sel * 1e-3) / 1e9, 1),
                                       "ms_without_inputs_ready": round(ms_sel_plain, 4),
                                       "ms_one_layer_repeated": round(ms_sel_same, 4),
                                       "launch": "16 layers' selections (each its own scores, 134 MB) in one CUDA "
                                                 "graph, inputs_ready; ms_one_layer_repeated: one layer's scores "
                                                 "selected 10 times without the declaration"}
    del layer_scores, sel_layer
    cmp_launch = (f"{n_cmp} layers' compactions (each its own source and compact pool) x 3 in one CUDA graph, "
                  "inputs_ready")
    res["sparse_layer_compact"] = {"ms": round(ms_cmp, 4), "gbs": round(cmp_bytes / (ms_cmp * 1e-3) / 1e9, 1),
                                   "ms_without_inputs_ready": round(ms_cmp_plain, 4), "launch": cmp_launch}
    del cmp_layer
    res["sparse_layer_gather_decode"] = {"ms": round(ms_gat, 4),
                                         "gbs": round(sparse_bytes / (ms_gat * 1e-3) / 1e9, 1),
                                         "frac": round(sparse_bytes / (ms_gat * 1e-3) / 1e9 / hbm, 4),
                                         "ms_without_inputs_ready": round(ms_gat_plain, 4),
                                         "launch": "10 calls in one CUDA graph, inputs_ready"}
    with torch.cuda.stream(gstream):
        res.update(_rolling_rows(pkv, wl, dev, gstream, lens, scores, comp[:4], dbt, klens, ws, out))
    # the same layer over INT8 pools (random codes, row scales ~ Exp): compaction and rolling
    gq = torch.Generator(device=dev).manual_seed(43)
    codes = lambda n: torch.randint(1, 256, (n, hkv, 16, d), generator=gq, device=dev, dtype=torch.uint8)
    rscales = lambda n: torch.empty((n, hkv, 16), device=dev).exponential_(generator=gq) * 0.02
    snb = src["k_cache"].shape[0]
    s8 = {"kq": codes(snb), "vq": codes(snb), "ks": rscales(snb), "vs": rscales(snb)}
    d8 = {"q": comp[0]["q"], "kq": codes(dnb), "vq": codes(dnb), "ks": rscales(dnb), "vs": rscales(dnb)}
    tables = [(c["block_tables"], c["context_lens"]) for c in full]
    del full, comp
    torch.cuda.empty_cache()
    # INT8 compactions as the bf16 ones: n_cmp layers, each its own source and compact pools
    s8l = [s8] + [{"kq": codes(snb), "vq": codes(snb), "ks": rscales(snb), "vs": rscales(snb)}
                  for _ in range(n_cmp - 1)]
    d8l = [d8] + [{"q": d8["q"], "kq": codes(dnb), "vq": codes(dnb), "ks": rscales(dnb), "vs": rscales(dnb)}
                  for _ in range(n_cmp - 1)]
    cmp8_layer = [lambda s_=s_, d_=d_, t_=t_, r=r: pkv.kv_compact_q8(d_["kq"], d_["vq"], d_["ks"], d_["vs"], dbt,
                                                                     s_["kq"], s_["vq"], s_["ks"], s_["vs"], t_[0],
                                                                     t_[1], kept, kl, inputs_ready=r, stream=cur())
                  for r in (True, False) for s_, d_, t_ in zip(s8l, d8l, tables)]
    gat8 = lambda: pkv.sparse_decode_attention_q8(src["q"], s8["kq"], s8["vq"], s8["ks"], s8["vs"],
                                                  src["block_tables"], src["context_lens"], kept, kl, wl.scale,
                                                  out=out, workspace=ws_s, stream=cur(), inputs_ready=True)
    with torch.cuda.stream(gstream):
        ms_gat8 = _graph_time([gat8] * 10, args.warmup, 5, dev, gstream) / 10
        ms_cmp8 = _graph_time(cmp8_layer[:n_cmp] * 3, args.warmup, 5, dev, gstream) / (3 * n_cmp)
        ms_cmp8_plain = _graph_time(cmp8_layer[n_cmp:] * 3, args.warmup, 5, dev, gstream) / (3 * n_cmp)
        res.update(_rolling_rows(pkv, wl, dev, gstream, lens, scores, d8l, dbt, klens, ws, out, q8=True))
    cmp8_bytes = B * hkv * K * (d + 4) * 2 * 2
    gat8_bytes = B * hkv * K * (d + 4) * 2 + 2 * B * hq * d * 2
    res["sparse_layer_gather_decode_int8"] = {"ms": round(ms_gat8, 4), "bytes": gat8_bytes,
                                              "gbs": round(gat8_bytes / (ms_gat8 * 1e-3) / 1e9, 1),
                                              "ms_bf16": round(ms_gat, 4)}
    res["sparse_layer_compact_int8"] = {"ms": round(ms_cmp8, 4), "bytes": cmp8_bytes,
                                        "gbs": round(cmp8_bytes / (ms_cmp8 * 1e-3) / 1e9, 1),
                                        "ms_without_inputs_ready": round(ms_cmp8_plain, 4),
                                        "ms_bf16": round(ms_cmp, 4), "launch": cmp_launch}
    del s8, d8, s8l, d8l, cmp8_layer, scores
    return res


def _rolling_rows(pkv, wl, dev, gstream, lens, scores, pools, dbt, klens, ws, out, calls=10, trials=5, q8=False):
    """Sparse layers kept at their fixed budget by rolling admission, stepped as a decode step
    steps them: `pools` are the layers' compact pools (each its own; q8: kq, vq, ks, vs), each
    layer's state a top-k selection over the first L - 1 tokens.  Step i admits token L - 1 + i
    (its own row of context lengths) into every layer, then, in the layer step, attends over
    that layer's compact pool with the scores added to its slot scores.  The admissions declare
    their inputs ready: a layer's slot state was last written by its own score pass of the
    previous step, with the other layers' work in between (the undeclared calls beside).
    Admission changes the state, so the calls are one CUDA graph replayed once per trial from a
    restored state.  Rows named *_int8 for q8."""
    B, hq, hkv, d, K = wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim, wl.keep_max
    prev = (lens - 1).to(dev)
    kept = torch.empty((B, hkv, K), dtype=torch.int32, device=dev)
    kl = torch.empty((B,), dtype=torch.int32, device=dev)
    pkv.kv_select_topk(scores, prev, wl.n_sink, wl.n_recent, wl.k_top, kept_out=kept, kept_lens_out=kl,
                       stream=gstream)
    pos0 = kept.clone()
    sc0 = torch.gather(scores, 2, kept.to(torch.int64))
    kl0 = kl.clone()
    g = torch.Generator(device=dev).manual_seed(11)
    n_layers = len(pools)
    news = [(torch.randn((B, hkv, d), generator=g, device=dev).to(torch.bfloat16),
             torch.randn((B, hkv, d), generator=g, device=dev).to(torch.bfloat16)) for _ in pools]
    lens_rows = (lens.to(dev).view(1, B) + torch.arange(calls, dtype=torch.int32, device=dev).view(-1, 1)).contiguous()
    states = [(pos0.clone(), sc0.clone(), kl0.clone()) for _ in pools]
    lse = torch.empty((B, hq), dtype=torch.float32, device=dev)
    logits = torch.empty((B, hq, K), dtype=torch.float32, device=dev)
    err = pkv.new_error_word(dev)

    cur = lambda: torch.cuda.current_stream(dev)

    def admit(i, l, ready):
        c, (pos, sc, kls), (k_new, v_new) = pools[l], states[l], news[l]
        if q8:
            pkv.kv_rolling_admit_q8(c["kq"], c["vq"], c["ks"], c["vs"], dbt, pos, sc, kls, lens_rows[i], k_new,
                                    v_new, wl.n_sink, wl.n_recent, error_word=err, inputs_ready=ready, stream=cur())
        else:
            pkv.kv_rolling_admit(c["k_cache"], c["v_cache"], dbt, pos, sc, kls, lens_rows[i], k_new, v_new,
                                 wl.n_sink, wl.n_recent, error_word=err, inputs_ready=ready, stream=cur())

    def decode_scores(l):
        c, sc = pools[l], states[l][1]
        if q8:
            pkv.paged_decode_attention_scores_q8(c["q"], c["kq"], c["vq"], c["ks"], c["vs"], dbt, klens, wl.scale,
                                                 sc, out=out, lse=lse, logits=logits, workspace=ws, error_word=err,
                                                 stream=cur())
        else:
            pkv.paged_decode_attention_scores(c["q"], c["k_cache"], c["v_cache"], dbt, klens, wl.scale, sc,
                                              out=out, lse=lse, logits=logits, workspace=ws, error_word=err,
                                              stream=cur())

    def plain(l):
        c = pools[l]
        if q8:
            pkv.paged_decode_attention_q8(c["q"], c["kq"], c["vq"], c["ks"], c["vs"], dbt, klens, wl.scale, out=out,
                                          workspace=ws, stream=cur())
        else:
            pkv.paged_decode_attention(c["q"], c["k_cache"], c["v_cache"], dbt, klens, wl.scale, out=out,
                                       workspace=ws, stream=cur())

    def restore():
        for pos, sc, kls in states:
            pos.copy_(pos0)
            sc.copy_(sc0)
            kls.copy_(kl0)
        torch.cuda.synchronize(dev)

    def series(body):
        """body(i, l) enqueues layer l's work of step i; returns ms per (step, layer)."""
        restore()
        for l in range(n_layers):            # one eager pass: any lazy setup happens outside the capture
            body(0, l)
        restore()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=gstream):
            for i in range(calls):
                for l in range(n_layers):
                    body(i, l)
        times = []
        for _ in range(trials + 1):          # the first replay is a warm-up
            restore()
            e0 = torch.cuda.Event(enable_timing=True)
            e1 = torch.cuda.Event(enable_timing=True)
            e0.record(gstream)
            gr.replay()
            e1.record(gstream)
            torch.cuda.synchronize(dev)
            times.append(e0.elapsed_time(e1) / (calls * n_layers))
        return sorted(times[1:])[trials // 2]
    ms_adm = series(lambda i, l: admit(i, l, True))
    ms_adm_plain = series(lambda i, l: admit(i, l, False))
    ms_layer = series(lambda i, l: (admit(i, l, True), decode_scores(l)))
    ms_layer_plain = series(lambda i, l: (admit(i, l, False), decode_scores(l)))
    ms_plain = series(lambda i, l: plain(l))
    if pkv.read_error(err) != 0:
        raise RuntimeError(f"rolling admission reported device error {pkv.read_error(err)}")
    segs = B * hkv
    row_out = (d + 4) * 2 if q8 else d * 2 * 2     # one K and one V row written: codes + scale, or bf16
    adm_bytes = segs * (K * 8 + 2 * d * 2 + row_out + 8)  # slot positions+scores read, new rows in, rows out
    if q8:
        tok = int(klens.to(torch.int64).sum().item())
        kv = tok * hkv * (d + 4) * 2 + 2 * B * hq * d * 2
    else:
        kv = decode_bytes(klens.cpu(), B, hq, hkv, d)
    sfx = "_int8" if q8 else ""
    launch = (f"{calls} steps of {n_layers} layers (each its own pool and state) in one CUDA graph, median of "
              f"{trials}; admissions declaring their inputs ready")
    return {"sparse_layer_rolling_admit" + sfx: {"ms": round(ms_adm, 4), "bytes": adm_bytes,
                                                 "gbs": round(adm_bytes / (ms_adm * 1e-3) / 1e9, 1),
                                                 "ms_without_inputs_ready": round(ms_adm_plain, 4),
                                                 "launch": launch},
            "sparse_layer_rolling_step" + sfx: {
                "ms": round(ms_layer, 4), "ms_without_inputs_ready": round(ms_layer_plain, 4),
                "ms_plain_compact_decode": round(ms_plain, 4),
                "gbs": round((kv + adm_bytes) / (ms_layer * 1e-3) / 1e9, 1),
                "what": "admit + score-emitting decode over 1540 slots per (b, kv head)",
                "launch": launch}}


def _time(fn, warmup, steps, dev, stream):
    for _ in range(warmup):
        fn()
    torch.cuda.synchronize(dev)
    e0 = torch.cuda.Event(enable_timing=True)
    e1 = torch.cuda.Event(enable_timing=True)
    e0.record(stream)
    for _ in range(steps):
        fn()
    e1.record(stream)
    torch.cuda.synchronize(dev)
    return e0.elapsed_time(e1) / steps


# ------------------------------------------------------------------------- reference arm

def run_reference(args):
    """The fp64 CPU oracle timed on the host cores as the reference arm: each step runs the
    oracle over a bounded sample of the same workload (4 of the 32 sequences, all heads)."""
    dist, rank, world = _dist()
    if rank != 0:
        if dist is not None:
            dist.destroy_process_group()
        return
    import oracle
    from paged_kv_cache_mapped_gb300 import inputs as W
    wl = W.WORKLOADS[WORKLOAD]
    host0 = W.make_layer(wl, layer=0, device="cpu")
    n_seq = 4
    q = host0["q"][:n_seq].contiguous().view(torch.int16).numpy().view(np.uint16)
    kc = host0["k_cache"].view(torch.int16).numpy().view(np.uint16)
    vc = host0["v_cache"].view(torch.int16).numpy().view(np.uint16)
    bt = host0["block_tables"][:n_seq].contiguous().numpy()
    ln = host0["context_lens"][:n_seq].contiguous().numpy()
    for _ in range(args.warmup):
        oracle.paged_decode(q, kc, vc, bt, ln, wl.scale)
    t0 = time.perf_counter()
    for _ in range(args.steps):
        oracle.paged_decode(q, kc, vc, bt, ln, wl.scale)
    dt = (time.perf_counter() - t0) / args.steps
    value = round(n_seq / dt, 2)
    line = {
        "impl": "reference",
        "metric": METRIC, "value": value, "unit": "tokens/s", "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": round(dt * 1e3, 4), "higher_is_better": True,
        "scaling": "weak", "vs_baseline": None, "dtype": "f64", "data": "synthetic",
        "config": arm_config(wl, W.context_lengths(wl), host0["num_blocks"], world),
        "cpu_baseline": {"value": value, "unit": "tokens/s", "cores": oracle.num_threads(),
                         "cpu": cpu_model(), "os_cpu_count": os.cpu_count(), "kind": "oracle",
                         "sample": f"each step: the oracle's decode of {n_seq} of the {wl.batch} sequences "
                                   f"(all {wl.num_q_heads} heads, their full contexts); tokens/s counts "
                                   f"those {n_seq} sequences"},
        "e2e": {"value": value, "unit": "tokens/s", "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
    }
    print(json.dumps(line), flush=True)
    if dist is not None:
        dist.destroy_process_group()


# ------------------------------------------------------------------- small profiling cases

CASES = ("q8", "gather", "gather_q8", "prefill", "kvops", "layers", "append", "qwen8", "qwen8_plain",
         "chunk", "step")


def run_case(name: str, calls: int = 3):
    """One small, self-contained case for an ncu capture: the named path called `calls` times
    on one layer of its workload (a few GB on the device at most), then exit.  Nothing is
    timed here; the profiles name these commands.

      q8       llama8b-shaped layer over INT8 pools: paged_decode_attention_q8
      gather   one sparse layer: kv_select_topk, then sparse_decode_attention (gather form)
      gather_q8  the same over INT8 pools: sparse_decode_attention_q8
      prefill  one sparse layer: prefill_window_scores with the lse computed, then given
      kvops    one sparse layer: kv_select_topk, kv_compact, kv_compact_q8 in turn
      layers   a qwen1p5b layer (append + decode), a full sparse layer, a compacted sparse layer
      append   llama8b layer: kv_append, kv_append_q8 in turn
      qwen8    eight qwen1p5b layers (each with its own pools: append + decode, the calls declaring
               their inputs ready) captured in one CUDA graph and replayed `calls` times
      qwen8_plain  the same graph with calls that do not declare their inputs ready
      chunk    a sparse layer's first sequence, its last 4096 of 16384 tokens: paged_prefill_attention,
               plain, then with capped scores
      step     llama8b-shaped prompts into FP8 pools: kv_step_tables, kv_append_f8, then one token a
               sequence by paged_decode_attention_f8, and over bf16 pools by paged_decode_attention_rules
    """
    import paged_kv_cache_mapped_gb300 as pkv
    from paged_kv_cache_mapped_gb300 import inputs as W
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)

    def q8_pools(nb, hkv, d, seed, scale_fn):
        g = torch.Generator(device=dev).manual_seed(seed)
        codes = [torch.randint(1, 256, (nb, hkv, 16, d), generator=g, device=dev, dtype=torch.uint8)
                 for _ in range(2)]
        return codes + [scale_fn(g, (nb, hkv, 16)) for _ in range(2)]
    exp_scales = lambda g, shape: torch.empty(shape, device=dev).exponential_(generator=g) * 0.02
    uni_scales = lambda g, shape: torch.rand(shape, generator=g, device=dev)

    def ws_for(wl, c):
        return torch.zeros(pkv.decode_workspace_bytes(wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim,
                                                      c["num_blocks"], c["max_blocks_per_seq"]),
                           dtype=torch.uint8, device=dev)

    if name in ("q8", "append"):
        wl = W.WORKLOADS["llama8b"]
        c = W.make_layer(wl, device=dev, device_rng=True)
        nb, hkv, _, d = c["k_cache"].shape
        kq, vq, ks, vs = q8_pools(nb, hkv, d, 41, exp_scales)
        for _ in range(calls):
            if name == "q8":
                pkv.paged_decode_attention_q8(c["q"], kq, vq, ks, vs, c["block_tables"], c["context_lens"],
                                              c["scale"])
            else:
                pkv.kv_append(c["k_cache"], c["v_cache"], c["k_new"], c["v_new"], c["slot_mapping"])
                pkv.kv_append_q8(kq, vq, ks, vs, c["k_new"], c["v_new"], c["slot_mapping"])
    elif name in ("gather", "gather_q8", "kvops"):
        wl = W.WORKLOADS["sparse"]
        lens = W.context_lengths(wl)
        B, hkv, d, K = wl.batch, wl.num_kv_heads, wl.head_dim, wl.keep_max
        src = W.make_layer(wl, layer=0, device=dev, device_rng=True)
        scores = W.make_scores(wl, wl.full_layers, lens, device=dev, device_rng=True)
        kept = torch.empty((B, hkv, K), dtype=torch.int32, device=dev)
        kl = torch.empty((B,), dtype=torch.int32, device=dev)
        if name == "gather":
            pkv.kv_select_topk(scores, src["context_lens"], wl.n_sink, wl.n_recent, wl.k_top,
                               kept_out=kept, kept_lens_out=kl)
            for _ in range(calls):
                pkv.sparse_decode_attention(src["q"], src["k_cache"], src["v_cache"], src["block_tables"],
                                            src["context_lens"], kept, kl, wl.scale)
        elif name == "gather_q8":
            pkv.kv_select_topk(scores, src["context_lens"], wl.n_sink, wl.n_recent, wl.k_top,
                               kept_out=kept, kept_lens_out=kl)
            kq, vq, ks, vs = q8_pools(src["k_cache"].shape[0], hkv, d, 43, exp_scales)
            del src["k_cache"], src["v_cache"]
            for _ in range(calls):
                pkv.sparse_decode_attention_q8(src["q"], kq, vq, ks, vs, src["block_tables"], src["context_lens"],
                                               kept, kl, wl.scale)
        else:
            dbt_cpu, dnb = W.compact_tables(K, B, seed=5)
            dbt = dbt_cpu.to(dev)
            dk = torch.empty((dnb, hkv, 16, d), dtype=torch.bfloat16, device=dev)
            dv = torch.empty_like(dk)
            sq, svq, ss, svs = q8_pools(src["k_cache"].shape[0], hkv, d, 3, uni_scales)
            dq, dvq, ds, dvs = q8_pools(dnb, hkv, d, 4, uni_scales)
            for _ in range(calls):
                pkv.kv_select_topk(scores, src["context_lens"], wl.n_sink, wl.n_recent, wl.k_top,
                                   kept_out=kept, kept_lens_out=kl)
                pkv.kv_compact(dk, dv, dbt, src["k_cache"], src["v_cache"], src["block_tables"],
                               src["context_lens"], kept, kl)
                pkv.kv_compact_q8(dq, dvq, ds, dvs, dbt, sq, svq, ss, svs, src["block_tables"],
                                  src["context_lens"], kept, kl)
    elif name == "prefill":
        wl = W.WORKLOADS["sparse"]
        c = W.make_layer(wl, device=dev, device_rng=True)
        del c["v_cache"]
        alpha = 256
        g = torch.Generator(device=dev).manual_seed(51)
        q_win = torch.randn((wl.batch, alpha, wl.num_q_heads, wl.head_dim), generator=g,
                            device=dev).to(torch.bfloat16)
        acc = torch.zeros((wl.batch, wl.num_kv_heads, c["max_blocks_per_seq"] * 16), dtype=torch.float32,
                          device=dev)
        lse = pkv.prefill_window_scores(q_win, c["k_cache"], c["block_tables"], c["context_lens"], wl.scale, acc)
        pkv.prefill_window_scores(q_win, c["k_cache"], c["block_tables"], c["context_lens"], wl.scale, acc,
                                  lse=lse, lse_given=True)
    elif name == "layers":
        wl = W.WORKLOADS["qwen1p5b"]
        c = W.make_layer(wl, layer=0, device=dev, device_rng=True)
        ws = ws_for(wl, c)
        for _ in range(calls):
            pkv.paged_decode_attention_append(c["q"], c["k_cache"], c["v_cache"], c["k_new"], c["v_new"],
                                              c["block_tables"], c["context_lens"], c["scale"], workspace=ws)
        torch.cuda.synchronize(dev)
        del c, ws
        torch.cuda.empty_cache()
        wl = W.WORKLOADS["sparse"]
        c = W.make_layer(wl, layer=0, device=dev, device_rng=True)
        ws = ws_for(wl, c)
        for _ in range(calls):
            pkv.paged_decode_attention(c["q"], c["k_cache"], c["v_cache"], c["block_tables"], c["context_lens"],
                                       c["scale"], workspace=ws)
        torch.cuda.synchronize(dev)
        del c
        torch.cuda.empty_cache()
        K = wl.keep_max
        dbt, dnb = W.compact_tables(K, wl.batch, seed=5)
        g = torch.Generator(device=dev).manual_seed(9)
        kc = torch.randn((dnb, wl.num_kv_heads, 16, wl.head_dim), generator=g, device=dev).to(torch.bfloat16)
        vc = torch.randn((dnb, wl.num_kv_heads, 16, wl.head_dim), generator=g, device=dev).to(torch.bfloat16)
        q = torch.randn((wl.batch, wl.num_q_heads, wl.head_dim), generator=g, device=dev).to(torch.bfloat16)
        kl = torch.full((wl.batch,), K, dtype=torch.int32, device=dev)
        for _ in range(calls):
            pkv.paged_decode_attention(q, kc, vc, dbt.to(dev), kl, wl.scale, workspace=ws)
    elif name in ("qwen8", "qwen8_plain"):
        wl = W.WORKLOADS["qwen1p5b"]
        layers = [W.make_layer(wl, layer=l, device=dev, device_rng=True) for l in range(8)]
        ws = torch.zeros(max(pkv.decode_workspace_bytes(wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim,
                                                        c["num_blocks"], c["max_blocks_per_seq"]) for c in layers),
                         dtype=torch.uint8, device=dev)
        out = torch.empty_like(layers[0]["q"])
        ready = name == "qwen8"
        s = torch.cuda.Stream(dev)

        def step():
            for c in layers:
                pkv.paged_decode_attention_append(c["q"], c["k_cache"], c["v_cache"], c["k_new"], c["v_new"],
                                                  c["block_tables"], c["context_lens"], c["scale"], out=out,
                                                  workspace=ws, stream=torch.cuda.current_stream(dev),
                                                  inputs_ready=ready)
        with torch.cuda.stream(s):
            step()
            torch.cuda.synchronize(dev)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
            graph.replay()
            torch.cuda.synchronize(dev)
            # the replays alone are in the profiler's range (ncu --profile-from-start off)
            torch.cuda.cudart().cudaProfilerStart()
            for _ in range(calls):
                graph.replay()
            torch.cuda.synchronize(dev)
            torch.cuda.cudart().cudaProfilerStop()
    elif name == "chunk":
        wl = W.WORKLOADS["sparse"]
        c = W.make_layer(wl, device=dev, device_rng=True)
        n = 4096
        g = torch.Generator(device=dev).manual_seed(61)
        q = torch.randn((n, wl.num_q_heads, wl.head_dim), generator=g, device=dev).to(torch.bfloat16)
        starts = torch.tensor([0, n], dtype=torch.int32, device=dev)
        for cap in (0.0, 30.0):
            pkv.paged_prefill_attention(q, c["k_cache"], c["v_cache"], c["block_tables"][:1].contiguous(),
                                        c["context_lens"][:1].contiguous(), starts, wl.scale, softcap=cap)
    elif name == "step":
        wl = W.WORKLOADS["llama8b"]
        c = W.make_layer(wl, device=dev, device_rng=True)
        B, (nb, hkv, _, d) = wl.batch, c["k_cache"].shape
        T = int(c["context_lens"].sum())
        bt = torch.full_like(c["block_tables"], -1)
        free, count = torch.randperm(nb, dtype=torch.int32, device=dev), torch.tensor([nb], dtype=torch.int32, device=dev)
        lens, _, slots, _, _ = pkv.kv_step_tables(bt, torch.zeros_like(c["context_lens"]), c["context_lens"], free, count, T)
        g = torch.Generator(device=dev).manual_seed(62)
        k, v = (torch.randn((T, hkv, d), generator=g, device=dev).to(torch.bfloat16) for _ in range(2))
        kq, vq = (torch.zeros((nb, hkv, 16, d), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.zeros((nb, hkv), device=dev) for _ in range(2))
        for _ in range(calls):
            pkv.kv_append_f8(kq, vq, ks, vs, k, v, slots)
            pkv.paged_decode_attention_f8(c["q"], kq, vq, ks, vs, bt, lens, c["scale"])
            pkv.paged_decode_attention_rules(c["q"], c["k_cache"], c["v_cache"], c["block_tables"], c["context_lens"],
                                             c["scale"], softcap=30.0)
    else:
        raise SystemExit(f"unknown case {name!r}; one of {', '.join(CASES)}")
    torch.cuda.synchronize(dev)
    print(json.dumps({"case": name, "calls": calls, "ok": True}))


def _free_port() -> int:
    import socket
    with socket.socket() as sk:
        sk.bind(("127.0.0.1", 0))
        return sk.getsockname()[1]


def launch_replicas(n: int) -> int:
    """`--gpus N` run directly (no WORLD_SIZE in the environment): start N ranks of this script,
    one per GPU, through torch.distributed.run on 127.0.0.1, and return their exit status.  Each
    rank runs an independent replica (the path shards by sequence with no exchange); rank 0
    prints the JSON line."""
    cmd = [sys.executable, "-m", "torch.distributed.run", "--nnodes=1", f"--nproc-per-node={n}",
           "--master-addr", "127.0.0.1", "--master-port", str(_free_port()), os.path.abspath(__file__),
           *sys.argv[1:]]
    return subprocess.run(cmd).returncode


def dist_check():
    """The multi-rank launch checked without a GPU (PKV_DIST_BACKEND=gloo): every rank joins,
    the barrier passes, and rank 0 prints the ranks seen and the max over ranks of a value that
    differs per rank (the reduction the timed region uses)."""
    dist, rank, world = _dist()
    dev = torch.device("cpu")
    _barrier(dist)
    ranks = [rank]
    if dist is not None:
        gathered = [None] * world
        dist.all_gather_object(gathered, rank)
        ranks = sorted(gathered)
    mx = _max_over_ranks(dist, 1.0 + rank, dev)
    if rank == 0:
        print(json.dumps({"dist_check": {"world": world, "ranks": ranks, "max_over_ranks": mx}}), flush=True)
    if dist is not None:
        dist.destroy_process_group()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=2000)
    ap.add_argument("--warmup", type=int, default=10)
    ap.add_argument("--impl", choices=["ours", "reference"], default="ours")
    ap.add_argument("--no-secondary", dest="secondary", action="store_false",
                    help="skip the other workloads' measurements")
    ap.add_argument("--no-baseline", dest="baseline", action="store_false",
                    help="skip the CPU oracle baseline")
    ap.add_argument("--no-e2e", dest="e2e", action="store_false",
                    help="skip the end-to-end (host buffers) measurement")
    ap.add_argument("--preload-s", type=float, default=0.8,
                    help="seconds of untimed identical load before the timed region (clock sampling)")
    ap.add_argument("--rotate", type=int, default=ROTATE,
                    help="independent pool copies the timed steps rotate over")
    ap.add_argument("--case", choices=CASES, default=None,
                    help="run one small profiling case (no timing, no JSON metric line) and exit")
    ap.add_argument("--dist-check", action="store_true",
                    help="check the multi-rank launch (ranks, barrier, max over ranks) and exit")
    args = ap.parse_args()
    if args.case is not None:
        run_case(args.case)
        return
    if args.gpus < 1:
        sys.exit("--gpus must be at least 1")
    world = os.environ.get("WORLD_SIZE")
    if world is None and args.gpus > 1:
        sys.exit(launch_replicas(args.gpus))
    if world is not None and int(world) != args.gpus:
        sys.exit(f"--gpus {args.gpus} but WORLD_SIZE={world}: launch one rank per requested GPU")
    if args.dist_check:
        dist_check()
        return
    if args.warmup < 3:
        args.warmup = 3
    if args.impl == "reference":
        run_reference(args)
    else:
        run_ours(args)


if __name__ == "__main__":
    main()
