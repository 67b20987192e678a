"""The headline run's JSON line fits into the last 3000 characters of the output, with every other
workload's value in it."""
import json

import bench

# a headline run's line on one GPU, without its workloads
LINE = {
    "metric": bench.METRIC, "value": 2067.35, "unit": "TFLOP/s", "n_gpus": 1, "steps": 20, "warmup": 5,
    "repeats": 250, "timed_s": 1.018, "ms_per_step": 0.2036, "higher_is_better": True, "scaling": "weak",
    "vs_baseline": None, "dtype": "fp8_e4m3 (fp32 accumulate)", "data": "synthetic",
    "config": {"workload": "fprop_4096x7168x7168", "M": 4096, "N": 7168, "K": 7168,
               "step": "quant_act(X) + quant_weight(W) + fp8_gemm -> bf16",
               "l2": "inputs 161.5 MB, under twice the L2: steps cycle through 3 copies of the step's buffers "
                     "(484 MB of inputs); no flush", "parallelism": "replicas x1"},
    "roofline": {"bound": "tensor", "achieved": 2564.0, "peak": 3807.8, "unit": "TFLOP/s", "frac": 0.6734,
                 "peak_source": "measured: bf16 burst 1903.9 TFLOP/s x 2.0 (nominal fp8/bf16 ratio)",
                 "traffic": 121122816.0, "kernel": "fp8q_gemm_kernel", "work_per_launch": 420906795008.0},
    "timing": {"mode": "cuda_graph", "kernel_events": "recorded on a side stream at every kernel boundary",
               "graphs": 3},
    "kernels": {"quant_act_kernel": {"ms": 0.01351, "gbs": 6585.6, "frac_hbm": 0.9702},
                "quant_weight_kernel": {"ms": 0.02493, "gbs": 6183.6, "frac_hbm": 0.911},
                "fp8q_gemm_kernel": {"ms": 0.16416, "tflops": 2564.0, "frac_fp8_peak": 0.6734},
                "hbm_peak_gbs": 6787.6, "fp8_peak_tflops": 3807.8, "peak_source": "measured"},
    "e2e": {"value": 488.13, "unit": "TFLOP/s", "h2d_bytes_per_step": 161480704,
            "d2h_bytes_per_step": 58720256, "ms_per_step": 0.8623, "steps": 20},
    "gpu_launches": 15000, "buffer_copies": 3,
    "clocks": {"sm_mhz": 2017.5, "sm_max_mhz": 2070.0, "power_w_max": 1221.05, "reasons": ["sw_power_cap"],
               "samples": 10},
    "cpu_baseline": {"value": 0.031796, "unit": "TFLOP/s", "cores": 16, "kind": "oracle",
                     "sample": "quant_weight 7168x7168 in full (0.05 s); quant_act and GEMM in full "
                               "(0.03 s + 13.16 s)", "seconds": 13.24},
    "errors": {"rows_checked": 4096, "cols": 7168, "max_err_over_tol": 0.832,
               "tolerance": "|C - C_ref| <= 2e-4 * sum_k |a_k b_k| + 0.5 ulp_bf16",
               "rel_fro_err_vs_bf16_gemm": 0.027893, "rel_fro_err_vs_bf16_gemm_oracle": 0.027844,
               "bf16_rows": 256},
}


def test_the_headline_line_is_short():
    others = {name: {"value": 12345.67, "kernels": {"k": {"ms": 1.0}}, "clocks": {}}
              for _, name in bench.CONFIG_WORKLOADS}
    line = json.dumps(dict(LINE, workloads=bench.short_values(others)))
    assert len(line) < 2900
    assert set(json.loads(line)["workloads"]) == {name for _, name in bench.CONFIG_WORKLOADS}


def test_short_values_keep_three_digits():
    values = {"a": 6.2345, "b": 0.012345, "c": 99.96, "d": 2303.4}
    assert bench.short_values({k: {"value": v} for k, v in values.items()}) == \
        {"a": 6.23, "b": 0.0123, "c": 100.0, "d": 2303}
