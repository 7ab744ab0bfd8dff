"""The benchmark's line on stdout is short: a reader of a log's end gets all of it (CPU only)."""
import json
import math


def _workload(i):
    number = 1234.5678901234567 + i
    kernels = {f"some_kernel_of_the_step_{k}": {"ms_per_step": number / 3, "share": 0.0625} for k in range(20)}
    stages = {f"stage_{k}": {"kernels": ["router_logits", "topk_softmax", "permute"], "bytes": 10 ** 10 + i,
                             "ms_per_step": number / 7, "gbs": number * 3, "frac_of_hbm": number / 9999} for k in range(4)}
    return {"workload": f"w{i}: T=32768 d=1536 E=512 n=256 K=8", "ms_per_step": number, "tflops": number, "pct_of_peak_bf16": 33.3,
            "tokens_per_s": number * 1e5, "pairs": 262144, "roofline": dict(stages["stage_0"], kernel="k", tflops=number),
            "hbm_stages": stages, "kernels": kernels, "activation_memory": dict(stages["stage_1"]), "steps": 10}


def test_line_keeps_its_keys_and_figures_and_is_short():
    import bench
    main = _workload(0)
    line = {"metric": "m", "value": 570.8491214988177, "unit": "TFLOP/s", "n_gpus": 1, "steps": 20, "warmup": 5,
            "ms_per_step": 1.0834303975105286, "higher_is_better": True, "vs_baseline": None, "config": {"workload": "c2"},
            "gpu_launches": 320, "clocks": {"sm_mhz": 2070.0, "reasons": ["sw_power_cap"]}, **{k: main[k] for k in (
                "roofline", "hbm_stages", "kernels", "activation_memory")},
            "e4m3_forward": {f"some_time_of_a_form_{k}_ms": 0.1234567890123456 for k in range(60)},
            "per_workload": {f"w{i}": _workload(i) for i in range(4)}}
    whole, text = json.dumps(line), json.dumps(bench.short_line(line))
    assert len(whole) > 16000 and len(text) < 10000
    short = json.loads(text)
    assert set(short) == set(line) and set(short["per_workload"]) == set(line["per_workload"])

    def same(a, b):
        if isinstance(b, dict):
            return all(same(a[k], b[k]) for k in b)
        if isinstance(b, float):
            return math.isclose(a, b, rel_tol=5e-6)
        return a == b and type(a) is type(b)

    assert all(same(line[k], short[k]) for k in line)
    for w in short["per_workload"].values():
        assert set(w) == {"workload", "ms_per_step", "tflops", "pct_of_peak_bf16", "tokens_per_s", "steps"}


def test_line_without_further_workloads():
    import bench
    for none in (None, {}):
        assert bench.short_line({"value": 1.0, "per_workload": none}) == {"value": 1.0, "per_workload": none}
