"""The line that bench.py prints, with the workloads stood in for by records of
the size that real ones have."""

import importlib.util
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# keys and lengths of a measured record
RECORD = {
    "workload": "decode32",
    "config": {"workload": "decode32: 32 token(s), hidden 4096, 256 routed experts (mxfp4) + 1 "
                           "shared (mxfp4), intermediate 2048, top-6, learned routing, bf16 "
                           "activations, 8 cold layer copies",
               "n_tokens": 32, "packed_experts": True},
    "routed_slots_per_step": 192.0, "value": 115617.76096197456, "unit": "tokens/s",
    "steps": 400, "warmup": 20, "ms_per_step": 0.27677408500000666,
    "step_stats": {"reps": 5, "steps_per_rep": [80] * 5, "us_per_step_median": 276.5861749649048,
                   "us_per_step_min": 276.29170417785645, "us_per_step_max": 277.38709449768066,
                   "spread_over_15pct": False},
    "roofline": {"kernel": "routed gate/up kernel of moe_ffn_forward (+ SwiGLU), with the shared "
                           "expert's items",
                 "bound": "hbm", "achieved": 5836.342671792411, "peak": 8000.0, "unit": "GB/s",
                 "frac": 0.7295428339740514, "traffic": 984323636.1031737,
                 "bytes_per_launch": 966509199.36, "flops_per_launch": 7516192768.0,
                 "flop_per_byte": 7.776638621729672, "avg_launch_us": 165.60185953974724,
                 "timed_launches": 100,
                 "timing": "dispatch-recorded HIP events on every step of a 100-step pass right "
                           "after the timed steps (same rotation, cold)",
                 "hbm_frac": 0.7295428339740514, "mfma_bf16_frac": 0.018154851132443927,
                 "peak_note": "bf16-equivalent: " + 180 * "x",
                 "issued_flops_per_launch": 15032385536.0,
                 "issued_frac_of_fp8_peak": 0.018154851132443927},
    "path": {"bytes_per_step": 1448887808.0, "achieved_GBps": 5234.911382689477,
             "hbm_frac": 0.6543639228361846, "flops_per_step": 11274289152.0,
             "achieved_TFLOPs": 40.73462713100371, "mfma_bf16_frac": 0.016293850852401485},
    "down_kernel": {"kernel": "routed down kernel of moe_ffn_forward, with the shared expert's "
                              "items",
                    "bytes_per_launch": 483647815.68, "flops_per_launch": 3758096384.0,
                    "avg_launch_us": 91.26989006996153, "achieved_GBps": 5299.094973263003,
                    "achieved_TFLOPs": 41.17564271326819, "mfma_bf16_frac": 0.016470257085307277,
                    "issued_frac_of_fp8_peak": 0.024705385627960912},
    "cpu_baseline": {"value": 2.1593798280999956, "unit": "tokens/s", "cores": 16,
                     "kind": "oracle", "sample": 130 * "x"},
}


@pytest.fixture
def bench(monkeypatch):
    spec = importlib.util.spec_from_file_location("bench", os.path.join(ROOT, "bench.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    asked = []

    def run_workload(name, steps, warmup, *_, variant=None):
        asked.append(variant or name)
        return dict(RECORD, workload=variant or name, steps=steps, warmup=warmup)

    monkeypatch.setattr(module, "run_workload", run_workload)
    monkeypatch.setattr(module, "read_ceiling", lambda dev: {"kernel": 200 * "x"})
    monkeypatch.setattr(module, "mfma_ceiling", lambda dev: {"kernel": 300 * "x"})
    module.asked = asked
    return module


def _line(bench, monkeypatch, capsys, *argv):
    monkeypatch.setattr(sys, "argv", ["bench.py", *argv])
    bench.main()
    out = capsys.readouterr().out
    assert out.count("\n") == 1 and out.endswith("\n")
    return out, json.loads(out)


def test_the_line_is_short_and_has_the_contracts_keys(bench, monkeypatch, capsys):
    # where a few KB of a run's output are kept, a line of 22 KB lost its beginning
    out, line = _line(bench, monkeypatch, capsys, "--gpus", "1", "--steps", "20", "--warmup", "5")
    assert len(out) < 6000
    want = {"metric": bench.METRIC, "value": RECORD["value"], "unit": "tokens/s", "n_gpus": 1,
            "steps": 20, "warmup": 5, "ms_per_step": RECORD["ms_per_step"],
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "data": "synthetic",
            "roofline": RECORD["roofline"], "step_stats": RECORD["step_stats"]}
    assert {k: line[k] for k in want} == want
    nested = bench.NESTED + list(bench.VARIANTS)
    assert list(line["configs"]) == nested and bench.asked == nested + [bench.HEADLINE]
    for rec in line["configs"].values():
        assert rec["value"] == 115617.8 and rec["ms_per_step"] == 0.276774
        assert rec["roofline"] == {"bound": "hbm", "frac": 0.7295, "avg_launch_us": 165.6}
        assert rec["cpu_tokens_per_s"] == 2.159


def test_records_are_kept_in_full_in_a_file(bench, monkeypatch, capsys, tmp_path):
    path = tmp_path / "records.json"
    _, line = _line(bench, monkeypatch, capsys, "--records", str(path))
    full = json.loads(path.read_text())
    assert {k: v for k, v in full.items() if k != "configs"} == {
        k: v for k, v in line.items() if k != "configs"}
    st, wu = bench.DEFAULTS["decode32"][:2]
    assert full["configs"]["decode32"] == dict(RECORD, steps=st, warmup=wu)


def test_one_workload_alone_has_no_configs(bench, monkeypatch, capsys):
    _, line = _line(bench, monkeypatch, capsys, "--workload", "decode1_top4", "--steps", "3")
    assert "configs" not in line and line["steps"] == 3 and bench.asked == ["decode1_top4"]
