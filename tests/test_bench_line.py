"""The benchmark's printed result line (no GPU)."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_result_line_stays_short():
    """The printed line keeps the headline's figures as they are and a few
    kilobytes of length; the secondary legs' full figures go beside it."""
    x = 1234.5678901234567
    metrics = dict(us_per_call=x, p10_us=x, p90_us=x, cv_pct=x, gbs=x, frac_of_hbm_peak=x, tflops=x, frac_of_tensor_peak=x,
                   frac_of_tensor_peak_sustained=x, roofline_us=x, frac_of_roofline=x, bound="hbm")
    sweep = {M: {"library_choice": "rows", "paths": {p: metrics for p in ("rows", "tc", "tile", "pair", "auto", "cublas_addmm")}}
             for M in ("32", "64", "128")}
    low = {"per_m": [dict(m=m, kernel="w8_rows_kernel", us=x, gbs=x, frac_of_hbm_peak=x) for m in (1, 2, 4, 16)], "note": "n" * 200}
    line = {"metric": bench.METRIC, "value": x, "ms_per_step": x, "config": {"workload": "w" * 250}, "headline": {"note": "h" * 330},
            "per_m": {str(M): {**metrics, "path": "rows", "cublas_addmm": metrics, "measured_again_last": metrics}
                      for M in bench.M_LIST},
            "transition": sweep, "compute_bound": sweep, "roofline": {"note": "r" * 520}, "cpu_baseline": {"sample": "c" * 500},
            "e2e": {"value": x, "unit": "GB/s", "note": "e" * 230}, "chain": dict(us_per_layer=x, us_per_layer_no_pdl=x, note="n"),
            "grouped": None, "w8": low, "w4": low,
            "down_projection": {"per_m": [dict(m=m, us=x, p10_us=x, cublas_addmm_us=x) for m in (1, 4, 16, 32, 64)]},
            "gpu_launches": 1, "clocks": {"sm_mhz": x}, "peaks": {"hbm_gbs": x}}
    short, legs = bench.short_line(line)
    assert len(json.dumps(short)) < 5000
    assert list(short) == list(line) and short["grouped"] is None
    for k in ("metric", "value", "ms_per_step", "config", "headline", "roofline", "cpu_baseline", "e2e", "gpu_launches", "clocks", "peaks"):
        assert short[k] == line[k]
    assert legs == {k: line[k] for k in bench.LEGS if k != "grouped"}
    assert short["per_m"]["4"] == {"us": 1234.6, "cublas_us": 1234.6, "gbs": 1234.6, "path": "rows"}
    assert short["transition"]["64"] == {"path": "rows", "us": 1234.6, "cublas_us": 1234.6}
    assert short["w4"]["16"] == 1234.6 and short["down_projection"]["32"] == {"us": 1234.6, "cublas_us": 1234.6}
