"""The benchmark's line: what it says of the variants, and that it stays short."""
import json


def layer(ms, **more):
    return {"workload": "qwen30b-128k", "dtype": "bf16", "logit_scale": 16.0, "alpha": 0.1, "mean_correction": True,
            "ms_per_layer": ms, "dense_equiv_tflops": 14216.66,
            "stages_ms": {"discover": 1.839, "select": 0.0189, "sparse_attn": 8.046, "discover_select_fused": 1.9543},
            "timing": "medians of 10 event-timed calls", "density": 0.06019, "attn_tflops": 1182.41, "attn_peak_tflops": 1729.8,
            "attn_frac": 0.6836, "dense_attn_ms": 90.0498, "speedup_vs_own_dense": 9.096, "device_status": 0, **more}


def point(alpha):
    return {"logit_scale": 1.0, "alpha": alpha, "mean_correction": False, "density": 0.99999, "ms_per_layer": 358.6851,
            "stages_ms": {"discover": 6.4787, "select": 0.045, "sparse_attn": 352.1615},
            "err_vs_oracle": {"max_abs": 4e-05, "mean_abs": 6e-06}, "err_vs_dense": {"max_abs": 4e-05, "rel_fro": 0.00235},
            "index_flips_outside_band": 0, "mean_correction_overhead_ms": 8.0057}


def test_variants_are_tables():
    import bench
    rules = {f"rule_{i}": {"density": 0.06, "attn_ms": 8.04, "rel_err_vs_dense": 1.09} for i in range(5)}
    variants = {"a": layer(9.9, selection_ablation=rules, mean_correction_overhead_ms=1.54)}
    variants.update({f"v{i}": layer(10.0 + i) for i in range(5)})
    variants["chunk"] = {"workload": "chunk-512", "auto_split": layer(0.95, kv_splits=7), "no_split": layer(1.79, kv_splits=1),
                         "attn_speedup_from_split": 2.097}
    variants["32k"] = {"workload": "llama8b-32k", **{k: layer(5.9) for k in ("x", "y", "z", "w")}}
    variants["varlen"] = {"workload": "varlen", **{k: layer(35.4) for k in ("x", "y")}}
    variants["sweep"] = {t: {"workload": "qwen30b-256k", "dtype": t, "alphas": [0.2], "oracle_seconds": 26.7,
                             "points": [point(0.2 / (1 + i)) for i in range(20)]} for t in ("bf16", "e4m3")}
    got = bench.packed(variants)
    rows = [{**got["layers"]["all"], **dict(zip(got["layers"]["columns"], r))} for r in got["layers"]["rows"]]
    assert [r["variant"] for r in rows] == ["a"] + [f"v{i}" for i in range(5)] + ["chunk.auto_split", "chunk.no_split"] + [
        f"32k.{k}" for k in "xyzw"] + ["varlen.x", "varlen.y"]
    assert rows[0]["ms_per_layer"] == 9.9 and rows[0]["stages_ms.sparse_attn"] == 8.046 and rows[0]["kv_splits"] is None
    assert rows[6]["kv_splits"] == 7 and got["chunk.attn_speedup_from_split"] == 2.097
    assert rows[0]["timing"] == "medians of 10 event-timed calls" and "timing" not in got["layers"]["columns"]
    assert got["selection_ablation"]["rows"][4] == ["rule_4"] and got["selection_ablation"]["all"]["attn_ms"] == 8.04
    sweep = got["sweeps"]["sweep.e4m3"]
    assert sweep["dtype"] == "e4m3" and len(sweep["points"]["rows"]) == 20
    last = {**sweep["points"]["all"], **dict(zip(sweep["points"]["columns"], sweep["points"]["rows"][19]))}
    assert last["alpha"] == 0.01 and last["err_vs_dense.rel_fro"] == 0.00235
    assert len(json.dumps(got)) < 9000 < len(json.dumps(variants))
