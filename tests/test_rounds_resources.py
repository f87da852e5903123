"""Register and scratch budgets of the kernels around a round for gfx950 (a device-only compile;
no GPU needed): nothing in scratch memory, no spilled vector registers, and two workgroups of the
attention on a CU (its loads in flight are what the plan of pieces counts on)."""

from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_resources import _hipcc_available, _remarks

SOURCES = ["rules.hip", "history.hip", "attend.hip", "pages.hip"]


@pytest.fixture(scope="module")
def resources(tmp_path_factory):
    if not _hipcc_available():
        pytest.skip("hipcc is not available")
    d = tmp_path_factory.mktemp("res")
    with ThreadPoolExecutor(max_workers=4) as pool:
        futures = {s: pool.submit(_remarks, s, str(d / (s + ".o"))) for s in SOURCES}
        return {s: f.result() for s, f in futures.items()}


def test_no_scratch_and_no_vector_spills(resources):
    for src, kernels in resources.items():
        assert kernels, f"no kernel remarks for {src}"
        for name, r in kernels.items():
            assert r["ScratchSize [bytes/lane]"] == "0", f"{name} uses scratch"
            assert r["VGPRs Spill"] == "0", f"{name} spills vector registers"


def test_attention_keeps_two_workgroups_a_cu(resources):
    seen = 0
    for name, r in resources["attend.hip"].items():
        if "attend_kernel" in name or "attend_wide_kernel" in name:
            seen += 1
            assert int(r["Occupancy [waves/SIMD]"]) >= 2, f"{name}: {r}"
            assert int(r["LDS Size [bytes/block]"]) <= 80 * 1024, f"{name}: {r}"
    assert seen >= 8
