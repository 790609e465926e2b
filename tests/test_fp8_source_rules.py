"""Rules of the e4m3 product's kernels that a wrong run would show only by luck, read off their source."""

import ctypes
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "post_weight_quantization_tcgen05_b200", "csrc")
PRODUCTS = ("fp8_gemm.cu", "fp8_gemm_few.cu")


def code(name):
    """A source file without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_every_cluster_barrier_is_reached_by_whole_warps():
    """The cluster barriers are .aligned: all lanes of a warp execute them together.  So the statement
    before one is a barrier that brings the warp together, of the warp, the CTA or the cluster."""
    whole = re.compile(r"(?:__syncwarp|__syncthreads|ptx::cluster_sync(?:_relaxed)?)\(\)$")
    found = 0
    for name in PRODUCTS:
        before = ""
        for statement in re.split(r"[;{}]", code(name)):
            statement = re.sub(r"^if constexpr \(\w+\) ", "", " ".join(statement.split()))
            if re.fullmatch(r"ptx::cluster_sync(?:_relaxed)?\(\)", statement):
                found += 1
                assert whole.search(before), f"{name}: {statement} after '{before}'"
            if statement:
                before = statement
    assert found == 6


def test_scales_of_a_running_quantiser_are_not_read_as_constants():
    """hq_fp8_linear launches the product while the kernel that writes the activations' scales still runs.
    ld.global.nc (__ldg) is for data that nothing writes while the kernel runs, so no such load may take
    an address made from a_scales; the weights' scales are constants."""
    for name in PRODUCTS:
        src = code(name)
        made = {"a_scales"} | set(re.findall(r"(\w+)\s*=\s*[^;=]*\ba_scales\b", src))
        loads = re.findall(r"(\w+)\(([^()]*(?:\([^()]*\)[^()]*)*)\)", src)
        constant = [arg for f, arg in loads if f == "__ldg" and made & set(re.findall(r"\w+", arg))]
        assert not constant, f"{name}: __ldg({constant[0]})"
        assert any(f == "__ldcg" and made & set(re.findall(r"\w+", arg)) for f, arg in loads), name


def test_every_wait_of_the_products_takes_the_call_s_limit():
    """A wait that gave up only after the library's own limit would hold up a call that was given a shorter
    one.  The waits without an abort flag (nullptr) drain what the CTA issued itself."""
    for name in PRODUCTS:
        waits = re.findall(r"ptx::mbar_wait\(((?:[^()]|\((?:[^()]|\([^()]*\))*\))*)\)", code(name))
        assert len(waits) == 8 and all(w.endswith(("abort_flag, limit", "nullptr")) for w in waits), waits
        assert sum(w.endswith("nullptr") for w in waits) == 2


def test_bad_limits_and_stages_are_refused_before_a_launch():
    import post_weight_quantization_tcgen05_b200 as hq
    p = ctypes.c_void_p(4096)  # never dereferenced

    def call(limit=1_000_000, stage=-1, status=p, impl=1, rows=2, offsets=None, E=1, dt=0):
        return hq.lib.hq_debug_fp8_gemm_timeout(p, p, rows, offsets, p, p, E, 4, 8, p, dt, status, impl, limit, stage, None)
    assert call(rows=0) == hq.HQ_OK
    for kw in ({"limit": 99_999}, {"limit": 4_000_000_001}, {"stage": -2}, {"stage": 4}, {"status": None}, {"impl": 5},
               {"impl": -1}, {"E": 2}, {"dt": 2}):
        assert call(**kw) == hq.HQ_ERR_INVALID, kw
    assert call(dt=1) == hq.HQ_ERR_UNSUPPORTED
