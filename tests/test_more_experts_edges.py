"""What of the int8 product's pipeline can be looked over without a GPU: how its warps leave their loops after an
abort, and that a CTA leaves only when nothing can arrive in its shared memory any more."""
import re

import pytest
from test_experts_edges import code, unvoted


def kernel():
    text = code("int8_product.cu")
    body = text[text.index("int8_product_kernel(const __grid_constant__") :]
    return body[: body.index("\n}\n")]


def part(begin, end):
    body = kernel()
    body = body[body.index(begin) :]
    return body[: body.index(end)]


COPIES = ("if (warp == 0) {\n    const bool leader", "} else if (warp == 1) {")
MMAS = ("} else if (warp == 1) {", "} else if (warp < kWidenWarp")
WIDENING = ("} else if (warp < kWidenWarp", "} else {\n    const uint32_t q = warp & 3;")
EPILOGUE = ("} else {\n    const uint32_t q = warp & 3;", "\n  __syncthreads();")


def test_accumulators_go_back_only_to_units_that_wait_for_them():
    """The other CTA's epilogue arrives on the first one's barriers: an arrival that no MMA waits for could come when that
    CTA has left, which the closing barrier of the cluster, that releases nothing, does not prevent."""
    loop = part(*EPILOGUE)
    arrivals = re.findall(r"if \(([^()]*)\) mbar_arrive_cluster\(empty0 \+ buf \* 8\);", loop)
    assert len(arrivals) == loop.count("mbar_arrive_cluster(") == 2
    assert all(a == "lane == 0 && taken_again" for a in arrivals)
    # two accumulators in turn, a pair's units as many apart as there are pairs
    assert "const bool taken_again = at.u + 2 * (int)(gridDim.x >> 1) < units;" in loop
    assert "u += gridDim.x >> 1;" in code("int8_product.cu")


def test_widening_sets_wait_for_the_commit_of_their_last_slot():
    """It arrives in both CTAs from the first one's tensor cores."""
    body = part(*WIDENING)
    behind = body[body.rindex("for (; kb >= KB && at.u < units; kb -= KB) at.next();") :]
    assert "if (ok) int8_wait(wide_empty0 + set * 8, slot_phase, ab);" in behind
    # a set without a stage asks for the phase before the first one, which is there
    assert "raw_phase = 0, slot_phase = 1;" in body and "slot_phase ^= 1;" in body


@pytest.mark.parametrize("where", [WIDENING, EPILOGUE], ids=["widening", "epilogue"])
def test_warps_leave_their_loops_whole(where):
    """Their tensor-memory loads and stores want all lanes: no lane decides by itself."""
    loop = part(*where)
    assert unvoted(loop) == []
    assert re.findall(r"int8_(?:sleep|wait_one|wait_long)\(", loop) == []
    text = code("int8_product.cu")
    for name in ("int8_wait", "int8_wait2"):
        body = text[text.index(f"bool {name}(") :]
        last = body[: body.index("\n}")].strip().splitlines()[-1]
        assert re.fullmatch(r"\s*return __all_sync\(0xffffffffu, int8_wait_long\([^()]*\)\);", last) or last.count("int8_wait(") == 2, name


@pytest.mark.parametrize("where", [COPIES, MMAS], ids=["copies", "mmas"])
def test_issuing_warps_agree_on_an_abort(where):
    """One thread issues; the warp goes on to the next unit only with its answer."""
    loop = part(*where)
    assert "at.u < units && ok;" in loop and "ok = __all_sync(0xffffffffu, ok);" in loop


def test_every_wait_ends_and_copies_in_flight_are_given_time():
    text = code("int8_product.cu")
    long = text[text.index("bool int8_wait_long(") :]
    long = long[: long.index("\n}")]
    assert "if (*flag) return false;" in long and re.search(r"globaltimer_ns\(\) - t0 > limit", long)
    # what asks for a phase outside of those waits has a limit of its own
    tail = kernel()
    tail = tail[tail.rindex("if (threadIdx.x == 0) {") : tail.index("tmem_dealloc_pair(")]
    assert len(re.findall(r"while \([^{]*globaltimer_ns\(\) - t0 < 1000000ull\)", tail)) == 2
    assert "if (s_abort)" in tail
    body = kernel()[: -len(tail)]
    assert "mbar_try_wait(" not in body[: body.rindex("if (threadIdx.x == 0) {")]
    # tensor memory goes back behind the cluster's barrier
    assert "cluster_sync();" in tail
