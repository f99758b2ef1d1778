"""What of the operators around the experts can be looked over without a GPU,
beside test_experts_abi.py: how their kernels leave a loop after an abort."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_route_scan_gb300", "csrc")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def unvoted(text):
    """Reads of the abort flag, and waits, that each lane decides on by itself."""
    bare = re.sub(r"__(?:any|all)_sync\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\)", "vote", text)
    return re.findall(r"[^;{}]*(?<!&)\bs_abort\b[^;{}]*", bare) + re.findall(r"\b(?:product_wait|wait_or_abort)\(", bare)


def test_product_epilogue_leaves_its_loop_as_a_whole_warp():
    """Its loop has ballots over all lanes: lanes that see the abort flag at different times would part
    there for good."""
    text = code("expert_product.cu")
    body = text[text.index("} else if (warp >= kEpilogueWarp) {") :]
    loop = body[: body.index("__syncthreads();")]
    assert "product_unit(" in loop and "product_wait_warp(" in loop
    assert unvoted(loop) == []


def test_product_waits_end_with_one_answer_for_the_warp():
    text = code("expert_product.cu")
    for name in ("product_wait_warp", "product_wait_all"):
        body = text[text.index(f"bool {name}(") :]
        body = body[: body.index("\n}")]
        assert re.search(r"return __all_sync\(0xffffffffu, \w+(\([^()]*\))?\);$", body.strip()), name
