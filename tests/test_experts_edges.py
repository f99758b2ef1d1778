"""What of the operators around the experts can be looked over without a GPU,
beside test_experts_abi.py: how their kernels leave a loop after an abort, and
where their binding is needed."""
import os
import re
import subprocess
import sys

import pytest

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


def test_ffn_epilogue_leaves_its_loops_as_a_whole_warp():
    """Its tensor-memory loads want all lanes, as the product's votes do; and a unit that an abort cut off
    is not counted as stored."""
    text = code("ffn.cu")
    body = text[text.index("const int feat = 32 * q + lane;") :]
    loop = body[: body.index("tmem_dealloc(")]
    loop = loop[: loop.rindex("__syncthreads();")]
    assert "tc_ld16(" in loop and "wait_or_abort(" in loop
    assert unvoted(loop) == []
    assert loop.index("if (cut) break;") < loop.index("red.release")


def test_ffn_lets_its_copies_end_after_an_abort():
    """Nobody waits for the copies and MMAs under way then: the block does, for a bounded time, before its
    shared and tensor memory are given back."""
    text = code("ffn.cu")
    end = text[text.index("const int feat = 32 * q + lane;") : text.index("tmem_dealloc(tmem, kTmemCols);")]
    behind = end[end.rindex("__syncthreads();") :]
    assert re.search(r"if \(s_abort\) \{[^}]*globaltimer_ns\(\) - t0 < \d+ull", behind)


def test_product_waits_end_with_one_answer_for_the_warp():
    text = code("expert_product.cu")
    for name in ("product_wait_warp", "product_wait_all"):
        body = text[text.index(f"bool {name}(") :]
        body = body[: body.index("\n}")]
        assert re.search(r"return __all_sync\(0xffffffffu, \w+(\([^()]*\))?\);$", body.strip()), name


def test_product_waits_for_every_arrival_of_its_scale_warps():
    """Each of their commits arrives on a barrier in shared memory: the last one before the block ends, too."""
    text = code("expert_product.cu")
    body = text[text.index("} else if (warp < 2 + kScaleWarps) {") : text.index("} else if (warp >= kEpilogueWarp) {")]
    behind = body[body.rindex("tc_commit_if(leader, smem_u32(&taken[mine]));") :]
    assert "product_wait_all(smem_u32(&taken[mine]), taken_phase, ab)" in behind


# ------------------------------------------------------------------ the native binding

def child(program):
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


@pytest.fixture(scope="module")
def build():
    from combine_route_scan_gb300 import build
    build.build()
    return build


def test_dispatch_and_combine_do_without_the_native_binding(build):
    """The calls of include/moe.h need the library alone; those of include/moe_experts.h say what is missing."""
    out = child("""
import os.path, torch
there = os.path.exists
os.path.exists = lambda p: "_bind" not in str(p) and there(p)
from combine_route_scan_gb300 import moe
print(moe.workspace_size(moe.config(2, 4, 64, 2, 4, torch.bfloat16))[1])
try:
    moe.route(moe.router_config(4, 64, 8, torch.float32), torch.zeros(4, 64), None, None, None)
except RuntimeError as e:
    print("missing" in str(e))
""")
    assert out.split() == ["16", "True"]


def test_library_is_built_where_the_binding_cannot_be(build, monkeypatch):
    def fail():
        raise RuntimeError("no Python.h")

    monkeypatch.setattr(build, "_bind_stale", lambda: True)
    monkeypatch.setattr(build, "build_bind", fail)
    with pytest.warns(RuntimeWarning, match="no Python.h"):
        assert build.build() == build.LIB


def test_binding_of_another_torch_is_not_taken_for_this_one(build, monkeypatch):
    import torch
    assert not build._bind_stale()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert build._bind_stale()


def test_binding_of_another_python_is_not_taken_for_this_one(build, monkeypatch):
    there = build.sysconfig.get_config_var
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else there(name))
    assert build._bind_stale()
