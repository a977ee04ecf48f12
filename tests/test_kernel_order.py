"""Orders of instructions that no run can show to be wrong without hanging or racing, read from the
kernels' sources."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_head_gb300", "csrc")


def _sources():
    """{file: text without comments}"""
    out = {}
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h", ".cpp")):
            with open(os.path.join(CSRC, name)) as f:
                out[name] = re.sub(r"//[^\n]*", "", f.read())
    return out


def _body(text, at):
    """The block in braces that begins behind `at`."""
    begin = text.index("{", at)
    depth = 0
    for i in range(begin, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[begin:i + 1]
    raise AssertionError("unbalanced braces")


def test_no_tmem_is_held_across_the_wait_for_the_kernel_before():
    """A kernel that may begin before the one ahead of it has finished allocates TMEM behind its
    wait: the other one may yet have to allocate its own."""
    kernels = 0
    for name, text in _sources().items():
        if "launch_after(kernel" not in text:
            continue
        for m in re.finditer(r"__global__ void", text):
            body = _body(text, text.index("(", text.index("bsa_", m.end())))
            assert "wait_before();" in body, name
            if "tmem_alloc(" in body:
                kernels += 1
                assert body.index("wait_before();") < body.index("tmem_alloc("), name
                # by the allocating warp itself, not by others beside it
                warp = body[body.rindex("if (warp ==", 0, body.index("tmem_alloc(")):]
                assert "wait_before();" in _body(warp, 0)
    assert kernels == 2  # the differential forward and backward


def test_a_warp_learns_of_other_blocks_writes_behind_a_barrier():
    """One lane's acquire orders the other lanes' loads only through a barrier between them: whoever
    asks a count for a warp uses the wrappers that have it, or a barrier of the block."""
    text = _sources()
    ptx = text["bsa_ptx.cuh"]
    for name, asked in (("warp_load_acquire", "load_acquire("), ("warp_add_acq_rel", "add_acq_rel(")):
        body = _body(ptx, ptx.index(f"int {name}("))
        ask, tell = body.index(asked), body.index("__shfl_sync")
        assert "__syncwarp();" in body[ask:tell], name
        if name == "warp_add_acq_rel":  # the other lanes' writes before lane 0 announces them
            assert "__syncwarp();" in body[:ask]
    for call in re.findall(r"\w*(?:load_acquire|add_acq_rel)\(", text["bsa_diff_bwd_kernel.cuh"]):
        assert call.startswith("warp_"), call
