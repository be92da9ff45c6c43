"""What the library's sources keep to, where no call can show it: failures that cannot be made to order."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def sources():
    out = {}
    for path in sorted(glob.glob(os.path.join(ROOT, "persistent_kv_cache_gb300", "csrc", "*.cu*"))):
        with open(path) as f:
            out[os.path.basename(path)] = re.sub(r"//[^\n]*", "", f.read())
    assert len(out) >= 12
    return out


def test_errors_of_cuda_are_read_where_they_are_returned():
    """A call that fails leaves no error behind for the next one to find."""
    for name, text in sources().items():
        if name == "kvc_common.cuh":
            # launch_status and cuda_failed read it
            assert len(re.findall(r"KVC_ERR_CUDA", text)) == text.count("cudaGetLastError()") == 2
        else:
            assert not re.findall(r"return\s+KVC_ERR_CUDA", text) and not re.findall(r"[?:]\s*KVC_ERR_CUDA\b\s*[;)]", text), name


def test_ragged_kernels_load_by_ordinary_loads():
    """The kernels of a ragged step may start before the kernel in front of them has ended: what that one may write (a
    plan the table, an append the queries) was not read-only for their whole life, as the non-coherent path wants it."""
    text = sources()
    for name in ("kvc_ragged.cu", "kvc_ragged_attn.cu"):
        assert "launch_chained" in text[name]
        assert not re.findall(r"__ldg|__ldnc|ld\.global(\.\w+)*\.nc|__restrict__ (?!cos_t|sin_t)", text[name]), name


def test_waits_of_whole_warps_have_one_answer():
    """A warp that loads and stores tensor memory, votes and shuffles as a whole decides as a whole whether it does: in
    the softmax warps of the ragged attention a vote comes between the last wait and every such question."""
    text = sources()["kvc_ragged_attn.cu"]
    kernel = text[text.index("ragged_attn_kernel(const"):text.index("ragged_merge_kernel(const")]
    softmax = kernel[kernel.index("quad = warp & 3"):]
    assert "tcgen05" not in softmax and "mbar_wait" not in softmax
    asked = [m.start() for m in re.finditer(r"\bactive && ok\b", softmax)]
    assert len(asked) == 3 and not re.findall(r"\bok && active\b|if \(ok\)", softmax)
    given = [(m.start(), m.group(1)) for m in re.finditer(r"\bok = ([^;]*);", softmax)]
    for at in asked:
        last = [what for begin, what in given if begin < at][-1]
        assert "warp_wait_or_abort(ok, " in last or "__all_sync(0xffffffffu, ok)" in last, last


def test_chained_kernels_wait_before_they_write_or_end():
    """A kernel that may start before the one in front has ended waits for that in every block, also in one that has
    nothing to do: the kernel behind counts on all before it having ended too."""
    text = sources()
    kernels = {"kvc_ragged.cu": ("page_release_kernel", "ragged_plan_kernel", "ragged_append_kernel"),
               "kvc_ragged_attn.cu": ("ragged_attn_kernel", "ragged_merge_kernel")}
    for name, ones in kernels.items():
        for kernel in ones:
            body = re.search(kernel + r"\(const .*?\n\}\n", text[name], re.S).group(0)
            before = body[:body.index("grid_dep_wait()")]
            assert "return" not in before and "raise_status" not in before and not re.findall(r"\ba\.\w+\[[^\]]*\] = ", before), kernel
