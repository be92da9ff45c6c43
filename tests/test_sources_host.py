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


def test_what_the_first_kernel_of_a_call_writes_is_loaded_by_ordinary_loads():
    """The same where a call's second kernel begins while its first one runs."""
    text = sources()
    assert not re.findall(r"__ldg\(see_words", text["kvc_tree.cu"]) and text["kvc_tree.cu"].count("see_words[") == 2
    decode = text["kvc_sparse.cu"][text["kvc_sparse.cu"].index("sparse_decode_kernel(const"):]
    assert "a.sub_table" in decode and not re.findall(r"__ldg\((?!a\.(cos|sin)_t)", decode)


def test_nothing_hangs_on_what_a_wait_of_softmax_warps_answers():
    """Lanes whose bounded wait runs out do so one by one, and what follows wants whole warps (tensor memory) and every
    warp (barriers without a limit): the answer, which is the flag that the lane has set or found, is asked for at the
    stores alone."""
    text = sources()
    kernel = text["kvc_ragged_attn.cu"]
    softmax = kernel[kernel.index("quad = warp & 3"):kernel.index("ragged_merge_kernel(const")]
    prefill = text["kvc_prefill.cu"]
    tiles = prefill[prefill.index("float m_run", prefill.index("pair_bar = 1 + quad")):prefill.index("prefill_combine_kernel(")]
    for section, waits in ((softmax, 7), (tiles, 4)):
        assert "tcgen05" not in section
        # (each a statement of its own)
        assert len(re.findall(r"wait_or_abort\(", section)) == len(re.findall(r"(?<=[;{})])\s*(else\s+)?wait_or_abort\([^;]*\);", section)) == waits
    # the flag: a store's condition, where no load or barrier follows that not all come to; a vote
    assert re.findall(r".*\*abort_flag", softmax) == ["            const bool there = tok < a.toks && first + tok < seg.n && !*abort_flag"]
    stores = softmax[softmax.index("if (!there)"):softmax.index("if (!whole && there && col0 == 0)")]
    assert "kvc_tc::ld" not in stores and "sync(" not in stores and softmax.count("!there") == 1
    assert "const bool have_o = __all_sync(0xffffffffu, !*abort_flag);" in tiles
    assert re.search(r"if \(sw == 0 && lane == 0 && !\*abort_flag\)", tiles)


def test_decode_warps_leave_their_tiles_whole():
    """The decodes' tiles are the work of whole warps (shuffles, products): a lane's answer to a wait goes through a vote
    before a branch hangs on it."""
    text = sources()["kvc_decode.cu"]
    tiles = text[text.index("bool timed_out = false;"):text.index("if (timed_out) {")]
    assert len(re.findall(r"\bthere = kvc::mbar_wait\(", tiles)) == 2 and tiles.count("mbar_wait(") == 3
    assert len(re.findall(r"\bthere\b", tiles)) == 4 and len(re.findall(r"if \(!__all_sync\(0xffffffffu, there\)\) \{\s*timed_out = true;\s*break;", tiles)) == 1
    # (and the loads in flight land before the warps meet)
    left = text[text.index("if (timed_out) {"):]
    left = left[:left.index("consumer_sync();")]
    assert left.index("atomicExch(abort_flag, 1);") < left.index("kvc::mbar_wait(&full[(at + k) % NBAR], (uint32_t)((at + k) / NBAR) & 1u);")
    step = text[text.index("window_step_kernel("):]
    step = step[:step.index("__syncthreads_and(ok)")]
    assert re.findall(r"(?<!_)\bok = [^;]*;", step) == ["ok = true;", "ok = __all_sync(0xffffffffu, kvc::mbar_wait(&bar[t], 0)) && ok;"]


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
