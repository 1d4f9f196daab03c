"""Rules of the device code that no result on a GPU shows until they are broken at the wrong
moment: read from the sources, without a GPU."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "lvlm_kv_cache_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, head):
    """The braces' contents behind the first `head`."""
    at = text.index("{", text.index(head))
    depth, i = 1, at + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at + 1:i - 1]


def test_warps_meet_before_a_cluster_barrier():
    # barrier.cluster.*.aligned is undefined for a warp whose lanes have not reconverged
    for name in sorted(os.listdir(CSRC)):
        if name != "ptx.cuh":
            assert "barrier.cluster" not in source(name), name
    text = source("ptx.cuh")
    assert text.count("barrier.cluster.arrive") == 1
    assert body(text, "void cluster_sync_all()").strip().startswith("__syncwarp();")


def test_waits_of_the_paged_decode_end_for_whole_warps_and_after_its_copies():
    text = source("paged_decode.cu")
    assert "mbar_wait(" not in text and "__all_sync" in body(source("ptx.cuh"), "bool mbar_wait_warp(")
    producer = body(text, "if (warp == kPdWarps) {")
    assert producer.rindex("mbar_wait_warp(&full[") > producer.rindex("tma_load_5d(")


def test_shared_memory_that_is_read_in_pieces_is_aligned_for_them():
    # dynamic shared memory that is cast to 16-byte vectors says so itself, whatever static arrays lie before it
    for name in ("evict.cu", "elite.cu", "compact.cu"):
        text = source(name)
        assert "uint4*" in text or "float4*" in text
        for decl in re.findall(r"extern __shared__[^;]*;", text):
            assert re.search(r"__align__\((16|32|64|128|1024)\)|alignas\((16|32|64|128|1024)\)|uint4|float4", decl), (name, decl)


def test_host_code_keeps_nothing_that_two_threads_could_set_at_once():
    # a function's static is constant, one to a thread, or of a type that threads may share
    plain = r"^ +static (?!const\b|constexpr\b|thread_local\b|std::mutex\b|std::once_flag\b|std::atomic<|__device__)[^()]*;"
    guarded = {"budget.cu": "std::call_once(", "api.cu": "std::lock_guard<std::mutex> lock(mu);"}
    for name in sorted(os.listdir(CSRC)):
        found = re.findall(plain, source(name), re.M)
        assert not found or guarded.get(name, "nothing") in source(name), (name, found)


def test_kernels_let_the_next_one_start_behind_their_own_wait():
    # a decode with AIRCACHE_DECODE_EARLY_CACHE reads its rows when the kernel before it lets it start: that kernel's
    # predecessors, which may write the rows, have then to be complete
    for name in ("rotate.cu", "paged_decode.cu", "evict.cu", "decode.cu"):
        text = source(name)
        kernels = text.split("__global__")[1:]
        assert kernels, name
        for k in kernels:
            if "pdl_trigger();" in k:
                assert -1 < k.rindex("pdl_wait();") < k.index("pdl_trigger();"), name


def test_every_tile_of_the_paged_decode_is_noted():
    # the mass kernel takes each tile's pages from the workspace: a producer whose wait ran out notes the tiles that it
    # does not copy as not there, or another call's pages would be found in their place
    producer = body(source("paged_decode.cu"), "if (warp == kPdWarps) {")
    gave_up = body(producer, "if (!mbar_wait_warp(&empty")
    assert ".page[lane] = -1;" in gave_up and "while (next_run(" in gave_up
    assert producer.count("break;") == gave_up.count("break;") == 1
