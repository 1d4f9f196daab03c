"""Rules of the device code that no result on a GPU shows until they are broken at the wrong
moment: read from the sources, without a GPU."""
import os
import re
import subprocess

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


def test_paged_attention_lets_the_next_kernel_start_behind_its_own_wait():
    # (its join may let one start before, where that is the same call's: results that are a part of another's)
    kernels = source("paged_attend.cu").split("__global__")[1:]
    assert len(kernels) == 3
    for k in kernels:
        waits, starts = k.index("pdl_wait();"), [m.start() for m in re.finditer(r"pdl_trigger\(\);", k)]
        early = [s for s in starts if s < waits]
        assert starts and max(starts) > waits
        assert [k[s - 19:s].strip() for s in early] == ["if (a.part.out)"] * len(early)
    text = source("shared_decode.cu")
    assert text.index("attend_launch(&pl.at") < text.rindex("paged_decode_run(&p->own, prior")


def test_a_decode_that_starts_early_waits_before_it_ends_and_before_it_joins():
    text = source("paged_decode.cu")
    kernel = text[text.index("paged_decode_kernel(const"):text.index("struct Joined {")]
    assert kernel.count("if (late) prior_wait();") == kernel.count("return;") + 1  # at each way out
    assert body(text, "Joint joint(").strip().startswith("prior_wait();")
    assert "if (!late) pdl_wait();" in kernel and "if (!late || !SHORT) pdl_trigger();" in kernel


def test_waits_of_the_paged_attention_end_for_whole_warps():
    text = source("paged_attend.cu")
    assert "mbar_wait(" not in text and "named_bar_sync" not in text and "bar.sync" not in text
    # each wait's answer is looked at, but for those that let copies and products end
    for line in text.split("\n"):
        if "mbar_wait_warp(" in line and "(void)" not in line:
            assert re.search(r"ok = |&& |return |if \(!", line) or "mbar_wait_warp(&ctl->turn" in line, line


def test_registers_that_the_paged_attention_shares_out():
    # what setmaxnreg adds up to may not pass what the launch brings, or it waits for ever: stated in the source, and the
    # launch compares the built kernel's registers with it
    text = source("paged_attend.cu")
    assert "256 * kRegsSoft + (kThreads - 256) * kRegsOther <= kThreads * kRegs" in text
    assert "if (regs < C::kRegs) return AIRCACHE_ERR_CUDA;" in text
    assert text.count("setmaxnreg") == 2


def test_division_by_a_constant_holds_over_its_range(tmp_path):
    # rows of a sequence (of 16, to its pages) run up to 2^31: a product that passes 64 bits would name another page
    with open(os.path.join(CSRC, "paged_attend.cu")) as f:
        text = f.read()
    at = text.index("struct AtDivisor {")
    code = text[at:text.index("struct AtArgs {", at)]
    main = """
#include <cstdint>
#include <cstdio>
#define __host__
#define __device__
#define __forceinline__ inline
%s
int main() {
  long bad = 0;
  for (int d = 1; d <= 304; ++d) {
    const AtDivisor by = divisor(d);
    auto check = [&](int64_t x) { bad += x >= 0 && x < (1ll << 31) && by.quotient((int)x) != x / d; };
    for (int64_t x = 0; x < 3000; ++x) check(x), check((1ll << 31) - 1 - x);
    for (int b = 10; b < 31; ++b)
      for (int64_t k = -40; k <= 40; ++k) check((1ll << b) + k), check(((1ll << b) / d + k) * d), check(((1ll << b) / d + k) * d - 1);
  }
  printf("%%ld\\n", bad);
}
""" % code
    src, exe = tmp_path / "divide.cpp", tmp_path / "divide"
    src.write_text(main)
    subprocess.run(["g++", "-O1", "-std=c++17", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.strip() == "0"


def test_the_second_walk_waits_for_the_columns_that_it_clears():
    # tcgen05.ld is ordered behind an earlier tcgen05.st of the same columns by tcgen05.wait::st alone
    text = source("paged_attend.cu")
    walk = body(text, "if (clean) {")
    cleared = body(walk, "if (it == 0) {")
    assert cleared.index("tmem_st16(") < cleared.index("tmem_wait_st();")
    assert walk.index("tmem_wait_st();") < walk.index("add_odd<")
    # and what adds to them leaves them ready for the next that does
    add = body(text, "void add_odd(")
    assert add.index("tmem_st16(") < add.rindex("tmem_wait_st();")


def test_lanes_meet_before_the_paged_attention_moves_tensor_memory():
    # tcgen05.ld and .st are .sync.aligned: what lets a warp's lanes part in front of one is followed by __syncwarp, or
    # is an instruction under a predicate instead of a branch
    text = source("paged_attend.cu")
    result = text[text.index("for (int c = c0; c < c1; c += 16) {"):]
    loop = body(result, "for (int c = c0; c < c1; c += 16) {")
    assert "continue;" not in loop and loop.strip().endswith("__syncwarp();")
    half_done = body(text, "auto half_done = [&] {")
    assert "if (" not in half_done and "mbar_arrive_if(lane == 0," in half_done
    assert "@p mbarrier.arrive" in body(text, "void mbar_arrive_if(")
    add = body(text, "void add_odd(")
    assert add.index("if (sees &&") < add.index("__syncwarp();") < add.index("tmem_st16(")


def test_a_warp_that_the_others_do_not_meet_says_so():
    # without the second walk outputs are left as the first made them: that is an error, not a result
    onward = body(source("paged_attend.cu"), "auto onward = [&](bool& clean) {")
    assert "set_error(a.error, AIRCACHE_ERR_DEVICE_TIMEOUT);" in body(onward, "if (!mbar_wait_warp(&ctl->again")


def test_a_failed_query_of_a_kernel_is_asked_again():
    # a static that takes its value from the first call alone would refuse every later one
    text = source("paged_attend.cu")
    assert "static const int regs" not in text
    query = body(text, "if (regs == 0) {")
    assert query.index("return AIRCACHE_ERR_CUDA;") < query.index("known.store(")
