"""Rules that every kernel of the library keeps, read from its sources."""
import glob
import os
import re
import subprocess

from decode_gemm_e8_b200 import build as e8build

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_gemm_e8_b200", "csrc")


def _sources():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                   glob.glob(os.path.join(CSRC, "*.h")))
    assert len(files) > 10
    return {os.path.basename(f): open(f).read() for f in files}


def test_no_copy_is_multicast_to_a_cluster():
    """Every bulk and tensor copy fills the shared memory of its own CTA: one library serves
    every rank of a run on several GPUs.  (A commit signals barriers and copies nothing.)"""
    for name, text in _sources().items():
        text = re.sub(r'"\s*\n\s*"', "", text)   # an instruction may be cut into several literals
        for line in text.splitlines():
            if "multicast::cluster" in line:
                assert "tcgen05.commit" in line and "cp.async" not in line, (name, line)


# kernels that let the next kernel of the stream start before they have ended: they write
# workspaces, fp32 results, codes or scales, but nothing that a call takes as X or as indices
RELEASE = {"k_act_rht_fast", "k_act_q8", "k_gemm_q8", "k_mx4_encode", "k_moe_route"}


def test_kernels_whose_output_is_an_input_of_e8_gemm_end_before_the_next_starts():
    """e8_gemm reads X, idx1 and idx2 before it waits for the kernel in front of it, so a
    kernel that writes tokens (bf16) may not release its dependents early."""
    found = set()
    for name, text in _sources().items():
        text = re.sub(r"//[^\n]*", "", text)
        kernel = None
        for m in re.finditer(r"__global__[^;{]*?\b(k_\w+)\s*\(|\bgrid_dep_launch\(\);", text):
            if m.group(1):
                kernel = m.group(1)
            else:
                found.add(kernel)
    assert found == RELEASE


def test_the_experts_ring_is_not_written_without_a_proxy_fence():
    """The lists' scratch space lies where copies of the async proxy land next: ordinary
    writes to it happen only on the path that ends with a fence of the two."""
    text = _sources()["e8_moe.cu"]
    lists = text[text.index("void build_lists("):text.index("// A unit as the scheduler")]
    assert lists.rstrip().endswith("fence_proxy_async_smem();   // the scratch space becomes the copies' ring\n"
                                   "  __syncthreads();\n}")
    kernel = text[text.index("k_moe_experts(const"):]
    assert kernel.count("mask[") == 1
    assert re.search(r"if \(slots > 32\)\s*for \([^)]*\) mask\[i\] = 0ull;", kernel)
    assert re.search(r"if \(slots > 32\)\s*build_lists\(", kernel)


def test_a_timer_that_reads_backwards_ends_no_wait(tmp_path):
    """Every bounded wait measures its time with ns_between, which answers 0 when the later
    reading is the smaller one."""
    for name, text in _sources().items():
        assert not re.search(r"global_timer_ns\(\)\s*-", text), name
        assert not re.search(r"\bt - t0\b", text), name
    src = tmp_path / "t.cu"
    src.write_text('''#include <cstdio>
#include "e8_common.cuh"
int main() {
  const uint64_t top = 1ull << 63;
  const uint64_t pair[][2] = {{5, 5}, {5, 9}, {9, 5}, {1ull << 60, (1ull << 60) - 1}, {7, 7 + e8::kWaitLimitNs},
                              {top - 2, top + 3}, {~0ull, 2}};
  for (const auto& p : pair) std::printf("%llu\\n", (unsigned long long)e8::ns_between(p[0], p[1]));
}
''')
    exe = tmp_path / "t"
    root = os.path.dirname(os.path.dirname(CSRC))
    subprocess.run([e8build.NVCC, *e8build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", CSRC, "-I",
                    os.path.join(root, "include"), "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [0, 4, 0, 0, 2000000000, 5, 3]


def test_tile_counts_at_the_largest_sizes(tmp_path):
    """Sizes go up to 2^31 - 1; the product's kernels count their tiles in 32 bits."""
    text = re.sub(r"//[^\n]*", "", _sources()["e8_mx4_gemm.cu"])
    assert not re.search(r"\(a\.[MNK] \+ ", text)
    src = tmp_path / "t.cu"
    src.write_text('''#include <cstdio>
#include "e8_mx4.cuh"
int main() {
  for (int n : {1, 256, 257, 2147483391, 2147483392, 2147483393, 2147483647})
    std::printf("%d\\n", e8::mx4::tiles_of(n, 256));
}
''')
    exe = tmp_path / "t"
    subprocess.run([e8build.NVCC, *e8build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", CSRC, "-I",
                    e8build.INCLUDE, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [1, 1, 2, 2 ** 23 - 1, 2 ** 23 - 1, 2 ** 23, 2 ** 23]
