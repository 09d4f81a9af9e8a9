"""Chunk and windowed attention and the page operators on the host: sizes at their limits, and what the sources promise of every call."""
import os
import re
import subprocess

import split_kv_decode_decoding_gb300 as da
from test_paged_more_host import fork

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "split_kv_decode_decoding_gb300", "csrc")


def test_pages_of_the_longest_sequences(tmp_path):
    """Every page size, at the longest sequence that the checks admit and around it: no sum passes what its type holds."""
    src = tmp_path / "pages.cpp"
    src.write_text(r"""
#include <cstdio>
#include "geometry.h"
int main() {
    for (int page = 16; page <= 1024; page += 16) {
        const int64_t most = 0x7fffff00ll / page * page;      // max_pages * page_size
        const int64_t lengths[] = {0, 1, page - 1, page, page + 1, most / 2, most - page, most - page + 1, most - 1, most};
        for (int64_t n : lengths) {
            const int64_t want = n / page + (n % page != 0), got = da_impl::pages_of(static_cast<int>(n), page);
            if (got != want) return std::printf("%lld tokens in pages of %d: %lld, not %lld\n", (long long)n, page, (long long)got, (long long)want), 1;
        }
    }
    return 0;
}
""")
    exe = str(tmp_path / "pages")
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC, "-o", exe, str(src)], check=True)
    got = subprocess.run([exe], capture_output=True, text=True)
    assert got.returncode == 0, got.stdout + got.stderr


def test_the_page_operators_count_pages_in_one_place():
    text = open(os.path.join(CSRC, "paged_pages.cu")).read()
    assert text.count("pages_of(") >= 2 and "P - 1) /" not in text


def test_a_fork_refuses_pages_whose_parts_pass_32_bits():
    """Refused on the host, before any device work (the addresses are never followed)."""
    da.build()
    lib = da.load()
    for heads, D, kv in ((1 << 17, 128, da.DA_F16), (1 << 18, 64, da.DA_BF16), (1 << 18, 128, da.DA_E4M3), (5 << 20, 64, da.DA_E4M3)):
        assert fork(lib, cache=dict(page_size=1024, Hkv=heads, D=D, kv_dtype=kv), page_size=1024) == da.DA_ERR_UNSUPPORTED


def functions(text):
    """Bodies of the device functions of a source file, with their heads."""
    found = []
    for head in re.finditer(r"^ *(?:template[^\n]*\n *)?(?:static )?__device__[^;{]*\{|^__global__[^;{]*\{", text, re.M):
        depth, at = 1, head.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        found.append(text[head.start():at])
    return found


def test_a_wait_that_ends_some_lanes_ends_their_warp():
    """The lanes of a warp look at their own clocks. Where the answer of a wait is used, the warp votes on it, so that a time-out
    that some lanes saw cannot leave the others alone at the next instruction for a whole warp."""
    used = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.startswith("paged_"):
            continue
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for body in functions(text):
            if re.match(r"[^{]*\bwait_lane\(", body):
                continue                                                   # its own definition
            for call in re.finditer(r"\bwait_lane\(", body):
                before = body[:call.start()].rstrip()
                if before.endswith((";", "{", "}", ")")):
                    continue                                               # a statement: nothing is done with the answer
                used += 1
                assert re.search(r"__(all|any)_sync\(0xffffffffu,", body[call.end():]), (name, body[:200])
    assert used >= 2


def test_no_kernel_reads_past_the_coherent_path():
    """Every kernel may begin while the one before it in the stream still writes, so none of its inputs is read as constant."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
            assert not re.search(r"\b__ldg\b|ld\.global(\.\w+)*\.nc\b|\b__restrict__\b", text), name


def test_every_block_of_a_chunk_leaves_the_second_kernel_its_list():
    """Whichever way a block of the first kernel ends, it has written its entry of the list of parts to join."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "paged_chunk.cu")).read())
    body = re.search(r"\nchunk_kernel\(.*?\n\}\n", text, re.S).group(0)
    assert "leave_join(p, plan);" in body
    for leave in re.finditer(r"\breturn;", body):
        assert re.search(r"p\.join\[blockIdx\.x\] = |leave_join\(", body[:leave.start()])
