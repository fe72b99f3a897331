"""Rules of the 4-bit cache's kernels that hold by their sources, checked without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "q8_int8_block_gb300", "csrc")


def source(name):
    """A source file without its comments, and whatever of csrc it includes."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    return text, [h for h in re.findall(r'#include "([^"]+)"', text) if os.path.exists(os.path.join(CSRC, h))]


@pytest.mark.parametrize("name", ["q8_kv4.cu", "q8_kv4_attn.cu"])
def test_kernels_that_start_early_use_no_read_only_loads(name):
    """A kernel launched as the dependent of the one in front starts while that still writes; ld.global.nc
    (__ldg, or what const __restrict__ allows) asks for data that is constant while the kernel runs, and
    may be moved across the wait."""
    seen, todo = set(), [name]
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        text, more = source(at)
        todo += more
        found = re.findall(r"__ldg|ld\.global[.\w:]*\.nc|__restrict__", text)
        assert not found, (at, found)
    assert "griddepcontrol.wait" in "".join(source(f)[0] for f in seen)


def test_linears_that_start_early_use_no_read_only_loads_of_what_is_in_front():
    """The same for the decode kernel (its norm's weights, its epilogue's input) and for the factor that the
    batch kernel's quantiser takes from the kernel in front."""
    decode, batch = source("q8_decode.cu")[0], source("q8_batch.cu")[0]
    assert not re.search(r"__ldg|ld\.global[.\w:]*\.nc|__restrict__|epi_aux", decode) and "late_aux(p.epi" in decode
    assert "return e.op == kEpiNone ? 0.0f : e.aux[i];" in decode
    args = re.search(r"void __launch_bounds__\(256\) quantize_batch_kernel\((.*?)\) \{", batch, flags=re.S)[1]
    assert re.search(r"const float\* r$", args)
    reads = re.findall(r"[^\n]*(?:\br ?\+ m\b|\br\[m\])[^\n]*", batch)
    assert reads == ["        d = __fmul_rn(d, *static_cast<const volatile float*>(r + m));"]


def test_the_batch_kernel_knows_its_epilogue_input_only_behind_the_wait():
    """Its loads of aux may be read-only ones, which move freely: the address they take comes out of a statement
    that stays behind the wait."""
    kernel = source("q8_batch.cu")[0]
    wait = re.search(r"pdl_wait\(\);\s*if constexpr \(!kBlockSums && kFused\)", kernel).start()
    known = kernel.index('asm volatile("" : "+l"(epi.aux));')
    assert wait < known < kernel.index("epi_aux(epi,") and "epi_aux(p.epi" not in kernel


RING = """
#include "q8_kv4_ring.h"
// Bit k: the copy of tile at + k is waited for when the wait for tile `at` of a run of `tiles` gives up; of
// every third tile the page is missing.
extern "C" unsigned waited_for(int tiles, int stages, int at) {
  int held[32];
  auto fill = [&](int i) { held[i % stages] = q8::stage_state(i < tiles, i % 3 != 2); };
  for (int i = 0; i < stages; ++i) fill(i);
  for (int i = 0; i < at; ++i) fill(i + stages);
  unsigned bits = 0;
  for (int k = 0; k < stages; ++k) bits |= static_cast<unsigned>(q8::stage_completes(held[(at + k) % stages])) << k;
  return bits;
}
"""


def test_a_wait_that_gives_up_waits_for_the_copies_under_way(tmp_path):
    """Those of the run's tiles from the one that did not come to a ring ahead of it, and no others: nobody
    would complete their phases."""
    (tmp_path / "ring.cpp").write_text(RING)
    lib = str(tmp_path / "ring.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I" + CSRC, str(tmp_path / "ring.cpp"), "-o", lib], check=True)
    waited_for = ctypes.CDLL(lib).waited_for
    for stages in (2, 3, 4, 7, 10):
        for tiles in range(1, 101):
            for at in range(tiles):
                want = sum(1 << k for k in range(stages) if at + k < tiles)
                assert waited_for(tiles, stages, at) == want, (stages, tiles, at)
    text, _ = source("q8_kv4_attn.cu")
    assert re.search(r"held = stage_state\(in_run, src != nullptr\);", text) and "held_s[st] = held;" in text
    assert re.search(r"if \(stage_completes\(held_s\[k % S\]\)\) mbar_wait\(&bars\[k % S\]", text)


def test_the_header_names_the_heads_that_have_a_prompt_path():
    """q8_kv4_attention's notes send chunks of a prompt to q8_prompt_attention, which takes heads of 64 and 128
    channels and refuses 256."""
    import __graft_entry__ as g
    g.build()
    import q8_int8_block_gb300 as q8
    # 0 q 1 k 2 v 3 cu_q 4 cu_k 5 o 6 B 7 Tq 8 Tk 9 H 10 Hkv 11 d 12 scale 13 strides 14 workspace 15 bytes 16 stream
    at = ctypes.c_void_p(0x10000)
    refused = {d: q8.lib().q8_prompt_attention(None, at, at, at, at, at, 1, 4, 4, 2, 1, d, 0.1, None, None, 0, None) for d in (64, 128, 256)}
    assert refused == {64: 1, 128: 1, 256: 2}  # a missing pointer, a size
    note = open(os.path.join(ROOT, "include", "q8.h")).read().split("q8_kv4_attention --")[1].split("*/")[0]
    note = " ".join(note.replace("*", " ").split())
    assert "with heads of 64 or 128 channels: q8_prompt_attention takes no heads of 256" in note
