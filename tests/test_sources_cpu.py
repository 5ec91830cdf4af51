"""What the kernels' sources may not hold, read as text: forms that are safe on one GPU alone, and reads whose order the
language does not promise."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_232_gb300", "csrc")


def sources():
    """(file name, text without comments) of every kernel source."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if path.endswith((".cu", ".cuh", ".h")):
            with open(path) as f:
                yield os.path.basename(path), re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def instructions(text):
    """The string literals of each asm statement, joined."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(((?:\s*\"(?:[^\"\\]|\\.)*\")+)", text):
        yield "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))


def test_no_load_is_sent_to_several_blocks():
    """The library is loaded by every rank of a run over several GPUs, and a cache may lie in another GPU's memory: no tensor
    load writes the shared memory of more than one block."""
    seen = 0
    for name, text in sources():
        for code in instructions(text):
            for line in code.split("\\n\\t"):
                if "cp.async.bulk" in line:
                    seen += 1
                    assert "multi" + "cast" not in line, f"{name}: {line}"
    assert seen >= 4      # the loads were found at all


def test_no_read_of_changing_data_through_the_non_coherent_path():
    """A kernel that waits for the one before it (griddepcontrol.wait) is resident while that one still writes, so what it
    reads may change while it runs: the read-only path is not defined for that, nor may a load be moved ahead of the wait."""
    waiting = []
    for name, text in sources():
        if "griddepcontrol.wait" in text:
            waiting.append(name)
            for form in ("__ldg(", "__ldcg(", "ldg_nc_128(", "ldg_f4(", "ld.global.nc", "__restrict__"):
                assert form not in text, f"{name}: {form}"
    assert {"decode.cuh", "latent_kernel.cuh", "pages.cuh", "prefill_kernel.cuh", "tree_kernel.cuh"} <= set(waiting)
