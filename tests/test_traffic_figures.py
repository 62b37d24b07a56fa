"""The DRAM figures that the benchmark's line reports are of the kernels in the tree (no GPU)."""
import re

import bench
from tests.test_bench_host import CSRC


def _local_headers(name):
    """The files beside it that `name` includes, and theirs (the C header declares, and holds no code)."""
    found, todo = set(), [name]
    while todo:
        at = todo.pop()
        if at not in found:
            found.add(at)
            todo += [h for h in re.findall(r'^#include "([^"/]+)"', (CSRC / at).read_text(), flags=re.M) if (CSRC / h).exists()]
    return found


def test_the_hash_covers_every_header_of_the_kernels(monkeypatch):
    for grouped, sources in ((False, ["decode.cu"]), (True, ["decode.cu", "group_prefix.cu"])):
        read = []
        monkeypatch.setattr(bench, "_code_only", lambda text: read.append(text) or text)
        bench.decode_source_hash(grouped=grouped)
        monkeypatch.undo()
        assert {(CSRC / n).read_text() for s in sources for n in _local_headers(s)} <= set(read), sources


def test_every_figure_is_of_these_sources():
    lines = [l.split() for l in bench.TRAFFIC_FILE.read_text().splitlines() if l and not l.startswith("#")]
    assert len(lines) == 4
    assert [l[0] for l in lines if bench.traffic_per_launch(l[0]) is None] == []
