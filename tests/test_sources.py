"""What the kernels' sources may name (nothing is compiled here)."""
from pathlib import Path

import paged_kv_cache_11_gb300 as pkv

PACKAGE = Path(pkv.__file__).resolve().parent
SOURCES = sorted(p for d in (PACKAGE, PACKAGE.parent / "include") for p in d.rglob("*") if p.suffix in (".cu", ".cuh", ".h", ".cpp", ".c"))


def test_no_copy_or_arrival_goes_to_several_ctas():
    """The library also runs as replicas on several GPUs, and its calls take whatever device pointer they are given: none of
    its copies may go to more than one CTA's shared memory, where memory of another GPU behind the pointer would hang."""
    word = "multi" + "cast"
    assert len(SOURCES) > 15
    assert [p.name for p in SOURCES if word in p.read_text().lower()] == []
