"""The rules of test_source_rules.py for the C++ sources, which its lists of endings leave out.  CPU only."""
import re

from tests.test_source_rules import _files, _read


def test_cpp_sources_keep_the_rules():
    files = _files((".cpp", ".cc", ".cxx", ".hpp"))
    assert any(p.endswith("requests_binding.cpp") for p in files)
    # (assembled here, so that this file does not contain the names either)
    names = [a + "Batch" + "Async" for a in ("cudaMemcpy", "cudaMemcpy3D", "cuMemcpy", "cuMemcpy3D")]
    for p in files:
        text = _read(p)
        assert ".multicast::cluster" not in text, p
        assert not any(n in text for n in names), p
        assert "__trap" not in text and not re.search(r"\b(abort|trap|exit)\s*\(", text), p
        assert not re.search(r"^\s*assert\s*\(", text, flags=re.M), p
