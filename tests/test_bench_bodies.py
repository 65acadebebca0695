"""The recorded traffic of a kernel follows the headers that hold its body, too."""
import os
import re
import shutil

import bench


def test_a_change_of_a_body_changes_the_hash(tmp_path, monkeypatch):
    for source, names in bench.BODIES.items():
        kind = next(k for k, v in bench.SOURCES.items() if v == source)
        sha = bench.gemm_source_sha(kind)
        for name in names:
            shutil.copy(os.path.join(bench._CSRC, name), tmp_path / name)
        with monkeypatch.context() as m:
            m.setattr(bench, "_BODY_DIR", str(tmp_path))
            assert bench.gemm_source_sha(kind) == sha
            for name in names:
                text = (tmp_path / name).read_text()
                (tmp_path / name).write_text("// a comment\n" + text)
                assert bench.gemm_source_sha(kind) == sha
                (tmp_path / name).write_text(text + "\nint extra_symbol;\n")
                assert bench.gemm_source_sha(kind) != sha
                (tmp_path / name).write_text(text)


def test_every_body_is_listed():
    """A header that a source includes and that holds a kernel's body is one of its BODIES."""
    for source in set(bench.SOURCES.values()):
        text = open(os.path.join(bench._CSRC, source)).read()
        for name in re.findall(r'#include "([^"]+)"', text):
            path = os.path.join(bench._CSRC, name)
            if os.path.exists(path) and "_body(" in open(path).read():
                assert name in bench.BODIES.get(source, ()), (source, name)
