"""What build() puts in place, with compilers that only write their output file (no GPU)."""
import os
import warnings

import pytest

import combine_moe_route_06_gb300 as m

WRITER = """#!/bin/sh
while [ $# -gt 0 ]; do
    if [ "$1" = -o ]; then echo built > "$2"; fi
    shift
done
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty build folder; tree(False) makes the C++ compiler fail."""
    b = m._build
    for name, ok in (("cuda/bin/nvcc", True), ("good", True), ("bad", False)):
        path = tmp_path / name
        path.parent.mkdir(parents=True, exist_ok=True)
        path.write_text(WRITER if ok else "#!/bin/sh\necho no such header >&2\nexit 1\n")
        path.chmod(0o755)
    monkeypatch.setenv("CUDA_HOME", str(tmp_path / "cuda"))
    out = tmp_path / "out"
    monkeypatch.setattr(b, "OUT_DIR", str(out))
    monkeypatch.setattr(b, "LIB_PATH", str(out / "libmoeroute.so"))
    monkeypatch.setattr(b, "OPS_PATH", str(out / "_moe_ops.so"))
    monkeypatch.setattr(b, "OPS_FOR_PATH", str(out / "_moe_ops.for"), raising=False)
    monkeypatch.setattr(m, "_ops_module", None)
    monkeypatch.setattr(m, "load_library", lambda: None)     # (what is built here is no library)

    def compiler(works):
        monkeypatch.setenv("CXX", str(tmp_path / ("good" if works else "bad")))

    compiler(True)
    return b, compiler


def stamp(path):
    return os.stat(path).st_mtime_ns


def age(path):
    os.utime(path, (1, 1))


def test_the_library_does_not_need_the_entry_points(tree):
    b, compiler = tree
    compiler(False)
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert b.build() == b.LIB_PATH
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.OPS_PATH)
    with pytest.raises(m.MoeLibraryMissing, match="_moe_ops.so is not built"):
        m._ops()
    # the next call tries the entry points again, and them only
    before = stamp(b.LIB_PATH)
    compiler(True)
    assert b.build() == b.LIB_PATH
    assert os.path.exists(b.OPS_PATH) and stamp(b.LIB_PATH) == before


def test_what_is_fresh_is_not_built_again(tree):
    b, _ = tree
    b.build()
    for touched, other in ((b.OPS_PATH, b.LIB_PATH), (b.LIB_PATH, b.OPS_PATH)):
        age(touched)
        before = stamp(other)
        b.build()
        assert stamp(touched) > 10 ** 12 and stamp(other) == before
    before = stamp(b.LIB_PATH), stamp(b.OPS_PATH)
    b.build()
    assert (stamp(b.LIB_PATH), stamp(b.OPS_PATH)) == before


def test_entry_points_that_no_longer_build_do_not_stay(tree):
    b, compiler = tree
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        b.build()
    age(b.OPS_PATH)
    compiler(False)
    with pytest.warns(RuntimeWarning, match="were not built"):
        b.build()
    assert not os.path.exists(b.OPS_PATH)


def test_entry_points_of_another_torch_are_built_again_and_not_loaded(tree, monkeypatch):
    b, _ = tree
    monkeypatch.setattr(b.torch, "__version__", "1.0")
    b.build()
    monkeypatch.setattr(b.torch, "__version__", "1.1")
    with pytest.raises(m.MoeLibraryMissing, match="torch 1.0.*torch 1.1"):
        m._ops()
    before = stamp(b.LIB_PATH)
    with open(b.OPS_PATH, "w") as f:
        f.write("of torch 1.0")
    b.build()
    with open(b.OPS_PATH) as f:
        assert f.read() == "built\n"
    assert stamp(b.LIB_PATH) == before
    with pytest.raises(ImportError):            # (what the writer wrote is no module)
        m._ops()
