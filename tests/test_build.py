"""How many compilers the build starts."""
import pytest

from differentiable_rasterization_amd import build


@pytest.mark.parametrize("value,want", [(None, 8), ("", 8), ("0", 8), ("-3", 8), ("many", 8),
                                        ("2.5", 8), ("1", 1), ("5", 5), ("16", 8), (" 4 ", 4)])
def test_jobs(monkeypatch, value, want):
    if value is None:
        monkeypatch.delenv("MAX_JOBS", raising=False)
    else:
        monkeypatch.setenv("MAX_JOBS", value)
    assert build.jobs() == want


@pytest.mark.parametrize("value", ["0", "-1", "many"])
def test_a_build_starts_whatever_the_variable_says(monkeypatch, tmp_path, value):
    """A compiler that only writes its output stands in for the real one."""
    fake = tmp_path / "hipcc"
    fake.write_text("#!/bin/sh\nwhile [ \"$1\" != -o ]; do shift; done\necho built > \"$2\"\n")
    fake.chmod(0o755)
    monkeypatch.setenv("MAX_JOBS", value)
    monkeypatch.setenv("HIPCC", str(fake))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "HASH_FILE", str(tmp_path / "hash"))
    build.build()
    assert (tmp_path / "lib.so").read_text() == "built\n"
