"""The bench line's profiled figures belong to the sources the products are
built from: other operators' files leave them valid (no GPU)."""
import os
import re
import shutil

import pytest

import bench
from few_row_quantized_amd import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of csrc/ that bench.py looks at."""
    csrc = tmp_path / "few_row_quantized_amd" / "csrc"
    shutil.copytree(os.path.join(bench.ROOT, "few_row_quantized_amd", "csrc"), csrc)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return csrc


def test_files_of_other_operators_do_not_count(tree):
    before = bench.csrc_sha256()
    (tree / "qgemv_new_operator.hip").write_text("int another;\n")
    assert bench.csrc_sha256() == before
    for name in ("qgemv_append.hip", "qgemv_attend_impl.h", "qgemv_kv.h", "qgemv_torch.cpp", "qgemv_verify.hip"):
        path = tree / name
        path.write_text(path.read_text() + "int more;\n")
        assert bench.csrc_sha256() == before, name


@pytest.mark.parametrize("name", ["qgemv_mfma.hip", "qgemv_mfma_impl.h", "qgemv_device.h", "qgemv_select_table.h",
                                  "qgemv_api.cpp", "qgemv_gather_route.h"])
def test_the_products_own_files_do(tree, name):
    before = bench.csrc_sha256()
    path = tree / name
    path.write_text(path.read_text() + "// a comment\n\n")
    assert bench.csrc_sha256() == before
    path.write_text(path.read_text() + "int more;\n")
    assert bench.csrc_sha256() != before


def test_every_source_is_built_once_and_every_include_counts():
    assert sorted(build.SOURCES) == sorted(set(build.SOURCES))
    names = bench.product_sources()
    assert set(build.PRODUCTS) <= set(names) and not set(build.VERIFY_STEP) & set(names)
    for name in names:
        text = open(os.path.join(bench.ROOT, "few_row_quantized_amd", "csrc", name), encoding="utf-8").read()
        for other in re.findall(r'#include "([^"/]+)"', text):
            assert other in names
