"""The plan of the products of rows, on the CPU: the host code of linear.hip in
a program of its own that prints what a call of given sizes would launch."""
import os
import subprocess

import pytest

import submanifold_sparse_convolution_device_amd.build as lib_build

PROGRAM = """
#include "linear.hip"
#include <cstdio>
namespace spconv {
hipError_t launch_product_f32(const ProductArgs&, ProductForm, ProductShape, hipStream_t) { return hipSuccess; }
hipError_t launch_product_f16(const ProductArgs&, ProductForm, ProductShape, hipStream_t) { return hipSuccess; }
hipError_t launch_product_bf16(const ProductArgs&, ProductForm, ProductShape, hipStream_t) { return hipSuccess; }
}
int main() {
  int dtype, rows, k, n;
  while (scanf("%d %d %d %d", &dtype, &rows, &k, &n) == 4) {
    spconv::Carver c{nullptr};
    const spconv::ByRows b = spconv::plan_all_rows(spconv::kByRows, dtype, nullptr, rows, 1, k, n, &c);
    printf("%d %d %d %zu\\n", b.head, b.p.shape == spconv::kLargeShape, b.head == 0 ? rows : b.p.a.rows + b.rest.a.rows, c.at);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """(rows of the first of two launches or 0, whether it takes the largest
    tiles, rows of both, bytes of workspace) for (dtype, rows, k, n)."""
    if not os.path.exists(lib_build.HIPCC):
        pytest.skip("no hipcc")
    at = tmp_path_factory.mktemp("plan")
    source, program = str(at / "plan.hip"), str(at / "plan")
    with open(source, "w") as f:
        f.write(PROGRAM)
    flags = [f for f in lib_build.FLAGS if f != "-O3"]
    subprocess.run([lib_build.HIPCC, "-O1", *flags, "-I", lib_build.CSRC, source, "-o", program], check=True, capture_output=True, timeout=300)

    def ask(sizes):
        text = "".join("%d %d %d %d\n" % s for s in sizes)
        out = subprocess.run([program], input=text, check=True, capture_output=True, text=True, timeout=60).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]

    return ask


def test_two_launches_only_for_the_largest_tiles(plan):
    """A product goes by two launches where the first one fills rounds of the
    largest tiles: 65,537 rows by 256 columns.  With so many columns that whole
    rows of tiles are a part of a round, the first one would not take them, and
    the weights would be read twice."""
    sizes = [(2, rows, k, n) for rows in (257, 300, 400, 512, 513, 700, 4097, 13057, 65537, 70000, 131073)
             for k in (512, 1024, 2048, 4096) for n in (192, 256, 1024, 4096, 20000, 22100, 24000, 33000, 36000, 40704, 48000, 100000)]
    got = plan(sizes)
    assert len(got) == len(sizes)
    for size, (head, largest, rows, _) in zip(sizes, got):
        assert head == 0 or largest, size
        assert rows == size[1] and head % 256 == 0 and head < size[1], size
    by_size = dict(zip(sizes, got))
    assert by_size[(2, 65537, 1024, 256)][0] == 65536
    assert by_size[(2, 4097, 4096, 4096)][0] == 4096
    assert by_size[(2, 300, 1024, 33000)][0] == 0
