"""What runs beside what in a stream: a product reads its weight before the kernel ahead has ended, so every kernel of
the family lets the next one start only after its own wait, and the one that writes weights not at all.  Read from the
sources; the calls themselves are in test_w4a4_order_gpu.py."""
import os
import re

import pytest

import nvfp4_block_scaled_linear_gb300 as pkg

HERE = os.path.join(os.path.dirname(os.path.abspath(pkg.__file__)), "csrc_w4a4")


def code(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(HERE, name)).read())
    return re.sub(r"\s+", " ", text)


def body(text, kernel):
    """From the kernel's name to the end of its braces."""
    at = text.index("{", text.index(kernel + "("))
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
        if depth == 0:
            return text[at:end]


KERNELS = [("rows.cu", "norm_kernel"), ("rows.cu", "quantize_rows_kernel"), ("product_narrow.cu", "narrow_kernel"),
           ("product_few.cu", "few_kernel"), ("product_many.cu", "many_kernel")]


@pytest.mark.parametrize("name, kernel", KERNELS)
def test_the_next_kernel_starts_after_the_wait(name, kernel):
    b = body(code(name), kernel)
    assert b.count("griddep_launch_dependents()") == 1
    # in the producer's branch, or at the kernel's begin: the wait is ahead of it, and no branch ends between them
    wait, start = b.index("griddep_wait()"), b.index("griddep_launch_dependents()")
    assert wait < start
    between = b[wait:start]
    depth = least = 0
    for c in between:
        depth += {"{": 1, "}": -1}.get(c, 0)
        least = min(least, depth)
    assert least == 0


def test_the_layout_of_scales_lets_nothing_start():
    b = body(code("rows.cu"), "scale_layout_kernel")
    assert "griddep_wait()" in b and "griddep_launch_dependents" not in b


def test_every_kernel_is_listed():
    found = []
    for name in sorted(os.listdir(HERE)):
        found += [(name, k) for k in re.findall(r"__global__ void (?:__launch_bounds__\([^()]*\) )?(\w+)\(", code(name))]
    assert sorted(found) == sorted(KERNELS + [("rows.cu", "scale_layout_kernel"), ("api.cu", "read_w4a4_error_kernel")])
