"""What the products with block scales read of the kernel in front of them, from the sources: these orders hold by the
memory model or not at all, and a run that keeps them by chance looks like one that must."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "quantized_speculative_decoding_shared_gb300", "csrc")


def source(name):
    """A file of csrc without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def body(text, name):
    """The body of the function `name`, braces included."""
    start = text.index("{", re.search(r"\b%s\([^;{]*\)\s*\{" % name, text).start())
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(name)


@pytest.mark.parametrize("file,kernel", [("fp8_block_stream.cu", "stream_kernel"), ("fp8_block_tile.cu", "tile_kernel")])
def test_scales_are_read_coherently(file, kernel):
    """The kernel in front may still write them while this one is resident: nothing that is read-only by declaration
    only (ld.global.nc) reads them, and what does is behind the dependency wait."""
    text = body(source(file), kernel)
    assert "__ldg(" not in text and ".nc" not in text
    reads = [m.start() for m in re.finditer(r"__ldcg\(", text)]
    warp = text.index("warp == kScaleWarp")
    wait = text.index("pdl_wait()", warp)
    assert len(reads) >= 2 and all(r > wait for r in reads)


@pytest.mark.parametrize("file,kernel", [("fp8_block.cu", "quant_weights_kernel"), ("fp8.cu", "quant_rows_kernel")])
def test_quantisers_of_weights_end_before_the_next_kernel_begins(file, kernel):
    """Linears read their weights ahead of the dependency wait: their maker never lets them begin early, and ends with
    its codes performed for the device and ordered before asynchronous copies."""
    text = body(source(file), kernel)
    early = [line.strip() for line in text.splitlines() if "pdl_launch_dependents" in line]
    assert early == ([] if kernel == "quant_weights_kernel" else ["if (!kHalf) pdl_launch_dependents();"])
    stored, fence, proxy = (text.rindex(s) for s in ("store_codes" if early == [] else "make_uint2(lo, hi)", "__threadfence();",
                                                     "umma::fence_proxy_async_global();"))
    assert stored < fence < proxy


@pytest.mark.parametrize("file,kernel,first", [("fp8_block_stream.cu", "stream_kernel", "i < pre; ++i) load_weights("),
                                               ("fp8_block_tile.cu", "tile_kernel", "i < early; ++i) load_weights("),
                                               ("fp8.cu", "fp8_umma_kernel", "umma::tma_load_2d(")])
def test_early_weights_are_read_behind_a_fence_of_the_proxies(file, kernel, first):
    text = body(source(file), kernel)
    assert 0 <= text.find("umma::fence_proxy_async_global();") < text.index(first)


def test_scales_and_rows_of_the_per_token_linear_are_read_coherently():
    text = source("fp8.cu")
    quant, linear = body(text, "quant_rows_kernel"), body(text, "fp8_umma_kernel")
    assert not re.search(r"\brow\[", quant) and quant.count("ld_written(row + i)") == 2
    assert not re.search(r"\b(sa|s8)\[", linear) and "ld_written(sa +" in linear and "ld_written(s8 +" in linear
    assert quant.index("pdl_wait()") < quant.index("ld_written(") and linear.rindex("pdl_wait()") < linear.index("ld_written(")
    assert "asm volatile(\"ld.global.f32" in source("qspec_device.cuh")
