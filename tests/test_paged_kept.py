"""How sage_paged_compact orders the items of a long list: read from the kernel's source."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "video_diffusion_transformer_sage_gb300", "csrc", "paged_move.cu")


def test_the_rings_numbers_have_an_order():
    """An item's number is put behind a fence of the GPU's scope that comes after its rows were read, a writer goes on behind
    one that comes after it saw the numbers, and bulk stores behind a fence between the proxies."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    assert "fence.acq_rel.gpu" in text and "fence.proxy.async.global" in text
    kernel = text[text.index("paged_compact_long_kernel(const"):]
    assert "volatile uint16_t" not in kernel and "*at" not in kernel and not re.search(r"ring\[", kernel)
    read, fence, put, go = (kernel.index(x) for x in ("wait(full, k, B) &&", "fence_gpu();", "ring_put(", "pass(go, k, B)"))
    assert read < fence < put < go and kernel.count("ring_put(") == 1
    late = kernel[put:go]
    assert late.index("clear()") < late.index("fence_gpu();")
    write = kernel[kernel.index("bulk_store(") - 250:kernel.index("bulk_store(")]
    assert "fence_proxy_async_global();" in write
