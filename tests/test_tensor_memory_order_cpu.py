"""The order of tensor-memory allocations and of the waits between kernels.  An allocation waits for free columns; a CTA that
holds some while it waits for the grid ahead must not keep a CTA of that grid, which counts as triggered, waiting for its own.
So a kernel triggers the next one only behind a barrier after its allocation, and a kernel whose CTAs leave an SM room for other
kernels' allocates after its wait.  Read from the sources: on a GPU the fault is a hang."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_recurrence_sequence_gb300", "csrc")
ALLOC = re.compile(r"\btmem_alloc2?\(&")


def _kernels():
    """(file, body) of every kernel that allocates tensor memory: a function from its __global__ to the brace that ends it."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"__global__", text):
            end = text.find("\n}", m.start())
            body = text[m.start():end]
            if ALLOC.search(body):
                yield name, body


KERNELS = list(_kernels())


def test_the_kernels_are_found():
    assert {n for n, _ in KERNELS} == {"block_gemm.cu", "ce_gemm.cu", "proj_gemm.cu", "rglru.cu", "ssm_scan_bwd.cu"}


IDS = [f"{i}-{n}" for i, (n, _) in enumerate(KERNELS)]


def _places(body, call):
    return [m.start() for m in re.finditer(r"\b" + re.escape(call), body)]


@pytest.mark.parametrize("name,body", KERNELS, ids=IDS)
def test_the_next_kernel_starts_after_every_allocation(name, body):
    alloc = ALLOC.search(body).start()
    for trigger in _places(body, "pdl_trigger()"):
        assert any(alloc < sync < trigger for sync in _places(body, "__syncthreads()"))


def test_the_scan_allocates_after_its_wait():
    """Its CTAs take a quarter of an SM's shared memory or less where channels are few."""
    bodies = [b for n, b in KERNELS if n == "ssm_scan_bwd.cu"]
    assert bodies
    for body in bodies:
        assert max(_places(body, "pdl_wait()")) < ALLOC.search(body).start()


def test_the_rglru_scans_start_in_stream_order():
    for body in (b for n, b in KERNELS if n == "rglru.cu"):
        assert not _places(body, "pdl_wait()") and not _places(body, "pdl_trigger()")
