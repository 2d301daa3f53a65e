"""Which kernels let the next one of the stream start early, read from the
source: a race cannot be provoked safely, and need not show when it is there."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_inner_product_b200", "csrc")


def _body(source, kernel):
    """The body of a __global__ function, without comments."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, source)).read())
    at = re.search(r"__global__[^;{]*?\b%s\(" % kernel, text)
    assert at, kernel
    start = text.index("{", text.index(")", at.end() - 1))
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError(kernel)


# the last kernels of the training calls: what they write may be a search's rows or queries
LAST = {"k_softmax_grad.cu": ["k6_finish"], "k_embedding.cu": ["k8_lookup", "k8_join"],
        "k_rownorm.cu": ["k7_layernorm", "k7_normalize_grad", "k7_columns"], "k_clip.cu": ["k9_scale", "k9_norm"],
        "k_normalize.cu": ["k1_normalize", "k0_cast_bf16"]}


def test_a_calls_last_kernel_does_not_signal_early():
    """The search reads its corpus and queries before it waits for its predecessors (k2_stream, DEFER)."""
    for source, kernels in LAST.items():
        for kernel in kernels:
            assert "pdl_trigger" not in _body(source, kernel), kernel
    # the runs are the last kernel where one block holds them all
    runs = _body("k_embedding.cu", "k8_runs")
    assert runs.count("pdl_trigger") == 1 and "if (gridDim.x > 1) pdl_trigger();" in runs


def test_what_the_call_wrote_is_not_read_as_read_only_data():
    """__ldg is for data that nothing writes while the kernel lives, and these kernels may be there before
    an earlier one of the call has written what they read."""
    for source, kernels in {"k_softmax_grad.cu": ["k6_finish"], "k_embedding.cu": ["k8_scan", "k8_heads", "k8_join"],
                            "k_rownorm.cu": ["k7_columns"]}.items():
        for kernel in kernels:
            body = _body(source, kernel)
            assert "__ldg(" not in body and ".load(" not in body, kernel


def test_memory_is_touched_after_the_wait():
    """Kernels that may start early: nothing of the call's arguments is read or written before the wait."""
    for source, kernels in {"k_softmax_grad.cu": ["k6_prepare", "k6_products", "k6_finish"], "k_rownorm.cu": ["k7_columns"],
                            "k_embedding.cu": ["k8_count", "k8_scan", "k8_scatter", "k8_heads", "k8_runs", "k8_join"]}.items():
        for kernel in kernels:
            before = _body(source, kernel).split("pdl_wait();")[0]
            assert len(before) < len(_body(source, kernel)), kernel
            touched = re.search(r"__ldc?g\(|\*\s*[pa]\.\w+|\b[pa]\.\w+(\.\w+)?\s*\[|load_token", before)
            assert not touched, (kernel, touched.group(0))
